"""Grouped expert products, row grouping and the MXFP4 quantizer in float64
-- TEST INFRASTRUCTURE ONLY.

Parity pinned: tests/test_experts_cpu.py works the grouping, the products'
gradients (central differences) and the quantizer (every rounding case of the
E2M1 grid by hand) out on small inputs.

Definitions:
- grouping: rows with ids in [0, n) sorted by id, ties by row; the others in
  no group, positions behind the last group holding -1;
- products: Y[y(s)] = X[x(s)] W_e, dX[p(s)] = dY[y(s)] W_e^T, dW_e = sum over
  e's grouped rows s of X[x(s)]^T dY[y(s)], where x(s) = order[s] // top_k or
  s, y(s) and p(s) = order[s] or s;
- MXFP4: per block of 32 the shared exponent floor(log2 max|x|) - 2 clamped to
  [-127, 127] (-127 for zeros); x 2^-exponent to the nearest of 0, 0.5, 1,
  1.5, 2, 3, 4, 6, a tie to the one of even code, past 6 to 6; a block with a
  NaN or an infinity has scale code 255 and element codes 0.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def group_rows(ids, n):
    ids = np.asarray(ids, dtype=np.int64)
    rows = [np.flatnonzero(ids == g) for g in range(n)]
    offsets = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
    order = np.full(ids.shape[0], -1, dtype=np.int32)
    flat = np.concatenate(rows) if rows else np.zeros(0, dtype=np.int64)
    order[:flat.shape[0]] = flat
    return offsets, order


def _rows(offsets, order, e, top_k, x_order, y_order):
    s = np.arange(offsets[e], offsets[e + 1])
    o = np.asarray(order)[s].astype(np.int64) if (x_order or y_order) else s
    return (o // top_k if x_order else s), (o if y_order else s), (o if x_order else s)


def forward(X, W, offsets, order, rows, top_k=1, x_order=False, y_order=False):
    """W: [E][d_in][d_out].  Returns (Y, S, owned): the product, the sums of
    magnitudes |x||w| that bound its rounding, and the rows that have an owner."""
    Y = np.zeros((rows, W.shape[2]))
    S = np.zeros_like(Y)
    owned = np.zeros(rows, dtype=bool)
    for e in range(W.shape[0]):
        xi, yi, _ = _rows(offsets, order, e, top_k, x_order, y_order)
        Y[yi] = X[xi] @ W[e]
        S[yi] = np.abs(X[xi]) @ np.abs(W[e])
        owned[yi] = True
    return Y, S, owned


def backward(dY, X, W, offsets, order, rows, top_k=1, x_order=False, y_order=False):
    """Returns dX, its magnitude sums, the owned rows, dW, its magnitude sums."""
    dX = np.zeros((rows, W.shape[1]))
    SX = np.zeros_like(dX)
    owned = np.zeros(rows, dtype=bool)
    dW = np.zeros(W.shape)
    SW = np.zeros_like(dW)
    for e in range(W.shape[0]):
        xi, yi, pi = _rows(offsets, order, e, top_k, x_order, y_order)
        dX[pi] = dY[yi] @ W[e].T
        SX[pi] = np.abs(dY[yi]) @ np.abs(W[e].T)
        owned[pi] = True
        if X is not None:
            dW[e] = X[xi].T @ dY[yi]
            SW[e] = np.abs(X[xi]).T @ np.abs(dY[yi])
    return dX, SX, owned, dW, SW


def quantize(x):
    """x [rows][cols] (blocks along a row) -> element codes [rows][cols]
    (0..15) and scale codes [rows][cols / 32]."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    amax = np.abs(np.where(bad[:, :, None], 0.0, b)).max(axis=2)
    _, ex = np.frexp(np.where(amax > 0, amax, 1.0))
    shared = np.where(amax > 0, np.clip(ex - 1 - 2, -127, 127), -127)
    a = np.abs(np.where(bad[:, :, None], 0.0, b)) / np.exp2(shared.astype(np.float64))[:, :, None]
    d = np.abs(a[..., None] - GRID)
    # nearest point; of two equally near ones the even code
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    code = np.where(a >= 6.0, 7, code)
    code = code | (np.signbit(b).astype(np.int64) << 3)
    code = np.where(bad[:, :, None], 0, code).reshape(rows, cols).astype(np.uint8)
    return code, np.where(bad, 255, shared + 127).astype(np.uint8)


def decode(codes, scales):
    """float64 values of codes [rows][cols] with scale codes [rows][cols / 32]."""
    c = np.asarray(codes).astype(np.int64)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    sc = np.asarray(scales).astype(np.float64)
    s = np.where(sc == 255, np.nan, np.exp2(sc - 127.0))
    return v * np.repeat(s, 32, axis=1)


def pack(codes, scales):
    """The packed buffer: codes two per byte along a row (even element low), then the scales."""
    c = np.asarray(codes, dtype=np.uint8)
    return np.concatenate([(c[:, 0::2] | (c[:, 1::2] << 4)).reshape(-1), np.asarray(scales, dtype=np.uint8).reshape(-1)])
