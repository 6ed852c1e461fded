"""4-bit codes with a scale and a zero point per group -- TEST INFRASTRUCTURE
ONLY.

Parity pinned: tests/test_affine_cpu.py works roundings, zero points and the
packing out by hand.

Definitions: per group of consecutive elements of a row, in float32 steps, lo =
min(0, smallest), hi = max(0, largest), s = bf16(hi / 15 - lo / 15), z =
round(-lo / s) in 0 .. 15 (symmetric: s = bf16(max|x| / 7), z = 8), c = round(x /
s) + z in 0 .. 15; s = 0 takes c = z; a group with a value that is not finite has
s = NaN, z = 0, c = 0.  An element is s (c - z).
"""
from __future__ import annotations

import numpy as np


def bf16(x):
    """float32 rounded to bf16's values, ties to even (NaN stays)."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7fff + ((b >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16) << np.uint64(16)).astype(np.uint32)
    return np.where(np.isnan(x), np.float32(np.nan), r.view(np.float32)).astype(np.float32)


def quantize(x, group, symmetric=False):
    """x [rows][cols] float32 -> codes [rows][cols] uint8, zeros and scales [rows][cols / group] float32."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    b = x.reshape(rows, cols // group, group)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], np.float32(0), b)
    f = np.float32
    if symmetric:
        s = bf16(np.abs(b).max(axis=2) / f(7))
        z = np.full_like(s, 8)
    else:
        lo, hi = np.minimum(b.min(axis=2), f(0)), np.maximum(b.max(axis=2), f(0))
        s = bf16(hi / f(15) - lo / f(15))
        z = np.clip(np.rint(-lo / np.where(s == 0, f(1), s)), 0, 15).astype(f)
        z = np.where(s == 0, f(0), z)
    t = np.where((s == 0)[:, :, None], f(0), np.rint(b / np.where(s == 0, f(1), s)[:, :, None]))
    c = np.clip(t + z[:, :, None], 0, 15)
    c = np.where(bad[:, :, None], 0, c).reshape(rows, cols).astype(np.uint8)
    return c, np.where(bad, f(0), z).astype(f), np.where(bad, f(np.nan), s).astype(f)


def decode(codes, zeros, scales):
    """float64 values."""
    g = codes.shape[1] // scales.shape[1]
    r = lambda v: np.repeat(np.asarray(v, dtype=np.float64), g, axis=1)
    return r(scales) * (np.asarray(codes, dtype=np.float64) - r(zeros))


def pack(codes, zeros, scales):
    c = np.asarray(codes, dtype=np.uint8)
    half = lambda v: (np.ascontiguousarray(v, dtype=np.float32).view(np.uint32) >> np.uint32(16)).astype(np.uint16)
    params = np.stack([half(zeros), half(scales)], axis=-1)
    return np.concatenate([(c[:, 0::2] | (c[:, 1::2] << 4)).reshape(-1), params.reshape(-1).view(np.uint8)])


def unpack(buf, rows, cols, group):
    n = rows * cols // 2
    b = np.asarray(buf[:n]).reshape(rows, cols // 2)
    codes = np.empty((rows, cols), dtype=np.uint8)
    codes[:, 0::2], codes[:, 1::2] = b & 15, b >> 4
    p = np.ascontiguousarray(buf[n:]).view(np.uint16).reshape(rows, cols // group, 2).astype(np.uint32) << np.uint32(16)
    p = np.ascontiguousarray(p).view(np.float32)
    return codes, p[:, :, 0], p[:, :, 1]
