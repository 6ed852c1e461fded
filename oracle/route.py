"""Routing to experts and combining their rows in float64 -- TEST
INFRASTRUCTURE ONLY.

Parity pinned: tests/test_route_cpu.py works choices, weights and drops out by
hand and checks every gradient against central differences.

Definitions, per row: s = softmax or sigmoid of the logits in float64; c = s in
float32 plus the float32 bias; experts at -infinity (logit or c) are never
chosen; with top_groups < groups, the groups of the largest group score (largest
c, or the sum of the two largest in float32) are kept, equal scores to the
lowest; ids = the k largest c, falling, equal ones to the lowest, NaN first, -1
where none is left; weights = scale s (/ the sum of the chosen s).  (In float64:
softmax scores below e^-700, which only a bias chooses, are not this oracle's.)
"""
from __future__ import annotations

import numpy as np


def scores(x, score):
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        out = x == -np.inf
        top = np.where(out, -np.inf, x).max(axis=1, keepdims=True)
        e = np.where(out, 0.0, np.exp(x - np.where(top == -np.inf, 0.0, top)))
        t = e.sum(axis=1, keepdims=True)
        return np.where(t == 0, 0.0, e / np.where(t == 0, 1.0, t))




def _order(c):
    """Indexes by falling c, NaN first, ties to the lowest."""
    return sorted(range(len(c)), key=lambda i: (0 if np.isnan(c[i]) else 1, 0.0 if np.isnan(c[i]) else -float(c[i]), i))


def choose(x, s, k, bias=None, groups=1, top_groups=1, group_score="max"):
    rows, E = s.shape
    ids = np.full((rows, k), -1, dtype=np.int32)
    with np.errstate(all="ignore"):
        c = s.astype(np.float32)
        if bias is not None:
            c = c + np.asarray(bias, dtype=np.float32)
    c = np.where(np.asarray(x) == -np.inf, np.float32(-np.inf), c)
    per = E // groups
    for r in range(rows):
        cr = c[r].copy()
        if top_groups < groups:
            of = []
            for g in range(groups):
                m = [cr[g * per + i] for i in _order(cr[g * per:(g + 1) * per])]
                two = group_score == "top2" and per > 1 and m[1] != -np.inf
                with np.errstate(all="ignore"):
                    of.append(np.float32(m[0] + m[1]) if two else m[0])
            for g in _order(np.array(of, dtype=np.float32))[top_groups:]:
                cr[g * per:(g + 1) * per] = -np.inf
        best = [i for i in _order(cr) if cr[i] != -np.inf][:k]
        ids[r, :len(best)] = best
    return ids


def weights(s, ids, renorm=True, scale=1.0):
    on = ids >= 0
    u = np.where(on, np.take_along_axis(s, np.maximum(ids, 0), axis=1), 0.0)
    if renorm:
        t = u.sum(axis=1, keepdims=True)
        with np.errstate(all="ignore"):
            u = u / np.where(t == 0, 1.0, t)
    return u * np.float64(np.float32(scale))


def route(x, k, score="softmax", bias=None, groups=1, top_groups=1, group_score="max", renorm=True, scale=1.0):
    s = scores(x, score)
    ids = choose(x, s, k, bias, groups, top_groups, group_score)
    return ids, weights(s, ids, renorm, scale)


def route_backward(x, ids, dw, score="softmax", renorm=True, scale=1.0):
    """dlogits, the |s du| that bounds what rounding du to float32 costs, and the
    size s sum |scale dw| (1 + 1 / S) of the terms that cancel in 64 bits."""
    s = scores(x, score)
    rows, E = s.shape
    scale = np.float64(np.float32(scale))
    dl, mag, terms = np.zeros_like(s), np.zeros_like(s), np.zeros_like(s)
    for r in range(rows):
        on = [(int(e), float(g)) for e, g in zip(ids[r], dw[r]) if 0 <= e < E]
        S = sum(s[r, e] for e, _ in on)
        dot = sum(g * s[r, e] for e, g in on)
        du = np.zeros(E)
        for e, g in on:
            du[e] += scale * (g - dot / S) / S if renorm and S != 0 else scale * g
        if score == "sigmoid":
            dl[r] = du * s[r] * (1 - s[r])
        else:
            dl[r] = s[r] * (du - (0.0 if renorm and S != 0 else scale * dot))
        mag[r] = np.abs(s[r] * du)
        terms[r] = s[r] * sum(abs(scale * g) for _, g in on) * (1 + (1 / S if renorm and S != 0 else 0))
    off = np.asarray(x) == -np.inf
    return np.where(off, 0.0, dl), mag, terms


def combine(Y, k, ids=None, w=None, add=None, n_experts=0):
    """out and the sums of magnitudes that bound its rounding."""
    T, d = Y.shape[0] // k, Y.shape[1]
    y = Y.reshape(T, k, d)
    on = counts(ids, (T, k), n_experts)
    w = np.ones((T, k)) if w is None else w
    p = np.where(on[:, :, None], y * w[:, :, None], 0.0)
    out, S = p.sum(axis=1), np.abs(p).sum(axis=1)
    if add is not None:
        out, S = out + add, S + np.abs(add)
    return out, S


def counts(ids, shape, n_experts=0):
    if ids is None:
        return np.ones(shape, dtype=bool)
    return (ids >= 0) & (ids < n_experts) if n_experts else ids >= 0


def combine_backward(dout, Y, k, ids=None, w=None, n_experts=0):
    """dY, dweights and the magnitude sums of the latter."""
    T, d = dout.shape
    on = counts(ids, (T, k), n_experts)
    w = np.ones((T, k)) if w is None else w
    dY = np.where(on[:, :, None], w[:, :, None] * dout[:, None, :], 0.0).reshape(T * k, d)
    p = np.where(on[:, :, None], dout[:, None, :] * Y.reshape(T, k, d), 0.0)
    return dY, p.sum(axis=2), np.abs(p).sum(axis=2)
