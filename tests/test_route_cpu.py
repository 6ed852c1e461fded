"""Routing and combining without a GPU: the oracle on hand-worked rows and
against central differences, and every refusal of the C interface and the
binding (no launch happens: the pointers are host addresses that no call
reaches)."""
import ctypes

import numpy as np
import pytest

from adapter_lora_segments_amd import _lib
from adapter_lora_segments_amd import binding as b
from oracle import route as orc

NEG = -np.inf


# ---- the oracle ----

def test_choice_by_hand():
    x = np.log(np.array([[0.1, 0.4, 0.3, 0.2], [0.25, 0.25, 0.25, 0.25]]))
    ids, w = orc.route(x, 2)
    assert ids.tolist() == [[1, 2], [0, 1]]
    assert np.allclose(w, [[4 / 7, 3 / 7], [0.5, 0.5]], rtol=1e-14)
    ids, w = orc.route(x, 2, renorm=False, scale=2.0)
    assert np.allclose(w, [[0.8, 0.6], [0.5, 0.5]], rtol=1e-14)
    # the bias moves the choice, not the weight
    ids, w = orc.route(x, 1, bias=[1, 0, 0, 0], renorm=False)
    assert ids.tolist() == [[0], [0]] and np.allclose(w[:, 0], [0.1, 0.25])


def test_masks_by_hand():
    x = np.array([[NEG, 0.0, NEG, 0.0], [NEG] * 4, [0.0, np.nan, 1.0, NEG]])
    ids, w = orc.route(x, 3)
    assert ids[:2].tolist() == [[1, 3, -1], [-1, -1, -1]]
    assert w[:2].tolist() == [[0.5, 0.5, 0.0], [0.0, 0.0, 0.0]]
    assert ids[2].tolist() == [0, 1, 2] and np.isnan(w[2]).all()          # every score of the row is NaN
    ids, w = orc.route(x, 2, score="sigmoid", renorm=False)
    assert ids[2].tolist() == [1, 2] and np.isnan(w[2, 0]) and w[2, 1] == 1 / (1 + np.exp(-1.0))


def test_groups_by_hand():
    # sigmoid scores of three groups of two; sums 0.9 + 0.1, 0.6 + 0.5, 0.7 + 0.05
    p = np.array([[0.9, 0.1, 0.6, 0.5, 0.7, 0.05]])
    x = np.log(p / (1 - p))
    kw = dict(score="sigmoid", groups=3, renorm=False)
    assert orc.route(x, 1, top_groups=1, **kw)[0].tolist() == [[0]]
    assert orc.route(x, 1, top_groups=1, group_score="top2", **kw)[0].tolist() == [[2]]
    assert orc.route(x, 3, top_groups=2, **kw)[0].tolist() == [[0, 4, 1]]
    assert orc.route(x, 3, top_groups=2, group_score="top2", **kw)[0].tolist() == [[0, 2, 3]]
    # one expert of a group left: its score alone
    x[0, 3] = NEG
    assert orc.route(x, 1, top_groups=1, group_score="top2", **kw)[0].tolist() == [[0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_against_differences(score, renorm):
    """Central differences with h = 1e-5 are off by h^2 f''' / 6 (below 1e-9 of
    O(1) functions) and by rounding 2^-52 / h = 2e-11."""
    rng = np.random.default_rng(7)
    T, E, k = 5, 9, 3
    x, dw = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    x[2, 4] = NEG
    ids = orc.choose(x, orc.scores(x, score), k)
    ids[3, 1] = -1                                    # a dropped slot
    ids[4] = [2, 2, 5]                                # an expert named twice
    f = lambda x: (orc.weights(orc.scores(x, score), ids, renorm, 2.5) * np.where(ids >= 0, dw, 0.0)).sum()
    got, _, _ = orc.route_backward(x, ids, dw, score, renorm, 2.5)
    for i in np.ndindex(T, E):
        if x[i] == NEG:
            assert got[i] == 0
            continue
        up, down = x.copy(), x.copy()
        up[i] += 1e-5
        down[i] -= 1e-5
        assert abs((f(up) - f(down)) / 2e-5 - got[i]) < 1e-8, i


def test_combine_by_hand_and_differences():
    Y = np.array([[1.0, 2], [10, 20], [np.nan, np.nan], [3, 4]])
    ids, w = np.array([[5, 0], [-1, 7]]), np.array([[0.5, 2.0], [9.0, -1.0]])
    out, _ = orc.combine(Y, 2, ids, w)
    assert out.tolist() == [[20.5, 41], [-3, -4]]
    assert orc.combine(Y, 2, ids, w, add=np.ones((2, 2)), n_experts=6)[0].tolist() == [[21.5, 42], [1, 1]]
    rng = np.random.default_rng(1)
    Y, w, G = rng.standard_normal((12, 4)), rng.standard_normal((4, 3)), rng.standard_normal((4, 4))
    ids = rng.integers(-1, 3, size=(4, 3))
    dY, dw, _ = orc.combine_backward(G, Y, 3, ids, w)
    f = lambda Y, w: (orc.combine(Y, 3, ids, w)[0] * G).sum()
    for arr, grad in ((Y, dY), (w, dw)):              # bilinear: exact up to rounding
        for i in np.ndindex(arr.shape):
            old = arr[i]
            arr[i] = old + 0.5
            up = f(Y, w)
            arr[i] = old - 0.5
            down = f(Y, w)
            arr[i] = old
            assert abs(up - down - grad[i]) < 1e-12


# ---- refusals of the C interface ----

BUF = ctypes.create_string_buffer(1 << 12)
P16 = ctypes.addressof(BUF) + (-ctypes.addressof(BUF)) % 16
V = ctypes.c_void_p


def router(**kw):
    d = dict(n_experts=64, top_k=4, score=0, expert_groups=1, top_groups=1, group_score=0, renormalize=1, scale=1.0)
    d.update(kw)
    return _lib.Router(**d)


BAD_ROUTERS = [dict(n_experts=0), dict(n_experts=4097), dict(score=2), dict(score=-1), dict(expert_groups=0),
               dict(expert_groups=65, n_experts=65), dict(expert_groups=5), dict(top_groups=0), dict(top_groups=2),
               dict(group_score=2), dict(top_k=0), dict(top_k=65, n_experts=128), dict(top_k=5, n_experts=4),
               dict(expert_groups=32, top_groups=1, top_k=3), dict(renormalize=2)]


def _route(r, logits=P16, dt=1, rows=8, ld=64, bias=P16, ids=P16, w=P16):
    return _lib.lib().mlora_route(ctypes.byref(r) if r else None, V(logits), dt, rows, ld, V(bias), V(ids), V(w), None)


def _route_back(r, logits=P16, dt=1, rows=8, ld=64, ids=P16, dw=P16, dl=P16):
    return _lib.lib().mlora_route_backward(ctypes.byref(r) if r else None, V(logits), dt, rows, ld, V(ids), V(dw), V(dl),
                                           None)


@pytest.mark.parametrize("bad", BAD_ROUTERS)
def test_malformed_routers(bad):
    r = router(**bad)
    assert _route(r, ld=5000) == -1 and _route_back(r, ld=5000) == -1 and _route(r, rows=0, ld=5000) == -1
    assert _lib.lib().mlora_last_error().decode().startswith("route")


def test_malformed_route_calls():
    r = router()
    for f in (_route, _route_back):
        assert f(None) == -1 and f(r, dt=2) == -1 and f(r, rows=-1) == -1 and f(r, rows=1 << 31) == -1
        assert f(r, ld=63) == -1 and f(r, logits=0) == -1 and f(r, logits=P16 + 1) == -1 and f(r, ids=0) == -1
        assert f(r, ids=P16 + 2) == -1 and f(r, dt=0, logits=P16 + 2) == -1
        assert f(r, rows=1 << 30) == -2 and f(router(n_experts=4096), rows=1 << 24, ld=4096) == -2
    assert _route(r, w=0) == -1 and _route(r, w=P16 + 2) == -1 and _route(r, bias=P16 + 1) == -1
    assert _route_back(r, dw=0) == -1 and _route_back(r, dl=0) == -1 and _route_back(r, dw=P16 + 2) == -1
    assert _route_back(r, dl=P16 + 1) == -1
    assert _route(r, rows=0, logits=0, ids=0, w=0) == 0 and _route_back(r, rows=0, logits=0, ids=0, dw=0, dl=0) == 0


def _combine(Y=P16, dt=1, tokens=4, k=2, d=64, ids=P16, n=0, w=P16, add=P16, out=P16):
    return _lib.lib().mlora_combine(V(Y), dt, tokens, k, d, V(ids), n, V(w), V(add), V(out), None)


def _combine_back(dout=P16, Y=P16, dt=1, tokens=4, k=2, d=64, ids=P16, n=0, w=P16, dY=P16, dw=P16):
    return _lib.lib().mlora_combine_backward(V(dout), V(Y), dt, tokens, k, d, V(ids), n, V(w), V(dY), V(dw), None)


def test_malformed_combines():
    for f in (_combine, _combine_back):
        for bad in (dict(dt=3), dict(k=0), dict(k=65), dict(tokens=-1), dict(tokens=1 << 30), dict(d=0), dict(d=-8),
                    dict(d=12), dict(dt=0, d=6), dict(n=-1), dict(Y=P16 + 8), dict(ids=P16 + 1), dict(w=P16 + 2)):
            assert f(**bad) == -1, bad
        assert f(d=(1 << 20) + 8) == -2 and f(tokens=1 << 24, k=1, d=4096) == -2
        assert f(tokens=0) == 0
    assert _combine(Y=0) == -1 and _combine(out=0) == -1 and _combine(add=P16 + 4) == -1 and _combine(out=P16 + 4) == -1
    assert _combine_back(dout=0) == -1 and _combine_back(Y=0) == -1 and _combine_back(dout=P16 + 4) == -1
    assert _combine_back(dY=P16 + 4) == -1 and _combine_back(dw=P16 + 2) == -1
    assert _combine_back(dY=0, dw=0, dout=0, Y=0) == 0                     # nothing asked for


# ---- refusals of the binding ----

def test_binding_refusals():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="score"):
        b.Router(8, 2, score="tanh")
    with pytest.raises(ValueError, match="group_score"):
        b.Router(8, 2, group_score="mean")
    with pytest.raises(_lib.MloraError, match="top_k"):
        b.Router(8, 9)
    with pytest.raises(_lib.MloraError, match="divide"):
        b.Router(8, 2, expert_groups=3)
    r = b.Router(8, 2)
    z = torch.zeros
    with pytest.raises(ValueError, match="device"):
        r.route(z(3, 8))
    with pytest.raises(ValueError, match="2-d"):
        r.route(z(3, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="device"):
        r.backward(z(3, 8), z(3, 2, dtype=torch.int32), z(3, 2))
    with pytest.raises(ValueError, match="multiple of top_k"):
        b.mlora_combine(z(7, 8), 2)
    with pytest.raises(ValueError, match="device"):
        b.mlora_combine(z(8, 8), 2)
    with pytest.raises(ValueError, match="2-d"):
        b.mlora_combine(z(8, 8, dtype=torch.float64), 2)
    with pytest.raises(ValueError, match="dweights needs Y"):
        b.mlora_combine_backward(z(4, 8), None, 2, weights=z(4, 2))
    with pytest.raises(ValueError, match="device"):
        b.mlora_combine_backward(z(4, 8), z(8, 8), 2)
