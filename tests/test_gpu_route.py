"""Routing and combining on the GPU against the float64 oracle
(oracle/route.py).

Tolerances.  Ids are equal: scores are rounded to fp32 from 64 bits on both
sides, which differ (by at most 2^-50 of a score) for none of these inputs.
Weights are computed in 64 bits and rounded once: half a step, 2^-24 (and half
the smallest denormal).  A router's gradient: half a step of its type plus 2^-24
of the value (a bf16 gradient is rounded to fp32 before) plus 2^-24 of s |du|, du
being kept in fp32, plus 2^-47 of the terms that cancel (kernel and oracle each
take at most k + 9 = 15 operations of 2^-53 of them: 30 2^-53 < 2^-48).  Combining: as the grouped products, a sum of n products off
by at most (n + 2) 2^-23 of the sum of magnitudes, and half a step at the end."""
import numpy as np
import pytest

from oracle import route as orc
from tests.gpu_harness import say

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
NEG = -np.inf


def _t(dt):
    import torch
    return torch.bfloat16 if dt == "bf16" else torch.float32


def host(t):
    return t.detach().double().cpu().numpy()


def logits_of(T, E, dt, seed=0, masked=0.0, std=1.5):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * std
    if masked:
        x[torch.rand(T, E, generator=g) < masked] = NEG
    return x.to(_t(dt)).cuda()


def same_weights(got, want):
    bound = 2.0 ** -24 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -150
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    assert (np.abs(got - want)[~nan] <= bound[~nan]).all(), np.abs(got - want)[~nan].max()


def check_route(x, k, bias=None, **kw):
    from adapter_lora_segments_amd import Router
    opts = dict(score=kw.get("score", "softmax"), expert_groups=kw.get("groups", 1), top_groups=kw.get("top_groups", 1),
                group_score=kw.get("group_score", "max"), renormalize=kw.get("renorm", True), scale=kw.get("scale", 1.0))
    r = Router(x.shape[1], k, **opts)
    ids, w = r.route(x, bias)
    want, ww = orc.route(host(x), k, bias=None if bias is None else bias.cpu().numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), want)
    same_weights(host(w), ww)
    return r, ids, w


@pytest.mark.parametrize("E", [1, 2, 7, 8, 9, 16, 33, 64, 100, 128, 250, 256, 400, 512, 777, 1024, 2000, 4096])
@pytest.mark.parametrize("T", [1, 5, 67])
def test_route(E, T):
    say(f"route {T} x {E}")
    import torch
    for n, (dt, score) in enumerate((d, s) for d in ("bf16", "fp32") for s in ("softmax", "sigmoid")):
        k = min(E, (1, 2, 8, 64)[(n + T) % 4])
        bias = torch.randn(E, device="cuda") * 0.1 if n % 2 else None
        check_route(logits_of(T, E, dt, seed=E + n), k, bias, score=score, renorm=n != 2, scale=(1.0, 2.5)[n % 2])


@pytest.mark.parametrize("E,G,tg", [(8, 8, 3), (16, 4, 2), (60, 5, 2), (64, 8, 4), (256, 8, 4), (256, 64, 7), (320, 5, 1),
                                    (1024, 16, 3), (4096, 64, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(E, G, tg, score):
    import torch
    say(f"route groups {E} {G} {tg} {score}")
    for gs in ("max", "top2"):
        for masked in (0.0, 0.5):
            bias = torch.randn(E, device="cuda") * 0.2
            check_route(logits_of(37, E, "bf16" if gs == "max" else "fp32", seed=E, masked=masked),
                        min(8, E // G * tg), bias, score=score, groups=G, top_groups=tg, group_score=gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [6, 64, 300, 4096])
def test_route_ties_and_masks(E, score):
    """Few different logits (ties everywhere), rows with little or nothing
    left, the type's lowest value, NaN and infinities."""
    import torch
    say(f"route ties {E} {score}")
    rng = np.random.default_rng(E)
    x = torch.from_numpy(rng.integers(-2, 3, size=(40, E)).astype(np.float32))
    x[1] = 0
    x[2] = NEG
    x[3, 1:] = NEG
    x[4] = torch.finfo(torch.bfloat16).min
    x[5, ::2] = torch.finfo(torch.bfloat16).min
    x[6, 3] = np.nan
    x[7, 2] = np.inf
    x[8] = 1000
    x[9] = -1000
    x[10, ::3] = 90
    x[11, 1::2] = NEG
    x[12, 2:] = np.nan
    for dt in ("bf16", "fp32"):
        for renorm in (True, False):
            check_route(x.to(_t(dt)).cuda(), min(4, E), score=score, renorm=renorm)
    bias = torch.zeros(E)
    bias[0], bias[1], bias[2] = NEG, np.inf, np.nan
    check_route(x[:2].cuda(), min(4, E), bias.cuda(), score=score)


def test_route_all_groups_equal():
    import torch
    check_route(torch.zeros(3, 64, device="cuda"), 8, groups=8, top_groups=3, group_score="top2")
    x = torch.full((2, 64), NEG, device="cuda")
    x[1, 40] = 1.0
    check_route(x, 8, groups=8, top_groups=3, group_score="top2")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_route_strided(dt):
    """Rows with a stride, starting at any element."""
    x = logits_of(50, 90, dt, seed=1)
    for lo in (0, 1, 3):
        v = x[:, lo:lo + 64]
        r, ids, w = check_route(v, 4)
        d2 = r.backward(v, ids, w)
        d1 = r.backward(v.contiguous(), ids, w)
        import torch
        assert torch.equal(d1, d2)
    check_route(x[::7, :64], 4)
    check_route(x[:1, 5:69], 4)
    check_route(x[:0, 5:69], 4)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [2, 9, 64, 100, 256, 512, 1000, 2048, 4095])
def test_route_backward(E, renorm, score, dt):
    import torch
    from adapter_lora_segments_amd import Router
    say(f"route backward {E} {score} {dt} {renorm}")
    T, k = 33, min(E, 6)
    x = logits_of(T, E, dt, seed=E, masked=0.2)
    x[3] = NEG
    r = Router(E, k, score=score, renormalize=renorm, scale=1.5)
    ids, _ = r.route(x)
    ids[5, -1] = -1                          # dropped slots, ids of no expert, an expert named twice and oftener
    ids[6, 0] = E
    ids[7] = -2 ** 31
    ids[8, 1:] = ids[8, 0]
    ids[9, 1] = ids[9, 0]
    dw = torch.randn(T, k, device="cuda")
    dw[5, -1] = np.nan                       # (no part in anything)
    got = r.backward(x, ids, dw)
    h = np.where(np.isnan(host(dw)), 0.0, host(dw))
    want, mag, terms = orc.route_backward(host(x), ids.cpu().numpy(), h, score, renorm, 1.5)
    bound = (HALF[dt] + 2.0 ** -24) * np.abs(want) + 2.0 ** -24 * mag * (1 + 2.0 ** -8) + 2.0 ** -47 * terms + 2.0 ** -140
    err = np.abs(host(got) - want)
    assert (err <= bound).all(), (err / bound).max()
    assert torch.equal(r.backward(x, ids, dw), got)                      # repeatable
    y = x.clone()
    assert torch.equal(r.backward(y, ids, dw, dlogits=y), got)           # in place


def test_route_backward_not_finite():
    import torch
    from adapter_lora_segments_amd import Router
    x = torch.zeros(2, 8, device="cuda")
    x[0, 3], x[0, 5] = np.nan, NEG
    r = Router(8, 2, renormalize=False)
    ids, w = r.route(x)
    g = r.backward(x, ids, torch.ones_like(w))
    assert torch.isnan(g[0, :5]).all() and g[0, 5] == 0 and not torch.isnan(g[1]).any()


def test_route_past_32_bit_offsets():
    import torch
    from adapter_lora_segments_amd import Router
    say("route 600000 x 4096 bf16")
    T, E = 600_000, 4096
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    tail = logits_of(40, E, "bf16", seed=3)
    x[-40:] = tail
    r = Router(E, 8)
    ids, w = r.route(x)
    i2, w2 = r.route(tail)
    assert torch.equal(ids[-40:], i2) and torch.equal(w[-40:], w2) and (ids[:-40] == torch.arange(8, device="cuda")).all()
    d = r.backward(x, ids, w)
    assert torch.equal(d[-40:], r.backward(tail, i2, w2))


# ---- combining ----

def _combine_case(T, k, d, dt, ids, weights, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    Y = torch.randn(T * k, d, generator=g).to(_t(dt)).cuda()
    w = torch.randn(T, k, generator=g).cuda() if weights else None
    i = torch.randint(-1, 5, (T, k), generator=g, dtype=torch.int32).cuda() if ids else None
    if ids and T > 1:
        i[1] = -1                                        # a token of no expert
    if ids:
        Y[(i < 0).reshape(-1)] = np.nan                  # rows of dropped slots hold anything
    return Y, i, w


@pytest.mark.parametrize("d", [8, 24, 520, 1024, 2056, 4104, 9000])
@pytest.mark.parametrize("k", [1, 2, 3, 8, 9, 64])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_combine(d, k, dt):
    import torch
    from adapter_lora_segments_amd import mlora_combine, mlora_combine_backward
    say(f"combine {d} {k} {dt}")
    for n, T in enumerate((1, 3, 70)):
        has_ids, has_w, has_add = n != 0, n != 2 or k == 3, n == 2
        Y, ids, w = _combine_case(T, k, d, dt, has_ids, has_w, seed=n)
        add = torch.randn(T, d, device="cuda").to(_t(dt)) if has_add else None
        lim = 4 if n == 2 and has_ids else 0
        hid, hw = (None if t is None else t.cpu().numpy() for t in (ids, w))
        hw = None if hw is None else hw.astype(np.float64)
        out = mlora_combine(Y, k, ids, w, add=add, n_experts=lim)
        want, S = orc.combine(host(Y), k, hid, hw, None if add is None else host(add), lim)
        err = np.abs(host(out) - want)
        assert (err <= HALF[dt] * np.abs(want) + (k + 3) * 2.0 ** -23 * S * (1 + 2.0 ** -8)).all()
        dout = torch.randn(T, d, device="cuda").to(_t(dt))
        dY, dw = mlora_combine_backward(dout, Y, k, ids, w, n_experts=lim, want_dweights=True)
        wy, wd, SD = orc.combine_backward(host(dout), host(Y), k, hid, hw, lim)
        assert (np.abs(host(dY) - wy) <= (HALF[dt] + 2.0 ** -24) * np.abs(wy)).all()
        assert (np.abs(host(dw) - wd) <= 2.0 ** -24 * np.abs(wd) + (d + 2) * 2.0 ** -23 * SD).all()
        only, none = mlora_combine_backward(dout, None, k, ids, w, want_dweights=False, n_experts=lim)
        assert none is None and torch.equal(only, dY)
        none, only = mlora_combine_backward(dout, Y, k, ids, w, want_dy=False, want_dweights=True, n_experts=lim)
        assert none is None and torch.equal(only, dw)


def test_combine_in_place_and_empty():
    import torch
    from adapter_lora_segments_amd import mlora_combine, mlora_combine_backward
    Y, ids, w = _combine_case(50, 4, 264, "bf16", True, True)
    add = torch.randn(50, 264, device="cuda").to(torch.bfloat16)
    want = mlora_combine(Y, 4, ids, w, add=add)
    out = add.clone()
    assert mlora_combine(Y, 4, ids, w, add=out, out=out) is out and torch.equal(out, want)
    e = torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")
    assert mlora_combine(e, 4).shape == (0, 264)
    dY, dw = mlora_combine_backward(e, e, 4, None, torch.empty(0, 4, device="cuda"))
    assert dY.shape == (0, 264) and dw.shape == (0, 4)


def test_combine_sums_a_tokens_gradients():
    """Without weights: what the dX of a product with x_by_order needs."""
    import torch
    from adapter_lora_segments_amd import mlora_combine
    dX = torch.randn(21, 40, device="cuda")
    assert torch.allclose(mlora_combine(dX, 3), dX.reshape(7, 3, 40).sum(1), rtol=1e-6, atol=1e-6)


def test_combine_past_32_bit_offsets():
    import torch
    from adapter_lora_segments_amd import mlora_combine, mlora_combine_backward
    say("combine 300000 x 2 x 4096 bf16")
    T, k, d = 300_000, 2, 4096
    Y = torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda")
    Y[-6:] = torch.randn(6, d, device="cuda").to(torch.bfloat16)
    w = torch.rand(T, k, device="cuda")
    out = mlora_combine(Y, k, None, w)
    assert torch.equal(out[-3:], mlora_combine(Y[-6:], k, None, w[-3:])) and not out[:-3].any()
    dout = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    dout[-3:] = 1.5
    dY, dw = mlora_combine_backward(dout, Y, k, None, w)
    y3, w3 = mlora_combine_backward(dout[-3:], Y[-6:], k, None, w[-3:])
    assert torch.equal(dY[-6:], y3) and torch.equal(dw[-3:], w3) and not dY[:-6].any() and not dw[:-3].any()
