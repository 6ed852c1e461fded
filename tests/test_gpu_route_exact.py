"""Routing where 64-bit sums decide: gradients that nearly cancel, sums that do not
depend on how many lanes a row takes, scores far below 1.  Tolerances count the
roundings of test_gpu_route.py."""
import numpy as np
import pytest

from oracle import route as orc
from tests.gpu_harness import say
from tests.test_gpu_route import HALF, _t, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [9, 1100])
@pytest.mark.parametrize("E,k", [(8, 1), (64, 2), (256, 8)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_dense_gradient_of_saturated_rows(E, k, rows, dt):
    """One expert far above the others: du - sum du u cancels to 1 - s of itself, so
    du enters the difference unrounded (an expert named once: dweights, in fp32, times
    the scale in 64 bits).  Half a step of the result's type, 2^-24 of the rounding to
    fp32 before, 2^-47 of the terms that cancel."""
    import torch
    from adapter_lora_segments_amd import Router
    say(f"saturated rows {E} {k} {rows} {dt}")
    g = torch.Generator().manual_seed(E)
    x = torch.randn(rows, E, generator=g)
    at = torch.arange(rows) * 7 % E
    x[torch.arange(rows), at] = 12.0 + torch.arange(rows) % 9
    x = x.to(_t(dt)).cuda()
    r = Router(E, k, renormalize=False, scale=1.3)
    ids, _ = r.route(x)
    assert torch.equal(ids[:, 0].cpu().long(), at)
    dw = torch.randn(rows, k, generator=g).cuda()
    want, _, terms = orc.route_backward(host(x), ids.cpu().numpy(), host(dw), "softmax", False, 1.3)
    bound = (HALF[dt] + 2.0 ** -24) * np.abs(want) + 2.0 ** -47 * terms + 2.0 ** -140
    err = np.abs(host(r.backward(x, ids, dw)) - want)
    assert (err <= bound).all(), (err / bound).max()


# Rows of 64 logits in eighths and a scale 1 + m 2^-23 whose scores lie so near a
# border of fp32 that a sum of the 64 terms in another order rounds to the other side.
NEAR = [(False, 4190641, [
    -13, 19, 10, -11, 8, -12, -17, 0, 11, -5, -9, 3, -8, 6, 28, -5, 8, 3, -2, 12, 11, 3, -3, 21, -24, -17, 15, -8, 0, 20, -8,
    0, 3, 4, 24, 29, -20, -13, 5, -8, 8, -1, 0, -21, 20, -10, 19, 3, 6, -10, 0, 23, 1, -21, -5, -12, -5, -3, -4, 0, 11, 10,
    15, -27]), (False, 6911962, [
    10, 7, 14, 19, -18, 8, -6, -5, -18, -3, 9, -8, 7, 3, -2, 6, 11, -13, 0, 11, -18, -5, 12, -9, -20, -27, 9, 16, -10, -12,
    -13, -25, 0, 6, 16, 2, -5, -4, -8, -11, 31, -11, -8, -5, 23, -1, -22, -9, -8, 10, -22, -11, 17, 10, 3, -1, 11, 16, 23, 4,
    2, 1, 21, -4]), (True, 2010098, [
    5, -8, 8, 23, 12, -11, 6, 7, 14, -5, -9, 5, -2, -17, 16, 1, -2, 9, 10, 11, 7, 19, 11, -17, -7, -4, 5, -13, -15, 16, 8,
    -7, -3, 15, -23, 6, -26, -15, 5, 7, 4, -25, -4, -11, -4, -5, -5, -9, 8, -25, 13, 3, -10, 11, 2, 11, 3, 7, -8, 2, 18, 4,
    -8, -8]), (True, 6250845, [
    -14, 11, -4, -22, -10, 14, -5, 12, 28, 15, -21, 24, -9, -25, 3, 12, -5, -9, 3, -9, 6, -23, -5, -27, -21, -18, 3, 3, -3,
    -7, -7, -20, -6, -4, 1, 13, 9, -3, 14, -23, -2, -7, 6, 17, -11, -2, 10, -8, -10, -19, -23, 6, 1, 6, 14, 18, 14, 12, -6,
    10, -8, -4, -16, -16])]


@pytest.mark.parametrize("case", range(len(NEAR)))
def test_sums_do_not_depend_on_lanes(case):
    """All 64 experts chosen, in a call of 3 rows (64 lanes a row) and of 1100 (8
    lanes): the same bits."""
    import torch
    from adapter_lora_segments_amd import Router
    renorm, m, eighths = NEAR[case]
    x = torch.tensor([eighths], dtype=torch.float32, device="cuda") / 8
    r = Router(64, 64, renormalize=renorm, scale=1 + m * 2.0 ** -23)
    ids, w = r.route(x.expand(3, 64).contiguous())
    i2, w2 = r.route(x.expand(1100, 64).contiguous())
    assert torch.equal(i2, ids[:1].expand(1100, 64)) and torch.equal(w2, w[:1].expand(1100, 64))
    dw = torch.randn(1, 64, device="cuda")
    d = r.backward(x.expand(3, 64).contiguous(), ids, dw.expand(3, 64).contiguous())
    d2 = r.backward(x.expand(1100, 64).contiguous(), i2, dw.expand(1100, 64).contiguous())
    assert torch.equal(d2, d[:1].expand(1100, 64))


@pytest.mark.parametrize("rows", [4, 1100])
@pytest.mark.parametrize("low", [-80.0, -600.0, -699.0])
def test_sigmoid_gradient_of_tiny_sums(low, rows):
    """Renormalised sigmoid scores of e^-699, chosen by a bias (in fp32 they are all
    zero): a score over their sum is of ordinary size, whatever the sum is.  As
    before, with the terms p sum |g| that cancel."""
    import torch
    from adapter_lora_segments_amd import Router
    E, k = 12, 3
    x = torch.full((rows, E), low)
    x[:, 2], x[:, 7] = low + 0.5, low + 0.25
    r = Router(E, k, score="sigmoid", scale=2.5)
    bias = torch.zeros(E)
    bias[2], bias[7], bias[0] = 3, 2, 1
    ids, w = r.route(x.cuda(), bias.cuda())
    assert (ids.cpu() == torch.tensor([2, 7, 0])).all()
    at = [2, 7, 0]
    s = 1 / (1 + np.exp(-host(x)[:, at]))
    p = s / s.sum(axis=1, keepdims=True)
    dw = torch.randn(rows, k, device="cuda") * 1e6
    h = host(dw)
    want, terms = np.zeros((rows, E)), np.zeros((rows, E))
    want[:, at] = 2.5 * p * (1 - s) * (h - (h * p).sum(axis=1, keepdims=True))
    terms[:, at] = 2.5 * p * 2 * np.abs(h).sum(axis=1, keepdims=True)
    err = np.abs(host(r.backward(x.cuda(), ids, dw)) - want)
    assert (err <= 2.0 ** -24 * np.abs(want) + 2.0 ** -47 * terms).all()


@pytest.mark.parametrize("rows", [4, 1100])
@pytest.mark.parametrize("gap", [3.0, 690.0, 720.0, 744.0, 760.0, 1e30])
def test_chosen_scores_far_below_the_largest(gap, rows):
    """A bias that chooses experts whose scores are next to nothing beside the row's
    largest: renormalised weights are the softmax of the chosen logits however far
    down they lie, and the gradient is those weights'."""
    import torch
    from adapter_lora_segments_amd import Router
    E, k = 16, 3
    x = torch.zeros(rows, E)
    d = torch.tensor([0.0, 1.5, -2.0]) if gap < 1e3 else torch.zeros(3)
    x[:, 4:7] = d - gap
    bias = torch.zeros(E)
    bias[4:7] = torch.tensor([4.0, 3.0, 2.0])
    r = Router(E, k, scale=1.5)
    ids, w = r.route(x.cuda(), bias.cuda())
    assert (ids.cpu() == torch.tensor([4, 5, 6])).all()
    p = np.exp(host(x[:, 4:7]) - host(x[:, 4:7]).max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    assert (np.abs(host(w) - 1.5 * p) <= 2.0 ** -24 * 1.5 * p * (1 + 2.0 ** -20)).all()
    dw = torch.randn(rows, k, device="cuda")
    h = host(dw)
    want = np.zeros((rows, E))
    want[:, 4:7] = 1.5 * p * (h - (h * p).sum(axis=1, keepdims=True))
    terms = np.zeros((rows, E))
    terms[:, 4:7] = 1.5 * p * 2 * np.abs(h).sum(axis=1, keepdims=True)
    err = np.abs(host(r.backward(x.cuda(), ids, dw)) - want)
    assert (err <= 2.0 ** -24 * np.abs(want) + 2.0 ** -47 * terms).all()


@pytest.mark.parametrize("rows", [2, 1100])
def test_renormalised_softmax_of_a_row_that_is_not_finite(rows):
    """A NaN or an infinity among the logits makes every weight of the row NaN, chosen
    or not; the gradient is of the chosen logits alone."""
    import torch
    from adapter_lora_segments_amd import Router
    x = torch.zeros(rows, 16)
    x[:, 3] = torch.tensor([float("nan"), float("inf")] * (rows // 2))
    x[rows - 1] = 0.0
    r = Router(16, 3)
    ids, w = r.route(x.cuda())
    assert torch.isnan(w[:-1]).all() and (ids.cpu() == torch.tensor([0, 1, 2])).all()
    assert torch.equal(w[-1], w.new_full((3,), 1 / 3))
    d = r.backward(x.cuda(), ids, torch.tensor([[3.0, 0.0, 0.0]], device="cuda").expand(rows, 3).contiguous())
    want = torch.zeros(16)
    want[:3] = torch.tensor([2 / 3, -1 / 3, -1 / 3])
    assert torch.allclose(d.cpu(), want.expand(rows, 16), rtol=1e-6, atol=0)


@pytest.mark.parametrize("E,k", [(16, 13), (30, 30), (64, 33), (100, 17), (128, 64), (200, 40), (256, 64), (400, 33), (512, 64)])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_more_slots_than_lanes(E, k, renorm, score):
    """Many rows with more chosen experts than a row has lanes, against the oracle and
    against calls of few rows, which have a lane for every slot."""
    import torch
    from adapter_lora_segments_amd import Router
    say(f"more slots than lanes {E} {k} {score} {renorm}")
    rows = 1030
    r = Router(E, k, score=score, renormalize=renorm, scale=1.3)
    for dt in ("bf16", "fp32"):
        g = torch.Generator().manual_seed(E)
        x = torch.randn(rows, E, generator=g)
        x[5, k // 2:] = -np.inf                          # fewer experts than slots
        x = x.to(_t(dt)).cuda()
        ids, w = r.route(x)
        some = [0, 5, 17, 700, rows - 1]
        want, ww = orc.route(host(x)[some], k, score=score, renorm=renorm, scale=1.3)
        assert np.array_equal(ids.cpu().numpy()[some], want)
        assert (np.abs(host(w)[some] - ww) <= 2.0 ** -24 * np.abs(ww) * (1 + 2.0 ** -20) + 2.0 ** -150).all()
        i2, w2 = r.route(x[:1024])
        assert torch.equal(i2, ids[:1024]) and torch.equal(w2, w[:1024])
        dw = torch.randn(rows, k, generator=g).cuda()
        d = r.backward(x, ids, dw)
        want, _, terms = orc.route_backward(host(x)[some], ids.cpu().numpy()[some], host(dw)[some], score, renorm, 1.3)
        # (up to k + 9 = 73 operations of 2^-53 on either side: 2^-45)
        bound = (HALF[dt] + 2.0 ** -24) * np.abs(want) + 2.0 ** -45 * terms + 2.0 ** -140
        assert (np.abs(host(d)[some] - want) <= bound).all()
        assert torch.equal(r.backward(x[:1024], ids[:1024], dw[:1024]), d[:1024])


@pytest.mark.parametrize("rows", [9, 1100])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_sigmoid_gradient_of_saturated_scores(dt, renorm, rows):
    """Logits from 5 to 80, where 1 - s is e^-logit, which a rounded s no longer holds:
    s (1 - s) du with 1 - s = 1 / (1 + e^logit).  Tolerances as above, the terms that
    cancel times 1 - s."""
    import torch
    from adapter_lora_segments_amd import Router
    E, k = 16, 4
    g = torch.Generator().manual_seed(rows)
    x = (torch.rand(rows, E, generator=g) * 75 + 5).to(_t(dt)).cuda()
    r = Router(E, k, score="sigmoid", renormalize=renorm, scale=1.3)
    ids, _ = r.route(x)
    dw = torch.randn(rows, k, generator=g).cuda()
    at, h = ids.cpu().numpy().astype(np.int64), host(dw)
    l = np.take_along_axis(host(x), at, axis=1)
    s, rest = 1 / (1 + np.exp(-l)), 1 / (1 + np.exp(l))
    scale = float(np.float32(1.3))
    p = s / s.sum(axis=1, keepdims=True) if renorm else s
    du = h - (h * p).sum(axis=1, keepdims=True) if renorm else h
    want, terms = np.zeros((rows, E)), np.zeros((rows, E))
    np.put_along_axis(want, at, scale * p * rest * du, axis=1)
    np.put_along_axis(terms, at, scale * p * rest * 2 * np.abs(h).sum(axis=1, keepdims=True), axis=1)
    bound = (HALF[dt] + 2.0 ** -24) * np.abs(want) + 2.0 ** -47 * terms + 2.0 ** -140
    err = np.abs(host(r.backward(x, ids, dw)) - want)
    assert (err <= bound).all(), (err / bound).max()
