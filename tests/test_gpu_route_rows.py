"""Routing of many rows, where a row has fewer lanes than a wave (from 1025 rows
on, other kernels than those of a few), and choices between scores plus biases of
any sign and size.  Oracle and tolerances as in test_gpu_route.py."""
import numpy as np
import pytest

from oracle import route as orc
from tests.gpu_harness import say
from tests.test_gpu_route import HALF, NEG, host, logits_of, same_weights

pytestmark = pytest.mark.gpu


def check(x, k, bias=None, **kw):
    """Of many rows every eleventh, the last and the first few against the oracle."""
    from adapter_lora_segments_amd import Router
    r = Router(x.shape[1], k, score=kw.get("score", "softmax"), expert_groups=kw.get("groups", 1),
               top_groups=kw.get("top_groups", 1), group_score=kw.get("group_score", "max"),
               renormalize=kw.get("renorm", True), scale=kw.get("scale", 1.0))
    ids, w = r.route(x, bias)
    T = x.shape[0]
    rows = sorted({*range(min(T, 9)), *range(0, T, 11), T // 2, T // 3, T // 4, T - 1})
    want, ww = orc.route(host(x)[rows], k, bias=None if bias is None else bias.cpu().numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy()[rows], want)
    same_weights(host(w)[rows], ww)
    return r, ids, w


@pytest.mark.parametrize("E", [1, 5, 8, 13, 16, 31, 32, 40, 60, 64, 97, 128, 160, 192, 200, 256, 384, 500, 512])
def test_many_rows(E):
    import torch
    say(f"route many rows {E}")
    for n, (dt, score) in enumerate((d, s) for d in ("bf16", "fp32") for s in ("softmax", "sigmoid")):
        k = min(E, (2, 8, 6, 11)[n])
        bias = torch.randn(E, device="cuda") * 0.1 if n % 2 else None
        r, ids, w = check(logits_of(1031, E, dt, seed=E + n, masked=0.1), k, bias, score=score, renorm=n != 2)
        # any number of rows: the same bits
        x = logits_of(1031, E, dt, seed=E + n, masked=0.1)
        i2, w2 = r.route(x[:1024], bias)
        assert torch.equal(i2, ids[:1024]) and torch.equal(w2, w[:1024])


@pytest.mark.parametrize("E,G,tg", [(8, 4, 2), (12, 3, 1), (24, 8, 4), (60, 5, 2), (64, 8, 4), (64, 32, 5), (128, 8, 3),
                                    (256, 8, 4), (256, 64, 9), (480, 6, 2), (512, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_rows_in_groups(E, G, tg, score):
    import torch
    say(f"route many rows in groups {E} {G} {tg} {score}")
    for gs in ("max", "top2"):
        check(logits_of(1025, E, "fp32", seed=E, masked=0.3), min(8, E // G * tg),
                    torch.randn(E, device="cuda") * 0.2, score=score, groups=G, top_groups=tg, group_score=gs)


@pytest.mark.parametrize("E", [8, 30, 48, 64, 128, 192, 256, 384, 512])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_rows_backward(E, renorm, score):
    import torch
    from adapter_lora_segments_amd import Router
    say(f"route backward many rows {E} {score} {renorm}")
    T, k = 1033, min(E, 6)
    for dt in ("bf16", "fp32"):
        x = logits_of(T, E, dt, seed=E, masked=0.1)
        r = Router(E, k, score=score, renormalize=renorm, scale=1.5)
        ids, _ = r.route(x)
        dw = torch.randn(T, k, device="cuda")
        want, mag, terms = orc.route_backward(host(x), ids.cpu().numpy(), host(dw), score=score, renorm=renorm, scale=1.5)
        got = host(r.backward(x, ids, dw))
        bound = (HALF[dt] + 2.0 ** -24) * np.abs(want) + 2.0 ** -24 * mag * (1 + 2.0 ** -8) + 2.0 ** -47 * terms + 2.0 ** -140
        assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("rows", [7, 1040])
@pytest.mark.parametrize("E", [6, 16, 60, 128, 256, 400, 1000])
def test_biases_of_any_size(E, rows):
    """Scores plus biases that are negative, tie, pass fp32's ends or are not
    numbers: the order of fp32 sums, infinity above the largest number, NaN first."""
    import torch
    say(f"route biases {E} {rows}")
    rng = np.random.default_rng(E)
    top = float(np.finfo(np.float32).max)
    specials = [-0.0, 0.0, -1.0, -1.0, 1.0, -0.5, top, -top, np.inf, NEG, np.nan, 1e-40, -1e-40, 3e-39, -2.0 ** 20]
    x = torch.from_numpy(rng.integers(-1, 2, size=(rows, E)).astype(np.float32) * 40).cuda()
    x[rows // 2] = NEG
    x[rows // 3, ::2] = NEG
    x[rows // 4, 1] = np.nan
    for n in range(3):
        bias = torch.from_numpy(rng.choice(specials[:8 + 4 * n - (n == 2)], size=E).astype(np.float32)).cuda()
        for score in ("softmax", "sigmoid"):
            for k in sorted({1, min(E, 6), min(E, 20)}):
                check(x, k, bias, score=score, renorm=False)
                if E % 4 == 0:
                    check(x, min(k, E // 2), bias, score=score, groups=4, top_groups=2, group_score="top2",
                                renorm=False)
                    check(x, min(k, E // 2), bias, score=score, groups=4, top_groups=2, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_of_any_size(score):
    """Logits to both ends of fp32, with scores that leave its range."""
    import torch
    for T in (50, 1100):
        g = torch.Generator().manual_seed(T)
        x = torch.randn(T, 64, generator=g) * torch.exp2(torch.randint(-30, 8, (T, 1), generator=g).float())
        x[3] *= 1e36
        x[4] -= 500
        x[5] += 500
        x[6, :60] = -200
        check(x.cuda(), 6, score=score, renorm=False)


@pytest.mark.parametrize("k,d", [(1, 64), (3, 1032), (8, 4104)])
def test_combine_backward_in_place(k, d):
    """dY over Y, and the same bits for any number of tokens."""
    import torch
    from adapter_lora_segments_amd import mlora_combine_backward
    Y = torch.randn(300 * k, d, device="cuda").to(torch.bfloat16)
    dout, w = torch.randn(300, d, device="cuda").to(torch.bfloat16), torch.rand(300, k, device="cuda")
    ids = torch.randint(-1, 9, (300, k), device="cuda", dtype=torch.int32)
    dY, dw = mlora_combine_backward(dout, Y, k, ids, w)
    y2, w2 = mlora_combine_backward(dout[:5], Y[:5 * k], k, ids[:5], w[:5])
    assert torch.equal(y2, dY[:5 * k]) and torch.equal(w2, dw[:5])
    same, w3 = mlora_combine_backward(dout, Y, k, ids, w, dY=Y)
    assert same is Y and torch.equal(Y, dY) and torch.equal(w3, dw)


def test_combine_backward_of_more_slots_than_a_launch_has_waves():
    import torch
    from adapter_lora_segments_amd import mlora_combine_backward
    T, k, d = (1 << 20) + 3, 64, 264
    say(f"combine backward {T} x {k} x {d}")
    dout = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    dY, none = mlora_combine_backward(dout, None, k)
    assert none is None
    for lo in (0, T // 2, T - 4):
        assert torch.equal(dY.view(T, k, d)[lo:lo + 4], dout[lo:lo + 4, None].expand(4, k, d))
    assert torch.equal(dY.view(T, k, d)[:, 63], dout)
