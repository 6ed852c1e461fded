"""MXFP4 blocks at the ends of the scale codes' range, and blocks that are not
finite, through the products.

Every scale code whose six largest-element values are finite in bf16 (0 to 252;
the quantizer writes no other but 255) is one output column of the weight, or
one row of the activations.  The other operand is scaled by a power of two that
keeps the products in fp32's normal range, so the bounds are those of
tests/test_gpu_experts.py."""
import numpy as np
import pytest

from oracle import experts as ox
from tests.gpu_harness import say
from tests.test_gpu_experts import check

pytestmark = pytest.mark.gpu

DI = 256
ENDS = {"low": (np.arange(0, 64), 60), "high": (np.arange(189, 253), -60)}     # codes, exponent of the other operand


def weight(codes_of_scale, experts, do, rng):
    """A packed weight whose column j has scale codes_of_scale[j], and its values."""
    import torch
    codes = rng.integers(0, 16, size=(experts * do, DI), dtype=np.uint8)
    scales = np.tile(np.repeat(codes_of_scale.astype(np.uint8)[:, None], DI // 32, axis=1), (experts, 1))
    return (torch.from_numpy(ox.pack(codes, scales)).cuda(),
            ox.decode(codes, scales).reshape(experts, do, DI).transpose(0, 2, 1))


def per_column(got, want, S, K):
    """Columns differ by up to 2^63 in size: each is scaled to itself first (exact)."""
    up = np.exp2(-np.floor(np.log2(S.max(axis=0))))
    check(got * up, want * up, S * up, K, "bf16")


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("end", list(ENDS))
# one tile form each: 16, 32 few-row; 64, 128, 256 rows a tile
@pytest.mark.parametrize("rows,experts,wide", [(1, 1, 1), (40, 3, 2), (150, 3, 4), (600, 2, 8), (3000, 2, 8),
                                               (16384, 1, 16)])
def test_weight_scales(rows, experts, wide, end, act):
    import torch
    from adapter_lora_segments_amd import ExpertLinear
    say(f"scales {end} {rows} rows {experts} experts {act}")
    codes, shift = ENDS[end]
    do = 64 * wide
    rng = np.random.default_rng(rows + wide)
    W, Wm = weight(np.tile(codes, wide), experts, do, rng)
    X = torch.from_numpy(rng.standard_normal((rows, DI)).astype(np.float32)).cuda().to(torch.bfloat16) * 2.0 ** shift
    cut = np.linspace(0, rows, experts + 1).astype(np.int32)
    Y = ExpertLinear(W, experts, DI, do, rows, w_layout="nk", w_format="mxfp4", act_format=act).forward(
        X, torch.from_numpy(cut).cuda())
    Xh = X.double().cpu().numpy()
    Xh = Xh if act == "bf16" else ox.decode(*ox.quantize(Xh))
    want, S, _ = ox.forward(Xh, Wm, cut, None, rows)
    per_column(Y.double().cpu().numpy(), want, S, DI)


@pytest.mark.parametrize("end", list(ENDS))
@pytest.mark.parametrize("rows", [3, 150, 700])
def test_dx_scales(rows, end):
    """dX sums over the columns: one scale code for a whole weight at a time."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear
    codes, shift = ENDS[end]
    do, at = 72, codes[::9]
    say(f"dX scales {end} {rows}")
    rng = np.random.default_rng(rows)
    n = at.shape[0]
    W, Wm = weight(np.zeros(do, dtype=np.int64), n, do, rng)
    one = DI * do // 2
    W[n * one:] = torch.from_numpy(np.repeat(at.astype(np.uint8), do * DI // 32)).cuda()
    Wm = Wm * np.exp2(at.astype(np.float64))[:, None, None]
    dY = torch.from_numpy(rng.standard_normal((n * rows, do)).astype(np.float32)).cuda().to(torch.bfloat16) * 2.0 ** shift
    cut = (rows * np.arange(n + 1)).astype(np.int32)
    L = ExpertLinear(W, n, DI, do, n * rows, w_layout="nk", w_format="mxfp4")
    dX = L.backward(dY, None, torch.from_numpy(cut).cuda()).double().cpu().numpy()
    want, SX, _, _, _ = ox.backward(dY.double().cpu().numpy(), None, Wm, cut, None, n * rows)
    for e in range(n):
        r = slice(cut[e], cut[e + 1])
        up = 2.0 ** -np.floor(np.log2(SX[r].max()))
        check(dX[r] * up, want[r] * up, SX[r] * up, do, "bf16", f"scale code {at[e]}")


@pytest.mark.parametrize("end", list(ENDS))
@pytest.mark.parametrize("rows", [64, 128, 640])
def test_activation_scales(rows, end):
    """Activations whose own blocks quantize to every code of either end."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear
    codes, shift = ENDS[end]
    say(f"activation scales {end} {rows}")
    rng = np.random.default_rng(rows)
    x = rng.choice([1.0, -1.5, 0.5, 3.0, -6.0, 4.0, 0.0], size=(rows, DI))
    x[:, ::32] = 6.0                                                  # every block's maximum: its scale is the row's
    ex = np.tile(codes, rows // 64).astype(np.float64) - 127
    X = torch.from_numpy(np.ldexp(x, ex[:, None].astype(np.int64)).astype(np.float32)).cuda().to(torch.bfloat16)
    Xh = X.double().cpu().numpy()
    c, s = ox.quantize(Xh)
    assert np.array_equal(s[:, 0], np.tile(codes, rows // 64)) and np.array_equal(ox.decode(c, s), Xh)
    do = 136
    W, Wm = weight(np.full(do, 127 + shift), 1, do, rng)
    Y = ExpertLinear(W, 1, DI, do, rows, w_layout="nk", w_format="mxfp4", act_format="mxfp4").forward(X)
    want, S, _ = ox.forward(Xh, Wm, np.array([0, rows]), None, rows)
    up = np.exp2(-np.floor(np.log2(S.max(axis=1))))[:, None]
    check(Y.double().cpu().numpy() * up, want * up, S * up, DI, "bf16")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows", [5, 40, 200, 900])
def test_rows_that_are_not_finite(rows, bad):
    """Quantized activations: a row with a NaN or an infinity has a NaN result,
    the rows beside it what they have without it, bit for bit."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear
    say(f"not finite {rows} {bad}")
    rng = np.random.default_rng(rows)
    do = 264
    W, _ = weight(np.full(do, 120), 1, do, rng)
    X = torch.from_numpy(rng.standard_normal((rows, DI)).astype(np.float32)).cuda().to(torch.bfloat16)
    L = ExpertLinear(W, 1, DI, do, rows, w_layout="nk", w_format="mxfp4", act_format="mxfp4")
    Y = L.forward(X)
    at = rows // 2
    X[at, 77] = bad
    got = L.forward(X)
    rest = torch.arange(rows, device="cuda") != at
    assert torch.isnan(got[at]).all() and torch.equal(got[rest], Y[rest]) and not torch.isnan(Y).any()
