"""Few rows over 4-bit weights, whose codes are multiplied as they are: a group's part
is 16 s (P - (1 + z / 16) Q), P = sum x (1 + c / 16), Q = sum x, in fp32."""
import numpy as np
import pytest

from oracle import affine as oa
from oracle import experts as ox
from tests.gpu_harness import say
from tests.test_gpu_affine import Case, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 3, 8, 16, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_zero_weights(group, rows):
    """Activations of five bits' spread: whole numbers up to 255 2^5, whose sums over
    a group times 16 + 15 stay below 2^24 (128 of mean 2016: 8 10^6; largest drawn sum
    asserted), so that the sums with and without codes are exact and the weights' zero
    stays zero."""
    import torch
    from adapter_lora_segments_amd import AffineLinear
    say(f"zero weights {group} {rows}")
    rng = np.random.default_rng(group + rows)
    di, do = 1024, 200
    zeros = rng.integers(0, 16, size=(do, di // group)).astype(np.float32)
    codes = np.repeat(zeros, group, axis=1).astype(np.uint8)
    scales = oa.bf16(np.exp2(rng.uniform(-9, 0, size=zeros.shape)).astype(np.float32))
    x = rng.choice(np.arange(129, 256, 2), size=(rows, di)) * np.exp2(rng.integers(0, 6, size=(rows, di)))
    assert x.reshape(rows, -1, group).sum(axis=2).max() * 31 < 2 ** 24
    X = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
    assert np.array_equal(X.double().cpu().numpy(), x)
    L = AffineLinear(torch.from_numpy(oa.pack(codes, zeros, scales)).cuda(), 1, di, do, rows, group=group)
    assert not L.forward(X).any()


@pytest.mark.parametrize("rows", [1, 4, 7, 16])
@pytest.mark.parametrize("group,di", [(32, 4096), (64, 1088), (128, 14336)])
def test_sums(group, di, rows):
    """P and Q off by at most G 2^-23 of their sums of magnitudes each, a few roundings
    of 2^-24 more, the K / G parts added in fp32: half a bf16 step and (G + K / G + 16)
    2^-23 of sum |x| 16 |s| (1.94 + |1 + z / 16|), which bounds every partial sum."""
    say(f"affine sums {group} {di} {rows}")
    c = Case([rows], di, 136, group, seed=rows, odd_zero=rows == 7)
    codes, zeros, scales = oa.unpack(c.q.cpu().numpy(), c.do, di, group)
    z, s = (np.repeat(v.astype(np.float64), group, axis=1) for v in (zeros, scales))
    M = (16 * np.abs(s) * (1.94 + np.abs(1 + z / 16))).reshape(1, c.do, di).transpose(0, 2, 1)
    want, _, _ = ox.forward(c.Xh, c.W, c.off, c.order, rows, **c.kw)
    _, B, _ = ox.forward(c.Xh, M, c.off, c.order, rows, **c.kw)
    bound = 2.0 ** -8 * np.abs(want) + (group + di // group + 16) * 2.0 ** -23 * B * (1 + 2.0 ** -8)
    err = np.abs(host(c.layer().forward(c.X)) - want)
    assert (err <= bound).all(), (err / bound).max()
