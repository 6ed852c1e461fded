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
