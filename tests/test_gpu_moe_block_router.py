"""The last step of a mixture-of-experts block's way back: the router's gradient, from
the weights' gradients that the block itself made, against float64."""
import numpy as np
import pytest

from oracle import route as orc
from tests.gpu_harness import say
from tests.test_gpu_moe_block import KINDS, Block, n64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 5, 300, 1100])
def test_block_router_gradient(T, dt, kind):
    """Half a step of the logits' type, 2^-24 of the rounding to fp32 before, 2^-47 of
    the terms that cancel in 64 bits."""
    import torch
    say(f"moe block router {T} {dt} {kind}")
    opts = KINDS[kind]
    b = Block(T, 16, 4, 128, 320, **opts)
    ins = b.inputs(torch.bfloat16 if dt == "bf16" else torch.float32)
    r = b.step(*ins)
    want, _, terms = orc.route_backward(n64(ins[1]), r["ids"].cpu().numpy(), n64(r["dw"]), opts["score"],
                                        opts.get("renormalize", True), opts.get("scale", 1.0))
    half = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    bound = (half + 2.0 ** -24) * np.abs(want) + 2.0 ** -47 * terms + 2.0 ** -140
    assert r["dl"].dtype == ins[1].dtype
    assert (np.abs(n64(r["dl"]) - want) <= bound).all()
