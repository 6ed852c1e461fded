"""Memory of a frozen 4-bit expert layer: its codes and the forward's
workspace; a dX holds the decoded weight for the call."""
import pytest

from tests.gpu_harness import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_memory_of_a_frozen_layer(act):
    import torch
    from adapter_lora_segments_amd import ExpertLinear, mlora_expert_backward, mlora_microscale_quantize
    say(f"frozen layer {act}")
    E, di, do, rows = 16, 512, 1024, 96
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    W, X, dY = mlora_microscale_quantize(r(E * do, di)), r(rows, di), r(rows, do)
    off = torch.arange(0, rows + 1, rows // E, dtype=torch.int32, device="cuda")
    Y, dX = torch.empty_like(dY), torch.empty_like(X)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    start = torch.cuda.memory_allocated()
    L = ExpertLinear(W, E, di, do, rows, w_layout="nk", w_format="mxfp4", act_format=act)
    for _ in range(2):
        L.forward(X, off, None, Y)
    assert torch.cuda.max_memory_allocated() - start <= rows * di          # X's codes and scales
    for _ in range(2):
        L.backward(dY, None, off, None, dX)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - start <= rows * di
    assert torch.cuda.max_memory_allocated() - start <= rows * di + 2 * E * di * do
    ws = L.shape.alloc_workspace()
    want = mlora_expert_backward(L.shape, dY, None, W, off, None, torch.empty_like(X), None, ws)
    assert torch.equal(dX, want)
