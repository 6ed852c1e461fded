"""Grouped expert products over the most rows that the interface takes."""
import pytest

from tests.gpu_harness import say

pytestmark = pytest.mark.gpu


def test_most_rows():
    """One bf16 expert of 8 x 8 over 2^31 - 257 rows, 34 GB an operand: dW,
    which is summed in 256 chunks, and Y.  A few hundred rows hold small whole
    numbers (the ends of every chunk among them), the others zeros, so every
    sum is exact."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear
    R, d, C = 2 ** 31 - 257, 8, 2 ** 23
    if torch.cuda.mem_get_info()[0] < 3 * 2 * d * R + 2 ** 32:
        pytest.skip("needs 107 GB of free device memory")
    say("most rows: fill")
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randint(-4, 5, (1, d, d), generator=g, device="cuda").to(torch.bfloat16)
    X = torch.zeros(R, d, dtype=torch.bfloat16, device="cuda")
    dY = torch.zeros(R, d, dtype=torch.bfloat16, device="cuda")
    at = sorted({r for k in range(256) for r in (k * C, k * C + 12345, k * C + C - 1) if r < R} | {R - 1})
    x = torch.randint(-4, 5, (len(at), d), generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randint(-4, 5, (len(at), d), generator=g, device="cuda").to(torch.bfloat16)
    for i, r in enumerate(at):
        X[r].copy_(x[i])
        dY[r].copy_(dy[i])
    L = ExpertLinear(W, 1, d, d, R)
    assert L.ws is not None and L.ws.numel() >= 256 * d * d * 4
    torch.cuda.synchronize()
    say("most rows: dW")
    L.backward(dY, X, want_dx=False)
    torch.cuda.synchronize()
    assert torch.equal(L.dW[0].double(), x.double().t().contiguous() @ dy.double())
    del dY
    say("most rows: Y")
    Y = L.forward(X)
    torch.cuda.synchronize()
    want = (x.double() @ W[0].double()).to(torch.bfloat16)          # at most 128: exact
    assert torch.equal(torch.stack([Y[r] for r in at]), want)
    assert not Y[12346:100000].any() and not Y[R - C + 20000:R - 300].any()
    del X, Y
    torch.cuda.empty_cache()
