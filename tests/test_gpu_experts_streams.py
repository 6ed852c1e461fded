"""Grouped expert products and the MXFP4 quantizer with an explicit stream and
outputs of their own making, while earlier work still runs on the current
stream: the sequential results bit for bit, and nothing that the current stream
still reads is overwritten."""
import numpy as np
import pytest

from tests.gpu_harness import say
from tests.test_gpu_experts import Case

pytestmark = pytest.mark.gpu

SPIN = 100_000_000        # clock cycles: tens of milliseconds on the current stream


@pytest.mark.parametrize("form", ["bf16", "fp32", "mxfp4"])
@pytest.mark.parametrize("order", [False, True])
def test_outputs_made_on_a_given_stream(order, form):
    import torch
    say(f"given stream {form} {order}")
    w4 = form == "mxfp4"
    c = Case([100, 0, 260], 256, 264, dt="fp32" if form == "fp32" else "bf16", layout="nk", x_order=order,
             y_order=order, dropped=24, w4=w4)
    opts = dict(w_format="mxfp4", act_format="mxfp4") if w4 else {}
    seq, L = c.layer(**opts), c.layer(**opts)
    n = c.rows if order else int(c.off[-1])           # rows that a call writes or zeroes
    Y = seq.forward(c.X, c.d_off, c.d_order)
    dX = seq.backward(c.dY, None if w4 else c.X, c.d_off, c.d_order)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    y = L.forward(c.X, c.d_off, c.d_order, stream=s)
    dx = L.backward(c.dY, None if w4 else c.X, c.d_off, c.d_order, stream=s)
    torch.cuda.synchronize()                          # what was queued on the current stream ends too
    assert torch.equal(y[:n], Y[:n]) and torch.equal(dx[:n], dX[:n])
    if not w4:
        assert torch.equal(L.dW, seq.dW)


def test_outputs_do_not_take_memory_still_in_use():
    """Blocks freed to the current stream, which has yet to read them, are not
    what a call on another stream writes to."""
    import torch
    from adapter_lora_segments_amd import mlora_microscale_quantize
    c = Case([300], 256, 264, layout="nk")
    L = c.layer()
    wide = torch.randn(c.rows, 512, device="cuda").to(torch.bfloat16)
    q0 = mlora_microscale_quantize(wide)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls = {"Y": ((c.rows, 264), torch.bfloat16, lambda: L.forward(c.X, stream=s)),
             "dX": ((c.rows, 256), torch.bfloat16, lambda: L.backward(c.dY, None, want_dw=False, stream=s)),
             "dW": ((1, 264, 256), torch.float32, lambda: L.backward(c.dY, c.X, want_dx=False, stream=s)),
             "q": ((q0.numel(),), torch.uint8, lambda: mlora_microscale_quantize(wide, stream=s))}
    for name, (shape, dt, call) in calls.items():
        say(f"memory in use: {name}")
        held = torch.full(shape, 7, dtype=dt, device="cuda")
        out = torch.empty_like(held)
        torch.cuda.synchronize()
        torch.cuda._sleep(SPIN)
        out.copy_(held)
        del held
        call()
        torch.cuda.synchronize()
        assert (out == 7).all(), name


def test_outputs_freed_while_read_are_not_reused():
    """An output of a call on another stream that the current stream still has to
    read when it is freed: the next call there makes its own elsewhere."""
    import torch
    c = Case([300], 256, 264, layout="nk")
    L = c.layer()
    want = L.forward(c.X)
    other = (c.X * 0.5).contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(3):
        y = L.forward(c.X, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        out = torch.empty_like(want)
        torch.cuda._sleep(SPIN)
        out.copy_(y)
        del y
        L.forward(other, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
