"""Tensors that a call makes for itself (outputs not given, the first dW, the
quantizer's buffer) are made on the stream that the call's kernels run on, so
neither their fill nor the last use of their memory can meet the kernels.
Shown without a GPU: torch's makers are watched and no kernel is launched."""
import contextlib

import pytest

from adapter_lora_segments_amd import binding as b

torch = pytest.importorskip("torch")


@pytest.fixture
def made(monkeypatch):
    """[(maker, stream it ran on)] of the torch.zeros and torch.empty calls."""
    seen, at = [], [None]

    @contextlib.contextmanager
    def stream(s):
        was, at[0] = at[0], s
        yield
        at[0] = was

    def watch(name):
        make = getattr(torch, name)

        def run(*a, **k):
            seen.append((name, at[0]))
            return make(*a, **k)
        monkeypatch.setattr(torch, name, run)

    stream.at = lambda: at[0]
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: ("current", at[0]))
    # (only what was made on another stream is recorded, with the caller's)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append(("record", s)))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    watch("zeros")
    watch("empty")
    return seen


def layer(**opts):
    L = b.ExpertLinear.__new__(b.ExpertLinear)
    L.shape = b.ExpertShape(8, 2, 64, 64, **opts)
    L.W, L.ws, L.dW = torch.ones(2, 64, 64, dtype=torch.bfloat16), None, None
    return L


@pytest.mark.parametrize("given", [None, "side"])
@pytest.mark.parametrize("order", [False, True])
def test_outputs_are_made_on_the_calls_stream(made, monkeypatch, order, given):
    calls = []
    monkeypatch.setattr(b, "mlora_expert_forward", lambda *a: calls.append(a[-1]))
    monkeypatch.setattr(b, "mlora_expert_backward", lambda *a: calls.append(a[-1]))
    L = layer(x_order=order, y_order=order)
    x = torch.ones(8, 64, dtype=torch.bfloat16)
    del made[:]
    L.forward(x, stream=given)
    L.backward(x, x, stream=given)
    fill = "zeros" if order else "empty"
    assert calls == [given, given]
    kept = [("record", ("current", None))] if given else []
    assert made == [(fill, given)] + kept + [(fill, given)] + kept + [("empty", given)] + kept


@pytest.mark.parametrize("given", [None, "side"])
def test_quantizer_buffer_is_made_on_the_calls_stream(made, monkeypatch, given):
    class Matrix:
        dtype, is_cuda, shape, device = torch.bfloat16, True, (4, 64), torch.device("cpu")
        dim = staticmethod(lambda: 2)
        stride = staticmethod(lambda i: (64, 1)[i])
        data_ptr = staticmethod(lambda: 0)

    monkeypatch.setattr(b, "_need", lambda *a: None)
    monkeypatch.setattr(b, "_one_device", lambda *a: 0)
    monkeypatch.setattr(b, "_raw_stream", lambda *a: 0)
    monkeypatch.setattr(b, "_launch", lambda *a: None)
    b.mlora_microscale_quantize(Matrix(), stream=given)
    assert made == [("empty", given)] + ([("record", ("current", None))] if given else [])


@pytest.mark.parametrize("given", [None, "side"])
def test_packed_layer_outputs_are_made_on_the_calls_stream(made, monkeypatch, given):
    monkeypatch.setattr(b, "mlora_forward", lambda *a: None)
    monkeypatch.setattr(b, "mlora_backward", lambda *a: None)
    L = b.PackedLoRALinear.__new__(b.PackedLoRALinear)
    L.plan = type("Plan", (), dict(info=dict(T=8, d_in=64, d_out=64)))
    L.W0 = L.A_ptrs = L.B_ptrs = L.scales = L.Z = L.ws = L.dA_ptrs = L.dB_ptrs = None
    x = torch.ones(8, 64, dtype=torch.bfloat16)
    L.forward(x, stream=given)
    L.backward(x, x, stream=given)
    assert [m for m in made if m[0] != "record"] == [("empty", given)] * 2
    assert len(made) == (4 if given else 2)


def test_two_layout_base_is_copied_on_the_calls_stream(made, monkeypatch):
    """The copy beside the transpose kernel runs where the buffer is made."""
    at = []
    monkeypatch.setattr(b, "mlora_base_transpose", lambda W, out, stream: at.append(stream))
    copy = torch.Tensor.copy_
    monkeypatch.setattr(torch.Tensor, "copy_", lambda t, o: (made.append(("copy", torch.cuda.stream.at())), copy(t, o))[1])
    buf = b.base_both(torch.arange(64 * 64, dtype=torch.float32).view(64, 64), "side")
    assert buf.numel() == 2 * 64 * 64 and at == ["side"]
    assert made == [("empty", "side"), ("record", ("current", None)), ("copy", "side")]


@pytest.mark.parametrize("given", [None, "side"])
def test_optimizer_table_is_made_on_the_calls_stream(made, monkeypatch, given):
    monkeypatch.setattr(b, "adamw_hparams", lambda *a: made.append(("table", torch.cuda.stream.at())))
    monkeypatch.setattr(b, "mlora_adamw_step", lambda *a: None)
    opt = b.AdamW.__new__(b.AdamW)
    opt.layer = type("Layer", (), dict(plan=None, dA_ptrs=None, dB_ptrs=None, ws=torch.empty(0)))
    opt.A_ptrs = opt.B_ptrs = opt.mA_ptrs = opt.vA_ptrs = opt.mB_ptrs = opt.vB_ptrs = None
    opt.copies = (None, None)
    del made[:]
    opt.step([{}], stream=given)
    assert made == [("table", given)]
