"""What the routing, combining and 4-bit entry points make for themselves is made
on the stream that their kernels run on (as in test_experts_streams_cpu.py: torch's
makers are watched and no kernel is launched)."""
import pytest

from adapter_lora_segments_amd import binding as b
from tests.test_experts_streams_cpu import made  # noqa: F401  (a fixture)

torch = pytest.importorskip("torch")


@pytest.fixture
def quiet(monkeypatch):
    """No kernel is launched; the streams that were asked for."""
    asked = []
    monkeypatch.setattr(b, "_need", lambda *a: None)
    monkeypatch.setattr(b, "_one_device", lambda *a: 0)
    monkeypatch.setattr(b, "_raw_stream", lambda s, i: asked.append(s))
    monkeypatch.setattr(b, "_launch", lambda *a: None)
    return asked


def expect(given, *fills, returned=True):
    kept = [("record", ("current", None))] if given and returned else []
    return [m for f in fills for m in [(f, given)] + kept]


@pytest.mark.parametrize("given", [None, "side"])
def test_router(made, quiet, monkeypatch, given):  # noqa: F811
    monkeypatch.setattr(b, "_logits_of", lambda t, n: (t.shape[0], n, 0))
    r = b.Router(16, 4)
    x, ids, w = torch.ones(3, 16), torch.ones(3, 4, dtype=torch.int32), torch.ones(3, 4)
    del made[:]
    r.route(x, stream=given)
    r.backward(x, ids, w, stream=given)
    assert made == expect(given, "empty", "empty", "empty") and quiet == [given] * 2


@pytest.mark.parametrize("given", [None, "side"])
def test_combine(made, quiet, given):  # noqa: F811
    y, w = torch.ones(6, 8), torch.ones(3, 2)
    del made[:]
    b.mlora_combine(y, 2, None, w, stream=given)
    b.mlora_combine_backward(y[:3], y, 2, None, w, stream=given)
    assert made == expect(given, "empty", "empty", "empty") and quiet == [given] * 2


@pytest.mark.parametrize("given", [None, "side"])
def test_affine_quantizer(made, quiet, given):  # noqa: F811
    class Matrix:
        dtype, is_cuda, shape, device = torch.bfloat16, True, (4, 64), torch.device("cpu")
        dim = staticmethod(lambda: 2)
        stride = staticmethod(lambda i: (64, 1)[i])
        data_ptr = staticmethod(lambda: 0)

    b.mlora_affine_quantize(Matrix(), group=32, stream=given)
    assert made == expect(given, "empty") and quiet == [given]


@pytest.mark.parametrize("given", [None, "side"])
@pytest.mark.parametrize("order", [False, True])
@pytest.mark.parametrize("rows", [8, 4096])
def test_affine_linear(made, quiet, monkeypatch, rows, order, given):  # noqa: F811
    """Outputs, and the workspace of calls of many rows, which is freed to the
    stream it was used on."""
    monkeypatch.setattr(b, "_check_tables", lambda *a: None)
    L = b.AffineLinear.__new__(b.AffineLinear)
    L.shape = b.AffineShape(rows, 2, 64, 64, group=32, x_order=order, y_order=order)
    L.q = torch.ones(1)
    x = torch.ones(rows, 64, dtype=torch.bfloat16)
    del made[:]
    L.forward(x, stream=given)
    L.backward(x, stream=given)
    fill = expect(given, "zeros" if order else "empty")
    ws = expect(given, "empty", returned=False) if rows == 4096 else []
    assert made == (fill + ws) * 2 and quiet == [given] * 2
