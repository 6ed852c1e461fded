"""Workspaces of the grouped expert products by call, without a GPU: a frozen
4-bit layer that runs forward holds no 16-bit copy of its weights."""
import ctypes

import pytest

from adapter_lora_segments_amd import _lib
from adapter_lora_segments_amd import binding as b
from tests.test_experts_cpu import BAD_SHAPES, shape

torch = pytest.importorskip("torch")


@pytest.fixture
def on_cpu(monkeypatch):
    """Layers over host tensors: no call reaches the library's kernels."""
    calls = []
    monkeypatch.setattr(b, "_check_weight", lambda *a: None)
    monkeypatch.setattr(b, "mlora_expert_forward", lambda *a: calls.append(a[-2]))
    monkeypatch.setattr(b, "mlora_expert_backward", lambda *a: calls.append(a[-2]))
    return calls


def frozen(rows=64, **opts):
    W = torch.zeros(b.microscale_bytes(4 * 256, 128), dtype=torch.uint8)
    return b.ExpertLinear(W, 4, 128, 256, rows, w_layout="nk", w_format="mxfp4", **opts)


@pytest.mark.parametrize("act,need", [("bf16", 0), ("mxfp4", 64 * 64 + 64 * 4)])
def test_frozen_layer_keeps_the_forward_workspace_only(on_cpu, act, need):
    L = frozen(act_format=act)
    x = torch.zeros(64, 128, dtype=torch.bfloat16)
    assert (0 if L.ws is None else L.ws.numel()) == need
    L.forward(x)
    assert on_cpu[-1] is L.ws
    L.backward(torch.zeros(64, 256, dtype=torch.bfloat16), None)
    assert on_cpu[-1].numel() >= 2 * 4 * 128 * 256            # dX's decoded weight, for the call
    assert (0 if L.ws is None else L.ws.numel()) == need
    L.backward(torch.zeros(0, 256, dtype=torch.bfloat16), None)
    assert on_cpu[-1] is L.ws                                  # no rows: nothing is decoded


def test_workspace_of_gradient_sums_is_kept(on_cpu):
    W = torch.zeros(1, 128, 256, dtype=torch.bfloat16)
    L = b.ExpertLinear(W, 1, 128, 256, 4096)
    assert L.ws.numel() == L.shape.workspace_bytes > 0
    L.backward(torch.zeros(4096, 256, dtype=torch.bfloat16), torch.zeros(4096, 128, dtype=torch.bfloat16))
    assert on_cpu[-1] is L.ws


def test_forward_workspace():
    L, n, both = _lib.lib(), ctypes.c_int64(-7), ctypes.c_int64()
    for kw, want in ((dict(), 0), (dict(dtype=0), 0), (dict(w_format=2), 0),
                     (dict(w_format=2, act_format=2), 64 * 128 // 2 + 64 * 128 // 32),
                     (dict(w_format=2, act_format=2, rows=66, x_by_order=1, top_k=2), 33 * 128 // 2 + 144),
                     (dict(w_format=2, act_format=2, rows=0), 0)):
        s = shape(**kw)
        assert L.mlora_expert_forward_workspace(ctypes.byref(s), ctypes.byref(n)) == 0 and n.value == want, kw
        assert L.mlora_expert_workspace(ctypes.byref(s), ctypes.byref(both)) == 0 and both.value >= want


@pytest.mark.parametrize("bad,status", BAD_SHAPES)
def test_forward_workspace_refusals(bad, status):
    L, n = _lib.lib(), ctypes.c_int64(-7)
    s = shape(**bad)
    assert L.mlora_expert_forward_workspace(ctypes.byref(s), ctypes.byref(n)) == status and n.value == -7
    assert L.mlora_expert_forward_workspace(None, ctypes.byref(n)) == -1
    assert L.mlora_expert_forward_workspace(ctypes.byref(shape()), None) == -1
