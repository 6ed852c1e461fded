"""Grouped expert products, row grouping and MXFP4 quantization without a GPU:
the oracle on small hand-worked inputs, and every refusal of the C interface
and the binding (no launch happens: the pointers are host addresses that no
call reaches)."""
import ctypes

import numpy as np
import pytest

from adapter_lora_segments_amd import _lib
from adapter_lora_segments_amd import binding as b
from oracle import experts as ox


# ---- the oracle ----

def test_group_rows_by_hand():
    off, order = ox.group_rows([2, 0, -1, 2, 0, 7, 1, 2], 4)
    assert off.tolist() == [0, 2, 3, 6, 6]
    assert order.tolist() == [1, 4, 6, 0, 3, 7, -1, -1]
    off, order = ox.group_rows([], 3)
    assert off.tolist() == [0, 0, 0, 0] and order.size == 0


def test_products_by_hand():
    """Two experts, three tokens with two ids each; token 2's second id is dropped."""
    off, order = ox.group_rows([0, 1, 1, 0, 1, -1], 2)
    assert order.tolist() == [0, 3, 1, 2, 4, -1]
    X = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    W = np.array([[[1.0], [10.0]], [[100.0], [1000.0]]])
    Y, _, owned = ox.forward(X, W, off, order, 6, top_k=2, x_order=True, y_order=True)
    assert Y[:, 0].tolist() == [21, 2100, 4300, 43, 6500, 0] and owned.tolist() == [True] * 5 + [False]
    Yg, _, _ = ox.forward(X, W, off, order, 6, top_k=2, x_order=True)
    assert Yg[:, 0].tolist() == [21, 43, 2100, 4300, 6500, 0]


@pytest.mark.parametrize("x_order,y_order,top_k", [(False, False, 1), (True, False, 2), (True, True, 3), (False, True, 1)])
def test_gradients_against_differences(x_order, y_order, top_k):
    """The loss <Y, G> is bilinear in (X, W): central differences with any
    step are its gradient up to float64 rounding (here 1e-9 of O(10) values)."""
    rng = np.random.default_rng(3)
    E, di, do, T = 3, 4, 5, 6
    rows = T * top_k if x_order else T
    ids = rng.integers(-1, E, size=rows)
    off, order = ox.group_rows(ids, E)
    X, W = rng.standard_normal((T if x_order else rows, di)), rng.standard_normal((E, di, do))
    G = rng.standard_normal((rows, do))
    kw = dict(top_k=top_k, x_order=x_order, y_order=y_order)
    dXs, _, _, dW, _ = ox.backward(G, X, W, off, order, rows, **kw)
    dX = dXs.reshape(T, top_k, di).sum(1) if x_order else dXs
    loss = lambda X, W: (ox.forward(X, W, off, order, rows, **kw)[0] * G).sum()
    for arr, grad in ((X, dX), (W, dW)):
        for i in np.ndindex(arr.shape):
            old = arr[i]
            arr[i] = old + 0.5
            up = loss(X, W)
            arr[i] = old - 0.5
            down = loss(X, W)
            arr[i] = old
            assert abs(up - down - grad[i]) < 1e-9


def test_quantizer_rounding_by_hand():
    """A block whose maximum is 4..7.99 has scale 1: every midpoint of the
    E2M1 grid goes to the even code, and what passes 6 saturates."""
    x = np.zeros((1, 32))
    x[0, :15] = [7.9, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 0.26, 4.99, 5.01, -6.5, -0.0]
    c, s = ox.quantize(x)
    assert s[0, 0] == 127
    assert c[0, :15].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 14, 1, 6, 7, 15, 8]
    v = ox.decode(c, s)
    assert v[0, :5].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0]


def test_quantizer_scales_by_hand():
    x = np.zeros((6, 32))
    x[1, 3] = 4.0          # exponent 2: scale 2^0
    x[2, 3] = 3.99         # exponent 1: scale 2^-1
    x[3, 3] = 2.0 ** -140  # below the clamp: scale 2^-127, the element rounds to 0
    x[4, 3] = np.inf
    x[5, 3] = 2.0 ** 127   # scale 2^125
    c, s = ox.quantize(x)
    assert s[:, 0].tolist() == [0, 127, 126, 0, 255, 252]
    assert c[1, 3] == 6 and c[2, 3] == 7 and c[3, 3] == 0 and (c[4] == 0).all() and c[5, 3] == 6
    assert np.isnan(ox.decode(c, s)[4]).all()


# ---- refusals of the C interface ----

BUF = ctypes.create_string_buffer(1 << 12)
P16 = ctypes.addressof(BUF) + (-ctypes.addressof(BUF)) % 16


def shape(**kw):
    d = dict(rows=64, d_in=128, d_out=64, n_experts=4, dtype=1, w_layout=1, w_format=0, act_format=0, top_k=1,
             x_by_order=0, y_by_order=0, grad_accumulate=0)
    d.update(kw)
    return _lib.ExpertShape(**d)


BAD_SHAPES = [(dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(n_experts=0), -1), (dict(n_experts=4097), -1),
              (dict(dtype=2), -1), (dict(w_layout=2), -1), (dict(d_in=0), -1), (dict(d_in=100), -1),
              (dict(d_out=-8), -1), (dict(dtype=0, d_out=6), -1), (dict(top_k=0), -1), (dict(top_k=65), -1),
              (dict(top_k=3, x_by_order=1), -1), (dict(top_k=2), -1), (dict(x_by_order=2), -1),
              (dict(y_by_order=-1), -1), (dict(grad_accumulate=5), -1), (dict(w_format=1), -1),
              (dict(act_format=1), -1), (dict(d_in=(1 << 20) + 8), -2), (dict(w_format=2, d_in=64), -2),
              (dict(w_format=2, w_layout=0), -2), (dict(w_format=2, dtype=0), -2), (dict(act_format=2), -2),
              (dict(rows=(1 << 31) - 1, d_out=1 << 20), -2), (dict(rows=1 << 28, d_out=4096), -2),
              (dict(n_experts=4096, d_in=1 << 15, d_out=1 << 15), -2),
              (dict(w_format=2, act_format=2, rows=1 << 24, d_in=1 << 15, d_out=8), -2)]


@pytest.mark.parametrize("bad,status", BAD_SHAPES)
def test_malformed_shapes(bad, status):
    L = _lib.lib()
    s, n = shape(**bad), ctypes.c_int64(-7)
    assert L.mlora_expert_workspace(ctypes.byref(s), ctypes.byref(n)) == status and n.value == -7
    v = ctypes.c_void_p
    assert L.mlora_expert_forward(ctypes.byref(s), v(P16), v(P16), v(P16), v(P16), v(P16), v(P16), 1 << 60, None) == status
    assert L.mlora_expert_backward(ctypes.byref(s), v(P16), v(P16), v(P16), v(P16), v(P16), v(P16), v(P16), v(P16),
                                   1 << 60, None) == status
    assert L.mlora_last_error().decode().startswith("expert")


def _forward(s, X=P16, W=P16, off=P16, order=P16, Y=P16, ws=P16, n=1 << 60):
    v = ctypes.c_void_p
    return _lib.lib().mlora_expert_forward(ctypes.byref(s) if s else None, v(X), v(W), v(off), v(order), v(Y), v(ws),
                                           n, None)


def _backward(s, dY=P16, X=P16, W=P16, off=P16, order=P16, dX=P16, dW=P16, ws=P16, n=1 << 60):
    v = ctypes.c_void_p
    return _lib.lib().mlora_expert_backward(ctypes.byref(s) if s else None, v(dY), v(X), v(W), v(off), v(order), v(dX),
                                            v(dW), v(ws), n, None)


def test_malformed_calls():
    s = shape()
    assert _forward(None) == -1 and _backward(None) == -1
    for k in ("X", "W", "Y"):
        assert _forward(s, **{k: 0}) == -1 and _forward(s, **{k: P16 + 8}) == -1
    for k in ("dY", "X", "W"):
        assert _backward(s, **{k: 0}) == -1
    for k in ("dY", "X", "W", "dX", "dW"):
        assert _backward(s, **{k: P16 + 4}) == -1
    assert _forward(s, off=0) == -1 and _forward(s, off=P16 + 2) == -1 and _forward(s, order=P16 + 1) == -1
    assert _forward(shape(x_by_order=1), order=0) == -1 and _backward(shape(y_by_order=1), order=0) == -1
    q = shape(w_format=2, act_format=2)
    need = ctypes.c_int64()
    assert _lib.lib().mlora_expert_workspace(ctypes.byref(q), ctypes.byref(need)) == 0
    assert need.value == max(64 * 128 // 2 + 64 * 128 // 32, 2 * 4 * 128 * 64)
    assert _forward(q, ws=0) == -1 and _forward(q, ws=P16 + 4) == -1 and _forward(q, n=100) == -4
    assert _backward(shape(w_format=2)) == -2                          # a frozen weight has no dW
    assert _backward(shape(w_format=2), dW=0, n=2 * 4 * 128 * 64 - 1) == -4
    # no rows: nothing to launch, row-indexed buffers may be NULL
    assert _forward(shape(rows=0), X=0, Y=0) == 0
    assert _backward(shape(rows=0, grad_accumulate=1), dY=0, X=0) == 0


def test_group_rows_refusals():
    L, v, n = _lib.lib(), ctypes.c_void_p, ctypes.c_int64()
    for rows, g in ((-1, 4), (1 << 31, 4), (8, 0), (8, 4097)):
        assert L.mlora_group_rows_workspace(rows, g, ctypes.byref(n)) == -1
        assert L.mlora_group_rows(v(P16), rows, g, v(P16), v(P16), v(P16), 1 << 40, None) == -1
    assert L.mlora_group_rows_workspace(8, 4, None) == -1
    assert L.mlora_group_rows_workspace(100000, 8, ctypes.byref(n)) == 0 and n.value > 0
    args = dict(ids=P16, offsets=P16, order=P16, ws=P16)
    call = lambda rows, nb=1 << 40, **k: L.mlora_group_rows(*[v({**args, **k}["ids"]), rows, 8, v({**args, **k}["offsets"]),
                                                              v({**args, **k}["order"]), v({**args, **k}["ws"]), nb, None])
    for k in ("ids", "offsets", "order"):
        assert call(8, **{k: 0}) == -1 and call(8, **{k: P16 + 2}) == -1
    assert call(100000, ws=0) == -1 and call(100000, ws=P16 + 4) == -1 and call(100000, nb=n.value - 1) == -4


def test_group_rows_workspace_never_shrinks_with_rows():
    """The bytes for R rows cover every smaller number of rows (RowGroups relies on it)."""
    sizes = [1, 8192, 8193, 20000, 1 << 20, (1 << 20) + 1, 5 << 20, 1 << 30]
    got = [b.group_rows_workspace(r, 64) for r in sizes]
    assert got == sorted(got)
    for r, n in zip(sizes, got):      # parts the launch takes: group_part_rows
        part = max(4096, -(-(-(-r // 256)) // 1024) * 1024)
        assert r <= 8192 or 4 * 64 * -(-r // part) <= n


def test_quantize_refusals():
    L, v = _lib.lib(), ctypes.c_void_p
    ok = dict(X=P16, dtype=1, rows=32, cols=64, ld=64, down=0, q=P16, values=0)
    call = lambda **k: L.mlora_microscale_quantize(*[v({**ok, **k}[n]) if n in ("X", "q", "values") else {**ok, **k}[n]
                                                     for n in ok], None)
    for bad in (dict(dtype=3), dict(down=2), dict(rows=-32), dict(cols=0), dict(cols=48), dict(ld=56), dict(ld=68),
                dict(down=1, rows=33), dict(down=1, cols=36, ld=40), dict(X=0), dict(q=0), dict(X=P16 + 2),
                dict(q=P16 + 8), dict(values=P16 + 4)):
        assert call(**bad) == -1, bad
    assert call(cols=1 << 21, ld=1 << 21) == -2
    assert call(rows=0, X=0, q=0) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="w_layout"):
        b.ExpertShape(8, 2, 64, 64, w_layout="both")
    with pytest.raises(ValueError, match="w_format"):
        b.ExpertShape(8, 2, 64, 64, w_format="mxfp8")
    with pytest.raises(ValueError, match="act_format"):
        b.ExpertShape(8, 2, 64, 64, act_format="mxfp8")
    with pytest.raises(_lib.MloraError, match="MLORA_ERR_UNSUPPORTED"):
        b.ExpertShape(8, 2, 64, 64, w_layout="nk", w_format="mxfp4")
    sh = b.ExpertShape(8, 2, 64, 64)
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        b.mlora_expert_forward(sh, x, x, None, None, x)
    with pytest.raises(ValueError, match="along"):
        b.mlora_microscale_quantize(x, along="both")
    with pytest.raises(ValueError, match="2-d"):
        b.mlora_microscale_quantize(torch.zeros(8, 64, dtype=torch.float64))
    with pytest.raises(ValueError, match="device tensor"):
        b.mlora_microscale_quantize(x)
    with pytest.raises(ValueError, match="device tensor"):
        b.mlora_group_rows(torch.zeros(4, dtype=torch.int32), 2, None, None)


@pytest.mark.parametrize("dtype,least", [(1, 1024), (0, 256)])
def test_workspace_of_gradient_chunks(dtype, least):
    """The partial sums' room: none while no group can be cut, never less for
    more rows, and never past two slots per `least` rows; none once the tiles
    of all experts fill the chip."""
    L, n = _lib.lib(), ctypes.c_int64()

    def need(**kw):
        assert L.mlora_expert_workspace(ctypes.byref(shape(dtype=dtype, **kw)), ctypes.byref(n)) == 0
        return n.value

    for experts, di, do in ((1, 136, 864), (4, 72, 136), (7, 512, 1024)):
        last = 0
        for rows in list(range(0, 4 * least, 61)) + [10 ** 5, 10 ** 7, 10 ** 8]:
            v = need(rows=rows, n_experts=experts, d_in=di, d_out=do)
            assert v >= last and v <= 2 * rows // least * di * do * 4
            assert (v == 0) == (rows <= least)
            last = v
    assert need(rows=10 ** 6, n_experts=64, d_in=512, d_out=1024) == 0
