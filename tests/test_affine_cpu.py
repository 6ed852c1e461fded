"""4-bit weights with group scales without a GPU: the oracle by hand, packing,
and every refusal of the C interface and the binding."""
import ctypes

import numpy as np
import pytest

from adapter_lora_segments_amd import _lib
from adapter_lora_segments_amd import binding as b
from oracle import affine as oa


def test_quantizer_by_hand():
    x = np.zeros((4, 32), dtype=np.float32)
    x[0, :6] = [15, 0.5, 1.5, 2.5, 14.4, 0]           # s = 1, z = 0: ties to even
    x[1, :5] = [-7.5, 7.5, 0.5, -0.5, 1.4]            # s = 1, -lo / s = 7.5: z = 8
    x[2, :3] = [-30, -2, -31]                         # all below zero: s = 31 / 15 in bf16, z = 15
    c, z, s = oa.quantize(x, 32)
    assert s[0, 0] == 1 and z[0, 0] == 0 and c[0, :6].tolist() == [15, 0, 2, 2, 14, 0]
    assert s[1, 0] == 1 and z[1, 0] == 8 and c[1, :5].tolist() == [0, 15, 8, 8, 9]
    # 7.5 rounds to 8, clamped to 15 - 8; -7.5 to -8
    assert oa.decode(c, z, s)[1, :2].tolist() == [-8, 7]
    assert s[2, 0] == oa.bf16(np.float32(31) / np.float32(15)) and z[2, 0] == 15 and c[2, 3] == 15
    assert s[3, 0] == 0 and z[3, 0] == 0 and not c[3].any() and not oa.decode(c, z, s)[3].any()
    x[0, 0] = 7
    c, z, s = oa.quantize(x, 32, symmetric=True)
    assert (z == 8).all() and c[3].tolist() == [8] * 32 and not oa.decode(c, z, s)[3].any()
    x[1, 9], x[2, 1] = np.inf, np.nan
    c, z, s = oa.quantize(x, 32)
    assert np.isnan(s[1:3]).all() and not c[1:3].any() and np.isfinite(s[0]).all()


def test_pack_round_trip():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 192)).astype(np.float32)
    for g in (32, 64):
        c, z, s = oa.quantize(x, g)
        buf = oa.pack(c, z, s)
        assert buf.size == b.affine_bytes(6, 192, g)
        c2, z2, s2 = oa.unpack(buf, 6, 192, g)
        assert np.array_equal(c, c2) and np.array_equal(z, z2) and np.array_equal(s, s2)
        q = b.affine_pack(torch.from_numpy(c), torch.from_numpy(s), torch.from_numpy(z))
        assert np.array_equal(q.numpy(), buf)
        sym = b.affine_pack(torch.from_numpy(c.astype(np.int64)), torch.from_numpy(s))
        assert np.array_equal(sym.numpy(), oa.pack(c, np.full_like(z, 8), s))


def test_bf16_rounding():
    torch = pytest.importorskip("torch")
    r = np.random.default_rng(3).standard_normal(4000).astype(np.float32) * np.exp2(np.arange(4000) % 60 - 30).astype(np.float32)
    assert np.array_equal(oa.bf16(r), torch.from_numpy(r).to(torch.bfloat16).float().numpy())


BUF = ctypes.create_string_buffer(1 << 12)
P16 = ctypes.addressof(BUF) + (-ctypes.addressof(BUF)) % 16
V = ctypes.c_void_p


def shape(**kw):
    d = dict(rows=64, d_in=256, d_out=64, n_experts=4, group=64, top_k=1, x_by_order=0, y_by_order=0)
    d.update(kw)
    return _lib.AffineShape(**d)


BAD = [(dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(n_experts=0), -1), (dict(n_experts=4097), -1),
       (dict(group=16), -1), (dict(group=0), -1), (dict(group=256), -1), (dict(d_in=0), -1), (dict(d_in=96), -1),
       (dict(d_in=-64), -1), (dict(d_out=0), -1), (dict(d_out=12), -1), (dict(top_k=0), -1), (dict(top_k=65), -1),
       (dict(top_k=2), -1), (dict(top_k=3, x_by_order=1), -1), (dict(x_by_order=2), -1), (dict(y_by_order=-1), -1),
       (dict(d_in=(1 << 20) + 64), -2), (dict(d_out=(1 << 20) + 8), -2),
       (dict(rows=(1 << 31) - 1, d_out=1 << 20), -2), (dict(n_experts=4096, d_in=1 << 17, d_out=1 << 17), -2)]


def _forward(s, X=P16, q=P16, off=P16, order=P16, Y=P16, ws=P16, n=1 << 60):
    return _lib.lib().mlora_affine_forward(ctypes.byref(s) if s else None, V(X), V(q), V(off), V(order), V(Y), V(ws), n, None)


def _backward(s, dY=P16, q=P16, off=P16, order=P16, dX=P16, ws=P16, n=1 << 60):
    return _lib.lib().mlora_affine_backward(ctypes.byref(s) if s else None, V(dY), V(q), V(off), V(order), V(dX), V(ws), n,
                                          None)


@pytest.mark.parametrize("bad,status", BAD)
def test_malformed_shapes(bad, status):
    s, f = shape(**bad), ctypes.c_int64(-7)
    assert _lib.lib().mlora_affine_workspace(ctypes.byref(s), ctypes.byref(f), None) == status and f.value == -7
    assert _forward(s) == status and _backward(s) == status
    assert _lib.lib().mlora_last_error().decode().startswith("affine")


def test_malformed_calls():
    s = shape()
    assert _forward(None) == -1 and _backward(None) == -1
    for k in ("X", "q", "Y"):
        assert _forward(s, **{k: 0}) == -1 and _forward(s, **{k: P16 + 8}) == -1
    for k in ("dY", "q", "dX"):
        assert _backward(s, **{k: 0}) == -1 and _backward(s, **{k: P16 + 8}) == -1
    for f in (_forward, _backward):
        assert f(s, off=0) == -1 and f(s, off=P16 + 2) == -1 and f(s, order=P16 + 1) == -1
        assert f(shape(x_by_order=1), order=0) == -1 and f(shape(y_by_order=1), order=0) == -1
    big = shape(rows=1 << 20)
    f, w = ctypes.c_int64(), ctypes.c_int64()
    assert _lib.lib().mlora_affine_workspace(ctypes.byref(big), ctypes.byref(f), ctypes.byref(w)) == 0
    for call, need in ((_forward, f.value), (_backward, w.value)):
        if need:
            assert call(big, ws=0) == -1 and call(big, ws=P16 + 4) == -1 and call(big, n=need - 1) == -4
    # fewer rows never need more
    for rows in (1, 5, 64, 1000, 1 << 16):
        g, h = ctypes.c_int64(), ctypes.c_int64()
        assert _lib.lib().mlora_affine_workspace(ctypes.byref(shape(rows=rows)), ctypes.byref(g), ctypes.byref(h)) == 0
        assert g.value <= f.value and h.value <= w.value
    assert _forward(shape(rows=0), X=0, Y=0) == 0 and _backward(shape(rows=0), dY=0, dX=0) == 0


def test_quantize_refusals():
    L, n = _lib.lib(), ctypes.c_int64()
    for rows, cols, g, st in ((-1, 128, 128, -1), (4, 0, 128, -1), (4, 96, 64, -1), (4, 128, 48, -1), (4, 1 << 21, 128, -2)):
        assert L.mlora_affine_bytes(rows, cols, g, ctypes.byref(n)) == st
        assert L.mlora_affine_quantize(V(P16), 1, rows, cols, 1 << 22, g, 0, V(P16), V(0), None) == st
    assert L.mlora_affine_bytes(4, 128, 64, None) == -1
    q = lambda X=P16, dt=1, rows=4, cols=128, ld=128, g=64, sym=0, q=P16, v=0: L.mlora_affine_quantize(
        V(X), dt, rows, cols, ld, g, sym, V(q), V(v), None)
    assert q(dt=2) == -1 and q(sym=2) == -1 and q(ld=120) == -1 and q(ld=132) == -1 and q(dt=0, ld=130) == -1
    assert q(X=0) == -1 and q(q=0) == -1 and q(X=P16 + 8) == -1 and q(q=P16 + 4) == -1 and q(v=P16 + 8) == -1
    assert q(rows=1 << 40) == -2 and q(rows=0, X=0, q=0) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    with pytest.raises(_lib.MloraError, match="group"):
        b.affine_bytes(4, 128, 48)
    with pytest.raises(_lib.MloraError, match="group"):
        b.AffineShape(8, 2, 64, 64, group=128)
    with pytest.raises(ValueError, match="device"):
        b.AffineLinear(z(b.affine_bytes(128, 64, 64), dtype=torch.uint8), 2, 64, 64, 8, group=64)
    with pytest.raises(ValueError, match="device"):
        b.mlora_affine_quantize(z(4, 128))
    with pytest.raises(ValueError, match="2-d"):
        b.mlora_affine_quantize(z(4, 128, dtype=torch.float16))
    c, s = z(4, 128, dtype=torch.uint8), z(4, 2)
    with pytest.raises(ValueError, match="from 0 to 15"):
        b.affine_pack(c + 16, s)
    with pytest.raises(ValueError, match="from 0 to 15"):
        b.affine_pack(c.float(), s)
    with pytest.raises(ValueError, match="no group"):
        b.affine_pack(c, z(4, 8))
    with pytest.raises(ValueError, match="zeros"):
        b.affine_pack(c, s, z(4, 1))
    with pytest.raises(ValueError, match="codes must be"):
        b.affine_pack(c, z(3, 2))
