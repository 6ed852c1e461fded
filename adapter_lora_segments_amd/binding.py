"""Python binding of the C interface: argument marshalling only.

Names mirror include/mlora.h: ``mlora_plan`` builds a host plan,
``mlora_forward`` / ``mlora_backward`` launch the HIP kernels on torch
device tensors.  torch is used for device memory and the current stream;
every step of the layer runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
from typing import Sequence

import numpy as np

from . import _lib
from ._lib import check, lib


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch  # imported first so libmlora binds to torch's HIP runtime
        _torch_module = torch
    return _torch_module


class Plan:
    """Host plan for one packed layer (seg_offsets, ranks, d_in, d_out); through
    ``Plan.from_ids``, for rows in the caller's order with one adapter id per
    token; through ``Plan.multi``, for several projections sharing the input
    (ranks [n][n_proj], output widths per projection).

    ``ranks`` holds one rank per (adapter, projection) pair in the order
    i * n_proj + q, the order of the per-adapter pointer and scale arrays."""

    def __init__(self, seg_offsets, ranks, d_in: int, d_out: int, dtype: str = "bf16",
                 nano_rows: int = 0, n_streams: int = 0, chunk_min: int = 0, chunk_max: int = 0,
                 chunk_per_rank: int = 0, w0_layout: str = "kn", gemm_rows: int = 0, _ids=None,
                 _widths=None, w0_format: str = "bf16", act_format: str = "bf16", wg_overlap: str = "auto",
                 grad_accumulate: bool = False):
        rk = np.ascontiguousarray(np.asarray(ranks, dtype=np.int32))
        opts = _lib.PlanOpts(nano_rows, gemm_rows, n_streams, chunk_min, chunk_max, chunk_per_rank,
                             _lib.W0_LAYOUTS[w0_layout], _lib.W0_FORMATS[w0_format],
                             _lib.ACT_FORMATS[act_format], _lib.WG_OVERLAP[wg_overlap],
                             1 if grad_accumulate else 0)
        h = ctypes.c_void_p()
        widths = [int(d_out)] if _widths is None else [int(v) for v in _widths]
        if _widths is not None:
            P = len(widths)
            if rk.ndim != 2 or rk.shape[1] != P:
                raise ValueError("ranks must be [n][n_proj] for a multi-projection plan")
            n = int(rk.shape[0])
            rk = np.ascontiguousarray(rk.reshape(-1))
            w = np.ascontiguousarray(np.asarray(widths, dtype=np.int64))
            if _ids is not None:
                ids = np.ascontiguousarray(np.asarray(_ids, dtype=np.int32).reshape(-1))
                check(lib().mlora_plan_multi_from_ids(
                    n, int(ids.shape[0]), ids.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), P,
                    w.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                    rk.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), int(d_in), _lib.DTYPES[dtype],
                    ctypes.byref(opts), ctypes.byref(h)))
            else:
                off = np.ascontiguousarray(np.asarray(seg_offsets, dtype=np.int64))
                if off.shape != (n + 1,):
                    raise ValueError("seg_offsets must have n + 1 entries")
                check(lib().mlora_plan_multi(n, off.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), P,
                                             w.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                             rk.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), int(d_in),
                                             _lib.DTYPES[dtype], ctypes.byref(opts), ctypes.byref(h)))
        elif _ids is None:
            n = int(rk.shape[0])
            off = np.ascontiguousarray(np.asarray(seg_offsets, dtype=np.int64))
            if off.shape != (n + 1,):
                raise ValueError("seg_offsets must have len(ranks) + 1 entries")
            check(lib().mlora_plan(n, off.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                   rk.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), int(d_in),
                                   int(d_out), _lib.DTYPES[dtype], ctypes.byref(opts), ctypes.byref(h)))
        else:
            n = int(rk.shape[0])
            ids = np.ascontiguousarray(np.asarray(_ids, dtype=np.int32).reshape(-1))
            check(lib().mlora_plan_from_ids(n, int(ids.shape[0]),
                                            ids.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                            rk.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), int(d_in),
                                            int(d_out), _lib.DTYPES[dtype], ctypes.byref(opts),
                                            ctypes.byref(h)))
        self._L = lib()
        self._h = h
        inf = _lib.PlanInfo()
        check(lib().mlora_plan_get_info(h, ctypes.byref(inf)))
        self.info = {k: getattr(inf, k) for k, _ in _lib.PlanInfo._fields_}
        self.dtype = dtype
        self.w0_layout = w0_layout
        self.w0_format = w0_format
        self.act_format = act_format
        self.offsets = self.export("offsets") if _ids is not None else np.asarray(seg_offsets, dtype=np.int64)
        self.ranks = rk
        self.widths = widths
        self.n_proj = len(widths)
        # output width of each pair's B (the width of its projection)
        self.pair_widths = np.asarray([widths[v % len(widths)] for v in range(rk.shape[0])], dtype=np.int64)
        self._ws_uploaded = None

    @classmethod
    def from_ids(cls, token_adapter, ranks, d_in: int, d_out: int, dtype: str = "bf16", **opts):
        """mlora_plan_from_ids: token t belongs to adapter token_adapter[t]."""
        return cls(None, ranks, d_in, d_out, dtype, _ids=token_adapter, **opts)

    @classmethod
    def multi(cls, seg_offsets, ranks, d_in: int, widths, dtype: str = "bf16", **opts):
        """mlora_plan_multi: projections of output widths ``widths`` sharing
        the input; ranks [n][n_proj]."""
        return cls(seg_offsets, ranks, d_in, int(sum(widths)), dtype, _widths=widths, **opts)

    @classmethod
    def multi_from_ids(cls, token_adapter, ranks, d_in: int, widths, dtype: str = "bf16", **opts):
        """mlora_plan_multi_from_ids: projections sharing the input, rows in
        the caller's order with one adapter id per token."""
        return cls(None, ranks, d_in, int(sum(widths)), dtype, _widths=widths, _ids=token_adapter, **opts)

    @property
    def handle(self):
        return self._h

    def export(self, name: str) -> np.ndarray:
        tid = _lib.TABLES.index(name)
        nbytes = ctypes.c_size_t(0)
        check(lib().mlora_plan_export(self._h, tid, None, ctypes.byref(nbytes)))
        dt = np.int64 if name in _lib.TABLE_I64 else np.int32
        buf = np.zeros(nbytes.value // np.dtype(dt).itemsize, dtype=dt)
        check(lib().mlora_plan_export(self._h, tid, buf.ctypes.data_as(ctypes.c_void_p),
                                      ctypes.byref(nbytes)))
        if name in _lib.TABLE_COLS:
            buf = buf.reshape(-1, _lib.TABLE_COLS[name])
        return buf

    def __del__(self):
        # The library handle is held by the plan itself: at interpreter exit
        # the module globals lib() needs may already be gone.
        h = getattr(self, "_h", None)
        L = getattr(self, "_L", None)
        if h is not None and h.value and L is not None:
            L.mlora_plan_destroy(h)
            self._h = ctypes.c_void_p()

    # ---- device-side helpers (torch) ----
    def alloc_workspace(self, device="cuda"):
        torch = _torch()
        return torch.empty(max(1, self.info["workspace_bytes"]), dtype=torch.uint8, device=device)

    def alloc_z(self, device="cuda"):
        torch = _torch()
        dt = torch.bfloat16 if self.dtype == "bf16" else torch.float32
        return torch.empty(max(1, self.info["z_elems"]), dtype=dt, device=device)

    def upload(self, ws, stream=None):
        torch = _torch()
        s = stream if stream is not None else torch.cuda.current_stream()
        check(lib().mlora_plan_upload(self._h, ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                      ctypes.c_void_p(s.cuda_stream)))
        self._ws_uploaded = ws

    def profile_enable(self, on=True):
        """True: time every kernel kind; False: none; or an iterable of kind
        names (``_lib.KERNELS``) to time only those."""
        if on is True:
            mask = -1
        elif not on:
            mask = 0
        else:
            mask = 0
            for k in on:
                mask |= 1 << _lib.KERNELS.index(k)
        check(lib().mlora_profile_enable(self._h, mask))

    def profile_read(self) -> dict:
        n = len(_lib.KERNELS)
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_int64 * n)()
        check(lib().mlora_profile_read(self._h, ms, cnt))
        return {k: (ms[i], cnt[i]) for i, k in enumerate(_lib.KERNELS)}


def mlora_plan(seg_offsets, ranks, d_in, d_out, dtype="bf16", **opts) -> Plan:
    return Plan(seg_offsets, ranks, d_in, d_out, dtype, **opts)


def pointer_table(tensors: Sequence, device="cuda"):
    """Device int64 array of the data pointers of ``tensors``."""
    torch = _torch()
    return torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64, device=device)


def _p(t):
    return ctypes.c_void_p(t.data_ptr() if t is not None else 0)


def _check_t(t, name, shape, dtype, numel_min=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if numel_min is not None and t.numel() < numel_min:
        raise ValueError(f"{name} needs at least {numel_min} elements")


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _made(stream, make, shape, dtype, device, returned=True):
    """make(shape) on ``stream`` (None: the current stream): memory that a call
    hands to its kernels, and its fill, have to be ordered with them.  What is
    returned to the caller also waits, once freed, for what the caller's
    stream has queued by then."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    torch = _torch()
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _dt(plan):
    torch = _torch()
    return torch.bfloat16 if plan.dtype == "bf16" else torch.float32


def _npairs(plan):
    return plan.info["n"] * plan.info["n_proj"]


def _w0_shape(plan):
    i = plan.info
    if plan.w0_format == "mxfp8":  # element codes, then the block scale codes
        return (i["d_in"] * i["d_out"] + i["d_out"] * (i["d_in"] // 32),)
    if plan.w0_format == "mxfp4":  # element codes two to a byte, then the block scale codes
        return (i["d_in"] * i["d_out"] // 2 + i["d_out"] * (i["d_in"] // 32),)
    if plan.w0_layout == "both":   # [d_in][d_out], then its transpose
        return (2 * i["d_in"] * i["d_out"],)
    return (i["d_in"], i["d_out"]) if plan.w0_layout == "kn" else (i["d_out"], i["d_in"])


def mlora_base_transpose(W, out, stream=None):
    """out[c][r] = W[r][c] (bf16 or fp32, dimensions multiples of 64), by the
    library's transpose kernel."""
    torch = _torch()
    rows, cols = W.shape
    dt = _lib.DTYPES["bf16" if W.dtype == torch.bfloat16 else "fp32"]
    assert W.is_contiguous() and out.is_contiguous() and out.numel() == W.numel() and out.dtype == W.dtype
    check(lib().mlora_base_transpose(_p(W), _p(out), rows, cols, dt, _stream(stream)))
    return out


def base_both(W0_kn, stream=None):
    """The two-layout base buffer (MLORA_W0_BOTH) of a [d_in][d_out] weight:
    the weight, then its transpose [d_out][d_in] built by the library."""
    torch = _torch()
    d_in, d_out = W0_kn.shape
    buf = _made(stream, torch.empty, 2 * d_in * d_out, W0_kn.dtype, W0_kn.device)
    with torch.cuda.stream(stream):     # (None: the current one) the copies too
        buf[: d_in * d_out].view(d_in, d_out).copy_(W0_kn)
        mlora_base_transpose(W0_kn.contiguous(), buf[d_in * d_out:], stream)
    return buf


def _w0_dtype(plan):
    torch = _torch()
    return torch.uint8 if plan.w0_format in ("mxfp8", "mxfp4") else _dt(plan)


def mlora_forward(plan: Plan, X, W0, A_ptrs, B_ptrs, scales, Y, Z, ws, stream=None):
    """Y = X W0 + s_i (X A_i) B_i per segment; Z <- s_i X A_i (plan layout)."""
    torch = _torch()
    i = plan.info
    dt = _dt(plan)
    _check_t(X, "X", (i["T"], i["d_in"]), dt)
    _check_t(W0, "W0", _w0_shape(plan), _w0_dtype(plan))
    _check_t(Y, "Y", (i["T"], i["d_out"]), dt)
    _check_t(Z, "Z", None, dt, i["z_elems"])
    for nm, t in (("A_ptrs", A_ptrs), ("B_ptrs", B_ptrs)):
        _check_t(t, nm, (_npairs(plan),), torch.int64)
    _check_t(scales, "scales", (_npairs(plan),), torch.float32)
    check(lib().mlora_forward(plan.handle, _p(X), _p(W0), _p(A_ptrs), _p(B_ptrs), _p(scales),
                              _p(Y), _p(Z), _p(ws), ws.numel(), _stream(stream)))
    return Y, Z


def mlora_forward_noalloc(plan: Plan, X, W0, A_ptrs, B_ptrs, scales, Y, Z, stream=None):
    """mlora_forward with the library's static scratch instead of a
    workspace: nothing is allocated (layers whose buffers exceed the scratch
    are refused)."""
    torch = _torch()
    i = plan.info
    dt = _dt(plan)
    _check_t(X, "X", (i["T"], i["d_in"]), dt)
    _check_t(W0, "W0", _w0_shape(plan), _w0_dtype(plan))
    _check_t(Y, "Y", (i["T"], i["d_out"]), dt)
    _check_t(Z, "Z", None, dt, i["z_elems"])
    for nm, t in (("A_ptrs", A_ptrs), ("B_ptrs", B_ptrs)):
        _check_t(t, nm, (_npairs(plan),), torch.int64)
    _check_t(scales, "scales", (_npairs(plan),), torch.float32)
    check(lib().mlora_forward_noalloc(plan.handle, _p(X), _p(W0), _p(A_ptrs), _p(B_ptrs), _p(scales),
                                      _p(Y), _p(Z), _stream(stream)))
    return Y, Z


def mlora_backward(plan: Plan, dY, X, W0, A_ptrs, B_ptrs, scales, Z, dX, dA_ptrs, dB_ptrs, ws,
                   stream=None):
    """dX (optional) and fp32 dA_i, dB_i through the pointer tables."""
    torch = _torch()
    i = plan.info
    dt = _dt(plan)
    _check_t(dY, "dY", (i["T"], i["d_out"]), dt)
    _check_t(X, "X", (i["T"], i["d_in"]), dt)
    _check_t(W0, "W0", _w0_shape(plan), _w0_dtype(plan))
    _check_t(Z, "Z", None, dt, i["z_elems"])
    if dX is not None:
        _check_t(dX, "dX", (i["T"], i["d_in"]), dt)
    for nm, t in (("A_ptrs", A_ptrs), ("B_ptrs", B_ptrs), ("dA_ptrs", dA_ptrs), ("dB_ptrs", dB_ptrs)):
        _check_t(t, nm, (_npairs(plan),), torch.int64)
    _check_t(scales, "scales", (_npairs(plan),), torch.float32)
    check(lib().mlora_backward(plan.handle, _p(dY), _p(X), _p(W0), _p(A_ptrs), _p(B_ptrs),
                               _p(scales), _p(Z), _p(dX), _p(dA_ptrs), _p(dB_ptrs), _p(ws),
                               ws.numel(), _stream(stream)))
    return dX


def adamw_hparams(hparams: Sequence[dict], device="cuda"):
    """Device array of mlora_adamw_hparams from per-adapter mappings with
    lr, beta1, beta2, eps, weight_decay, step and optionally max_grad_norm."""
    torch = _torch()
    arr = (_lib.AdamwHparams * len(hparams))()
    for k, h in enumerate(hparams):
        arr[k] = _lib.AdamwHparams(h["lr"], h["beta1"], h["beta2"], h["eps"], h["weight_decay"],
                                   int(h["step"]), float(h.get("max_grad_norm", 0.0)))
    raw = np.frombuffer(bytes(arr), dtype=np.uint8).copy()
    return torch.from_numpy(raw).to(device)


def mlora_adamw_step(plan: Plan, hparams, A_ptrs, B_ptrs, dA_ptrs, dB_ptrs, mA_ptrs, vA_ptrs,
                     mB_ptrs, vB_ptrs, A_copy_ptrs, B_copy_ptrs, ws, stream=None, clip_grads=False):
    """One AdamW step of every adapter (fp32 masters and moments through the
    pointer tables; optional bf16 copies)."""
    torch = _torch()
    n = _npairs(plan)
    _check_t(hparams, "hparams", (n * ctypes.sizeof(_lib.AdamwHparams),), torch.uint8)
    for nm, t in (("A_ptrs", A_ptrs), ("B_ptrs", B_ptrs), ("dA_ptrs", dA_ptrs), ("dB_ptrs", dB_ptrs),
                  ("mA_ptrs", mA_ptrs), ("vA_ptrs", vA_ptrs), ("mB_ptrs", mB_ptrs), ("vB_ptrs", vB_ptrs)):
        _check_t(t, nm, (n,), torch.int64)
    for nm, t in (("A_copy_ptrs", A_copy_ptrs), ("B_copy_ptrs", B_copy_ptrs)):
        if t is not None:
            _check_t(t, nm, (n,), torch.int64)
    check(lib().mlora_adamw_step(plan.handle, _p(hparams), _p(A_ptrs), _p(B_ptrs), _p(dA_ptrs),
                                 _p(dB_ptrs), _p(mA_ptrs), _p(vA_ptrs), _p(mB_ptrs), _p(vB_ptrs),
                                 _p(A_copy_ptrs), _p(B_copy_ptrs), 1 if clip_grads else 0, _p(ws),
                                 ws.numel(), _stream(stream)))


def device_check() -> None:
    check(lib().mlora_device_check())


def _check_adapters(plan: Plan, A: Sequence, B: Sequence, scales) -> None:
    """The library reads A_i and B_i through raw device pointers with the
    plan's ranks and widths, so every tensor is checked here first: A_i is
    [d_in][r_i] and B_i is [r_i][w_i] (w_i its projection's width) in the
    plan's dtype, dense, on a GPU, 16-byte aligned."""
    n = _npairs(plan)
    if len(A) != n or len(B) != n:
        raise ValueError(f"expected {n} adapter tensors for A and for B, got {len(A)} and {len(B)}")
    if np.asarray(scales).size != n:
        raise ValueError(f"expected {n} scales, got {np.asarray(scales).size}")
    dt = _dt(plan)
    d_in = plan.info["d_in"]
    items = []
    for v in range(n):
        r, w = int(plan.ranks[v]), int(plan.pair_widths[v])
        items += [(f"A[{v}]", A[v], (d_in, r)), (f"B[{v}]", B[v], (r, w))]
    for name, t, shape in items:        # what the plan fixes, on every tensor first
        if t is None:
            raise ValueError(f"{name} is required")
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
        if t.dtype != dt:
            raise ValueError(f"{name} must be {dt}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for name, t, _ in items:            # then where the memory is
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if t.data_ptr() % 16 != 0:
            raise ValueError(f"{name} must be 16-byte aligned")


class PackedLoRALinear:
    """One packed layer with its adapters, buffers and pointer tables.

    Holds device tensors A_i, B_i (parameters), dA_i, dB_i (fp32 gradients),
    the saved activation Z and the workspace; ``forward``/``backward`` call the
    library.  Pointer tables are uploaded once at construction.
    """

    def __init__(self, plan: Plan, W0, A: Sequence, B: Sequence, scales, device="cuda"):
        torch = _torch()
        self.plan = plan
        both_2d = plan.w0_layout == "both" and W0 is not None and W0.dim() == 2
        if both_2d:
            want = (plan.info["d_in"], plan.info["d_out"])
            if tuple(W0.shape) != want:
                raise ValueError(f"a two-layout base is given as [d_in][d_out] = {want}, got {tuple(W0.shape)}")
        _check_adapters(plan, A, B, scales)
        if both_2d:
            W0 = base_both(W0)          # given as [d_in][d_out]: add its transpose once
        self.W0 = W0
        self.A = list(A)
        self.B = list(B)
        n = _npairs(plan)
        self.scales = torch.as_tensor(np.asarray(scales, dtype=np.float32).reshape(-1), device=device)
        self.dA = [torch.empty((plan.info["d_in"], int(r)), dtype=torch.float32, device=device)
                   for r in plan.ranks]
        self.dB = [torch.empty((int(r), int(w)), dtype=torch.float32, device=device)
                   for r, w in zip(plan.ranks, plan.pair_widths)]
        self.A_ptrs = pointer_table(self.A, device)
        self.B_ptrs = pointer_table(self.B, device)
        self.dA_ptrs = pointer_table(self.dA, device)
        self.dB_ptrs = pointer_table(self.dB, device)
        self.ws = plan.alloc_workspace(device)
        self.Z = plan.alloc_z(device)
        plan.upload(self.ws)

    def forward(self, X, Y=None, stream=None):
        torch = _torch()
        if Y is None:
            Y = _made(stream, torch.empty, (self.plan.info["T"], self.plan.info["d_out"]), X.dtype, X.device)
        mlora_forward(self.plan, X, self.W0, self.A_ptrs, self.B_ptrs, self.scales, Y, self.Z,
                      self.ws, stream)
        return Y

    def backward(self, dY, X, dX=None, want_dx=True, stream=None):
        torch = _torch()
        if want_dx and dX is None:
            dX = _made(stream, torch.empty, (self.plan.info["T"], self.plan.info["d_in"]), X.dtype, X.device)
        mlora_backward(self.plan, dY, X, self.W0, self.A_ptrs, self.B_ptrs, self.scales, self.Z,
                       dX if want_dx else None, self.dA_ptrs, self.dB_ptrs, self.ws, stream)
        return dX


class AdamW:
    """Per-adapter AdamW state of a PackedLoRALinear: fp32 master weights,
    first and second moments, and their pointer tables.

    For a bf16 layer the masters start as the fp32 values of the layer's bf16
    A_i and B_i, and every ``step`` writes the updated masters back into those
    bf16 tensors (rounded to nearest even), so the next forward uses them.
    For an fp32 layer the layer's own A_i and B_i are the masters.  Gradients
    are the layer's dA_i and dB_i as the last backward wrote them.
    """

    def __init__(self, layer: PackedLoRALinear, device="cuda"):
        torch = _torch()
        self.layer = layer
        bf16 = layer.plan.dtype == "bf16"
        self.A = [a.float().clone() for a in layer.A] if bf16 else layer.A
        self.B = [b.float().clone() for b in layer.B] if bf16 else layer.B
        self.mA = [torch.zeros_like(a) for a in self.A]
        self.vA = [torch.zeros_like(a) for a in self.A]
        self.mB = [torch.zeros_like(b) for b in self.B]
        self.vB = [torch.zeros_like(b) for b in self.B]
        tab = lambda ts: pointer_table(ts, device)
        self.A_ptrs, self.B_ptrs = tab(self.A), tab(self.B)
        self.mA_ptrs, self.vA_ptrs = tab(self.mA), tab(self.vA)
        self.mB_ptrs, self.vB_ptrs = tab(self.mB), tab(self.vB)
        self.copies = (layer.A_ptrs, layer.B_ptrs) if bf16 else (None, None)

    def step(self, hparams, stream=None, clip_grads=False):
        """hparams: per adapter a mapping (lr, beta1, beta2, eps,
        weight_decay, step, optionally max_grad_norm), or a device array
        from ``adamw_hparams``; clip_grads applies each adapter's
        max_grad_norm."""
        L = self.layer
        with _torch().cuda.stream(stream):  # (None: the current one) a table made here belongs to the call
            hp = hparams if hasattr(hparams, "data_ptr") else adamw_hparams(hparams, L.ws.device)
        mlora_adamw_step(L.plan, hp, self.A_ptrs, self.B_ptrs, L.dA_ptrs, L.dB_ptrs, self.mA_ptrs,
                         self.vA_ptrs, self.mB_ptrs, self.vB_ptrs, self.copies[0], self.copies[1],
                         L.ws, stream, clip_grads)
        return hp


# ---- grouped expert products, row grouping, MXFP4 quantization ----

# These calls run in decode steps, where the host's share of a call counts:
# the checks below look at each tensor once and build messages only to raise
# them, and pointers reach the library as plain integers.

def _need(t, name, shape, dtype):
    """_check_t, with the common case first."""
    if t is None or t.dtype != dtype or not t.is_cuda or (shape is not None and t.shape != shape) \
            or not t.is_contiguous():
        _check_t(t, name, shape, dtype)


def _raw_stream(stream, index):
    torch = _torch()
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    return stream.cuda_stream


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _one_device(*tensors):
    """Device index of ``tensors`` (None entries skipped), which must agree."""
    index = -1
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if index < 0:
                index = i
            elif i != index:
                raise ValueError(f"tensors are on different devices: cuda:{index} and cuda:{i}")
    return index


def _launch(index, fn, *args):
    """check(fn(*args)) with device ``index`` current."""
    torch = _torch()
    if index == torch._C._cuda_getDevice():
        status = fn(*args)
    else:
        with torch.cuda.device(index):
            status = fn(*args)
    if status:
        check(status)


def group_rows_workspace(rows: int, n_groups: int) -> int:
    """Workspace bytes of mlora_group_rows for up to ``rows`` rows."""
    n = ctypes.c_int64()
    check(lib().mlora_group_rows_workspace(rows, n_groups, ctypes.byref(n)))
    return n.value


def mlora_group_rows(ids, n_groups: int, offsets, order, ws=None, stream=None):
    """Stable grouping of rows by int32 ``ids`` (any value outside
    [0, n_groups): no group): offsets [n_groups + 1] and order [rows] int32;
    positions behind the last group hold -1."""
    torch = _torch()
    rows = ids.numel()
    _need(ids, "ids", (rows,), torch.int32)
    _need(offsets, "offsets", (n_groups + 1,), torch.int32)
    _need(order, "order", (rows,), torch.int32)
    if ws is not None:
        _need(ws, "ws", None, torch.uint8)
    i = _one_device(ids, offsets, order, ws)
    _launch(i, lib().mlora_group_rows, ids.data_ptr(), rows, n_groups, offsets.data_ptr(), order.data_ptr(), _ptr(ws),
            0 if ws is None else ws.numel(), _raw_stream(stream, i))
    return offsets, order


class RowGroups:
    """Buffers of mlora_group_rows for up to ``max_rows`` rows: ``group(ids)``
    returns (offsets, order), which the next call overwrites."""

    def __init__(self, max_rows: int, n_groups: int, device="cuda"):
        torch = _torch()
        need = group_rows_workspace(max_rows, n_groups)
        self.max_rows, self.n_groups = max_rows, n_groups
        self.offsets = torch.empty(n_groups + 1, dtype=torch.int32, device=device)
        self.order = torch.empty(max_rows, dtype=torch.int32, device=device)
        self.ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None

    def group(self, ids, stream=None):
        rows = ids.numel()
        if rows > self.max_rows:
            raise ValueError(f"{rows} ids for buffers of {self.max_rows} rows")
        order = self.order if rows == self.max_rows else self.order[:rows]
        return mlora_group_rows(ids, self.n_groups, self.offsets, order, self.ws, stream)


class ExpertShape:
    """Sizes, types and layouts of a grouped expert product
    (``mlora_expert_shape``).  ``rows`` is the most rows of a call; ``src_rows``
    is the number of rows X then has."""

    def __init__(self, rows: int, n_experts: int, d_in: int, d_out: int, dtype: str = "bf16", w_layout: str = "kn",
                 w_format: str = "bf16", act_format: str = "bf16", top_k: int = 1, x_order: bool = False,
                 y_order: bool = False, grad_accumulate: bool = False):
        if w_layout not in ("kn", "nk"):
            raise ValueError(f"w_layout must be 'kn' or 'nk', got {w_layout!r}")
        if w_format not in ("bf16", "mxfp4"):
            raise ValueError(f"w_format must be 'bf16' (the dtype's own values) or 'mxfp4', got {w_format!r}")
        if act_format not in _lib.EXPERT_ACT_FORMATS:
            raise ValueError(f"act_format must be 'bf16' or 'mxfp4', got {act_format!r}")
        self.rows, self.n_experts, self.d_in, self.d_out = int(rows), int(n_experts), int(d_in), int(d_out)
        self.dtype, self.w_layout, self.w_format, self.act_format = dtype, w_layout, w_format, act_format
        self.top_k, self.x_order, self.y_order = int(top_k), bool(x_order), bool(y_order)
        self.grad_accumulate = bool(grad_accumulate)
        self._c = _lib.ExpertShape(self.rows, self.d_in, self.d_out, self.n_experts, _lib.DTYPES[dtype],
                                   _lib.W0_LAYOUTS[w_layout], _lib.W0_FORMATS[w_format],
                                   _lib.EXPERT_ACT_FORMATS[act_format], self.top_k, int(self.x_order),
                                   int(self.y_order), int(self.grad_accumulate))
        n = ctypes.c_int64()
        check(lib().mlora_expert_workspace(ctypes.byref(self.struct(self.rows)), ctypes.byref(n)))
        self.workspace_bytes = n.value
        check(lib().mlora_expert_forward_workspace(ctypes.byref(self._c), ctypes.byref(n)))
        self.forward_workspace_bytes = n.value
        # shape of all experts' weights (MXFP4: of the packed buffer)
        if w_format == "mxfp4":
            self.w_shape = (microscale_bytes(self.n_experts * self.d_out, self.d_in),)
        else:
            self.w_shape = (self.n_experts,) + ((self.d_in, self.d_out) if w_layout == "kn" else (self.d_out, self.d_in))
        # torch's dtypes of the activations and of the weight
        torch = _torch()
        self.t_dtype = _dt(self)
        self.t_w_dtype = torch.uint8 if w_format == "mxfp4" else self.t_dtype

    def struct(self, rows: int):
        """The C structure for a call of ``rows`` rows (never changed once made:
        a call on another thread may be reading it)."""
        c = self._c
        if c.rows != rows:
            c = _lib.ExpertShape.from_buffer_copy(c)
            c.rows = rows
            self._c = c
        return c

    def src_rows(self, rows: int) -> int:
        return rows // self.top_k if self.x_order else rows

    def alloc_workspace(self, device="cuda"):
        torch = _torch()
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device) if self.workspace_bytes else None


def _check_weight(shape: ExpertShape, W):
    _need(W, "W", shape.w_shape, shape.t_w_dtype)


def _check_tables(shape: ExpertShape, rows: int, offsets, order, ws):
    torch = _torch()
    if rows > shape.rows:
        raise ValueError(f"{rows} rows for a shape of at most {shape.rows}")
    if offsets is not None:
        _need(offsets, "offsets", (shape.n_experts + 1,), torch.int32)
    if order is not None:
        _need(order, "order", (rows,), torch.int32)
    if ws is not None:
        _need(ws, "ws", None, torch.uint8)


def mlora_expert_forward(shape: ExpertShape, X, W, offsets, order, Y, ws=None, stream=None):
    """Y[y(s)] = X[x(s)] W_e for every expert e and its grouped rows s (rows
    of Y that belong to no group are left as they were)."""
    rows = Y.shape[0]
    dt = shape.t_dtype
    _need(X, "X", (shape.src_rows(rows), shape.d_in), dt)
    _need(Y, "Y", (rows, shape.d_out), dt)
    _check_weight(shape, W)
    _check_tables(shape, rows, offsets, order, ws)
    i = _one_device(X, W, offsets, order, Y, ws)
    _launch(i, lib().mlora_expert_forward, ctypes.byref(shape.struct(rows)), X.data_ptr(), W.data_ptr(), _ptr(offsets),
            _ptr(order), Y.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(), _raw_stream(stream, i))
    return Y


def mlora_expert_backward(shape: ExpertShape, dY, X, W, offsets, order, dX, dW, ws=None, stream=None):
    """dX[p(s)] = dY[y(s)] W_e^T and dW_e = sum_s X[x(s)]^T dY[y(s)] (fp32);
    dX or dW may be None to skip it."""
    torch = _torch()
    rows = dY.shape[0]
    dt = shape.t_dtype
    _need(dY, "dY", (rows, shape.d_out), dt)
    if X is not None:
        _need(X, "X", (shape.src_rows(rows), shape.d_in), dt)
    if W is not None:
        _check_weight(shape, W)
    if dX is not None:
        _need(dX, "dX", (rows, shape.d_in), dt)
    if dW is not None:
        _need(dW, "dW", shape.w_shape, torch.float32)
    _check_tables(shape, rows, offsets, order, ws)
    i = _one_device(dY, X, W, offsets, order, dX, dW, ws)
    _launch(i, lib().mlora_expert_backward, ctypes.byref(shape.struct(rows)), dY.data_ptr(), _ptr(X), _ptr(W),
            _ptr(offsets), _ptr(order), _ptr(dX), _ptr(dW), _ptr(ws), 0 if ws is None else ws.numel(),
            _raw_stream(stream, i))
    return dX


class ExpertLinear:
    """A base weight per expert with its buffers: ``W`` holds all experts'
    weights in the layout and format given ([n_experts][d_in][d_out] for "kn",
    [n_experts][d_out][d_in] for "nk", the packed buffer of
    ``mlora_microscale_quantize`` for "mxfp4").  ``forward`` and ``backward``
    take up to ``max_rows`` grouped rows; ``dW`` holds the fp32 gradients of
    the last backward (with grad_accumulate, their sum since it was zeroed).
    An MXFP4 layer keeps the forward's workspace only: a dX decodes the weight
    into memory of torch's allocator (2 bytes per weight) for the call.
    The calls share the workspace ``ws``: those that may overlap, on two streams,
    from two threads or in graphs that run at once, need an ExpertLinear each
    (over one W).
    A call given a ``stream`` runs there, and what it makes (Y, dX, the first
    ``dW``) is made there: the stream has to wait for the inputs and for what
    the constructor filled, and a reader on another stream for the results."""

    def __init__(self, W, n_experts: int, d_in: int, d_out: int, max_rows: int, **options):
        torch = _torch()
        self.shape = ExpertShape(max_rows, n_experts, d_in, d_out, **options)
        _check_weight(self.shape, W)
        self.W = W
        keep = self.shape.forward_workspace_bytes if self.shape.w_format == "mxfp4" else self.shape.workspace_bytes
        self.ws = torch.empty(keep, dtype=torch.uint8, device=W.device) if keep else None
        self.dW = None
        if self.shape.grad_accumulate and self.shape.w_format == "bf16":
            self.dW = torch.zeros(self.shape.w_shape, dtype=torch.float32, device=W.device)

    def forward(self, X, offsets=None, order=None, Y=None, stream=None):
        """Y [rows][d_out]; a Y made here is zero in rows of no group when an
        order names the rows."""
        torch = _torch()
        sh = self.shape
        if Y is None:
            rows = X.shape[0] * sh.top_k if sh.x_order else X.shape[0]
            make = torch.zeros if sh.y_order else torch.empty
            Y = _made(stream, make, (rows, sh.d_out), X.dtype, X.device)
        return mlora_expert_forward(sh, X, self.W, offsets, order, Y, self.ws, stream)

    def backward(self, dY, X, offsets=None, order=None, dX=None, want_dx=True, want_dw=True, stream=None):
        """dX [rows][d_in]; ``self.dW`` unless the weight is frozen (MXFP4) or
        want_dw is False.  A dX made here is zero in rows of no group when an
        order names the rows."""
        torch = _torch()
        sh = self.shape
        if want_dx and dX is None:
            make = torch.zeros if sh.x_order else torch.empty
            dX = _made(stream, make, (dY.shape[0], sh.d_in), dY.dtype, dY.device)
        want_dw = want_dw and sh.w_format == "bf16"
        if want_dw and self.dW is None:
            self.dW = _made(stream, torch.empty, sh.w_shape, torch.float32, self.W.device)
        ws = self.ws
        if want_dx and sh.w_format == "mxfp4" and dY.shape[0] > 0:
            ws = _made(stream, torch.empty, sh.workspace_bytes, torch.uint8, self.W.device, returned=False)
        mlora_expert_backward(sh, dY, X, self.W, offsets, order, dX if want_dx else None,
                              self.dW if want_dw else None, ws, stream)
        return dX if want_dx else None


def microscale_bytes(rows: int, cols: int) -> int:
    """Bytes of the packed MXFP4 buffer of a [rows][cols] matrix."""
    return rows * cols // 2 + rows * cols // 32


def mlora_microscale_quantize(X, q=None, values=None, along: str = "cols", stream=None):
    """X [rows][cols] (bf16 or fp32, rows contiguous) to MXFP4: q, the packed
    buffer of codes and scales, made if None (on ``stream`` if one is given).
    along: "cols", blocks of 32 along a row (a [d_out][d_in] weight or
    activations), or "rows", blocks down a column (a [d_in][d_out] weight).
    values: None or a dense tensor like X for the decoded elements."""
    torch = _torch()
    if along not in ("cols", "rows"):
        raise ValueError(f"along must be 'cols' or 'rows', got {along!r}")
    if X.dim() != 2 or X.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("X must be a 2-d bf16 or fp32 tensor")
    if not X.is_cuda:
        raise ValueError("X must be a device tensor")
    rows, cols = X.shape
    if X.stride(1) != 1 and cols > 1:
        raise ValueError("X's rows must be contiguous")
    n = microscale_bytes(rows, cols)
    if q is None:
        q = _made(stream, torch.empty, n, torch.uint8, X.device)
    _need(q, "q", (n,), torch.uint8)
    if values is not None:
        _need(values, "values", (rows, cols), X.dtype)
    i = _one_device(X, q, values)
    _launch(i, lib().mlora_microscale_quantize, X.data_ptr(), 1 if X.dtype == torch.bfloat16 else 0, rows, cols,
            X.stride(0) if rows > 1 else cols, 1 if along == "rows" else 0, q.data_ptr(), _ptr(values),
            _raw_stream(stream, i))
    return q
