"""What the grouped products and the MXFP4 operators are measured on.

Every case is one call (or the two calls that belong together) as a program
that runs mixture-of-experts layers or a 4-bit base makes it:

- ``group``: the rows of a router's answer sorted by expert on the device;
- ``forward``: one product per expert over ragged row groups;
- ``backward``: the gradients of such a product, dX and fp32 dW (dX alone
  over a frozen MXFP4 weight);
- ``quantize``: a matrix to MXFP4 codes and scales with its decoded values;
- ``mx4``: the product with MXFP4 weights, activations in bf16 or quantized
  to MXFP4 on the way.

With ``own`` false ``run`` computes the plain form in fp32 torch operations.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step's routing: 16 tokens, two experts each
        {"name": "group decode 32 of 16", "op": "group", "tokens": 16, "top_k": 2, "experts": 16, "zipf": 0.0,
         "dropped": 0.0},
        # a long prefill's routing: skewed experts, some slots dropped
        {"name": "group prefill 262144 of 64", "op": "group", "tokens": 32768, "top_k": 8, "experts": 64,
         "zipf": 1.1, "dropped": 0.02},
        # a decode step through the 4096x4096 projection of eight experts
        {"name": "forward decode bf16 nk", "op": "forward", "dtype": "bf16", "layout": "nk", "tokens": 4, "top_k": 2,
         "experts": 8, "zipf": 0.0, "d_in": 4096, "d_out": 4096, "x_order": True, "y_order": False},
        # 32768 routed rows over 64 experts of an up projection, skewed
        {"name": "forward prefill bf16 kn", "op": "forward", "dtype": "bf16", "layout": "kn", "tokens": 16384,
         "top_k": 2, "experts": 64, "zipf": 1.1, "d_in": 4096, "d_out": 14336, "x_order": True, "y_order": False},
        # small odd sizes in fp32, rows scattered back to the caller's order
        {"name": "forward odd fp32 nk", "op": "forward", "dtype": "fp32", "layout": "nk", "tokens": 517, "top_k": 1,
         "experts": 5, "zipf": 0.7, "d_in": 1000, "d_out": 264, "x_order": True, "y_order": True},
        # training step of four experts on the 4096x4096 projection
        {"name": "backward bf16 kn", "op": "backward", "dtype": "bf16", "layout": "kn", "tokens": 7680, "top_k": 1,
         "experts": 4, "zipf": 0.8, "d_in": 4096, "d_out": 4096, "x_order": False, "y_order": False, "w4": False},
        # many small experts of odd widths, routed twice, dY in slot order
        {"name": "backward ragged bf16 nk", "op": "backward", "dtype": "bf16", "layout": "nk", "tokens": 1501,
         "top_k": 2, "experts": 24, "zipf": 1.1, "d_in": 1032, "d_out": 2056, "x_order": True, "y_order": True,
         "w4": False},
        # a 14336x4096 weight quantized along its rows, decoded values kept
        {"name": "quantize weight bf16", "op": "quantize", "dtype": "bf16", "rows": 14336, "cols": 4096,
         "along": "cols"},
        # an fp32 master in the [d_in][d_out] layout, blocks down the columns
        {"name": "quantize kn fp32", "op": "quantize", "dtype": "fp32", "rows": 1024, "cols": 4096, "along": "rows"},
        # single-token serving: four rows against a 4-bit up projection
        {"name": "mx4 decode bf16 act", "op": "mx4", "act": "bf16", "tokens": 4, "top_k": 1, "experts": 1,
         "zipf": 0.0, "d_in": 4096, "d_out": 14336, "x_order": False, "y_order": False},
        # prefill on the 4-bit matrix cores, activations quantized in the call
        {"name": "mx4 prefill mxfp4 act", "op": "mx4", "act": "mxfp4", "tokens": 8192, "top_k": 1, "experts": 1,
         "zipf": 0.0, "d_in": 4096, "d_out": 14336, "x_order": False, "y_order": False},
        # routed rows over 32 experts with 4-bit weights, rows scattered back
        {"name": "mx4 experts bf16 act", "op": "mx4", "act": "bf16", "tokens": 2048, "top_k": 2, "experts": 32,
         "zipf": 0.9, "d_in": 4096, "d_out": 1024, "x_order": True, "y_order": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["group", "forward", "forward", "backward", "backward", "quantize", "mx4", "mx4"])
    if op == "group":
        top_k = rng.choice([1, 2, 4, 8])
        experts = max(top_k, _log(rng, 1, 256))
        return {"op": op, "tokens": _log(rng, 1, 32768), "top_k": top_k, "experts": experts,
                "zipf": rng.choice([0.0, 0.8, 1.1]), "dropped": rng.choice([0.0, 0.02, 0.3])}
    if op == "quantize":
        along = rng.choice(["cols", "rows"])
        rows, cols = _log(rng, 1, 14336), _log(rng, 32, 4096)
        if along == "cols":
            cols = 32 * max(1, cols // 32)
        else:
            rows, cols = 32 * max(1, rows // 32), 8 * max(1, cols // 8)
        return {"op": op, "dtype": rng.choice(["bf16", "fp32"]), "rows": rows, "cols": cols, "along": along}
    top_k = rng.choice([1, 1, 2, 4])
    experts = max(top_k, rng.choice([1, 2, 3, 5, 8, 16, 24, 64]))
    c = {"op": op, "top_k": top_k, "experts": experts, "zipf": rng.choice([0.0, 0.8, 1.1])}
    big = rng.random() < 0.3
    d_in, d_out = _log(rng, 64, 4096), _log(rng, 64, 14336 if big else 4096)
    tokens = _log(rng, 1, 16384 if big else 4096) // top_k + 1
    x_order = top_k > 1 or rng.random() < 0.5
    c.update(tokens=tokens, x_order=x_order, y_order=rng.random() < 0.5)
    if op == "mx4":
        c.update(act=rng.choice(["bf16", "mxfp4"]), d_in=128 * max(1, d_in // 128), d_out=8 * max(1, d_out // 8))
        return c
    fp32 = rng.random() < 0.3
    unit = 4 if fp32 else 8
    c.update(dtype="fp32" if fp32 else "bf16", layout=rng.choice(["kn", "nk"]), d_in=unit * (d_in // unit),
             d_out=unit * (d_out // unit))
    if fp32:
        c["tokens"] = min(tokens, 1024)
    if op == "backward":
        c["d_out"] = min(c["d_out"], 4096)
        w4 = not fp32 and rng.random() < 0.2
        if w4:
            c.update(layout="nk", d_in=128 * max(1, d_in // 128))
        c.update(w4=w4, tokens=min(c["tokens"], 4096))
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _probs(case):
    """Experts' shares: 1 / (rank + 1)^zipf."""
    p = [1.0 / (i + 1) ** case["zipf"] for i in range(case["experts"])]
    s = sum(p)
    return [v / s for v in p]


def _route(case, g):
    """Expert ids [tokens * top_k], the top_k of a token all different."""
    p = torch.tensor(_probs(case), device="cuda")
    p = p[torch.randperm(case["experts"], generator=g, device="cuda")]
    u = torch.rand((case["tokens"], case["experts"]), device="cuda", generator=g).clamp_min(1e-12)
    key = -torch.log(u) / p                      # the smallest keys: drawn without replacement
    ids = key.topk(case["top_k"], dim=1, largest=False).indices.reshape(-1).to(torch.int32)
    if case.get("dropped"):
        gone = torch.rand(ids.shape, device="cuda", generator=g) < case["dropped"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids


def _group_plain(ids, n):
    """offsets [n + 1] and order [rows]: a stable sort by id, ids outside [0, n) last and named -1."""
    key = torch.where((ids >= 0) & (ids < n), ids, torch.full_like(ids, n)).long()
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    edge = torch.arange(n + 1, device=ids.device)
    counts = (key[:, None] == edge[None, :n]).sum(0) if n <= 64 else torch.bincount(key, minlength=n + 1)[:n]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    at = torch.arange(ids.numel(), device=ids.device)
    order = torch.where(at < offsets[n], order, torch.full_like(order, -1))
    return offsets, order


def _state_rows(case, g):
    ids = _route(case, g)
    offsets, order = _group_plain(ids, case["experts"])
    return {"offsets": offsets, "order": order, "host": [int(v) for v in offsets.tolist()]}


def _mx4_weight(g, rows, cols):
    """Packed MXFP4 buffer (codes, then scales) of normal weights."""
    w = _rand(g, (rows, cols), torch.float32, 0.02)
    mags, shared = _quant_plain(w)
    return _pack(w, mags, shared)


def _pack(x, mags, shared):
    rows, cols = x.shape
    code = (2 * mags).clamp(max=4) + (mags > 2).float() + (mags > 3).float() + (mags > 4).float()
    # 0 .5 1 1.5 2 3 4 6 -> 0 1 2 3 4 5 6 7
    code = code.to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)
    pairs = code[:, 0::2] | (code[:, 1::2] << 4)
    return torch.cat([pairs.reshape(-1), (shared + 127).to(torch.uint8).reshape(-1)])


def _rows(case):
    return case["tokens"] * case["top_k"]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "group":
        s["ids"] = _route(case, g)
        if own:
            from adapter_lora_segments_amd import RowGroups
            s["groups"] = RowGroups(_rows(case), case["experts"])
        return s
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        x = _rand(g, (rows, cols), torch.float32, 0.02)
        x *= torch.exp2(_rand(g, (rows, 1), torch.float32, 1.5))      # rows of different sizes
        s["x"] = x.to(DT[case["dtype"]])
        if own:
            from adapter_lora_segments_amd import microscale_bytes
            s["q"] = torch.empty(microscale_bytes(rows, cols), dtype=torch.uint8, device="cuda")
            s["values"] = torch.empty_like(s["x"])
        return s
    s.update(_state_rows(case, g))
    R, E, di, do = _rows(case), case["experts"], case["d_in"], case["d_out"]
    dt = DT[case.get("dtype", "bf16")]
    w4 = op == "mx4" or case.get("w4", False)
    if w4:
        s["w"] = _mx4_weight(g, E * do, di)
    else:
        s["w"] = _rand(g, (E, di, do) if case["layout"] == "kn" else (E, do, di), dt, 0.02)
    if not (op == "backward" and w4):
        s["x"] = _rand(g, (case["tokens"] if case["x_order"] else R, di), dt)
    if op == "backward":
        s["dy"] = _rand(g, (R, do), dt)
    if own:
        from adapter_lora_segments_amd import ExpertLinear
        s["layer"] = ExpertLinear(s["w"], E, di, do, R, dtype=case.get("dtype", "bf16"),
                                  w_layout=case.get("layout", "nk"), w_format="mxfp4" if w4 else "bf16",
                                  act_format=case.get("act", "bf16"), top_k=case["top_k"],
                                  x_order=case["x_order"], y_order=case["y_order"])
    return s


# ---------------------------------------------------------------- plain form

def _pow2(e):
    """2^e in fp32 for integer e in the normal range, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quant_plain(x):
    """|element| values on the E2M1 grid and the shared exponents of blocks of 32 along the last axis."""
    rows, cols = x.shape
    b = x.float().reshape(rows, cols // 32, 32)
    amax = b.abs().amax(dim=2)
    _, ex = torch.frexp(amax)
    shared = torch.where(amax > 0, (ex - 1 - 2).clamp(-127, 127), torch.full_like(ex, -127))
    # two exact power-of-two factors: 2^-shared alone may pass fp32's range
    half = torch.div(shared, 2, rounding_mode="floor")
    a = b.abs() * _pow2(-half)[:, :, None] * _pow2(half - shared)[:, :, None]
    q = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return q.clamp(max=6.0).reshape(rows, cols), shared


def _scale_values(x, mags, shared):
    rows, cols = mags.shape
    half = torch.div(shared, 2, rounding_mode="floor")
    f = mags.reshape(rows, cols // 32, 32) * _pow2(half)[:, :, None] * _pow2(shared - half)[:, :, None]
    return torch.where(torch.signbit(x), -f.reshape(rows, cols), f.reshape(rows, cols))


def _decode_plain(buf, rows, cols, dtype=torch.float32):
    """Values of a packed MXFP4 buffer, [rows][cols]."""
    n = rows * cols // 2
    codes, sc = buf[:n].reshape(rows, cols // 2), buf[n:].reshape(rows, cols // 32)
    mags = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device=buf.device)
    mags = torch.cat([mags, -mags])
    v = torch.stack([mags[(codes & 15).long()], mags[(codes >> 4).long()]], dim=2).reshape(rows, cols // 32, 32)
    return (v * _pow2(sc.to(torch.int32) - 127).to(dtype)[:, :, None]).reshape(rows, cols)


def _products_plain(s, dtype, out_dtype, decode, quant=None):
    """forward and mx4: Y, rows outside every group zero."""
    c = s["case"]
    R, E, di, do = _rows(c), c["experts"], c["d_in"], c["d_out"]
    o, order = s["host"], s["order"].long()
    x = s["x"].to(dtype)
    if quant is not None:
        x = quant(s["x"]).to(dtype)
    y = torch.zeros((R, do), dtype=out_dtype, device="cuda")
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        if hi <= lo:
            continue
        idx = order[lo:hi]
        xe = x[torch.div(idx, c["top_k"], rounding_mode="floor")] if c["x_order"] else x[lo:hi]
        if c["op"] == "mx4":
            we = decode(_expert_buf(s["w"], E, do, di, e), do, di, dtype).t()
        else:
            we = s["w"][e].to(dtype)
            we = we if c["layout"] == "kn" else we.t()
        ye = (xe @ we).to(out_dtype)
        if c["y_order"]:
            y[idx] = ye
        else:
            y[lo:hi] = ye
    return y


def _expert_buf(buf, E, do, di, e):
    n = do * di
    return torch.cat([buf[e * n // 2:(e + 1) * n // 2], buf[E * n // 2 + e * n // 32:E * n // 2 + (e + 1) * n // 32]])


def _backward_plain(s, dtype, out_dtype, dw_dtype, decode):
    c = s["case"]
    R, E, di, do = _rows(c), c["experts"], c["d_in"], c["d_out"]
    o, order = s["host"], s["order"].long()
    dx = torch.zeros((R, di), dtype=out_dtype, device="cuda")
    dw = None
    if not c["w4"]:
        dw = torch.zeros((E, di, do) if c["layout"] == "kn" else (E, do, di), dtype=dw_dtype, device="cuda")
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        if hi <= lo:
            continue
        idx = order[lo:hi]
        dye = (s["dy"][idx] if c["y_order"] else s["dy"][lo:hi]).to(dtype)
        if c["w4"]:
            wt = decode(_expert_buf(s["w"], E, do, di, e), do, di, dtype)
        else:
            wt = s["w"][e].to(dtype)
            wt = wt.t() if c["layout"] == "kn" else wt
        dxe = (dye @ wt).to(out_dtype)
        if c["x_order"]:
            dx[idx] = dxe
        else:
            dx[lo:hi] = dxe
        if dw is not None:
            xe = s["x"][torch.div(idx, c["top_k"], rounding_mode="floor")] if c["x_order"] else s["x"][lo:hi]
            xe = xe.to(dtype)
            dw[e] = (xe.t() @ dye if c["layout"] == "kn" else dye.t() @ xe).to(dw_dtype)
    return {"dx": dx} if dw is None else {"dx": dx, "dw": dw}


def _run_plain(s):
    c, op = s["case"], s["op"]
    if op == "group":
        offsets, order = _group_plain(s["ids"], c["experts"])
        return {"offsets": offsets, "order": order}
    if op == "quantize":
        x = s["x"] if c["along"] == "cols" else s["x"].t().contiguous()
        v = _scale_values(x, *_quant_plain(x)).to(s["x"].dtype)
        return {"values": v if c["along"] == "cols" else v.t().contiguous()}
    if op == "forward":
        return {"y": _products_plain(s, torch.float32, DT[c["dtype"]], None)}
    if op == "backward":
        return _backward_plain(s, torch.float32, DT[c["dtype"]], torch.float32, _decode_plain)
    quant = (lambda x: _scale_values(x, *_quant_plain(x))) if c["act"] == "mxfp4" else None
    return {"y": _products_plain(s, torch.float32, torch.bfloat16, _decode_plain, quant)}


# ---------------------------------------------------------------- the framework's operators

def _run_own(s):
    from adapter_lora_segments_amd import mlora_microscale_quantize
    c, op = s["case"], s["op"]
    if op == "group":
        offsets, order = s["groups"].group(s["ids"])
        return {"offsets": offsets, "order": order}
    if op == "quantize":
        mlora_microscale_quantize(s["x"], s["q"], values=s["values"], along=c["along"])
        return {"values": s["values"]}
    layer = s["layer"]
    if op == "backward":
        dx = layer.backward(s["dy"], s.get("x"), s["offsets"], s["order"])
        return {"dx": dx} if c["w4"] else {"dx": dx, "dw": layer.dW}
    return {"y": layer.forward(s["x"], s["offsets"], s["order"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- work and exact values

def work(case):
    op = case["op"]
    if op == "group":
        return {"bytes": 8 * _rows(case) + 4 * (case["experts"] + 1), "flops": 0}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * (2 if case["dtype"] == "bf16" else 4) + 17 / 32), "flops": 0}
    R, E, di, do = _rows(case), case["experts"], case["d_in"], case["d_out"]
    sz = 4 if case.get("dtype") == "fp32" else 2
    active = sum(1 - (1 - p) ** R for p in _probs(case))
    w4 = op == "mx4" or case.get("w4", False)
    w = active * di * do * (17 / 32 if w4 else sz)
    x = (case["tokens"] if case["x_order"] else R) * di * sz
    if op == "backward":
        if w4:
            return {"bytes": w + R * (do + di) * sz, "flops": 2 * R * di * do}
        return {"bytes": w + x + R * (do + di) * sz + 4 * E * di * do, "flops": 4 * R * di * do}
    return {"bytes": w + x + R * do * sz, "flops": 2 * R * di * do}


def _two_to(e):
    """2^e in float64 for integer-valued e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid_values(x):
    """MXFP4 values of x (blocks along the last axis) in float64: each element takes the nearest of the grid's
    sixteen points, an equally near pair the one of even index."""
    rows, cols = x.shape
    b = x.double().reshape(-1, 32)
    amax = b.abs().amax(dim=1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    e = torch.where(_two_to(e) > amax, e - 1, e)
    e = torch.where(_two_to(e + 1) <= amax, e + 1, e) - 2
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))
    a = b.abs() / _two_to(e)
    pts = [0, .5, 1, 1.5, 2, 3, 4, 6]
    q = torch.zeros_like(a)
    for i in range(1, 8):
        mid = (pts[i - 1] + pts[i]) / 2
        q = torch.where((a > mid) | ((a == mid) & (i % 2 == 0)), torch.full_like(a, pts[i]), q)
    return (torch.sign(b) * q * _two_to(e)).reshape(rows, cols)


def exact(case, seed):
    op = case["op"]
    if op == "group":
        return None                    # whole numbers: nothing to round
    s = prepare(case, seed)
    if op == "quantize":
        if case["along"] == "cols":
            return {"values": _grid_values(s["x"])}
        return {"values": _grid_values(s["x"].t().contiguous()).t().contiguous()}
    R, E, di, do = _rows(case), case["experts"], case["d_in"], case["d_out"]
    order, o = s["order"].long(), s["host"]
    group = torch.bucketize(torch.arange(R, device="cuda"), s["offsets"][1:].long(), right=True)
    token = torch.div(order, case["top_k"], rounding_mode="floor")
    w4 = op == "mx4" or case.get("w4", False)

    def weight(e):                     # [d_in][d_out]
        if not w4:
            return s["w"][e].double() if case["layout"] == "kn" else s["w"][e].double().t()
        n = E * do * di // 2
        codes = s["w"][:n].reshape(E, do, di // 2)[e].int()
        sc = s["w"][n:].reshape(E, do, di // 32)[e].double()
        c = torch.empty((do, di), dtype=torch.int32, device="cuda")
        c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
        ex, man = ((c >> 1) & 3).double(), (c & 1).double()
        v = torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * _two_to(ex - 1))
        v = torch.where(c >= 8, -v, v)
        return (v * torch.repeat_interleave(_two_to(sc - 127), 32, dim=1)).t()

    if op == "backward":
        dx = torch.zeros((R, di), dtype=torch.float64, device="cuda")
        dw = []
        for e in range(E):
            at = torch.nonzero(group == e).reshape(-1)
            d = s["dy"][order[at] if case["y_order"] else at].double()
            dx[order[at] if case["x_order"] else at] = d @ weight(e).t()
            if not w4:
                x = s["x"][token[at] if case["x_order"] else at].double()
                dw.append(x.t() @ d if case["layout"] == "kn" else d.t() @ x)
        return {"dx": dx} if w4 else {"dx": dx, "dw": torch.stack(dw)}
    x = s["x"].double()
    if op == "mx4" and case["act"] == "mxfp4":
        x = _grid_values(s["x"])
    y = torch.zeros((R, do), dtype=torch.float64, device="cuda")
    for e in range(E):
        at = torch.nonzero(group == e).reshape(-1)
        y[order[at] if case["y_order"] else at] = x[token[at] if case["x_order"] else at] @ weight(e)
    return {"y": y}
