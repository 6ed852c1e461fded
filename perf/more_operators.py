"""What routing, combining and the 4-bit group-scaled products are measured on.

Every case is one call as a program that runs mixture-of-experts layers makes
it:

- ``route``: a router's logits to expert ids and weights: softmax or sigmoid
  scores, a bias for balance that only the choice sees, expert groups, the
  top_k of a token in falling order, renormalised weights;
- ``route_backward``: the gradient of the weights in the logits;
- ``combine``: the top_k expert rows of a token times their weights, summed
  into the token's row, a shared expert's output added;
- ``combine_backward``: the gradients of the rows and of the weights;
- ``int4``: the product with 4-bit codes, a scale and a zero point per group of
  inputs, one weight or one per expert, from a single row to a prefill;
- ``int4_backward``: its dX (the weight is frozen);
- ``int4_quantize``: a matrix to such codes, scales and zero points, with the
  decoded values.

With ``own`` false ``run`` computes the plain form in torch operations.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step's routing: 16 tokens, two of 64 experts each
        {"name": "route decode 16 of 64", "op": "route", "dtype": "bf16", "tokens": 16, "experts": 64, "top_k": 2,
         "score": "softmax", "groups": 1, "top_groups": 1, "group_score": "max", "bias": False, "renorm": True,
         "scale": 1.0, "masked": 0.0, "padded": 0},
        # a long prefill's: sigmoid scores with a balance bias, four of eight expert groups, eight experts a token
        {"name": "route prefill sigmoid 32768 of 256", "op": "route", "dtype": "fp32", "tokens": 32768, "experts": 256,
         "top_k": 8, "score": "sigmoid", "groups": 8, "top_groups": 4, "group_score": "top2", "bias": True,
         "renorm": True, "scale": 2.5, "masked": 0.0, "padded": 0},
        # a training step's: unnormalised softmax weights, so every logit has a gradient; rows of padding at the end
        {"name": "route backward softmax 16384 of 64", "op": "route_backward", "dtype": "bf16", "tokens": 16384,
         "experts": 64, "top_k": 8, "score": "softmax", "groups": 1, "top_groups": 1, "group_score": "max",
         "bias": False, "renorm": False, "scale": 1.0, "masked": 0.0, "padded": 200},
        # a decode step's expert rows back into 16 tokens, a shared expert's output added
        {"name": "combine decode 16", "op": "combine", "dtype": "bf16", "tokens": 16, "top_k": 2, "d": 4096,
         "weights": True, "add": True, "dropped": 0.0},
        # a long prefill's, some slots dropped
        {"name": "combine prefill 16384 x 8", "op": "combine", "dtype": "bf16", "tokens": 16384, "top_k": 8, "d": 4096,
         "weights": True, "add": False, "dropped": 0.02},
        # a training step's, an odd width
        {"name": "combine backward 7681 x 2", "op": "combine_backward", "dtype": "bf16", "tokens": 7681, "top_k": 2,
         "d": 4104, "weights": True, "dropped": 0.02},
        # single-token serving: one row against a 4-bit up projection
        {"name": "int4 one row", "op": "int4", "group": 128, "tokens": 1, "top_k": 1, "experts": 1, "zipf": 0.0,
         "d_in": 4096, "d_out": 14336, "x_order": False, "y_order": False},
        # a decode step of 16 tokens over eight experts, smaller groups
        {"name": "int4 decode experts", "op": "int4", "group": 64, "tokens": 16, "top_k": 2, "experts": 8, "zipf": 0.0,
         "d_in": 4096, "d_out": 4096, "x_order": True, "y_order": False},
        # routed rows of a short prefill over 32 experts, scattered back
        {"name": "int4 routed 4096 rows", "op": "int4", "group": 128, "tokens": 2048, "top_k": 2, "experts": 32,
         "zipf": 0.9, "d_in": 4096, "d_out": 1024, "x_order": True, "y_order": True},
        # a long prefill through one weight
        {"name": "int4 prefill 8192 rows", "op": "int4", "group": 128, "tokens": 8192, "top_k": 1, "experts": 1,
         "zipf": 0.0, "d_in": 4096, "d_out": 14336, "x_order": False, "y_order": False},
        # adapters trained over frozen 4-bit experts: the gradient that passes through
        {"name": "int4 backward 1501 rows", "op": "int4_backward", "group": 32, "tokens": 1501, "top_k": 1,
         "experts": 4, "zipf": 0.8, "d_in": 4096, "d_out": 4096, "x_order": False, "y_order": False},
        # a 14336 x 4096 weight quantized, decoded values kept
        {"name": "int4 quantize weight", "op": "int4_quantize", "dtype": "bf16", "group": 128, "symmetric": False,
         "rows": 14336, "cols": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "combine", "combine_backward", "int4", "int4", "int4",
                     "int4_backward", "int4_quantize"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        experts = groups * max(2, _log(rng, 1, 512) // groups)
        top_groups = rng.randint(1, groups)
        top_k = min(rng.choice([1, 2, 4, 6, 8]), experts // groups * top_groups)
        # a lone renormalised weight is constant: its gradient is zero, and what a plain form returns is rounding
        renorm = rng.random() < 0.6 and (op == "route" or top_k > 1)
        return {"op": op, "dtype": rng.choice(["bf16", "fp32"]), "tokens": _log(rng, 1, 16384), "experts": experts,
                "top_k": top_k, "score": rng.choice(["softmax", "sigmoid"]), "groups": groups,
                "top_groups": top_groups, "group_score": rng.choice(["max", "top2"]), "bias": rng.random() < 0.5,
                "renorm": renorm, "scale": rng.choice([1.0, 2.5]),
                "masked": rng.choice([0.0, 0.0, 0.1]) if experts // groups >= 8 else 0.0,
                "padded": rng.choice([0, 0, 3])}
    if op in ("combine", "combine_backward"):
        c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"]), "top_k": rng.choice([1, 2, 4, 6, 8]),
             "d": 8 * max(1, _log(rng, 8, 8192) // 8), "weights": rng.random() < 0.8,
             "dropped": rng.choice([0.0, 0.02, 0.3])}
        c["tokens"] = _log(rng, 1, 32768 // c["top_k"])
        if op == "combine":
            c["add"] = rng.random() < 0.5
        return c
    group = rng.choice([32, 64, 128])
    if op == "int4_quantize":
        return {"op": op, "dtype": rng.choice(["bf16", "fp32"]), "group": group, "symmetric": rng.random() < 0.3,
                "rows": _log(rng, 1, 14336), "cols": group * max(1, _log(rng, 32, 4096) // group)}
    top_k = rng.choice([1, 1, 2, 4])
    experts = max(top_k, rng.choice([1, 1, 2, 5, 8, 16, 32]))
    d_in, d_out = _log(rng, 64, 4096), _log(rng, 64, 14336 if experts < 8 else 4096)
    most = 4096 if rng.random() < 0.4 else 128
    x_order = top_k > 1 or rng.random() < 0.5
    return {"op": op, "group": group, "tokens": _log(rng, 1, most) // top_k + 1, "top_k": top_k, "experts": experts,
            "zipf": rng.choice([0.0, 0.8, 1.1]), "d_in": group * max(1, d_in // group), "d_out": 8 * max(1, d_out // 8),
            "x_order": x_order, "y_order": rng.random() < 0.5}


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


def _tables(case, g):
    """offsets and order of rows thrown at the experts, the top_k of a token all different."""
    p = torch.tensor(_probs(case), device="cuda")
    p = p[torch.randperm(case["experts"], generator=g, device="cuda")]
    u = torch.rand((case["tokens"], case["experts"]), device="cuda", generator=g).clamp_min(1e-12)
    ids = (-torch.log(u) / p).topk(case["top_k"], dim=1, largest=False).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices.to(torch.int32)
    counts = torch.bincount(ids, minlength=case["experts"])
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return {"offsets": offsets, "order": order, "host": [int(v) for v in offsets.tolist()]}


def _dropped_ids(case, g):
    """ids [tokens][top_k] of a router over 64 experts, a share of the slots dropped (-1)."""
    shape = (case["tokens"], case["top_k"])
    ids = torch.randint(0, 64, shape, generator=g, device="cuda", dtype=torch.int32)
    gone = torch.rand(shape, device="cuda", generator=g) < case["dropped"]
    return torch.where(gone, torch.full_like(ids, -1), ids)


def _rows(case):
    return case["tokens"] * case["top_k"]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("route", "route_backward"):
        T, E = case["tokens"], case["experts"]
        logits = _rand(g, (T, E), torch.float32, 1.5)
        if case["masked"]:                           # experts that this token may not take
            logits.masked_fill_(torch.rand((T, E), device="cuda", generator=g) < case["masked"], -math.inf)
        if case["padded"]:                           # rows of padding: nothing may be taken
            logits[max(0, T - case["padded"]):] = -math.inf
        s["logits"] = logits.to(DT[case["dtype"]])
        s["bias"] = _rand(g, (E,), torch.float32, 0.1) if case["bias"] else None
        if op == "route_backward":
            s["ids"] = _choose_plain(case, _scores_plain(case, s["logits"]), s["logits"], s["bias"]).to(torch.int32)
            s["dweights"] = _rand(g, (T, case["top_k"]), torch.float32)
        if own:
            from adapter_lora_segments_amd import Router
            s["router"] = Router(E, case["top_k"], score=case["score"], expert_groups=case["groups"],
                                 top_groups=case["top_groups"], group_score=case["group_score"],
                                 renormalize=case["renorm"], scale=case["scale"])
        return s
    if op in ("combine", "combine_backward"):
        T, k, d, dt = case["tokens"], case["top_k"], case["d"], DT[case["dtype"]]
        s["y"] = _rand(g, (T * k, d), dt)
        s["ids"] = _dropped_ids(case, g) if case["dropped"] else None
        s["weights"] = torch.rand((T, k), device="cuda", generator=g) if case["weights"] else None
        if op == "combine":
            s["add"] = _rand(g, (T, d), dt) if case["add"] else None
        else:
            s["dout"] = _rand(g, (T, d), dt)
        return s
    if op == "int4_quantize":
        x = _rand(g, (case["rows"], case["cols"]), torch.float32, 0.02)
        x *= torch.exp2(_rand(g, (case["rows"], 1), torch.float32, 1.5))      # rows of different sizes
        s["x"] = x.to(DT[case["dtype"]])
        if own:
            from adapter_lora_segments_amd import affine_bytes
            s["q"] = torch.empty(affine_bytes(case["rows"], case["cols"], case["group"]), dtype=torch.uint8,
                                 device="cuda")
            s["values"] = torch.empty_like(s["x"])
        return s
    s.update(_tables(case, g))
    R, E, di, do = _rows(case), case["experts"], case["d_in"], case["d_out"]
    s["w"] = _int4_weight(g, E * do, di, case["group"])
    if op == "int4":
        s["x"] = _rand(g, (case["tokens"] if case["x_order"] else R, di), torch.bfloat16)
    else:
        s["dy"] = _rand(g, (R, do), torch.bfloat16)
    if own:
        from adapter_lora_segments_amd import AffineLinear
        s["layer"] = AffineLinear(s["w"], E, di, do, R, group=case["group"], top_k=case["top_k"],
                                x_order=case["x_order"], y_order=case["y_order"])
    return s


def _int4_weight(g, rows, cols, group):
    """Packed buffer (codes, then a zero point and a scale per group) of normal weights."""
    codes, zero, scale = _quant_plain(_rand(g, (rows, cols), torch.float32, 0.02), group, False)
    c = codes.reshape(rows, cols).to(torch.uint8)
    pairs = c[:, 0::2] | (c[:, 1::2] << 4)
    params = torch.stack([zero, scale], dim=-1).to(torch.bfloat16).contiguous().view(torch.uint8)
    return torch.cat([pairs.reshape(-1), params.reshape(-1)])


# ---------------------------------------------------------------- plain form

def _scores_plain(case, logits):
    """Scores in 64 bits: what the choice rounds to 32 lies next to borders. Experts at -inf score 0."""
    x = logits.double()
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _choose_plain(case, scores, logits, bias):
    """ids [tokens][top_k] in falling order of score + bias in fp32, ties to the lowest; -1 where nothing is left."""
    c = scores.float()
    if bias is not None:
        c = c + bias
    c = torch.where(logits == -math.inf, torch.full_like(c, -math.inf), c)
    G = case["groups"]
    if G > 1:
        per = case["experts"] // G
        best = torch.sort(c.reshape(-1, G, per), dim=2, descending=True).values
        of = best[:, :, 0]
        if case["group_score"] == "top2" and per > 1:
            of = torch.where(best[:, :, 1] == -math.inf, of, of + best[:, :, 1])
        taken = torch.sort(of, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros_like(of, dtype=torch.bool).scatter_(1, taken, True)
        c = torch.where(keep.repeat_interleave(per, dim=1), c, torch.full_like(c, -math.inf))
    value, at = torch.sort(c, dim=1, descending=True, stable=True)
    k = case["top_k"]
    return torch.where(value[:, :k] == -math.inf, torch.full_like(at[:, :k], -1), at[:, :k])


def _route_plain(s):
    c = s["case"]
    scores = _scores_plain(c, s["logits"])
    ids = _choose_plain(c, scores, s["logits"], s["bias"])
    u = torch.where(ids < 0, torch.zeros((), dtype=scores.dtype, device="cuda"), scores.gather(1, ids.clamp_min(0)))
    if c["renorm"]:
        total = u.sum(dim=1, keepdim=True)
        u = u / torch.where(total == 0, torch.ones_like(total), total)
    return {"ids": ids.to(torch.int32), "weights": (u * c["scale"]).float()}


def _route_backward_plain(s):
    c = s["case"]
    x, ids, on = s["logits"].float(), s["ids"].long().clamp_min(0), s["ids"] >= 0
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(dim=1, keepdim=True)
        e = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        total = e.sum(dim=1, keepdim=True)
        p = e / torch.where(total == 0, torch.ones_like(total), total)
    u = torch.where(on, p.gather(1, ids), torch.zeros((), device="cuda"))
    du = torch.where(on, s["dweights"] * c["scale"], torch.zeros((), device="cuda"))
    if c["renorm"]:
        total = u.sum(dim=1, keepdim=True)
        total = torch.where(total == 0, torch.ones_like(total), total)
        du = torch.where(on, (du - (du * u).sum(dim=1, keepdim=True) / total) / total, du)
    dp = torch.zeros_like(p).scatter_add_(1, ids, du)
    if c["score"] == "sigmoid":
        dx = dp * p * (1 - p)
    else:
        dx = p * (dp - (du * u).sum(dim=1, keepdim=True))
    return {"dlogits": dx.to(s["logits"].dtype)}


def _combine_plain(s):
    c = s["case"]
    T, k = c["tokens"], c["top_k"]
    y = s["y"].float().reshape(T, k, c["d"])
    if s["weights"] is not None:
        y = y * s["weights"][:, :, None]
    if s["ids"] is not None:
        y = torch.where((s["ids"] >= 0)[:, :, None], y, torch.zeros((), device="cuda"))
    out = y.sum(dim=1)
    if s["add"] is not None:
        out = out + s["add"].float()
    return {"out": out.to(s["y"].dtype)}


def _combine_backward_plain(s):
    c = s["case"]
    T, k = c["tokens"], c["top_k"]
    dout = s["dout"].float()[:, None, :]
    on = torch.ones((T, k), dtype=torch.bool, device="cuda") if s["ids"] is None else s["ids"] >= 0
    w = on.float() if s["weights"] is None else torch.where(on, s["weights"], torch.zeros((), device="cuda"))
    r = {"dy": (dout * w[:, :, None]).to(s["y"].dtype).reshape(T * k, c["d"])}
    if s["weights"] is not None:
        dot = (dout * s["y"].float().reshape(T, k, c["d"])).sum(dim=2)
        r["dweights"] = torch.where(on, dot, torch.zeros((), device="cuda"))
    return r


def _quant_plain(x, group, symmetric):
    """codes [rows][groups][group], zero points and scales [rows][groups] in fp32 (bf16 values), steps in fp32."""
    rows, cols = x.shape
    b = x.float().reshape(rows, cols // group, group)
    if symmetric:
        seven = torch.full((), 7.0, device=x.device)
        scale = (b.abs().amax(dim=2) / seven).to(torch.bfloat16).float()
        zero = torch.full_like(scale, 8.0)
    else:
        n = torch.full((), 15.0, device=x.device)
        lo, hi = b.amin(dim=2).clamp_max(0), b.amax(dim=2).clamp_min(0)
        scale = (hi / n - lo / n).to(torch.bfloat16).float()
        by = torch.where(scale == 0, torch.ones_like(scale), scale)
        zero = torch.round(-lo / by).clamp(0, 15)
    by = torch.where(scale == 0, torch.ones_like(scale), scale)
    codes = (torch.round(b / by[:, :, None]) + zero[:, :, None]).clamp(0, 15)
    return codes, zero, scale


def _decode_plain(buf, rows, cols, group, first, count):
    """fp32 values of rows first .. first + count - 1 of a packed buffer of [rows][cols] weights."""
    n = rows * cols // 2
    codes = buf[:n].reshape(rows, cols // 2)[first:first + count]
    zs = buf[n:].view(torch.bfloat16).reshape(rows, cols // group, 2)[first:first + count].float()
    v = torch.stack([codes & 15, codes >> 4], dim=2).reshape(count, cols // group, group).float()
    return ((v - zs[:, :, :1]) * zs[:, :, 1:]).reshape(count, cols)


def _int4_plain(s, transposed):
    """Y = X W_e^T (or dX = dY W_e) over the groups' rows; rows outside every group zero."""
    c = s["case"]
    R, E, di, do = _rows(c), c["experts"], c["d_in"], c["d_out"]
    o, order = s["host"], s["order"].long()
    out = torch.zeros((R, di if transposed else do), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        lo, hi = o[e], o[e + 1]
        if hi <= lo:
            continue
        w, idx = _decode_plain(s["w"], E * do, di, c["group"], e * do, do), order[lo:hi]
        if transposed:
            v = (s["dy"][idx] if c["y_order"] else s["dy"][lo:hi]).float() @ w
            scatter = c["x_order"]
        else:
            x = s["x"][torch.div(idx, c["top_k"], rounding_mode="floor")] if c["x_order"] else s["x"][lo:hi]
            v = x.float() @ w.t()
            scatter = c["y_order"]
        if scatter:
            out[idx] = v.to(torch.bfloat16)
        else:
            out[lo:hi] = v.to(torch.bfloat16)
    return {"dx" if transposed else "y": out}


def _run_plain(s):
    c, op = s["case"], s["op"]
    if op == "route":
        return _route_plain(s)
    if op == "route_backward":
        return _route_backward_plain(s)
    if op == "combine":
        return _combine_plain(s)
    if op == "combine_backward":
        return _combine_backward_plain(s)
    if op == "int4_quantize":
        codes, zero, scale = _quant_plain(s["x"], c["group"], c["symmetric"])
        v = (codes - zero[:, :, None]) * scale[:, :, None]
        return {"values": v.reshape(s["x"].shape).to(s["x"].dtype)}
    return _int4_plain(s, op == "int4_backward")


# ---------------------------------------------------------------- the framework's operators

def _run_own(s):
    import adapter_lora_segments_amd as m
    c, op = s["case"], s["op"]
    if op == "route":
        ids, weights = s["router"].route(s["logits"], s["bias"])
        return {"ids": ids, "weights": weights}
    if op == "route_backward":
        return {"dlogits": s["router"].backward(s["logits"], s["ids"], s["dweights"])}
    if op == "combine":
        return {"out": m.mlora_combine(s["y"], c["top_k"], s["ids"], s["weights"], add=s["add"])}
    if op == "combine_backward":
        dy, dw = m.mlora_combine_backward(s["dout"], s["y"], c["top_k"], s["ids"], s["weights"])
        return {"dy": dy} if dw is None else {"dy": dy, "dweights": dw}
    if op == "int4_quantize":
        m.mlora_affine_quantize(s["x"], s["q"], values=s["values"], group=c["group"], symmetric=c["symmetric"])
        return {"values": s["values"]}
    if op == "int4_backward":
        return {"dx": s["layer"].backward(s["dy"], s["offsets"], s["order"])}
    return {"y": s["layer"].forward(s["x"], s["offsets"], s["order"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- work and exact values

def work(case):
    op = case["op"]
    sz = 4 if case.get("dtype") == "fp32" else 2
    if op in ("route", "route_backward"):
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        if op == "route":
            return {"bytes": T * E * sz + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 0}
        # scores of the chosen alone enter a sigmoid's gradient and a renormalised softmax's
        read = T * k if case["score"] == "sigmoid" or case["renorm"] else T * E
        return {"bytes": (read + T * E) * sz + 8 * T * k, "flops": 0}
    if op in ("combine", "combine_backward"):
        T, k, d = case["tokens"], case["top_k"], case["d"]
        kept = T * k * (1 - case["dropped"]) * d * sz
        small = T * k * ((4 if case["weights"] else 0) + (4 if case["dropped"] else 0))
        if op == "combine":
            return {"bytes": kept + T * d * sz * (2 if case["add"] else 1) + small, "flops": 0}
        read = kept if case["weights"] else 0
        return {"bytes": read + T * d * sz + T * k * d * sz + small + (4 * T * k if case["weights"] else 0), "flops": 0}
    if op == "int4_quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * sz + 0.5 + 4 / case["group"]), "flops": 0}
    R, E, di, do = _rows(case), case["experts"], case["d_in"], case["d_out"]
    active = sum(1 - (1 - p) ** R for p in _probs(case))
    w = active * di * do * (0.5 + 4 / case["group"])
    x = (case["tokens"] if case["x_order"] and op == "int4" else R) * di * 2
    return {"bytes": w + x + R * do * 2, "flops": 2 * R * di * do}


def _exact_scores(case, x):
    if case["score"] == "sigmoid":
        return torch.sigmoid(x)
    off = (x == -math.inf).all(dim=1, keepdim=True)
    return torch.where(off, torch.zeros_like(x), torch.softmax(torch.where(off, torch.zeros_like(x), x), dim=1))


def _exact_ids(case, p, x, bias):
    """The choice by whole-number keys, all different: (score + bias) as ordered bits, then the index from behind."""
    E = case["experts"]
    c = (p.float() if bias is None else p.float() + bias) + 0.0
    b = c.contiguous().view(torch.int32).long()
    key = torch.where(b < 0, -1 - (b & 0x7fffffff), b)                        # rises with c
    key = key * 8192 + (8191 - torch.arange(E, device="cuda"))
    out = -(1 << 60)
    key = torch.where(x == -math.inf, torch.full_like(key, out), key)
    G = case["groups"]
    if G > 1:
        per = E // G
        two = torch.topk(torch.where(x == -math.inf, -math.inf, c).reshape(-1, G, per), min(2, per), dim=2).values
        of = two[:, :, 0]
        if case["group_score"] == "top2" and per > 1:
            of = torch.where(torch.isinf(two[:, :, 1]), of, two[:, :, 0] + two[:, :, 1])
        g = torch.arange(G, device="cuda")
        ahead = (of[:, None, :] > of[:, :, None]) | ((of[:, None, :] == of[:, :, None]) & (g[None, None, :] < g[None, :, None]))
        keep = ahead.sum(dim=2) < case["top_groups"]
        key = torch.where(keep[:, :, None].expand(-1, G, per).reshape(-1, E), key, torch.full_like(key, out))
    v, at = torch.topk(key, case["top_k"], dim=1)
    return torch.where(v == out, torch.full_like(at, -1), at)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("route", "route_backward"):
        x = s["logits"].double()
        p = _exact_scores(case, x)
        ids = _exact_ids(case, p, x, s["bias"]) if op == "route" else s["ids"].long()
        hit = torch.zeros_like(p).scatter_add_(1, ids.clamp_min(0), (ids >= 0).double())     # 1 where chosen
        total = (p * hit).sum(dim=1, keepdim=True)
        some = total > 0
        safe = torch.where(some, total, torch.ones_like(total))
        if op == "route":
            w = p / safe if case["renorm"] else p
            w = w.gather(1, ids.clamp_min(0)) * (ids >= 0) * case["scale"]
            return {"ids": None, "weights": w}
        dw = torch.zeros_like(p).scatter_add_(1, ids.clamp_min(0), s["dweights"].double() * (ids >= 0)) * case["scale"]
        if case["renorm"]:       # w = p / sum of chosen p
            dp = hit * (dw - (dw * p).sum(dim=1, keepdim=True) / safe) / safe
        else:
            dp = dw
        inner = p * dp
        if case["score"] == "sigmoid":
            return {"dlogits": inner * torch.sigmoid(-x)}
        return {"dlogits": inner - p * inner.sum(dim=1, keepdim=True)}
    if op in ("combine", "combine_backward"):
        T, k, d = case["tokens"], case["top_k"], case["d"]
        w = torch.ones((T, k), dtype=torch.float64, device="cuda") if s["weights"] is None else s["weights"].double()
        if s["ids"] is not None:
            w = w * (s["ids"] >= 0)
        if op == "combine":
            out = torch.zeros((T, d), dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()
            for j in range(k):
                out = out + w[:, j:j + 1] * s["y"][j::k].double()
            return {"out": out}
        g = s["dout"].double()
        r = {"dy": torch.stack([w[:, j:j + 1] * g for j in range(k)], dim=1).reshape(T * k, d)}
        if s["weights"] is not None:
            dots = torch.stack([(g * s["y"][j::k].double()).sum(dim=1) for j in range(k)], dim=1)
            r["dweights"] = dots if s["ids"] is None else dots * (s["ids"] >= 0)
        return r
    if op == "int4_quantize":
        G = case["group"]
        x = s["x"].double().reshape(-1, G)
        if case["symmetric"]:
            scale, lo = x.abs().amax(dim=1) / 7, None
        else:
            lo = torch.minimum(x.amin(dim=1), torch.zeros((), dtype=torch.float64, device="cuda"))
            scale = (torch.maximum(x.amax(dim=1), torch.zeros((), dtype=torch.float64, device="cuda")) - lo) / 15
        scale = scale.float().to(torch.bfloat16).double()
        safe = torch.where(scale > 0, scale, torch.ones_like(scale))
        z = torch.full_like(scale, 8.0) if case["symmetric"] else torch.clamp(torch.round(-lo / safe), 0, 15)
        step = torch.clamp(torch.round(x / safe[:, None]), -z[:, None], (15 - z)[:, None])
        return {"values": (step * scale[:, None]).reshape(s["x"].shape)}
    R, E, di, do, G = _rows(case), case["experts"], case["d_in"], case["d_out"], case["group"]
    order = s["order"].long()
    group = torch.bucketize(torch.arange(R, device="cuda"), s["offsets"][1:].long(), right=True)
    n = E * do * di // 2
    params = s["w"][n:].view(torch.bfloat16).reshape(E, do, di // G, 2)

    def weight(e):                     # [d_out][d_in]
        b = s["w"][:n].reshape(E, do, di // 2)[e].to(torch.int16)
        c = torch.empty((do, di), dtype=torch.float64, device="cuda")
        c[:, 0::2], c[:, 1::2] = (b % 16).double(), torch.div(b, 16, rounding_mode="floor").double()
        z, sc = params[e, :, :, 0].double(), params[e, :, :, 1].double()
        return c * sc.repeat_interleave(G, dim=1) - (z * sc).repeat_interleave(G, dim=1)

    back = op == "int4_backward"
    out = torch.zeros((R, di if back else do), dtype=torch.float64, device="cuda")
    for e in range(E):
        at = torch.nonzero(group == e).reshape(-1)
        if back:
            v = s["dy"][order[at] if case["y_order"] else at].double() @ weight(e)
            out[order[at] if case["x_order"] else at] = v
        else:
            rows = torch.div(order[at], case["top_k"], rounding_mode="floor") if case["x_order"] else at
            out[order[at] if case["y_order"] else at] = s["x"][rows].double() @ weight(e).t()
    return {"dx" if back else "y": out}
