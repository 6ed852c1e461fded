"""A mixture-of-experts block as it is used: routing, grouping, products with
4-bit or bf16 weights, combining and the way back, against float64; the same
captured in a HIP graph; on a given stream; on two streams at once."""
import numpy as np
import pytest

from oracle import affine as oa
from oracle import experts as ox
from tests.gpu_harness import say

pytestmark = pytest.mark.gpu

SPIN = 100_000_000        # clock cycles: tens of milliseconds on the current stream


def n64(t):
    return t.detach().double().cpu().numpy()


class Block:
    """X -> router -> up -> ReLU -> down -> weighted sum, and back to X."""

    def __init__(self, T, E, k, di, dh, bits4=True, group=64, seed=0, **router):
        import torch
        from adapter_lora_segments_amd import AffineLinear, ExpertLinear, Router, RowGroups, mlora_affine_quantize
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.E, self.k, self.di, self.dh, self.bits4 = T, E, k, di, dh, bits4
        self.router = Router(E, k, **router)
        self.groups = RowGroups(T * k, E)
        w = lambda n, m: (torch.randn((E * n, m), generator=g, device="cuda") * m ** -0.5).to(torch.bfloat16)
        Wu, Wd = w(dh, di), w(di, dh)
        up, down = dict(top_k=k, x_order=True), dict(y_order=True)
        if bits4:
            Vu, Vd = torch.empty_like(Wu), torch.empty_like(Wd)
            self.up = AffineLinear(mlora_affine_quantize(Wu, values=Vu, group=group), E, di, dh, T * k, group=group, **up)
            self.down = AffineLinear(mlora_affine_quantize(Wd, values=Vd, group=group), E, dh, di, T * k, group=group, **down)
            # the weights that the products use are s (c - z), not yet rounded to bf16
            f = lambda q, n, m: oa.decode(*oa.unpack(q.cpu().numpy(), E * n, m, group)).reshape(E, n, m).transpose(0, 2, 1)
            self.Wu, self.Wd = f(self.up.q, dh, di), f(self.down.q, di, dh)
        else:
            self.up = ExpertLinear(Wu.view(E, dh, di), E, di, dh, T * k, w_layout="nk", **up)
            self.down = ExpertLinear(Wd.view(E, di, dh), E, dh, di, T * k, w_layout="nk", **down)
            self.Wu, self.Wd = (n64(v).reshape(E, n, m).transpose(0, 2, 1) for v, n, m in ((Wu, dh, di), (Wd, di, dh)))

    def inputs(self, dt=None):
        import torch
        r = lambda *s: torch.randn(s, generator=self.g, device="cuda")
        return (r(self.T, self.di).to(torch.bfloat16), r(self.T, self.E).to(dt or torch.float32),
                r(self.E) * 0.1, r(self.T, self.di).to(torch.bfloat16))

    def _back(self, L, dy, x, off, order):
        if self.bits4:
            return L.backward(dy, off, order)
        return L.backward(dy, x, off, order)

    def step(self, X, logits, bias, dout):
        """Every tensor on the way."""
        from adapter_lora_segments_amd import mlora_combine, mlora_combine_backward
        ids, w = self.router.route(logits, bias)
        off, order = self.groups.group(ids.view(-1))
        h = self.up.forward(X, off, order)
        a = h.clamp_min(0)
        y = self.down.forward(a, off, order)
        out = mlora_combine(y, self.k, ids, w, add=X, n_experts=self.E)
        dy, dw = mlora_combine_backward(dout, y, self.k, ids, w, n_experts=self.E)
        da = self._back(self.down, dy, a, off, order)
        dh = da * (h > 0)
        dx = mlora_combine(self._back(self.up, dh, X, off, order), self.k, ids, None, add=dout, n_experts=self.E)
        dl = self.router.backward(logits, ids, dw)
        return dict(ids=ids, w=w, off=off, order=order, h=h, a=a, y=y, out=out, dy=dy, dw=dw, da=da, dh=dh, dx=dx, dl=dl)


KINDS = [dict(bits4=True, score="sigmoid", expert_groups=4, top_groups=2, group_score="top2", scale=2.5),
         dict(bits4=True, score="softmax"), dict(bits4=False, score="softmax", renormalize=False)]


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("T", [1, 5, 300])
def test_block(T, kind):
    """Each step's output within its own rounding of the oracle's on the inputs
    that the step was given.  Of a product over 4-bit weights that is 2^-8 of the
    sum of magnitudes, S: the weights' rounding to bf16 where they are rounded,
    and more than the sums' own error where the codes are multiplied as they
    are ((64 + 5 + 16) 2^-23 of sum |x| 128 |s| 2.2, which is 0.003 sum |x| |s|,
    below 2^-8 S wherever the codes are three quarters of a step off the zero
    point on average)."""
    import torch
    E, k, di, dh = 16, 4, 128, 320
    say(f"moe block {T} {kind}")
    b = Block(T, E, k, di, dh, **KINDS[kind])
    X, logits, bias, dout = b.inputs()
    r = b.step(X, logits, bias, dout)
    off, order = r["off"].cpu().numpy(), r["order"].cpu().numpy()
    ids = r["ids"].cpu().numpy()
    assert (np.sort(ids, axis=1)[:, 1:] != np.sort(ids, axis=1)[:, :-1]).all() and (ids >= 0).all()
    assert np.array_equal(order, ox.group_rows(ids.reshape(-1), E)[1])
    N = T * k
    eps = 2.0 ** -8

    def near(got, want, S, n, name, wround=eps if b.bits4 else 0):
        bound = eps * np.abs(want) + (wround + (n + 8) * 2.0 ** -23) * S * 1.01
        assert (np.abs(n64(got) - want) <= bound).all(), name

    def slots(v):                                     # the sum over a token's slots
        return v.reshape(T, k, -1).sum(1)

    want, S, _ = ox.forward(n64(X), b.Wu, off, order, N, top_k=k, x_order=True)
    near(r["h"], want, S, di, "h")
    want, S, _ = ox.forward(n64(r["a"]), b.Wd, off, order, N, y_order=True)
    near(r["y"], want, S, dh, "y")
    w, y = n64(r["w"]), n64(r["y"])
    terms = y.reshape(T, k, di) * w[:, :, None]
    near(r["out"], n64(X) + terms.sum(1), np.abs(n64(X)) + np.abs(terms).sum(1), k, "out", 0)
    want = (n64(dout)[:, None] * w[:, :, None]).reshape(N, di)
    near(r["dy"], want, np.abs(want), 0, "dy", 0)
    t = n64(dout)[:, None] * y.reshape(T, k, di)
    err = np.abs(n64(r["dw"]) - t.sum(2))
    assert (err <= (di + 2) * 2.0 ** -23 * np.abs(t).sum(2)).all()
    want, S, _, _, _ = ox.backward(n64(r["dy"]), None, b.Wd, off, order, N, y_order=True)
    near(r["da"], want, S, di, "da")
    # each slot is rounded once, their sum and dout's once more
    want, S, _, _, _ = ox.backward(n64(r["dh"]), None, b.Wu, off, order, N, top_k=k, x_order=True)
    wr = eps if b.bits4 else 0
    slot_err = eps * np.abs(want) + (wr + (dh + 8) * 2.0 ** -23) * S
    total = n64(dout) + slots(want)
    bound = (slots(slot_err) + eps * np.abs(total)) * 1.01 + 8 * 2.0 ** -23 * (np.abs(n64(dout)) + slots(np.abs(want)))
    assert (np.abs(n64(r["dx"]) - total) <= bound).all()
    assert r["dl"].shape == (T, E) and torch.isfinite(r["dl"]).all()


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("T", [3, 150, 1100])
def test_captured_block(T, kind):
    """The whole step in one captured graph, replayed over new inputs with eager
    work between: every replay equals the eager step bit for bit.  With 1100
    tokens over two experts the weights are decoded first."""
    import torch
    E, k = (2, 2) if T == 1100 else (8, 2)
    opts = dict(KINDS[kind])
    if "expert_groups" in opts and E == 2:
        opts.update(expert_groups=1, top_groups=1)
    say(f"captured moe block {T} {kind}")
    cap, eager = (Block(T, E, k, 128, 320, seed=4, **opts) for _ in range(2))
    if cap.bits4:
        assert bool(cap.up.shape.forward_workspace_bytes) == (T == 1100)
    X, logits, bias, dout = ins = cap.inputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cap.step(*ins)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cap.step(*ins)
    for i in range(4):
        for t, v in zip(ins, cap.inputs()):
            t.copy_(v)
        graph.replay()
        want = eager.step(*ins)
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(out[name], want[name]), (i, name)


@pytest.mark.parametrize("T", [20, 1100])
def test_captured_quantizer_feeds_products(T):
    """New weights quantized and multiplied inside one graph."""
    import torch
    from adapter_lora_segments_amd import AffineLinear, affine_bytes, mlora_affine_quantize
    di, do = 256, 136
    W, X = torch.empty(do, di, device="cuda"), torch.empty(T, di, dtype=torch.bfloat16, device="cuda")
    qs = [torch.zeros(affine_bytes(do, di, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    L = [AffineLinear(q, 1, di, do, T, group=64) for q in qs]

    def step(i):
        mlora_affine_quantize(W, q=qs[i], group=64)
        y = L[i].forward(X)
        return y, L[i].backward(y)

    g = torch.Generator(device="cuda").manual_seed(3)
    fill = lambda: (W.normal_(generator=g), X.normal_(generator=g))
    fill()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(0)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(0)
    for i in range(4):
        fill()
        graph.replay()
        want = step(1)
        torch.cuda.synchronize()
        assert torch.equal(qs[0], qs[1]) and all(torch.equal(a, b) for a, b in zip(out, want))


def calls_of(b, ins, r, W):
    """{name: a call on a given stream whose outputs are its own}"""
    from adapter_lora_segments_amd import mlora_affine_quantize, mlora_combine, mlora_combine_backward
    X, logits, bias, dout = ins
    one = lambda t: t if isinstance(t, tuple) else (t,)
    k, E = b.k, b.E
    return {name: (lambda s, f=f: one(f(s))) for name, f in {
        "route": lambda s: b.router.route(logits, bias, stream=s),
        "route backward": lambda s: b.router.backward(logits, r["ids"], r["dw"], stream=s),
        "combine": lambda s: mlora_combine(r["y"], k, r["ids"], r["w"], add=X, n_experts=E, stream=s),
        "combine backward": lambda s: mlora_combine_backward(dout, r["y"], k, r["ids"], r["w"], n_experts=E, stream=s),
        "forward": lambda s: b.up.forward(X, r["off"], r["order"], stream=s),
        "forward, zeroed": lambda s: b.down.forward(r["a"], r["off"], r["order"], stream=s),
        "backward": lambda s: b.down.backward(r["dy"], r["off"], r["order"], stream=s),
        "backward, zeroed": lambda s: b.up.backward(r["dh"], r["off"], r["order"], stream=s),
        "quantize": lambda s: mlora_affine_quantize(W, group=64, stream=s)}.items()}


@pytest.mark.parametrize("T", [40, 1100])
def test_outputs_made_on_a_given_stream(T):
    """While the current stream is busy: the sequential results, made of memory
    that the current stream does not still use."""
    import torch
    say(f"given stream {T}")
    b = Block(T, 2, 2, 128, 320)
    ins = b.inputs()
    r = b.step(*ins)
    W = torch.randn(264, 256, device="cuda")
    calls = calls_of(b, ins, r, W)
    s = torch.cuda.Stream()
    for name, call in calls.items():
        say(f"  {name}")
        want = call(None)
        s.wait_stream(torch.cuda.current_stream())
        held = [torch.full_like(t, 7) for t in want]
        copies = [torch.empty_like(t) for t in held]
        torch.cuda.synchronize()
        torch.cuda._sleep(SPIN)
        for c, h in zip(copies, held):
            c.copy_(h)
        del h, held                                   # freed to the current stream, which has yet to read them
        got = call(s)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), name
        assert all((c == 7).all() for c in copies), name


@pytest.mark.parametrize("T", [5, 300, 1100])
def test_steps_on_two_streams(T):
    """The same layers on two streams at once: each call's workspace is its own."""
    import torch
    say(f"two streams {T}")
    b = Block(T, 2, 2, 128, 320)
    ins = [b.inputs(), b.inputs()]
    r = [b.step(*i) for i in ins]
    calls = [calls_of(b, i, x, torch.randn(264, 256, device="cuda")) for i, x in zip(ins, r)]
    want = [{n: f(None) for n, f in c.items()} for c in calls]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    out = [[], []]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                out[i].append({n: f(None) for n, f in calls[i].items()})
    torch.cuda.synchronize()
    for i in range(2):
        for o in out[i]:
            for n in o:
                assert all(torch.equal(x, y) for x, y in zip(o[n], want[i][n])), n
