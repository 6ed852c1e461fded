"""Grouped expert products, row grouping and MXFP4 quantization on the GPU
against the float64 oracle (oracle/experts.py).

Tolerances, per element.  A sum of K products in fp32 in any order is off by
at most K 2^-23 times the sum S of the products' magnitudes (each of the K
additions rounds once or truncates: at most 2^-23 of a partial sum, which is at
most S; products of bf16 or E2M1 values are exact in fp32, fp32 products add
one rounding of 2^-24 each).  The result is rounded once: half a step, 2^-8 of
a bf16 value, 2^-24 of an fp32 value.  So |got - exact| <= half |exact|
+ (K + 2) 2^-23 S (1 + 2^-8).  Integer results and quantized values are equal."""
import numpy as np
import pytest

from oracle import experts as ox
from tests.gpu_harness import say

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _t(dt):
    import torch
    return torch.bfloat16 if dt == "bf16" else torch.float32


def check(got, want, S, K, dt, what=""):
    import torch
    got = got.detach().double().cpu().numpy() if torch.is_tensor(got) else got
    bound = HALF[dt] * np.abs(want) + (K + 2) * 2.0 ** -23 * S * (1 + 2.0 ** -8)
    err = np.abs(got - want)
    ok = err <= bound                      # NaN fails
    assert ok.all(), f"{what}: {np.count_nonzero(~ok)} of {ok.size} past the bound, first {np.argwhere(~ok)[:3].tolist()}"


def ids_of(sizes, rng, dropped=0):
    """Shuffled ids with sizes[e] rows of expert e and `dropped` rows of none."""
    ids = np.concatenate([np.full(n, e) for e, n in enumerate(sizes)] + [np.full(dropped, -1)]).astype(np.int32)
    return rng.permutation(ids)


class Case:
    """Device tensors and their float64 values for one product."""

    def __init__(self, sizes, di, do, dt="bf16", layout="kn", top_k=1, x_order=False, y_order=False, dropped=0,
                 seed=0, w4=False):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.E, self.di, self.do, self.dt, self.layout = len(sizes), di, do, dt, layout
        pad = (-(sum(sizes) + dropped)) % top_k
        ids = ids_of(sizes, rng, dropped + pad)
        self.rows = ids.shape[0]
        self.off, self.order = ox.group_rows(ids, self.E)
        self.d_ids = torch.from_numpy(ids).cuda()
        self.d_off, self.d_order = torch.from_numpy(self.off).cuda(), torch.from_numpy(self.order).cuda()
        T = self.rows // top_k if x_order else self.rows
        r = lambda *s: torch.randn(s, generator=g, device="cuda").to(_t(dt))
        self.X, self.dY = r(T, di), r(self.rows, do)
        if w4:
            codes = rng.integers(0, 16, size=(self.E * do, di), dtype=np.uint8)
            scales = rng.integers(115, 126, size=(self.E * do, di // 32), dtype=np.uint8)
            self.W = torch.from_numpy(ox.pack(codes, scales)).cuda()
            self.Wm = ox.decode(codes, scales).reshape(self.E, do, di).transpose(0, 2, 1)
        else:
            self.W = r(*((self.E, di, do) if layout == "kn" else (self.E, do, di)))
            w = self.W.double().cpu().numpy()
            self.Wm = w if layout == "kn" else w.transpose(0, 2, 1)
        self.Xh, self.dYh = self.X.double().cpu().numpy(), self.dY.double().cpu().numpy()
        self.kw = dict(top_k=top_k, x_order=x_order, y_order=y_order)

    def layer(self, **more):
        from adapter_lora_segments_amd import ExpertLinear
        return ExpertLinear(self.W, self.E, self.di, self.do, self.rows, dtype=self.dt, w_layout=self.layout, **self.kw,
                            **more)

    def wdw(self, dw):
        return dw.transpose(0, 2, 1) if self.layout == "nk" else dw


# ---- grouping ----

@pytest.mark.parametrize("rows", [0, 1, 63, 64, 65, 1000, 8192, 8193, 20000, 300001])
@pytest.mark.parametrize("groups", [1, 2, 16, 65, 257, 1024, 4096])
def test_group_rows(rows, groups):
    import torch
    from adapter_lora_segments_amd import RowGroups
    say(f"group_rows {rows} rows of {groups}")
    rng = np.random.default_rng(rows + groups)
    # skewed ids, a tenth of them outside [0, groups), extremes of int32 among them
    ids = np.minimum(rng.geometric(min(0.9, 3.0 / groups), size=rows) - 1, groups - 1).astype(np.int32)
    out = rng.random(rows) < 0.1
    ids[out] = rng.choice(np.array([-1, groups, -2 ** 31, 2 ** 31 - 1]), size=int(out.sum())).astype(np.int32)
    gr = RowGroups(rows + 5, groups)
    for _ in range(2):                     # the second call meets the first one's workspace
        off, order = gr.group(torch.from_numpy(ids).cuda())
    want_off, want_order = ox.group_rows(ids, groups)
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(order.cpu().numpy(), want_order)


def test_group_rows_one_group_takes_all():
    import torch
    from adapter_lora_segments_amd import RowGroups
    for rows in (5000, 70000):
        off, order = RowGroups(rows, 64).group(torch.full((rows,), 37, dtype=torch.int32, device="cuda"))
        assert off.cpu().tolist() == [0] * 38 + [rows] * 27
        assert np.array_equal(order.cpu().numpy(), np.arange(rows))


# ---- products ----

# sizes reach every tile form: few rows (16 and 32 a tile), 64, 128 and 256 rows a tile
SIZES = {"one": [1], "few": [3, 0, 1, 7, 16, 5], "thirty": [31, 17, 0, 40, 25], "sixty": [64, 1, 130, 0, 65],
         "hundreds": [200, 129, 0, 301], "big": [513, 700]}
DIMS = [(8, 8), (64, 264), (200, 40), (328, 520)]


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("dt,layout", [("bf16", "kn"), ("bf16", "nk"), ("fp32", "kn"), ("fp32", "nk")])
def test_forward(sizes, dims, dt, layout):
    import torch
    say(f"forward {sizes} {dims} {dt} {layout}")
    x_order = sizes in ("few", "sixty", "big")
    y_order = sizes in ("few", "hundreds")
    di, do = dims if dt == "bf16" else (dims[0] + 4, dims[1] + 4)
    c = Case(SIZES[sizes], di, do, dt, layout, top_k=2 if x_order else 1, x_order=x_order, y_order=y_order, dropped=3)
    Y = torch.full((c.rows, do), 7.5, dtype=_t(dt), device="cuda")
    c.layer().forward(c.X, c.d_off, c.d_order, Y)
    want, S, owned = ox.forward(c.Xh, c.Wm, c.off, c.order, c.rows, **c.kw)
    y = Y.double().cpu().numpy()
    assert (y[~owned] == 7.5).all(), "rows of no group were written"
    check(y[owned], want[owned], S[owned], di, dt, "Y")


# Products (rows, experts, d_in, d_out), the smallest of a grid of sizes that
# between them take every few-row and tile form of each type and layout, over a
# short reduction and a long one.
FORMS = {
    "bf16 nk": [(1, 1, 128, 72), (1, 1, 1152, 72), (48, 32, 128, 264), (48, 32, 1152, 264), (384, 16, 128, 520),
                (384, 16, 1152, 520), (1024, 3, 256, 14336), (1024, 64, 1152, 264), (1536, 1, 128, 72),
                (1536, 1, 1152, 72), (1536, 64, 128, 72), (1536, 64, 1152, 72), (1536, 64, 1152, 136),
                (3000, 2, 256, 14336), (3000, 64, 128, 72), (3000, 64, 128, 520), (3000, 64, 1152, 72),
                (4096, 64, 256, 136), (8192, 1, 1152, 136), (16384, 1, 1152, 136), (16384, 8, 256, 264),
                (16384, 64, 1152, 136), (32768, 1, 128, 264), (32768, 64, 1152, 136)],
    "bf16 kn": [(1, 1, 128, 72), (1, 1, 1152, 72), (8, 3, 128, 2056), (8, 3, 1152, 2056), (768, 2, 1152, 14336),
                (1536, 64, 1280, 520), (2048, 8, 128, 14336), (3000, 1, 128, 72), (3000, 1, 1152, 72),
                (3000, 8, 256, 14336), (4096, 64, 1152, 72), (8192, 1, 1152, 136), (8192, 64, 256, 136),
                (16384, 1, 1152, 136), (16384, 64, 1152, 136), (32768, 1, 128, 72), (32768, 1, 128, 264),
                (32768, 1, 256, 72)],
    "fp32 nk": [(1, 1, 128, 72), (1, 1, 1152, 72), (48, 2, 1152, 14336), (64, 2, 128, 14336), (96, 3, 1152, 14336),
                (128, 2, 1152, 14336), (128, 3, 128, 14336), (128, 3, 1152, 4104), (128, 64, 128, 72),
                (128, 64, 1152, 72), (384, 2, 128, 14336), (384, 3, 256, 2056), (384, 16, 128, 264),
                (384, 16, 1152, 264), (768, 32, 128, 72), (768, 32, 1152, 72), (3000, 1, 128, 4104),
                (3000, 1, 1152, 4104), (3000, 64, 128, 72), (3000, 64, 1152, 72), (32768, 1, 128, 72),
                (32768, 1, 1152, 136)],
    "fp32 kn": [(1, 1, 128, 72), (1, 1, 1152, 72), (200, 2, 1152, 14336), (384, 2, 1152, 14336), (3000, 1, 128, 72),
                (3000, 1, 1152, 72), (3000, 1, 1152, 4104), (3000, 3, 128, 4104), (3000, 8, 128, 2056),
                (3000, 16, 128, 2056), (8192, 1, 128, 72), (8192, 1, 1152, 72), (16384, 1, 1152, 72),
                (32768, 1, 128, 72), (32768, 1, 1152, 72)],
    "w4 bf16": [(1, 1, 128, 72), (1, 1, 128, 14336), (1, 1, 1152, 72), (1, 1, 1152, 14336), (128, 8, 1152, 4104),
                (256, 8, 128, 14336), (384, 64, 128, 72), (384, 64, 1152, 72), (1536, 8, 128, 14336),
                (1536, 32, 128, 136), (1536, 32, 1152, 136), (2048, 1, 128, 72), (2048, 1, 1152, 72),
                (3000, 64, 1152, 136), (4096, 32, 1152, 264), (8192, 1, 128, 4104), (8192, 1, 128, 14336),
                (8192, 64, 1152, 264), (16384, 1, 128, 136), (16384, 1, 256, 72), (16384, 2, 1152, 136),
                (32768, 64, 1152, 136)],
    "w4 mxfp4": [(1, 1, 128, 72), (1, 1, 128, 14336), (1, 1, 1152, 72), (1, 1, 1152, 14336), (1, 1, 2048, 72),
                 (1, 1, 2048, 14336), (48, 32, 2048, 1032), (96, 64, 1152, 520), (128, 32, 1280, 520),
                 (128, 64, 2048, 264), (160, 64, 128, 72), (160, 64, 256, 1032), (160, 64, 1152, 72),
                 (160, 64, 2048, 72), (768, 32, 128, 264), (768, 32, 1152, 264), (1536, 1, 1280, 14336),
                 (1536, 32, 128, 72), (1536, 32, 1152, 72), (1536, 32, 2048, 72), (3000, 1, 256, 14336),
                 (3000, 1, 2048, 4104), (4096, 16, 1152, 264), (4096, 16, 2048, 264), (16384, 1, 128, 72),
                 (16384, 1, 128, 14336), (16384, 2, 128, 72), (16384, 2, 1152, 136), (16384, 2, 2048, 136)],
}


# bf16 and fp32 also with a reduction that ends inside a step.
ODD = [(f, (r, e, di + (8 if f < "f" else 4), do)) for f in FORMS if f[0] != "w" for r, e, di, do in FORMS[f]]


@pytest.mark.parametrize("form,size", [(f, s) for f in FORMS for s in FORMS[f]] + ODD)
def test_every_form(form, size):
    """Ragged groups, rows by order in two thirds of the cases, against float64
    products on the device."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear, mlora_microscale_quantize
    say(f"form {form} {size}")
    rows, E, di, do = size
    kind, how = form.split()
    dt = "fp32" if kind == "fp32" else "bf16"
    rng = np.random.default_rng(rows + E + di + do)
    p = 1.0 / (1 + np.arange(E))
    if E > 2:
        p[E // 2] = 0.0                                     # an expert without rows
    sizes = rng.permutation(rng.multinomial(rows, p / p.sum()))
    c = np.concatenate([[0], np.cumsum(sizes)])
    off = torch.from_numpy(c.astype(np.int32)).cuda()
    by = (rows + di) % 3 != 0
    order = torch.from_numpy(rng.permutation(rows).astype(np.int32)).cuda() if by else None
    g = torch.Generator(device="cuda").manual_seed(rows)
    X = torch.randn(rows, di, generator=g, device="cuda").to(_t(dt))
    opts = dict(dtype=dt, x_order=by, y_order=by)
    if kind == "w4":
        codes = rng.integers(0, 16, size=(E * do, di), dtype=np.uint8)
        scales = rng.integers(115, 126, size=(E * do, di // 32), dtype=np.uint8)
        W = torch.from_numpy(ox.pack(codes, scales)).cuda()
        Wd = torch.from_numpy(ox.decode(codes, scales).reshape(E, do, di)).cuda().transpose(1, 2)
        opts.update(w_layout="nk", w_format="mxfp4", act_format=how)
    else:
        W = torch.randn(*((E, do, di) if how == "nk" else (E, di, do)), generator=g, device="cuda").to(_t(dt))
        Wd = W.double().transpose(1, 2) if how == "nk" else W.double()
        opts.update(w_layout=how)
    Y = ExpertLinear(W, E, di, do, rows, **opts).forward(X, off, order)
    V = X
    if how == "mxfp4":
        V = torch.empty_like(X)
        mlora_microscale_quantize(X, values=V)
    V = V.double()
    for e in range(E):
        at = slice(int(c[e]), int(c[e + 1]))
        at = order[at].long() if by else at
        x, w = V[at], Wd[e].contiguous()
        want, S = x @ w, x.abs() @ w.abs()
        bound = HALF[dt] * want.abs() + (di + 2) * 2.0 ** -23 * S * (1 + 2.0 ** -8)
        ok = (Y[at].double() - want).abs() <= bound          # NaN fails
        assert ok.all(), f"expert {e}: {int((~ok).sum())} of {ok.numel()} past the bound"


@pytest.mark.parametrize("sizes", ["few", "sixty", "hundreds", "big"])
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("dt,layout", [("bf16", "kn"), ("bf16", "nk"), ("fp32", "kn"), ("fp32", "nk")])
def test_backward(sizes, dims, dt, layout):
    import torch
    say(f"backward {sizes} {dims} {dt} {layout}")
    x_order, y_order = sizes in ("few", "big"), sizes in ("sixty", "big")
    di, do = dims if dt == "bf16" else (dims[0] + 4, dims[1] + 4)
    c = Case(SIZES[sizes], di, do, dt, layout, top_k=2 if x_order else 1, x_order=x_order, y_order=y_order, dropped=5)
    L = c.layer()
    dX = torch.full((c.rows, di), -3.0, dtype=_t(dt), device="cuda")
    L.backward(c.dY, c.X, c.d_off, c.d_order, dX)
    want, SX, owned, dW, SW = ox.backward(c.dYh, c.Xh, c.Wm, c.off, c.order, c.rows, **c.kw)
    d = dX.double().cpu().numpy()
    assert (d[~owned] == -3.0).all(), "rows of no group were written"
    check(d[owned], want[owned], SX[owned], do, dt, "dX")
    n = max(SIZES[sizes])
    check(L.dW, c.wdw(dW), c.wdw(SW), n, "fp32", "dW")
    for e, k in enumerate(SIZES[sizes]):
        if k == 0:
            assert not L.dW[e].any(), "an expert without rows has a zero gradient"
    # alone, the same values
    first = L.dW.clone()
    assert torch.equal(L.backward(c.dY, None, c.d_off, c.d_order, dX.clone(), want_dw=False)[torch.from_numpy(owned).cuda()],
                       dX[torch.from_numpy(owned).cuda()])
    L.dW.fill_(9.0)
    assert L.backward(c.dY, c.X, c.d_off, c.d_order, want_dx=False) is None
    assert torch.equal(L.dW, first)


@pytest.mark.parametrize("x_order,y_order", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dt,di,do,sizes", [("bf16", 1032, 2056, [70, 0, 129, 1, 200]),
                                            ("fp32", 1540, 2052, [70, 1, 0]), ("fp32", 4100, 4100, [33, 0, 70])])
def test_gradients_of_wide_weights(dt, di, do, sizes, layout, x_order, y_order):
    """dW in the tiles that wide weights take (256 x 256, fp32 128 x 128), with
    either operand's rows by order, and dX beside it; accumulated once more."""
    import torch
    say(f"wide {dt} {di}x{do} {layout} {x_order} {y_order}")
    c = Case(sizes, di, do, dt, layout, top_k=2 if x_order and y_order else 1, x_order=x_order,
             y_order=y_order, dropped=5)
    A = c.layer(grad_accumulate=True)
    dX = A.backward(c.dY, c.X, c.d_off, c.d_order)
    want, SX, owned, dW, SW = ox.backward(c.dYh, c.Xh, c.Wm, c.off, c.order, c.rows, **c.kw)
    check(dX.double().cpu().numpy()[owned], want[owned], SX[owned], do, dt, "dX")
    check(A.dW, c.wdw(dW), c.wdw(SW), max(sizes), "fp32", "dW")
    one = A.dW.clone()
    A.backward(c.dY, c.X, c.d_off, c.d_order, want_dx=False)
    assert torch.equal(A.dW, one + one)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_accumulated_gradients(dt):
    """Two backwards into one dW: bit for bit the fp32 sums of two separate ones."""
    import torch
    c = Case([40, 0, 300], 72, 136, dt)
    L, A = c.layer(), c.layer(grad_accumulate=True)
    L.backward(c.dY, c.X, c.d_off, c.d_order)
    one = L.dW.clone()
    dY2 = (c.dY * 0.5 + 1).contiguous()
    L.backward(dY2, c.X, c.d_off, c.d_order)
    A.backward(c.dY, c.X, c.d_off, c.d_order)
    A.backward(dY2, c.X, c.d_off, c.d_order)
    assert torch.equal(A.dW, one + L.dW)
    A.backward(c.dY[:0], c.X[:0], torch.zeros_like(c.d_off), None)          # no rows: kept
    assert torch.equal(A.dW, one + L.dW)
    L.backward(c.dY[:0], c.X[:0], torch.zeros_like(c.d_off), None)          # no rows: zero
    assert not L.dW.any()


CHUNKS = {"skewed": [0, 700, 1, 300, 257, 2000, 256, 0],
          "one": [3000],
          "long": [5000, 20, 2500],
          "wide": [5 if e % 9 else 600 for e in range(80)]}


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("order", [False, True])
@pytest.mark.parametrize("sizes", list(CHUNKS))
def test_gradients_summed_in_chunks(sizes, order, dt):
    """Groups cut into pieces (of 256 rows, fp32, or 1024, bf16) whose sums are added by a second
    kernel: dW, its accumulation, the same bits twice, a captured one, and
    offsets out of order, which stay in the workspace."""
    import torch
    say(f"chunks {sizes} {order} {dt}")
    c = Case(CHUNKS[sizes], 72, 136, dt, "nk", x_order=order, y_order=order, dropped=3)
    L = c.layer()
    assert L.shape.workspace_bytes >= 4 * 72 * 136 * 2
    L.backward(c.dY, c.X, c.d_off, c.d_order, want_dx=False)
    _, _, _, dW, SW = ox.backward(c.dYh, c.Xh, c.Wm, c.off, c.order, c.rows, **c.kw)
    check(L.dW, c.wdw(dW), c.wdw(SW), max(CHUNKS[sizes]), "fp32", "dW")
    first = L.dW.clone()
    A = c.layer(grad_accumulate=True)
    A.dW.copy_(first)
    A.backward(c.dY, c.X, c.d_off, c.d_order, want_dx=False)
    assert torch.equal(A.dW, first + first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.backward(c.dY, c.X, c.d_off, c.d_order, want_dx=False)
    for _ in range(3):
        L.dW.fill_(9.0)
        A.ws.fill_(255)
        A.backward(c.dY, c.X, c.d_off, c.d_order, want_dx=False)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(L.dW, first)
    # every group is all rows: far more chunks than the workspace has room for
    n = L.ws.numel()
    pad = torch.full((n + 2 ** 20,), 7, dtype=torch.uint8, device="cuda")
    L.ws = pad[2 ** 19:2 ** 19 + n]
    off = c.d_off.clone()
    off[::2], off[1::2] = -4, 2 ** 31 - 1
    L.backward(c.dY, c.X, off, c.d_order, want_dx=False)
    assert (pad[:2 ** 19] == 7).all() and (pad[2 ** 19 + n:] == 7).all()


def test_single_expert_without_offsets():
    import torch
    c = Case([333], 136, 72)
    L = c.layer()
    assert torch.equal(L.forward(c.X), L.forward(c.X, c.d_off))
    a = L.backward(c.dY, c.X)
    w = L.dW.clone()
    assert torch.equal(a, L.backward(c.dY, c.X, c.d_off)) and torch.equal(w, L.dW)


def test_many_experts():
    """More experts than a wave has lanes, most of them empty."""
    rng = np.random.default_rng(1)
    sizes = [int(v) if rng.random() < 0.3 else 0 for v in rng.integers(1, 90, size=200)]
    c = Case(sizes, 72, 264, x_order=True, y_order=True)
    Y = c.layer().forward(c.X, c.d_off, c.d_order)
    want, S, _ = ox.forward(c.Xh, c.Wm, c.off, c.order, c.rows, **c.kw)
    check(Y, want, S, 72, "bf16")


@pytest.mark.parametrize("sizes", ["few", "sixty", "big"])
def test_values_of_other_groups_do_not_reach_a_group(sizes):
    """Rows of no group and a whole expert of NaN and infinity: the others are
    what they are without them, in Y, dX and dW."""
    import torch
    c = Case(SIZES[sizes], 72, 72, dropped=9)
    L = c.layer()
    Y0, dX0 = L.forward(c.X, c.d_off, c.d_order), L.backward(c.dY, c.X, c.d_off, c.d_order)
    dW0 = L.dW.clone()
    lo, hi = int(c.off[-2]), int(c.off[-1])
    for t in (c.X, c.dY):
        t[lo:hi:2] = float("nan")
        t[lo:] = torch.where(torch.isnan(t[lo:]), t[lo:], torch.full_like(t[lo:], float("inf")))
    c.W[-1] = float("nan")
    Y1, dX1 = L.forward(c.X, c.d_off, c.d_order), L.backward(c.dY, c.X, c.d_off, c.d_order)
    assert torch.equal(Y0[:lo], Y1[:lo]) and torch.equal(dX0[:lo], dX1[:lo]) and torch.equal(dW0[:-1], L.dW[:-1])
    assert torch.isnan(Y1[lo:hi]).all()


@pytest.mark.parametrize("n", [6, 700])
def test_damaged_tables_stay_in_the_buffers(n):
    """Offsets and order entries out of range: the buffers' neighbours and the
    rows that no valid entry names are untouched."""
    import torch
    say(f"damaged tables {n}")
    c = Case([n, n, n], 72, 72, x_order=True, y_order=True)
    R = c.rows
    pad = torch.full((R + 512, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    Y = pad[256:256 + R]
    order = c.d_order.clone()
    order[::2] = torch.tensor([-1, R, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda").repeat(R)[:order[::2].numel()]
    off = torch.tensor([-5, n, 2 * n, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    c.layer().forward(c.X, off, order, Y)
    good = order[(order >= 0) & (order < R)].long()
    touched = torch.zeros(R, dtype=torch.bool, device="cuda")
    touched[good] = True
    assert (pad[:256] == 5).all() and (pad[256 + R:] == 5).all() and (Y[~touched] == 5).all()
    want = c.layer().forward(c.X, c.d_off, c.d_order)
    assert torch.equal(Y[good], want[good])


# ---- MXFP4 weights ----

@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("dims", [(128, 8), (256, 264), (640, 72)])
@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
def test_mxfp4_forward(sizes, dims, act):
    import torch
    say(f"mxfp4 forward {sizes} {dims} {act}")
    x_order, y_order = sizes in ("few", "sixty"), sizes in ("few", "big")
    c = Case(SIZES[sizes], *dims, layout="nk", top_k=2 if x_order else 1, x_order=x_order, y_order=y_order, dropped=2,
             w4=True)
    Y = torch.full((c.rows, dims[1]), 7.5, dtype=torch.bfloat16, device="cuda")
    c.layer(w_format="mxfp4", act_format=act).forward(c.X, c.d_off, c.d_order, Y)
    X = c.Xh if act == "bf16" else ox.decode(*ox.quantize(c.Xh))
    want, S, owned = ox.forward(X, c.Wm, c.off, c.order, c.rows, **c.kw)
    y = Y.double().cpu().numpy()
    assert (y[~owned] == 7.5).all()
    check(y[owned], want[owned], S[owned], dims[0], "bf16", "Y")


@pytest.mark.parametrize("per,experts,do", [(3, 2, 40), (40, 4, 264), (64, 16, 1032), (130, 8, 520), (200, 3, 136),
                                            (600, 2, 264)])
@pytest.mark.parametrize("di", [2048, 2176, 3328])
@pytest.mark.parametrize("form", ["bf16", "w4 bf16", "w4 mxfp4"])
def test_long_reductions(per, experts, do, di, form):
    """Reductions of many steps, past every ring's depth, whole and with a
    partial last step."""
    say(f"long {per} x {experts} {di} -> {do} {form}")
    w4 = form.startswith("w4")
    act = form.split()[-1]
    c = Case([per, 0, per + 5, per - 2] if experts < 4 else [per + e % 3 for e in range(experts)], di, do, layout="nk",
             y_order=True, w4=w4)
    Y = c.layer(**(dict(w_format="mxfp4", act_format=act) if w4 else {})).forward(c.X, c.d_off, c.d_order)
    X = ox.decode(*ox.quantize(c.Xh)) if act == "mxfp4" else c.Xh
    want, S, _ = ox.forward(X, c.Wm, c.off, c.order, c.rows, **c.kw)
    check(Y, want, S, di, "bf16", "Y")


@pytest.mark.parametrize("sizes", ["few", "sixty", "big"])
def test_mxfp4_dx(sizes):
    import torch
    say(f"mxfp4 dX {sizes}")
    c = Case(SIZES[sizes], 256, 264, layout="nk", y_order=True, w4=True)
    dX = c.layer(w_format="mxfp4").backward(c.dY, None, c.d_off, c.d_order)
    want, SX, _, _, _ = ox.backward(c.dYh, None, c.Wm, c.off, c.order, c.rows, **c.kw)
    check(dX, want, SX, 264, "bf16", "dX")


def test_mxfp4_scales_over_the_whole_range():
    """Every scale code whose products bf16 and fp32 hold, small and large, and
    a NaN scale: its output column alone is NaN, in every form."""
    import torch
    di, do = 256, 256
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 16, size=(do, di), dtype=np.uint8)
    scales = np.repeat(np.arange(do).clip(20, 220).astype(np.uint8)[:, None], di // 32, axis=1)
    scales[100, 3] = 255
    W = torch.from_numpy(ox.pack(codes, scales)).cuda()
    Wm = ox.decode(codes, scales).T[None]
    from adapter_lora_segments_amd import ExpertLinear
    for rows in (5, 70, 300, 900):
        X = torch.randn(rows, di, device="cuda").to(torch.bfloat16)
        for act in ("bf16", "mxfp4"):
            say(f"scales {rows} {act}")
            Y = ExpertLinear(W, 1, di, do, rows, w_layout="nk", w_format="mxfp4", act_format=act).forward(X)
            Xh = X.double().cpu().numpy()
            Xh = Xh if act == "bf16" else ox.decode(*ox.quantize(Xh))
            off = np.array([0, rows])
            keep = np.arange(do) != 100
            want, S, _ = ox.forward(Xh, Wm[:, :, keep], off, None, rows)
            y = Y.double().cpu().numpy()
            assert np.isnan(y[:, 100]).all()
            check(y[:, keep], want, S, di, "bf16")


# ---- quantizer ----

def special_matrix(rng, rows, cols, dt):
    """Normal values of many sizes, exact ties, values that saturate, zeros,
    subnormals, and blocks with NaN or infinities."""
    import torch
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30, 30, size=(rows, 1)).astype(float))
    ties = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, 0.0, -0.0], size=(rows, cols))
    x = np.where(rng.random((rows, cols)) < 0.3, ties * rng.choice([-1, 1], size=(rows, cols)), x)
    x[:, : cols // 4] *= 2.0 ** -20
    x[rng.random((rows, cols)) < 0.002] = np.nan
    x[rng.random((rows, cols)) < 0.002] = -np.inf
    if rows > 3:
        x[1] = 0.0
        x[2] = rng.choice([0.0, 2.0 ** -126, -2.0 ** -130, 2.0 ** -133, 3 * 2.0 ** -128], size=cols)
        x[3] = rng.choice([2.0 ** 127, -1.5 * 2.0 ** 127, 2.0 ** 126, 1.0], size=cols)
    return torch.from_numpy(x.astype(np.float32)).cuda().to(_t(dt))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("along,rows,cols", [("cols", 1, 32), ("cols", 7, 96), ("cols", 130, 1056), ("rows", 32, 8),
                                             ("rows", 96, 200), ("rows", 320, 1032)])
def test_quantize(dt, along, rows, cols):
    import torch
    from adapter_lora_segments_amd import mlora_microscale_quantize
    say(f"quantize {dt} {along} {rows}x{cols}")
    full = special_matrix(np.random.default_rng(rows * cols), rows, cols + 16, dt)
    for x in (full[:, :cols].contiguous(), full[:, :cols]):      # dense, and rows of a wider matrix
        h = x.double().cpu().numpy()
        codes, scales = ox.quantize(h if along == "cols" else h.T)
        vals = ox.decode(codes, scales)
        if along == "rows":
            codes, vals = codes.T, vals.T
        v = torch.empty((rows, cols), dtype=x.dtype, device="cuda")
        q = mlora_microscale_quantize(x, values=v, along=along)
        assert np.array_equal(q.cpu().numpy(), ox.pack(codes, scales))
        got = v.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(vals))
        assert np.array_equal(got[~np.isnan(vals)], vals[~np.isnan(vals)])
        assert torch.equal(q, mlora_microscale_quantize(x, along=along))


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_quantized_base_of_a_packed_layer(layout):
    """The quantizer's buffer is an MXFP4 base of the multi-LoRA layer: the
    layer over it equals the layer over the decoded values, bit for bit."""
    import torch
    from adapter_lora_segments_amd import PackedLoRALinear, Plan, mlora_microscale_quantize
    di, do = 256, 320
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    W = r(di, do) if layout == "kn" else r(do, di)
    vals = torch.empty_like(W)
    q = mlora_microscale_quantize(W, values=vals, along="rows" if layout == "kn" else "cols")
    A, B, X = [r(di, 8), r(di, 16)], [r(8, do), r(16, do)], r(200, di)
    out = []
    for base, fmt in ((q, "mxfp4"), (vals, "bf16")):
        plan = Plan([0, 90, 200], [8, 16], di, do, "bf16", w0_layout=layout, w0_format=fmt)
        out.append(PackedLoRALinear(plan, base, A, B, [1.0, 0.5]).forward(X))
    assert torch.equal(out[0], out[1])


# ---- as they are used: together, on streams, in graphs ----

def block(ids, X, up, down, groups, T, k):
    """A two-product block over routed tokens: (token, id) results summed per token."""
    off, order = groups.group(ids)
    h = up.forward(X, off, order)
    a = h.relu()
    y = down.forward(a, off, order)
    return off, order, h, a, y.view(T, k, -1).sum(1)


@pytest.mark.parametrize("T", [3, 300])
def test_block_of_all_operators(T):
    """ids -> groups -> up product (rows read through the order) -> ReLU ->
    down product (rows written through it) -> sum per token, and the way back,
    against float64; then the same with both weights quantized."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear, RowGroups, mlora_microscale_quantize
    say(f"block {T}")
    E, k, di, dh = 6, 2, 128, 256
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    X, ids = r(T, di), torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32).reshape(-1)
    Wu, Wd = r(E, dh, di), r(E, di, dh)
    groups = RowGroups(T * k, E)
    mk = lambda Wa, Wb, f: (ExpertLinear(Wa, E, di, dh, T * k, w_layout="nk", w_format=f, top_k=k, x_order=True),
                            ExpertLinear(Wb, E, dh, di, T * k, w_layout="nk", w_format=f, y_order=True))
    up, down = mk(Wu, Wd, "bf16")
    off, order, h, a, y = block(ids, X, up, down, groups, T, k)
    n64 = lambda t: t.double().cpu().numpy()
    o, p = off.cpu().numpy(), order.cpu().numpy()
    assert np.array_equal(p, ox.group_rows(ids.cpu().numpy(), E)[1])
    Wu64, Wd64 = n64(Wu).transpose(0, 2, 1), n64(Wd).transpose(0, 2, 1)
    want_h, S, _ = ox.forward(n64(X), Wu64, o, p, T * k, top_k=k, x_order=True)
    check(h, want_h, S, di, "bf16", "h")
    want_y, S, _ = ox.forward(n64(a), Wd64, o, p, T * k, y_order=True)
    slots = down.forward(a, off, order)
    check(slots, want_y, S, dh, "bf16", "y slots")
    assert torch.equal(y, slots.view(T, k, -1).sum(1))
    # back: the token's gradient in every slot it has
    dy = r(T, di)
    dslots = dy[:, None].expand(T, k, di).reshape(T * k, di).contiguous()
    da = down.backward(dslots, a, off, order)
    dh_ = da * (h > 0)
    dx = up.backward(dh_, X, off, order).view(T, k, di).sum(1)
    w, SX, _, dW, SW = ox.backward(n64(dslots), n64(a), Wd64, o, p, T * k, y_order=True)
    check(da, w, SX, di, "bf16", "da")
    check(down.dW, dW.transpose(0, 2, 1), SW.transpose(0, 2, 1), T * k, "fp32", "dWd")
    w, SX, _, dW, SW = ox.backward(n64(dh_), n64(X), Wu64, o, p, T * k, top_k=k, x_order=True)
    check(up.dW, dW.transpose(0, 2, 1), SW.transpose(0, 2, 1), T * k, "fp32", "dWu")
    # the sum of k bf16 slots, rounded once more
    want = w.reshape(T, k, di).sum(1)
    S = SX.reshape(T, k, di).sum(1)
    got = n64(dx)
    assert (np.abs(got - want) <= 2.0 ** -8 * (np.abs(w.reshape(T, k, di)).sum(1) + np.abs(want)) * 1.01
            + (dh + 4) * 2.0 ** -23 * S * 1.01).all()
    # quantized weights
    vu, vd = torch.empty_like(Wu), torch.empty_like(Wd)
    qu = mlora_microscale_quantize(Wu.view(E * dh, di), values=vu.view(E * dh, di))
    qd = mlora_microscale_quantize(Wd.view(E * di, dh), values=vd.view(E * di, dh))
    upq, downq = mk(qu, qd, "mxfp4")
    hq, hv = upq.forward(X, off, order), mk(vu, vd, "bf16")[0].forward(X, off, order)
    want, S, _ = ox.forward(n64(X), n64(vu).transpose(0, 2, 1), o, p, T * k, top_k=k, x_order=True)
    check(hq, want, S, di, "bf16", "hq")
    check(hv, want, S, di, "bf16", "hv")
    dq = downq.backward(dslots, None, off, order)
    w, SX, _, _, _ = ox.backward(n64(dslots), None, n64(vd).transpose(0, 2, 1), o, p, T * k, y_order=True)
    check(dq, w, SX, di, "bf16", "da of quantized weights")


@pytest.mark.parametrize("T", [4, 200])
def test_captured_block(T):
    """Grouping, products and gradients in one captured graph, replayed over
    new ids and inputs with eager work between, every replay against the eager
    result bit for bit."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear, RowGroups
    say(f"captured block {T}")
    E, k, di, dh = 5, 2, 128, 256
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    Wu = torch.from_numpy(ox.pack(np.random.default_rng(1).integers(0, 16, size=(E * dh, di), dtype=np.uint8),
                                  np.full((E * dh, di // 32), 120, dtype=np.uint8))).cuda()
    Wd = r(E, dh, di)

    def parts():
        up = ExpertLinear(Wu, E, di, dh, T * k, w_layout="nk", w_format="mxfp4", act_format="mxfp4", top_k=k, x_order=True)
        down = ExpertLinear(Wd, E, dh, di, T * k, y_order=True)
        return up, down, RowGroups(T * k, E)

    X, dy = r(T, di), r(T * k, di)
    new_ids = lambda: torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32).reshape(-1)
    ids = new_ids()

    def step(p, X, ids, dy):
        up, down, groups = p
        off, order = groups.group(ids)
        h = up.forward(X, off, order)
        y = down.forward(h, off, order)
        da = down.backward(dy, h, off, order)
        dx = up.backward(da, None, off, order)
        return y, da, dx, down.dW

    cap, eager = parts(), parts()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(cap, X, ids, dy)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cap, X, ids, dy)
    for _ in range(4):
        X.copy_(r(T, di))
        dy.copy_(r(T * k, di))
        ids.copy_(new_ids())
        graph.replay()
        want = step(eager, X, ids, dy)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_calls_on_two_streams():
    """The same layer's weight used on two streams at once, each with its own
    workspace: both equal the sequential results."""
    import torch
    c = Case([100, 0, 260], 256, 264, layout="nk", w4=True)
    opts = dict(w_format="mxfp4", act_format="mxfp4")
    L = [c.layer(**opts) for _ in range(2)]
    X2 = (c.X * 0.5).contiguous()
    want = [L[0].forward(x, c.d_off, c.d_order) for x in (c.X, X2)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    out = [[], []]
    for _ in range(5):
        for i, x in enumerate((c.X, X2)):
            with torch.cuda.stream(st[i]):
                out[i].append(L[i].forward(x, c.d_off, c.d_order))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in out[i])
    # an explicit stream argument
    y = torch.empty_like(want[0])
    st[0].wait_stream(torch.cuda.current_stream())
    L[0].forward(c.X, c.d_off, c.d_order, y, stream=st[0])
    torch.cuda.current_stream().wait_stream(st[0])
    assert torch.equal(y, want[0])


def test_offsets_past_32_bits():
    """Rows of X and Y behind the 4 GiB mark, and an expert's weight behind it."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear
    say("past 32 bits")
    di, do, T = 64, 8192, 300000
    X = torch.randn(T, di, device="cuda").to(torch.bfloat16)
    E = 4200 // 2
    W = torch.randn(E, di, do, device="cuda", dtype=torch.bfloat16)      # 2.2 GB
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = 10
    off[E] = T
    L = ExpertLinear(W, E, di, do, T)
    Y = L.forward(X, off.cuda())                                          # 4.9 GB
    for lo, hi, e in ((0, 10, 0), (T - 1000, T, E - 1), (262000, 262300, E - 1)):
        x, w = X[lo:hi].double().cpu().numpy(), W[e].double().cpu().numpy()
        check(Y[lo:hi], x @ w, np.abs(x) @ np.abs(w), di, "bf16", f"rows {lo}")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_gradient_rows_past_32_bits(dt):
    """dW and dX whose rows lie behind the 4 GiB mark of X, dY and dX."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear
    say(f"gradient rows past 32 bits {dt}")
    di, do, T = (4096, 8, 600000) if dt == "bf16" else (4096, 8, 300000)
    X = torch.zeros(T, di, device="cuda", dtype=_t(dt))
    dY = torch.zeros(T, do, device="cuda", dtype=_t(dt))
    rows = torch.cat([torch.arange(T - 90, T), torch.arange(5), torch.arange(T - 300, T - 100)]).int()
    for t in (X, dY):
        t[rows.cuda().long()] = torch.randn(rows.numel(), t.shape[1], device="cuda").to(t.dtype)
    W = torch.randn(2, di, do, device="cuda").to(_t(dt))
    order = torch.full((T,), -1, dtype=torch.int32)
    order[:rows.numel()] = rows
    off = torch.tensor([0, 95, rows.numel()], dtype=torch.int32).cuda()
    L = ExpertLinear(W, 2, di, do, T, dtype=dt, x_order=True, y_order=True)
    dX = L.backward(dY, X, off, order.cuda())                                        # 4.9 GB each
    for e, (lo, hi) in enumerate(((0, 95), (95, rows.numel()))):
        at = rows[lo:hi].cuda().long()
        x, dy, w = (t.double().cpu().numpy() for t in (X[at], dY[at], W[e]))
        check(L.dW[e], x.T @ dy, np.abs(x).T @ np.abs(dy), hi - lo, "fp32", "dW")
        check(dX[at], dy @ w.T, np.abs(dy) @ np.abs(w).T, do, dt, "dX")


def test_as_many_experts_as_there_may_be():
    """4096 experts, most of them empty: forward, dX and dW."""
    rng = np.random.default_rng(3)
    sizes = [0] * 4096
    for e in rng.integers(0, 4096, size=37):
        sizes[e] += 3
    sizes[4095] += 1
    c = Case(sizes, 16, 8, x_order=True, dropped=2)
    L = c.layer()
    want, S, _ = ox.forward(c.Xh, c.Wm, c.off, c.order, c.rows, **c.kw)
    n = int(c.off[-1])
    check(L.forward(c.X, c.d_off, c.d_order)[:n], want[:n], S[:n], 16, "bf16", "Y")
    dX = L.backward(c.dY, c.X, c.d_off, c.d_order)
    want, SX, owned, dW, SW = ox.backward(c.dYh, c.Xh, c.Wm, c.off, c.order, c.rows, **c.kw)
    check(dX.double().cpu().numpy()[owned], want[owned], SX[owned], 8, "bf16", "dX")
    check(L.dW, dW, SW, max(sizes), "fp32", "dW")
