"""4-bit weights with group scales on the GPU against the float64 oracle
(oracle/affine.py, oracle/experts.py).

Tolerances, per element.  Where codes are multiplied as they are, a group's
part is 128 s (P - (1 + z / 128) Q), P = sum x (1 + c / 128) and Q = sum x in
fp32 over the group's G inputs, each off by at most G 2^-23 of its sum of
magnitudes, with a few roundings of 2^-24 more; the groups' parts are added in
fp32.  So the error is at most half a bf16 step of the value, 2^-8, plus
(G + K / G + 16) 2^-23 B, B = sum |x| 128 |s| (1.12 + |1 + z / 128|), which bounds
every partial sum (1 + 2^-8 for the step of a value that is off by that).  Where
the weights are rounded to bf16 first: 2^-8 of the sum of |x| |w| for that and (K +
2) 2^-23 of it for the sums.  The quantizer's buffer is equal."""
import numpy as np
import pytest

from oracle import affine as oa
from oracle import experts as ox
from tests.gpu_harness import say
from tests.test_gpu_experts import ids_of

pytestmark = pytest.mark.gpu


def host(t):
    return t.detach().double().cpu().numpy()


class Case:
    """A packed weight, rows and tables on the device with their float64 values."""

    def __init__(self, sizes, di, do, group, top_k=1, x_order=False, y_order=False, dropped=0, seed=0, odd_zero=False):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.E, self.di, self.do, self.group = len(sizes), di, do, group
        pad = (-(sum(sizes) + dropped)) % top_k
        ids = ids_of(sizes, rng, dropped + pad)
        self.rows = ids.shape[0]
        self.off, self.order = ox.group_rows(ids, self.E)
        self.d_off, self.d_order = torch.from_numpy(self.off).cuda(), torch.from_numpy(self.order).cuda()
        T = self.rows // top_k if x_order else self.rows
        r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
        self.X, self.dY = r(T, di), r(self.rows, do)
        codes = rng.integers(0, 16, size=(self.E * do, di), dtype=np.uint8)
        zeros = rng.integers(0, 16, size=(self.E * do, di // group)).astype(np.float32)
        if odd_zero:                                  # zero points of other quantizers: any value
            zeros = oa.bf16(zeros + rng.standard_normal(zeros.shape).astype(np.float32) * 4)
        scales = oa.bf16(np.exp2(rng.uniform(-9, -5, size=zeros.shape)).astype(np.float32))
        scales *= rng.choice([-1, 1, 1, 1], size=zeros.shape).astype(np.float32)
        self.q = torch.from_numpy(oa.pack(codes, zeros, scales)).cuda()
        W = oa.decode(codes, zeros, scales)
        z, s = (np.repeat(v.astype(np.float64), group, axis=1) for v in (zeros, scales))
        t = lambda w: w.reshape(self.E, do, di).transpose(0, 2, 1)
        self.W, self.M = t(W), t(128 * np.abs(s) * (1.12 + np.abs(1 + z / 128)))
        self.Xh, self.dYh = host(self.X), host(self.dY)
        self.kw = dict(top_k=top_k, x_order=x_order, y_order=y_order)

    def layer(self, rows=None):
        from adapter_lora_segments_amd import AffineLinear
        return AffineLinear(self.q, self.E, self.di, self.do, rows or self.rows, group=self.group, **self.kw)

    def check_y(self, Y, codes=None):
        if codes is None:                             # at most 16 rows a group: the codes as they are
            codes = self.rows <= 16 * min(self.E, self.rows)
        want, S, owned = ox.forward(self.Xh, self.W, self.off, self.order, self.rows, **self.kw)
        if codes:
            _, B, _ = ox.forward(self.Xh, self.M, self.off, self.order, self.rows, **self.kw)
            more = (self.group + self.di // self.group + 16) * 2.0 ** -23 * B
        else:
            more = (2.0 ** -8 + (self.di + 2) * 2.0 ** -23) * S
        bound = 2.0 ** -8 * np.abs(want) + more * (1 + 2.0 ** -8)
        err = np.abs(host(Y) - want)
        assert (err[owned] <= bound[owned]).all(), (err[owned] / bound[owned]).max()
        return owned

    def check_dx(self, dX):
        want, S, owned, _, _ = ox.backward(self.dYh, None, self.W, self.off, self.order, self.rows, **self.kw)
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + (self.do + 2) * 2.0 ** -23) * S * (1 + 2.0 ** -8)
        err = np.abs(host(dX) - want)
        assert (err[owned] <= bound[owned]).all(), (err[owned] / bound[owned]).max()
        return owned


SIZES = {"one": [1], "few": [3, 0, 1, 7, 16, 5], "thirty": [31, 17, 0, 40, 25], "sixty": [64, 1, 130, 0, 65],
         "hundreds": [200, 129, 0, 301], "big": [513, 700]}


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("group,di", [(32, 32), (32, 96), (32, 544), (64, 64), (64, 192), (64, 1088), (128, 128), (128, 640),
                                      (128, 4736)])
def test_products(sizes, group, di):
    import torch
    say(f"affine {sizes} {group} {di}")
    x_order = sizes in ("few", "sixty", "big")
    y_order = sizes in ("few", "hundreds")
    for n, do in enumerate((8, 264)):
        c = Case(SIZES[sizes], di, do, group, top_k=2 if x_order else 1, x_order=x_order, y_order=y_order, dropped=3,
                 odd_zero=n == 1)
        L = c.layer()
        Y = torch.full((c.rows, do), 7.5, dtype=torch.bfloat16, device="cuda")
        L.forward(c.X, c.d_off, c.d_order, Y)
        owned = c.check_y(Y)
        assert (Y[torch.from_numpy(~owned).cuda()] == 7.5).all(), "rows of no group were written"
        dX = torch.full((c.rows, di), 7.5, dtype=torch.bfloat16, device="cuda")
        L.backward(c.dY, c.d_off, c.d_order, dX)
        owned = c.check_dx(dX)
        assert (dX[torch.from_numpy(~owned).cuda()] == 7.5).all(), "rows of no group were written"


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 64, 65, 127, 300])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_weight(rows, group):
    """A weight without experts: no tables; wide outputs, a tile that ends inside."""
    say(f"affine one weight {rows} {group}")
    c = Case([rows], 512 + group, 1032, group, seed=rows)
    L = c.layer(rows=rows + 40)
    c.check_y(L.forward(c.X))
    c.check_dx(L.backward(c.dY))


def test_many_experts():
    c = Case([1, 0] * 2048, 64, 16, 64, x_order=True, top_k=2, y_order=True)
    L = c.layer()
    c.check_y(L.forward(c.X, c.d_off, c.d_order))
    c.check_dx(L.backward(c.dY, c.d_off, c.d_order))


def test_no_rows_and_fewer_rows():
    import torch
    c = Case([40, 30], 128, 64, 32)
    L = c.layer(rows=2000)
    assert L.forward(c.X[:0], c.d_off, c.d_order[:0]).shape == (0, 64)
    assert L.backward(c.dY[:0], c.d_off, c.d_order[:0]).shape == (0, 128)
    c.check_y(L.forward(c.X, c.d_off, c.d_order))
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    Y = torch.full((70, 64), 7.5, dtype=torch.bfloat16, device="cuda")
    L.forward(c.X, z, c.d_order, Y)
    assert (Y == 7.5).all()


def test_rows_that_are_not_finite_stay_alone():
    """A row with an infinity or a NaN is lost, its neighbours in the tile are not."""
    import torch
    for rows in (9, 200):
        c = Case([rows], 256, 72, 64)
        L = c.layer()
        want = L.forward(c.X)
        X = c.X.clone()
        X[2, 5], X[4, 100] = np.inf, np.nan
        got = L.forward(X)
        assert not torch.isfinite(got[2]).any() and torch.isnan(got[4]).all()
        keep = [i for i in range(rows) if i not in (2, 4)]
        assert torch.equal(got[keep], want[keep])


def test_groups_that_are_not_finite_stay_in_their_column():
    import torch
    c = Case([20], 256, 72, 64)
    want = c.layer().forward(c.X)
    q = c.q.clone()
    q[72 * 128 + (17 * 4 + 1) * 4 + 3] = 0x7f        # the scale of column 17's second group: NaN
    q[72 * 128 + (17 * 4 + 1) * 4 + 2] = 0xc0
    c.q = q
    got = c.layer().forward(c.X)
    assert torch.isnan(got[:, 17]).all()
    keep = [i for i in range(72) if i != 17]
    assert torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("rows", [12, 300])
def test_tables_that_name_no_row(rows):
    """Offsets past the rows and orders outside them reach no memory outside the buffers."""
    import torch
    c = Case([rows], 64, 64, 32, x_order=True, y_order=True)
    L = c.layer()
    Y = torch.full((rows, 64), 7.5, dtype=torch.bfloat16, device="cuda")
    order = c.d_order.clone()
    order[3], order[5] = -7, 2 ** 31 - 1
    off = torch.tensor([-5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    L.forward(c.X, off, order, Y)
    gone = sorted(int(c.order[i]) for i in (3, 5))
    assert (Y[gone] == 7.5).all()
    keep = [i for i in range(rows) if i not in gone]
    assert torch.equal(Y[keep], L.forward(c.X, c.d_off, c.d_order)[keep])


# ---- the quantizer ----

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("symmetric", [False, True])
def test_quantize(group, dt, symmetric):
    import torch
    from adapter_lora_segments_amd import mlora_affine_quantize
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    for rows, n in ((1, 1), (7, 3), (130, 5), (1000, 32)):
        say(f"quantize {rows} {n * group} {dt} {symmetric}")
        rng = np.random.default_rng(rows)
        x = rng.standard_normal((rows, n * group)) * np.exp2(rng.uniform(-20, 20, size=(rows, 1)))
        x = x + rng.choice([0, 0, 3, -3], size=(rows, 1)) * np.abs(x).max(axis=1, keepdims=True)
        if rows > 100:
            x[3] = 0
            x[4, :group] = 1e-44
            x[5, 2] = np.nan
            x[6, group - 1] = -np.inf
            x[7] = 3e38
            x[8, 1::2] = -3e38
            x[9] = np.abs(x[9])
            x[10] = -np.abs(x[10])
            x[11] = 1e-38 * rng.standard_normal(n * group)
            x[12] = rng.integers(-8, 8, size=n * group)
        X = torch.from_numpy(x.astype(np.float32)).to(t).cuda()
        V = torch.empty_like(X)
        q = mlora_affine_quantize(X, values=V, group=group, symmetric=symmetric)
        c, z, s = oa.quantize(X.float().cpu().numpy(), group, symmetric)
        gc, gz, gs = oa.unpack(q.cpu().numpy(), rows, n * group, group)
        assert np.array_equal(gs, s, equal_nan=True) and np.array_equal(gz, z) and np.array_equal(gc, c)
        v = torch.from_numpy(oa.decode(c, z, s)).to(torch.float32).to(t)
        assert torch.equal(torch.nan_to_num(V.cpu(), nan=12345.0), torch.nan_to_num(v, nan=12345.0))
        wide = torch.zeros(rows, n * group + 16, dtype=t, device="cuda")
        wide[:, 8:-8] = X
        assert torch.equal(mlora_affine_quantize(wide[:, 8:-8], group=group, symmetric=symmetric), q)


def test_quantize_then_multiply():
    """The buffer that the quantizer makes is the one that the products read."""
    import torch
    from adapter_lora_segments_amd import AffineLinear, mlora_affine_quantize
    W = torch.randn(264, 512, device="cuda") * 0.02
    V = torch.empty_like(W)
    q = mlora_affine_quantize(W, values=V, group=64)
    X = torch.randn(5, 512, device="cuda").to(torch.bfloat16)
    y = AffineLinear(q, 1, 512, 264, 5, group=64).forward(X)
    want = host(X) @ host(V).T
    assert np.abs(host(y) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-4
