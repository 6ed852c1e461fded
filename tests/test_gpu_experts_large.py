"""Grouped expert products, row grouping and the MXFP4 quantizer at the largest
sizes that the interface takes, and past 32-bit offsets."""
import pytest

from tests.gpu_harness import say

pytestmark = pytest.mark.gpu


def test_most_rows():
    """One bf16 expert of 8 x 8 over 2^31 - 257 rows, 34 GB an operand: dW,
    which is summed in 256 chunks, and Y.  A few hundred rows hold small whole
    numbers (the ends of every chunk among them), the others zeros, so every
    sum is exact."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear
    R, d, C = 2 ** 31 - 257, 8, 2 ** 23
    if torch.cuda.mem_get_info()[0] < 3 * 2 * d * R + 2 ** 32:
        pytest.skip("needs 107 GB of free device memory")
    say("most rows: fill")
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randint(-4, 5, (1, d, d), generator=g, device="cuda").to(torch.bfloat16)
    X = torch.zeros(R, d, dtype=torch.bfloat16, device="cuda")
    dY = torch.zeros(R, d, dtype=torch.bfloat16, device="cuda")
    at = sorted({r for k in range(256) for r in (k * C, k * C + 12345, k * C + C - 1) if r < R} | {R - 1})
    x = torch.randint(-4, 5, (len(at), d), generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randint(-4, 5, (len(at), d), generator=g, device="cuda").to(torch.bfloat16)
    for i, r in enumerate(at):
        X[r].copy_(x[i])
        dY[r].copy_(dy[i])
    L = ExpertLinear(W, 1, d, d, R)
    assert L.ws is not None and L.ws.numel() >= 256 * d * d * 4
    torch.cuda.synchronize()
    say("most rows: dW")
    L.backward(dY, X, want_dx=False)
    torch.cuda.synchronize()
    assert torch.equal(L.dW[0].double(), x.double().t().contiguous() @ dy.double())
    del dY
    say("most rows: Y")
    Y = L.forward(X)
    torch.cuda.synchronize()
    want = (x.double() @ W[0].double()).to(torch.bfloat16)          # at most 128: exact
    assert torch.equal(torch.stack([Y[r] for r in at]), want)
    assert not Y[12346:100000].any() and not Y[R - C + 20000:R - 300].any()
    del X, Y
    torch.cuda.empty_cache()


def test_group_most_rows():
    """The most rows that a grouping takes: counts, and the order checked piece by
    piece (ascending rows of the right id)."""
    import torch
    from adapter_lora_segments_amd import RowGroups
    R, G, step = 2 ** 31 - 1, 64, 2 ** 27
    say("group most rows: fill")
    ids = torch.empty(R, dtype=torch.int32, device="cuda")
    counts = torch.zeros(G, dtype=torch.int64, device="cuda")
    for lo in range(0, R, step):
        i = torch.arange(lo, min(R, lo + step), device="cuda")
        v = (i * 2654435761 >> 7) % 67 - 1                   # -1 and 64, 65: no group
        ids[lo:lo + step] = v.int()
        counts += torch.bincount(v[(v >= 0) & (v < G)], minlength=G)
    say("group most rows: call")
    off, order = RowGroups(R, G).group(ids)
    torch.cuda.synchronize()
    ends = counts.cumsum(0)
    assert off[0] == 0 and torch.equal(off[1:].long(), ends)
    say("group most rows: check")
    n = int(ends[-1])
    for lo in range(0, n, step):
        at = torch.arange(lo, min(n, lo + step), device="cuda")
        g, o = torch.bucketize(at, ends, right=True), order[lo:lo + at.numel()].long()
        assert (o >= 0).all() and torch.equal(ids[o].long(), g)
        assert ((o[1:] > o[:-1]) | (g[1:] != g[:-1])).all()
        if lo > 0 and ids[order[lo - 1]] == ids[order[lo]]:
            assert order[lo - 1] < order[lo]
    assert (order[n:] == -1).all()
    del ids, order, at, g, o, i, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("along", ["cols", "rows"])
def test_quantize_past_32_bits(along):
    """A matrix of 9.7 GB, whose codes end behind the 2 GiB mark."""
    import numpy as np
    import torch
    from adapter_lora_segments_amd import mlora_microscale_quantize
    from oracle import experts as ox
    say(f"quantize past 32 bits {along}")
    rows, cols = 296000, 16384
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    ends = (0, 131072 - 32, 262144 - 32, rows - 32)
    for r in ends:
        x[r:r + 32] = torch.randn(32, cols, generator=g, device="cuda").to(x.dtype)
    v = torch.empty_like(x)
    q = mlora_microscale_quantize(x, values=v, along=along)
    n = rows * cols // 2
    for r in ends:
        h = x[r:r + 32].double().cpu().numpy()
        codes, scales = ox.quantize(h if along == "cols" else h.T)
        vals = ox.decode(codes, scales)
        if along == "rows":
            codes, vals = codes.T, vals.T
            got = q[n:].view(cols, rows // 32)[:, r // 32:r // 32 + 1]
        else:
            got = q[n:].view(rows, cols // 32)[r:r + 32]
        assert np.array_equal(got.cpu().numpy(), scales)
        packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
        assert np.array_equal(q[:n].view(rows, cols // 2)[r:r + 32].cpu().numpy(), packed)
        assert np.array_equal(v[r:r + 32].double().cpu().numpy(), vals)
    assert not v[64:1000].any() and not q[64 * cols // 2:1000 * cols // 2].any()
    del x, v, q
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [5, 300])
def test_codes_past_32_bits(rows):
    """MXFP4 weights of 5.4 GB: the last expert's products and dX."""
    import torch
    from adapter_lora_segments_amd import ExpertLinear, mlora_microscale_quantize
    E, di, do = 10, 32768, 32768
    g = torch.Generator(device="cuda").manual_seed(3)
    W = torch.randint(0, 256, (E * di * do // 2 + E * di * do // 32,), generator=g, device="cuda", dtype=torch.uint8)
    n = E * di * do // 2
    W[n:] = 113 + W[n:] % 8
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = rows
    off[E] = 2 * rows                                       # the first and the last expert
    X = torch.randn(2 * rows, di, generator=g, device="cuda").to(torch.bfloat16)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")

    def weight(e, c0, c1):                                  # columns c0 .. c1 of expert e: [c1 - c0][di]
        b = W[(e * do + c0) * di // 2:(e * do + c1) * di // 2].view(c1 - c0, di // 2)
        s = W[n + (e * do + c0) * di // 32:n + (e * do + c1) * di // 32].view(c1 - c0, di // 32)
        v = torch.stack([grid[(b & 15).long()], grid[(b >> 4).long()]], dim=2).view(c1 - c0, di // 32, 32)
        return (v * torch.exp2(s.double() - 127)[:, :, None]).view(c1 - c0, di)

    def near(got, want, S, K):
        ok = (got.double() - want).abs() <= 2.0 ** -8 * want.abs() + (K + 2) * 2.0 ** -23 * S * (1 + 2.0 ** -8)
        assert ok.all()

    for act in ("bf16", "mxfp4"):
        say(f"codes past 32 bits {rows} {act}")
        L = ExpertLinear(W, E, di, do, 2 * rows, w_layout="nk", w_format="mxfp4", act_format=act)
        Y = L.forward(X, off.cuda())
        V = X
        if act == "mxfp4":
            V = torch.empty_like(X)
            mlora_microscale_quantize(X, values=V)
        for e, at in ((0, slice(0, rows)), (E - 1, slice(rows, 2 * rows))):
            for c0 in (0, do - 256):
                w, x = weight(e, c0, c0 + 256).t().contiguous(), V[at].double()
                near(Y[at, c0:c0 + 256], x @ w, x.abs() @ w.abs(), di)
    say(f"codes past 32 bits {rows} dX")
    # dY of the first and last 128 columns only
    dY = torch.zeros(2 * rows, do, dtype=torch.bfloat16, device="cuda")
    dY[:, :128] = torch.randn(2 * rows, 128, generator=g, device="cuda").to(dY.dtype)
    dY[:, -128:] = torch.randn(2 * rows, 128, generator=g, device="cuda").to(dY.dtype)
    dX = L.backward(dY, None, off.cuda())
    for e, at in ((0, slice(0, rows)), (E - 1, slice(rows, 2 * rows))):
        w = torch.cat([weight(e, 0, 128), weight(e, do - 128, do)])
        d = torch.cat([dY[at, :128], dY[at, -128:]], dim=1).double()
        near(dX[at], d @ w, d.abs() @ w.abs(), do)
    del W, L
    torch.cuda.empty_cache()
