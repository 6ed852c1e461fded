"""Every form of the 4-bit products (the entries of csrc/affine_choice.hpp and the
decoded path) against the float64 oracle, each at a size whose rule names it,
with uneven groups, rows of no group and tiles that end inside; rows, weights
and outputs behind 4 GiB; tables and tolerances as in test_gpu_affine.py."""
import numpy as np
import pytest

from tests.gpu_harness import say
from tests.test_gpu_affine import Case

pytestmark = pytest.mark.gpu

# form: (rows, experts, d_in, d_out)
FORMS = {"few 4x16x1": (3, 1, 128, 72), "few 8x16x1": (300, 1, 128, 72), "few 8x32x1": (150, 1, 128, 264),
         "few 16x16x1": (500, 1, 128, 72), "few 16x32x2": (700, 8, 128, 72), "few 16x64x2": (300, 2, 128, 520),
         "few 32x32x2": (2000, 2, 128, 72), "few 32x64x2": (3000, 3, 128, 72), "few 32x128x4": (2000, 8, 128, 264),
         "tile 64x128x1": (4000, 5, 128, 264), "tile 64x128x2": (4000, 5, 512, 264),
         "tile 128x128x1": (1500, 8, 128, 2056), "tile 128x128x2": (3000, 3, 1152, 1032)}
DX_FORMS = {"tile 32x128x2": (3, 1, 128, 72), "tile 64x128x1": (1500, 2, 1152, 72),
            "tile 128x128x1": (3000, 8, 1152, 72)}


def sizes_of(rows, E, kind):
    """Rows of E groups that leave some out: even, or most of them in one group and one group empty."""
    n = rows - min(3, rows - 1)
    if E == 1:
        return [n]
    if kind == "even":
        return [n // E + (i < n % E) for i in range(E)]
    return [n - (E - 2) * 5] + [5] * (E - 2) + [0]


@pytest.mark.parametrize("kind", ["even", "skewed"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("form", list(FORMS))
def test_every_form(form, group, kind):
    import torch
    rows, E, di, do = FORMS[form]
    say(f"affine form {form} {group} {kind}")
    sizes = sizes_of(rows, E, kind)
    c = Case(sizes, di, do, group, dropped=rows - sum(sizes), x_order=True, y_order=kind == "even", odd_zero=True)
    assert c.rows == rows
    Y = torch.full((rows, do), 7.5, dtype=torch.bfloat16, device="cuda")
    c.layer().forward(c.X, c.d_off, c.d_order, Y)
    owned = c.check_y(Y, codes=form.startswith("few"))
    assert (Y[torch.from_numpy(~owned).cuda()] == 7.5).all()


@pytest.mark.parametrize("kind", ["even", "skewed"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("form", list(DX_FORMS))
def test_every_dx_form(form, group, kind):
    import torch
    rows, E, di, do = DX_FORMS[form]
    say(f"affine dX form {form} {group} {kind}")
    sizes = sizes_of(rows, E, kind)
    c = Case(sizes, di, do, group, dropped=rows - sum(sizes), x_order=True, y_order=kind == "even")
    dX = torch.full((rows, di), 7.5, dtype=torch.bfloat16, device="cuda")
    c.layer().backward(c.dY, c.d_off, c.d_order, dX)
    owned = c.check_dx(dX)
    assert (dX[torch.from_numpy(~owned).cuda()] == 7.5).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("sizes", [[1024], [1500, 0, 700, 1100], [4000, 60, 40]])
def test_decoded(sizes, group):
    """1024 rows an expert and more: the weights are decoded first."""
    say(f"affine decoded {sizes} {group}")
    c = Case(sizes, 2 * group + 128, 136, group, y_order=len(sizes) > 1, dropped=0 if len(sizes) == 1 else 800)
    L = c.layer()
    assert L.shape.forward_workspace_bytes and L.shape.backward_workspace_bytes
    c.check_y(L.forward(c.X, c.d_off, c.d_order), codes=False)
    c.check_dx(L.backward(c.dY, c.d_off, c.d_order))


@pytest.mark.parametrize("rows", [5, 300])
def test_orders_do_not_change_a_row(rows):
    """Rows in place, and the same rows read and written through the order: the same bits."""
    import torch
    from adapter_lora_segments_amd import AffineLinear
    c = Case([rows, 0, 2 * rows, 1], 256, 136, 64)
    Y = c.layer().forward(c.X, c.d_off, c.d_order)
    L = AffineLinear(c.q, 4, 256, 136, c.rows, group=64, x_order=True, y_order=True)
    p = c.d_order.long()
    X = torch.empty_like(c.X)
    X[p] = c.X
    assert torch.equal(L.forward(X, c.d_off, c.d_order)[p], Y)


@pytest.mark.parametrize("di,do", [(131072, 8), (128, 131072)])
@pytest.mark.parametrize("E", [1, 17, 1100])
def test_offsets_past_32_bits(E, di, do):
    """Rows of X, Y, dY and dX behind 4 GiB, and with 1100 experts of 131072 outputs
    a weight's codes too, in the few-row kernel, in tiles and decoded."""
    import torch
    from adapter_lora_segments_amd import AffineLinear, affine_bytes
    say(f"affine past 32 bits {E} {di} {do}")
    rows, n = 17000, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.zeros(affine_bytes(E * do, di, 128), dtype=torch.uint8, device="cuda")
    nc, np_ = do * di // 2, do * (di // 128)
    last = torch.randint(0, 256, (nc,), generator=g, dtype=torch.uint8, device="cuda")
    q[(E - 1) * nc:E * nc] = last
    q[E * nc:].view(torch.int32)[-np_:] = (0x3c00 << 16) | 0x4100      # scale 2^-7, zero point 8
    w = torch.empty(do, di, dtype=torch.float64, device="cuda")
    pairs = last.view(do, di // 2)
    w[:, 0::2], w[:, 1::2] = (pairs & 15).double() - 8, (pairs >> 4).double() - 8
    w /= 128
    L = AffineLinear(q, E, di, do, rows, group=128, x_order=True, y_order=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = n
    order = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    for call, a, b, m in ((L.forward, di, do, w.T.contiguous()), (L.backward, do, di, w)):
        x = torch.zeros(rows, a, dtype=torch.bfloat16, device="cuda")
        x[-n:] = torch.randn(n, a, generator=g, device="cuda").to(torch.bfloat16)
        y = call(x, off, order)
        assert y.shape == (rows, b) and not y[:-n].any()
        want, S = x[-n:].double() @ m, x[-n:].double().abs() @ m.abs()
        bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + (a + 2) * 2.0 ** -23) * S * 1.01
        assert ((y[-n:].double() - want).abs() <= bound).all()
