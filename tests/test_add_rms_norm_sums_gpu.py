"""The norm's row sums, every column of them: inputs whose sums are exact, or of a single element.

A column lost from a sum of `cols` squares, or counted twice, moves the output by about 1 / (2 cols) of itself, which
no bound that grows with the width would see.
"""
import numpy as np
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
import step_ref as ref

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16", "f16"]
# a unit, a warp, several warps, every register form with vectors and without, rows that start anywhere, wide rows
WIDTHS = [1, 8, 40, 256, 257, 1000, 1537, 2048, 4096, 4097, 5003, 8192, 8200, 16384, 16385, 20480, 40000]
ROOT = 4 * 2.0**-23  # of s: the mean, a root and a division, and the product with it


def rows_of(values, kind, pad):
    """Rows `pad` elements apart (and as many from an aligned address)."""
    rows, cols = values.shape
    buf = torch.zeros(rows * (cols + pad) + pad + 16, dtype=ref.TDT[kind], device="cuda")
    view = buf.as_strided((rows, cols), (cols + pad, 1), pad)
    view.copy_(values)
    return buf.data_ptr() + pad * buf.element_size(), cols + pad, view


def some_columns(cols, n):
    """The first and last columns, those about multiples of what threads, warps and blocks take, and others."""
    near = [k * u + d for u in (8, 32, 256, 512, 1024, 4096, 8192, 16384) for k in (1, 2, 3) for d in (-1, 0, 1)]
    rng = np.random.default_rng(cols)
    c = list(range(min(cols, 10))) + [cols - 1 - i for i in range(min(cols, 10))] + near + rng.integers(0, cols, n).tolist()
    return sorted({x for x in c if 0 <= x < cols})


def norm(ctx, x, ld_x, rows, cols, kind, pad, codes=None, r=None, ld_r=0):
    ptr, ld, y = rows_of(torch.zeros(rows, cols, device="cuda"), kind, pad)
    sbt.add_rms_norm(ctx, x, ld_x, rows, cols, eps=0.0, y=ptr, ld_y=ld, dtype=kind, codes=codes, r=r, ld_r=ld_r)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("cols", WIDTHS)
def test_rows_of_ones(ctx, cols, pad, kind):
    """Rows of +-1 have the root 1: they come back as they are.  (In 16 bits a few lost columns would round away.)"""
    for rows in (3, 310):
        x = torch.ones(rows, cols, device="cuda")
        x[1::2, ::3] = -1
        ptr, ld, v = rows_of(x, kind, pad)
        assert torch.equal(norm(ctx, ptr, ld, rows, cols, kind, pad), v)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("cols", WIDTHS)
def test_every_column_counts_once(ctx, cols, pad, kind):
    """A single 1 in a row comes back as the root of the width; lost, it would be divided by zero."""
    at = some_columns(cols, 40)
    for repeat in (1, -(-310 // len(at))):  # few rows, and more than two for every SM
        rows = len(at) * repeat
        x = torch.zeros(rows, cols, device="cuda")
        x[torch.arange(rows), torch.tensor(at * repeat)] = 1
        ptr, ld, v = rows_of(x, kind, pad)
        y = norm(ctx, ptr, ld, rows, cols, kind, pad).double()
        want = v.double() * cols**0.5
        assert ((y - want).abs() <= (ROOT + ref.HALF_ULP[kind] * 1.01) * want).all()


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("cols", [32, 512, 4096, 8192, 16384, 16416, 40000])
def test_every_column_counts_once_under_codes(ctx, cols, pad):
    """The same with codes: the root of the width, rounded to E4M3 times the scale of its block; a residual of zeros."""
    at = some_columns(cols, 20)
    rows = len(at)
    x = torch.zeros(rows, cols, device="cuda")
    x[torch.arange(rows), torch.tensor(at)] = 1
    ptr, ld, v = rows_of(x, "bf16", pad)
    rp, ldr, _ = rows_of(torch.zeros(rows, cols, device="cuda"), "bf16", pad)
    codes, scales = (torch.empty((rows, n), dtype=torch.uint8, device="cuda") for n in (cols, cols // 16))
    handle = sbt.code_rows(codes, cols, scales, cols // 16, block=16)
    y = norm(ctx, ptr, ld, rows, cols, "bf16", pad, codes=handle, r=rp, ld_r=ldr).double()
    want = v.double() * cols**0.5
    assert ((y - want).abs() <= (ROOT + ref.HALF_ULP["bf16"] * 1.01) * want).all()
    got = (torch.from_numpy(ref.code_values(codes.cpu().numpy(), "e4m3"))
           * torch.from_numpy(ref.code_values(scales.cpu().numpy(), "e8m0")).repeat_interleave(16, 1)).cuda()
    assert ((got - want).abs() <= (ROOT + 2.0**-4) * want).all()  # half of E4M3's step


def backward(ctx, gy, h, kind, pad, weight=True):
    """dx and dweight with eps 0 and weights of one."""
    rows, cols = h.shape
    g, h = rows_of(gy, kind, pad), rows_of(h, kind, pad)
    dx = rows_of(torch.zeros(rows, cols, device="cuda"), kind, pad)
    w = torch.ones(cols, dtype=ref.TDT[kind], device="cuda") if weight else None
    dw = torch.empty(cols, device="cuda") if weight else None
    n = sbt.add_rms_norm_backward_workspace_size(ctx, rows, cols)
    ws = torch.full((n + (1 << 20),), 0xFF, dtype=torch.uint8, device="cuda")
    sbt.add_rms_norm_backward(ctx, *g[:2], *h[:2], rows, cols, *dx[:2], weight=w, eps=0.0, dweight=dw, workspace=ws,
                              workspace_bytes=n, dtype=kind)
    torch.cuda.synchronize()
    assert (ws[n:] == 0xFF).all()
    return dx[2].double(), dw


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("cols", WIDTHS)
def test_every_column_of_the_gradients_sums_counts_once(ctx, cols, pad, kind):
    """h = +-1 (so the root is 1) and gy one at a single column c: dx_j = [j = c] - h_j h_c / cols, and dweight counts."""
    at = some_columns(cols, 40)
    rows = len(at)
    i, c = torch.arange(rows), torch.tensor(at)
    sign = torch.where(torch.arange(cols, device="cuda") % 3 == 0, -1.0, 1.0)
    h, gy = sign.expand(rows, cols), torch.zeros(rows, cols, device="cuda")
    gy[i, c] = 1
    dx, dw = backward(ctx, gy, h, kind, pad)
    want = gy.double() - h.double() * h[i, c].double()[:, None] / cols
    # the mean is off by one rounding, its product with 1 by none, a difference by one of its larger term
    bound = (ref.HALF_ULP[kind] * 1.01 + ROOT) * want.abs() + 2.0**-24 * gy + ref.TINY[kind]
    assert ((dx - want).abs() <= bound).all()
    assert torch.equal(dw.double(), (gy * h).double().sum(0))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("cols", [w for w in WIDTHS if w > 1])
def test_every_square_of_the_gradients_sums_counts_once(ctx, cols, pad, kind):
    """h one at a single column c, gy zero there: dx = gy sqrt(cols); a lost square would divide by zero."""
    at = some_columns(cols, 40)
    rows = len(at)
    i, c = torch.arange(rows), torch.tensor(at)
    h, gy = torch.zeros(rows, cols, device="cuda"), torch.ones(rows, cols, device="cuda")
    h[i, c], gy[i, c] = 1, 0
    dx, dw = backward(ctx, gy, h, kind, pad)
    want = gy.double() * cols**0.5
    assert ((dx - want).abs() <= (ROOT + ref.HALF_ULP[kind] * 1.01) * want).all()
    assert (dw == 0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(3000, 256), (700, 512), (700, 4096), (700, 4097), (3000, 8192), (700, 8200), (700, 16384),
                                       (5000, 40)])
@pytest.mark.parametrize("pad", [0, 1])
def test_every_row_counts_once_in_dweight(ctx, rows, cols, pad, kind):
    """h = +-1 and whole numbers in gy: dweight is a sum of whole numbers, exact in any order."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    h = torch.randint(0, 2, (rows, cols), generator=g, device="cuda").float() * 2 - 1
    gy = torch.randint(-8, 9, (rows, cols), generator=g, device="cuda").float()
    _, dw = backward(ctx, gy, h, kind, pad)
    assert torch.equal(dw.double(), (gy * h).double().sum(0))
