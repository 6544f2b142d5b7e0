"""GPU parity of sbt_add_rms_norm and its gradient with their definitions in 64 bits.

Bounds.  h is one fp32 addition and one rounding to the type.  y is that
addition (2^-24 of h), a mean of C squares (C + 2 roundings, halved by the
root), a division, a root and two products: (C / 2 + 8) 2^-23 of |y| in fp32,
and one rounding to the type; rows of fp32 sums that are added in a tree stay
far below C / 2.  A code is y / 2^e to half a step: half of 2^-3 (E4M3) or 2^-2
(E5M2) of its value, or half of the smallest step, in units of the scale; y's
own fp32 error may move it to the next code where it is that close to a border,
so it is added.  dx is a difference of two terms of up to |g| s each, with the
row sums' errors; dweight a sum of `rows` terms.
"""
import numpy as np
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
import step_ref as ref
from gpu_helpers import Canvas

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16", "f16"]
EPS = 1e-6


class Rows:
    """A [rows][cols] input inside NaN padding, `offset` elements into its buffer, rows `pad` apart."""

    def __init__(self, values, kind, pad=0, offset=0):
        self.rows, self.cols = values.shape
        self.ld, self.offset, self.dt = self.cols + pad, offset, ref.TDT[kind]
        self.buf = torch.full((self.rows * self.ld + offset + 16,), float("nan"), dtype=self.dt)
        self.view = self.buf.as_strided((self.rows, self.cols), (self.ld, 1), offset)
        self.view.copy_(values.to(self.dt))
        self.dev = self.buf.cuda()
        self.ptr = self.dev.data_ptr() + offset * self.buf.element_size()

    def f64(self):
        return ref.f64(self.view)

    def back(self):
        """What the device buffer holds now; padding must still be NaN."""
        b = self.dev.cpu()
        got = b.as_strided((self.rows, self.cols), (self.ld, 1), self.offset).clone()
        b.as_strided((self.rows, self.cols), (self.ld, 1), self.offset).fill_(float("nan"))
        assert torch.isnan(b.float()).all()
        return ref.f64(got)


class Out:
    """An output of `rows` rows inside guard bands; bytes between rows must keep the canary."""

    def __init__(self, rows, cols, es, pad=0, offset=0):
        self.rows, self.cols, self.es, self.ld, self.offset = rows, cols, es, cols + pad, offset
        self.c = Canvas((rows * self.ld + offset) * es)
        self.ptr = self.c.ptr + offset * es

    def get(self, dt=None):
        assert self.c.guards_intact()
        n = self.rows * self.ld + self.offset
        b, o = (x[self.offset:].reshape(self.rows, self.ld, self.es)
                for x in (self.c.inner(np.uint8, (n, self.es)), self.c.original(np.uint8, (n, self.es))))
        assert np.array_equal(b[:, self.cols:], o[:, self.cols:])
        assert np.array_equal(self.c.inner(np.uint8, (n, self.es))[:self.offset],
                              self.c.original(np.uint8, (n, self.es))[:self.offset])
        raw = np.ascontiguousarray(b[:, :self.cols])
        return raw[..., 0] if dt is None else ref.f64(torch.from_numpy(raw).view(dt)[..., 0])


def inputs(seed, rows, cols, kind, pad=0, offset=0, r=True):
    g = torch.Generator().manual_seed(seed)
    x = Rows(torch.randn(rows, cols, generator=g) * 0.7, kind, pad, offset)
    res = Rows(torch.randn(rows, cols, generator=g) * 2.5, kind, pad, offset) if r else None
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(ref.TDT[kind])
    return x, res, w


def y_bound(y, kind, cols):
    with np.errstate(invalid="ignore"):
        return (ref.HALF_ULP[kind] * 1.01 + (cols / 2 + 8) * 2.0**-23) * np.abs(y) + ref.TINY[kind]


def check_h(got, h, kind):
    assert (np.abs(got - h) <= (ref.HALF_ULP[kind] * 1.01 + 2.0**-23) * np.abs(h) + ref.TINY[kind]).all()


def check_codes(codes, scales, y, fmt, block, cols):
    """Scales exactly (or next to the border that y's own error reaches), codes within half a step."""
    rows = y.shape[0]
    want = ref.scale_exponents(y, fmt, block)
    err = (cols / 2 + 8) * 2.0**-23
    lo, hi = ref.scale_exponents(y * (1 - err), fmt, block), ref.scale_exponents(y * (1 + err), fmt, block)
    for i in range(rows):
        for j in range(cols // block):
            if want[i, j] is None:
                assert scales[i, j] == 255
            else:
                assert lo[i, j] <= int(scales[i, j]) - 127 <= hi[i, j], (i, j, scales[i, j], want[i, j])
    s = np.repeat(ref.code_values(scales, "e8m0"), block, 1)
    v = ref.code_values(codes, fmt) * s
    nan = np.isnan(s)
    assert np.array_equal(np.isnan(v), nan)
    half = {"e4m3": 2.0**-4, "e5m2": 2.0**-3}[fmt]
    with np.errstate(invalid="ignore"):
        ok = np.abs(v - y) <= half * np.abs(y) * (1 + 2 * half) + ref.CODES[fmt][2] / 2 * s + err * np.abs(y)
    assert (ok | nan).all()


CASES = [  # rows, cols, pad, offset: one thread's unit, a warp, several warps, every register form, odd widths, wide rows
    (1, 1, 0, 0), (3, 8, 0, 0), (5, 16, 0, 0), (2, 64, 8, 0), (7, 100, 0, 0), (9, 256, 0, 0), (700, 256, 0, 0),
    (5, 257, 0, 0), (33, 1000, 24, 8), (4, 1000, 1, 3), (1, 4096, 0, 0), (610, 2048, 0, 0), (3, 5003, 0, 0),
    (400, 1537, 0, 0), (2, 8192, 0, 0), (311, 8192, 0, 0), (2, 16384, 0, 0), (2, 16385, 0, 0), (1, 40000, 0, 0),
    (2, 33000, 8, 0),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward(ctx, case, kind):
    rows, cols, pad, offset = CASES[case]
    x, r, w = inputs(case, rows, cols, kind, pad, offset)
    es = x.buf.element_size()
    h_out, y = Out(rows, cols, es, pad, offset), Out(rows, cols, es, pad, offset)
    wd = w.cuda()
    sbt.add_rms_norm(ctx, x.ptr, x.ld, rows, cols, weight=wd, eps=EPS, r=r.ptr, ld_r=r.ld, h_out=h_out.ptr,
                     ld_h=h_out.ld, y=y.ptr, ld_y=y.ld, dtype=kind)
    h64, y64 = ref.add_rms_norm(x.f64(), r.f64(), ref.f64(w), EPS)
    torch.cuda.synchronize()
    check_h(h_out.get(x.dt), h64, kind)
    assert (np.abs(y.get(x.dt) - y64) <= y_bound(y64, kind, cols)).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("parts", ["no residual", "no weight", "neither", "in place h", "in place y"])
def test_forms(ctx, parts, kind):
    rows, cols = 13, 520
    x, r, w = inputs(5, rows, cols, kind, pad=8)
    no_r, no_w = parts in ("no residual", "neither"), parts in ("no weight", "neither")
    h64, y64 = ref.add_rms_norm(x.f64(), None if no_r else r.f64(), None if no_w else ref.f64(w), EPS)
    out = Out(rows, cols, x.buf.element_size())
    wd = None if no_w else w.cuda()
    kw = dict(weight=wd, eps=EPS, dtype=kind)
    if not no_r:
        kw.update(r=r.ptr, ld_r=r.ld)
    if parts == "in place h":
        sbt.add_rms_norm(ctx, x.ptr, x.ld, rows, cols, h_out=r.ptr, ld_h=r.ld, y=out.ptr, ld_y=out.ld, **kw)
        check_h(r.back(), h64, kind)
    elif parts == "in place y":
        sbt.add_rms_norm(ctx, x.ptr, x.ld, rows, cols, h_out=out.ptr, ld_h=out.ld, y=x.ptr, ld_y=x.ld, **kw)
        check_h(out.get(x.dt), h64, kind)
    else:
        sbt.add_rms_norm(ctx, x.ptr, x.ld, rows, cols, y=out.ptr, ld_y=out.ld, **kw)
    got = x.back() if parts == "in place y" else out.get(x.dt)
    assert (np.abs(got - y64) <= y_bound(y64, kind, cols)).all()


CODE_CASES = [  # rows, cols, block, pad of inputs and codes, offset
    (3, 32, 32, 0, 0), (5, 64, 16, 0, 0), (4, 4096, 32, 0, 0), (700, 512, 32, 0, 0), (2, 384, 128, 0, 0),
    (9, 1024, 64, 8, 8), (3, 96, 32, 1, 3), (2, 1280, 128, 5, 1), (2, 48, 16, 3, 0), (1, 20480, 32, 0, 0),
    (320, 8192, 32, 0, 0),
]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", range(len(CODE_CASES)))
def test_codes(ctx, case, kind, fmt):
    rows, cols, block, pad, offset = CODE_CASES[case]
    x, r, w = inputs(40 + case, rows, cols, kind, pad, offset)
    x.view[:, :block] = 0
    r.view[:, :block] = 0     # a block of zeros
    if cols > 2 * block:      # and one far below the others
        x.view[0, block:2 * block] *= 2.0**-14
        r.view[0, block:2 * block] *= 2.0**-14
    for m in (x, r):
        m.dev.copy_(m.buf)
    codes, scales = Out(rows, cols, 1, pad, offset), Out(rows, cols // block, 1, 3, 1)
    h_out, y = Out(rows, cols, x.buf.element_size()), Out(rows, cols, x.buf.element_size())
    wd = w.cuda()
    handle = sbt.code_rows(codes.ptr, codes.ld, scales.ptr, scales.ld, fmt=fmt, block=block)
    sbt.add_rms_norm(ctx, x.ptr, x.ld, rows, cols, weight=wd, eps=EPS, r=r.ptr, ld_r=r.ld, h_out=h_out.ptr,
                     ld_h=h_out.ld, y=y.ptr, ld_y=y.ld, codes=handle, dtype=kind)
    torch.cuda.synchronize()
    h64, y64 = ref.add_rms_norm(x.f64(), r.f64(), ref.f64(w), EPS)
    check_h(h_out.get(x.dt), h64, kind)
    assert (np.abs(y.get(x.dt) - y64) <= y_bound(y64, kind, cols)).all()
    sc = scales.get()
    check_codes(codes.get(), sc, y64, fmt, block, cols)
    assert (sc[:, 0] == 127).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("aligned", [True, False])
def test_codes_at_the_borders(ctx, fmt, aligned):
    """y exact: rows of +-1 (eps 0, so the root is 1) times weights that are borders of scales and halves of steps."""
    block, largest = 16, ref.CODES[fmt][1]
    w = torch.tensor([largest, largest / 2, 1.0, 17.0, 18.0, 2.0**-9, 2.0**-10, 3 * 2.0**-10, 0.0, 2.0**-3, 9.5, 10.5, 300.0,
                      0.75, 1.0625, 1.1875,                                    # scale 1
                      largest * (1 + 2.0**-23), *([1.0] * 15),                 # just past it: scale 2
                      largest * 2.0**-130, *([2.0**-140] * 15),                # below the least scale
                      2.0**120, *([2.0**119 * 1.75] * 15)], dtype=torch.float64).to(torch.float32)
    cols = w.numel()
    x = torch.ones(2, cols)
    x[1, ::2] = -1
    x = Rows(x, "f32", 0 if aligned else 1)
    codes, scales = Out(2, cols, 1), Out(2, cols // block, 1)
    wd = w.cuda()
    sbt.add_rms_norm(ctx, x.ptr, x.ld, 2, cols, weight=wd, eps=0.0, dtype="f32",
                     codes=sbt.code_rows(codes.ptr, codes.ld, scales.ptr, scales.ld, fmt=fmt, block=block))
    torch.cuda.synchronize()
    y = x.f64() * ref.f64(w)
    want = ref.scale_exponents(y, fmt, block)
    assert [list(v) for v in scales.get().astype(int) - 127] == [list(v) for v in want]
    s = np.repeat(2.0 ** want.astype(np.float64), block, 1)
    exact = torch.from_numpy(y / s).float().to(ref.CODES[fmt][0]).view(torch.uint8).numpy()  # to nearest even
    assert np.array_equal(codes.get(), exact)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cols", [64, 96, 1040])
def test_infinities_and_nan(ctx, cols, kind):
    """A NaN fills its row; an infinity makes NaN of itself and zeros of the rest; other rows do not see them."""
    x, r, w = inputs(9, 4, cols, kind)
    x.view[1, 40], x.view[2, 3] = float("nan"), float("inf")
    x.dev.copy_(x.buf)
    y, codes, scales = Out(4, cols, x.buf.element_size()), Out(4, cols, 1), Out(4, cols // 16, 1)
    wd = w.cuda()
    sbt.add_rms_norm(ctx, x.ptr, x.ld, 4, cols, weight=wd, eps=EPS, r=r.ptr, ld_r=r.ld, y=y.ptr, ld_y=y.ld, dtype=kind,
                     codes=sbt.code_rows(codes.ptr, codes.ld, scales.ptr, scales.ld, block=16))
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        _, y64 = ref.add_rms_norm(x.f64(), r.f64(), ref.f64(w), EPS)
    got, sc = y.get(x.dt), scales.get()
    assert np.isnan(got[1]).all() and (sc[1] == 255).all()
    assert np.array_equal(np.isnan(got[2]), np.arange(cols) == 3) and (got[2][np.arange(cols) != 3] == 0).all()
    assert sc[2, 0] == 255 and (sc[2, 1:] == 127).all()
    check_codes(codes.get()[[0, 3]], sc[[0, 3]], y64[[0, 3]], "e4m3", 16, cols)
    assert (np.abs(got - y64)[[0, 3]] <= y_bound(y64, kind, cols)[[0, 3]]).all()


# ---------------------------------------------------------------------------- gradient

def dx_bound(gy, gh, h, w, dx, kind, cols):
    norm = np.sqrt((h**2).mean(-1, keepdims=True) + EPS)
    g = np.abs(gy) * (1 if w is None else np.abs(w))
    terms = (g + np.abs(h) / norm * (g * np.abs(h) / norm).mean(-1, keepdims=True)) / norm
    return (ref.HALF_ULP[kind] * 1.01 * np.abs(dx) + ref.TINY[kind] + (cols + 24) * 2.0**-23 * terms
            + 2.0**-22 * (0 if gh is None else np.abs(gh)))


def dw_bound(gy, h, rows, cols):
    n = h / np.sqrt((h**2).mean(-1, keepdims=True) + EPS)
    return (rows + cols / 2 + 16) * 2.0**-23 * (np.abs(gy) * np.abs(n)).sum(0) + 1e-30


BWD = [  # rows, cols, pad, offset
    (1, 1, 0, 0), (5, 16, 0, 0), (4, 64, 8, 0), (37, 100, 0, 0), (1000, 256, 0, 0), (7, 257, 0, 0), (3, 1000, 1, 3),
    (650, 1024, 0, 0), (2, 4096, 0, 0), (310, 4096, 0, 0), (33, 1537, 0, 0), (5, 4097, 0, 0), (2, 8192, 0, 0),
    (3, 8200, 0, 0), (2, 20001, 0, 0), (40, 512, 0, 1), (1300, 32, 0, 0),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form", ["all", "no gh", "no weight", "in place"])
@pytest.mark.parametrize("case", range(len(BWD)))
def test_backward(ctx, case, form, kind):
    rows, cols, pad, offset = BWD[case]
    h, gy, w = inputs(70 + case, rows, cols, kind, pad, offset)
    gh = inputs(90 + case, rows, cols, kind, pad, offset)[0] if form != "no gh" else None
    w = None if form == "no weight" else w
    es = h.buf.element_size()
    dx, dw = Out(rows, cols, es, pad, offset), Out(1, cols, 4)
    n = sbt.add_rms_norm_backward_workspace_size(ctx, rows, cols)
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    wd = None if w is None else w.cuda()
    target = (gh.ptr, gh.ld) if form == "in place" else (dx.ptr, dx.ld)
    sbt.add_rms_norm_backward(ctx, gy.ptr, gy.ld, h.ptr, h.ld, rows, cols, *target, gh=None if gh is None else gh.ptr,
                              ld_gh=0 if gh is None else gh.ld, weight=wd, eps=EPS,
                              dweight=None if w is None else dw.ptr, workspace=ws, workspace_bytes=n, dtype=kind)
    torch.cuda.synchronize()
    assert (ws[n:] == 0xFF).all()
    a = gy.f64(), None if gh is None else ref.f64(gh.view), h.f64(), None if w is None else ref.f64(w)
    dx64, dw64 = ref.add_rms_norm_backward(*a, EPS)
    got = gh.back() if form == "in place" else dx.get(h.dt)
    assert (np.abs(got - dx64) <= dx_bound(*a, dx64, kind, cols)).all()
    if w is not None:
        got = dw.get(torch.float32)[0]
        assert (np.abs(got - dw64) <= dw_bound(a[0], a[2], rows, cols)).all()


def test_backward_of_no_rows(ctx):
    dw, w = torch.full((64,), 7.0, device="cuda"), torch.ones(64, device="cuda")
    sbt.add_rms_norm_backward(ctx, None, 64, None, 64, 0, 64, None, 64, weight=w, dweight=dw, dtype="f32")
    assert (dw == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_against_differences(ctx, kind):
    """Along a direction, against central differences of the definition in 64 bits."""
    rows, cols = 6, 320
    h, gy, w = inputs(3, rows, cols, kind)
    gh = inputs(4, rows, cols, kind)[0]
    dx, dw = Out(rows, cols, h.buf.element_size()), Out(1, cols, 4)
    n = sbt.add_rms_norm_backward_workspace_size(ctx, rows, cols)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    wd = w.cuda()
    sbt.add_rms_norm_backward(ctx, gy.ptr, gy.ld, h.ptr, h.ld, rows, cols, dx.ptr, dx.ld, gh=gh.ptr, ld_gh=gh.ld,
                              weight=wd, eps=EPS, dweight=dw.ptr, workspace=ws, workspace_bytes=n, dtype=kind)
    torch.cuda.synchronize()
    rng, t = np.random.default_rng(0), 1e-6
    u, v = rng.standard_normal((rows, cols)), rng.standard_normal(cols)
    f = lambda s: ((ref.add_rms_norm(h.f64() + s * t * u, None, ref.f64(w) + s * t * v, EPS)[1] * gy.f64()).sum()
                   + ((h.f64() + s * t * u) * gh.f64()).sum())
    got = (dx.get(h.dt) * u).sum() + (dw.get(torch.float32)[0] * v).sum()
    # the gradient's roundings add up over rows * cols terms; differences: t^2, and 2^-52 of the values over t
    bound = ref.HALF_ULP[kind] * np.abs(dx.get(h.dt) * u).sum() + 1e-4 * np.abs(dw.get(torch.float32) * v).sum() + 1e-3
    assert abs((f(1) - f(-1)) / (2 * t) - got) <= bound


def test_same_bits_from_run_to_run(ctx):
    rows, cols = 3000, 768
    h, gy, w = inputs(8, rows, cols, "bf16")
    n = sbt.add_rms_norm_backward_workspace_size(ctx, rows, cols)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    wd, seen = w.cuda(), []
    for _ in range(4):
        dx, dw = torch.empty(rows, cols, dtype=h.dt, device="cuda"), torch.empty(cols, device="cuda")
        sbt.add_rms_norm_backward(ctx, gy.ptr, gy.ld, h.ptr, h.ld, rows, cols, dx, cols, weight=wd, dweight=dw,
                                  workspace=ws, workspace_bytes=n, dtype="bf16")
        seen.append((dx.clone(), dw.clone()))
    assert all(torch.equal(a, b) for s in seen for a, b in zip(s, seen[0]))


def test_codes_feed_the_block_scaled_gemm(ctx):
    """The codes and scales are the GEMM's A operand as they stand: the product against 64 bits of the codes' values."""
    rows, cols, N, block = 65, 256, 72, 32
    x, r, w = inputs(11, rows, cols, "bf16")
    codes, scales = (torch.empty((rows, c), dtype=torch.uint8, device="cuda") for c in (cols, cols // block))
    wd = w.cuda()
    sbt.add_rms_norm(ctx, x.ptr, x.ld, rows, cols, weight=wd, r=r.ptr, ld_r=r.ld, dtype="bf16",
                     codes=sbt.code_rows(codes, cols, scales, cols // block, block=block))
    g = torch.Generator().manual_seed(2)
    B = torch.randint(0, 256, (cols, N // 2), generator=g, dtype=torch.uint8)
    sb = torch.randint(120, 130, (cols // block, N), generator=g, dtype=torch.uint8)
    D, Bd, sbd = torch.empty((rows, N), device="cuda"), B.cuda(), sb.cuda()
    need = sbt.gemm_block_scaled_workspace_size(ctx, rows, N, cols)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    sbt.gemm_block_scaled(ctx, codes, cols, Bd, N, scales, cols // block, sbd, N, cols // block, D, N, rows, N, cols,
                          workspace=ws, workspace_bytes=need, a_fmt="e4m3", b_fmt="e2m1")
    a = ref.code_values(codes.cpu().numpy(), "e4m3") * np.repeat(ref.code_values(scales.cpu().numpy(), "e8m0"), block, 1)
    want, mag = ref.matvec(a, ref.unpack_e2m1(B.numpy(), cols, N, N), ref.code_values(sb.numpy(), "e8m0"), block, 1.0)
    assert (np.abs(ref.f64(D) - want) <= (cols + 8) * 2.0**-23 * mag).all()
