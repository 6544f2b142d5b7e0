"""GPU parity of sbt_matvec_e2m1 with its definition in 64 bits.

Bound: every product and sum is fp32 (K + 64 roundings, of the magnitudes that are
summed, at 2^-23 since the matrix unit truncates); x enters off by 2^-39 of its
row's largest (bf16) and also by 2^-21 of itself (fp32); one rounding to y's type.
"""
import numpy as np
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
import step_ref as ref
from gpu_helpers import Canvas

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, seed, kind, tokens, K, N, scale="e8m0", group=32, out=None, alpha=1.0, pad=(0, 0, 0, 0),
                 offset=(0, 0, 0, 0)):
        rng = np.random.default_rng(seed)
        self.kind, self.out, self.T, self.K, self.N = kind, out or kind, tokens, K, N
        self.scale, self.group, self.alpha, self.offset = scale, group, alpha, offset
        self.ld_x, self.ldb = K + pad[0], N + N % 2 + 2 * pad[1]
        self.ld_s, self.ld_y = N + pad[2], N + pad[3]
        x = torch.from_numpy(rng.standard_normal((tokens, K)))
        x[:, ::37] *= 12
        self.x = torch.full((tokens * self.ld_x + offset[0],), float("nan"), dtype=ref.TDT[kind])
        self.xv = self.x.as_strided((tokens, K), (self.ld_x, 1), offset[0])
        self.xv.copy_(x.to(ref.TDT[kind]))
        # bytes past a row's or the array's last code are 0xFF: their columns are not computed from
        self.packed = np.full((K, self.ldb // 2), 0xFF, np.uint8)
        self.packed[:, :(N + 1) // 2] = rng.integers(0, 256, (K, (N + 1) // 2))
        self.scales = np.full((K // group, self.ld_s), 0xFF, np.uint8)
        self.scales[:, :N] = (rng.integers(110, 121, (K // group, N)) if scale == "e8m0"
                              else rng.integers(0, 256, (K // group, N)))
        if scale == "e4m3":
            self.scales[:, :N][(self.scales[:, :N] & 0x7F) == 0x7F] = 0x38  # no NaN

    def dev(self, a, offset):
        """Bytes on the device, `offset` bytes past an aligned address."""
        b = np.ascontiguousarray(a).reshape(-1).view(np.uint8)
        t = torch.empty(b.size + offset, dtype=torch.uint8, device="cuda")
        t[offset:] = torch.from_numpy(b.copy())
        self.keep.append(t)
        return t.data_ptr() + offset

    def run(self, ctx):
        self.keep = []
        es = {"f32": 4, "bf16": 2, "f16": 2}
        xd = self.x.cuda()
        y = Canvas((self.T * self.ld_y + self.offset[3]) * es[self.out])
        sbt.matvec_e2m1(ctx, xd.data_ptr() + self.offset[0] * es[self.kind], self.ld_x, self.T,
                        self.dev(self.packed, self.offset[1]), self.ldb, self.dev(self.scales, self.offset[2]), self.ld_s,
                        self.K // self.group, y.ptr + self.offset[3] * es[self.out], self.ld_y, self.N, self.K,
                        s_fmt=self.scale, alpha=self.alpha, dtype=self.kind, y_dtype=self.out)
        torch.cuda.synchronize()
        assert y.guards_intact()
        n = self.T * self.ld_y + self.offset[3]
        got, was = (f(np.uint8, (n, es[self.out])) for f in (y.inner, y.original))
        assert np.array_equal(got[:self.offset[3]], was[:self.offset[3]])
        got, was = (v[self.offset[3]:].reshape(self.T, self.ld_y, -1) for v in (got, was))
        assert np.array_equal(got[:, self.N:], was[:, self.N:])
        return ref.f64(torch.from_numpy(np.ascontiguousarray(got[:, :self.N])).view(ref.TDT[self.out])[..., 0])

    def want(self):
        codes = ref.unpack_e2m1(self.packed, self.K, self.N, self.ldb)
        s = ref.code_values(self.scales[:, :self.N], self.scale)
        x = ref.f64(self.xv)
        y, mag = ref.matvec(x, codes, s, self.group, self.alpha)
        bound = (self.K + 64) * 2.0**-23 * mag + ref.HALF_ULP[self.out] * 1.01 * np.abs(y) + ref.TINY[self.out]
        if self.kind != "f16":
            w = np.abs(ref.E2M1[codes] * np.repeat(s, self.group, 0)).sum(0) * abs(self.alpha)
            bound = bound + 2.0**-39 * np.abs(x).max(1, keepdims=True) * w + (2.0**-21 * mag if self.kind == "f32" else 0)
        return y, bound

    def check(self, ctx):
        got, (y, bound) = self.run(ctx), self.want()
        # fp16 rounds values from 65520 on to infinity
        over = np.abs(y) + bound >= 65520 if self.out == "f16" else np.zeros(y.shape, bool)
        assert np.isfinite(got[~over]).all() and (np.sign(got) == np.sign(y))[over].all()
        assert np.isinf(got[np.abs(y) - bound >= 65520]).all() or self.out != "f16"
        bad = (np.abs(got - y) > bound) & ~over
        assert not bad.any(), (np.argwhere(bad)[:5], (np.abs(got - y) / bound).max())


SIZES = [  # tokens, K, N
    (1, 32, 1), (1, 32, 2), (2, 64, 31), (3, 96, 255), (1, 256, 256), (4, 512, 257), (8, 320, 300), (9, 352, 64),
    (16, 1024, 513), (17, 288, 40), (40, 160, 33), (1, 4096, 600), (5, 2080, 1030), (16, 4096, 2048), (7, 32, 20000),
]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale,group", [("e8m0", 32), ("e4m3", 16), ("e4m3", 32), ("e8m0", 16)])
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_sizes(ctx, size, scale, group, kind):
    T, K, N = SIZES[size]
    Case(size, kind, T, K, N, scale, group, alpha=0.75).check(ctx)


@pytest.mark.parametrize("group", [16, 48, 64, 96, 128, 160, 960])
@pytest.mark.parametrize("scale", ["e8m0", "e4m3"])
def test_groups(ctx, scale, group):
    K = 960 if 960 % group == 0 else group * 7
    Case(group, "bf16", 3, K, 200, scale, group, out="f32").check(ctx)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens", [1, 12])
def test_types(ctx, tokens, out, kind):
    Case(1, kind, tokens, 384, 300, "e4m3", 16, out=out, alpha=2.0**-6).check(ctx)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale,group", [("e8m0", 32), ("e4m3", 16)])
@pytest.mark.parametrize("offset", range(0, 17, 3))
def test_strides_and_addresses(ctx, offset, scale, group, kind):
    """Rows of weights, scales, x and y that start on any byte (element) and are any distance apart."""
    Case(offset, kind, 3, 256, 270, scale, group, pad=(offset % 5, offset, 2 * offset + 1, offset % 3),
         offset=(offset % 4, offset, offset + 1, offset % 2)).check(ctx)
    Case(offset, kind, 10, 128, 511, scale, group, pad=(0, 0, offset, 0), offset=(0, 16, offset, 0)).check(ctx)


@pytest.mark.parametrize("tokens", [1, 16])
@pytest.mark.parametrize("K,N", [(64, 256), (128, 512), (480, 256), (8192, 256), (8192, 300), (2048, 40000)])
def test_splits_with_exact_sums(ctx, K, N, tokens):
    """Whole numbers whose sums are exact in fp32 whatever their order: a stage lost or counted twice shows."""
    c = Case(K, "f16", tokens, K, N, "e8m0", 32, out="f32")
    rng = np.random.default_rng(N)
    c.xv.copy_(torch.from_numpy(rng.integers(-2, 3, (tokens, K))).to(c.xv.dtype))
    c.scales[:, :N] = rng.integers(127, 130, (K // 32, N))
    y, _ = c.want()
    assert np.abs(y).max() < 2**22 and np.array_equal(c.run(ctx), y)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_wide_ranges_of_x(ctx, order, kind):
    """Rows whose magnitudes run over 60 powers of two along k, up or down, and differ from row to row."""
    c = Case(6, kind, 5, 2048, 64, "e8m0", 32, out="f32")
    e = np.linspace(-30, 30, 2048)
    e = e if order == "rising" else e[::-1]
    shift = np.array([0, 60, -60, 20, -80])[:, None]
    c.xv.copy_(torch.from_numpy(np.random.default_rng(1).standard_normal((5, 2048)) * 2.0 ** (e + shift)).to(c.xv.dtype))
    c.check(ctx)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_zeros_and_tiny_rows(ctx, kind):
    c = Case(2, kind, 4, 256, 64, out="f32")
    c.xv[0] = 0
    c.xv[1, 1:] = 0
    c.xv[2] *= 2.0**-10 if kind == "f16" else 2.0**-100
    got, (y, bound) = c.run(ctx), c.want()
    assert (got[0] == 0).all() and (np.abs(got - y) <= bound + 2.0**-140).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_infinities_and_nan_stay_in_their_row(ctx, value, kind):
    c = Case(3, kind, 9, 512, 96, out="f32")
    c.packed[200] = 0x21                       # the weights that meet it are not zero
    codes = ref.unpack_e2m1(c.packed, 512, 96, c.ldb)
    assert (ref.E2M1[codes[200]] != 0).all()
    y, bound = c.want()
    c.xv[4, 200] = value
    got = c.run(ctx)
    want = np.full(96, value) if np.isnan(value) else value * np.sign(ref.E2M1[codes[200]])
    assert np.array_equal(got[4], want, equal_nan=True)
    rest = [i for i in range(9) if i != 4]
    assert (np.abs(got - y)[rest] <= bound[rest]).all()


@pytest.mark.parametrize("scale,group,byte", [("e8m0", 32, 255), ("e4m3", 16, 0x7F), ("e4m3", 16, 0xFF), ("e8m0", 16, 255)])
def test_nan_scales_stay_in_their_column(ctx, scale, group, byte):
    c = Case(4, "bf16", 3, 256, 90, scale, group, out="f32")
    y, bound = c.want()
    c.scales[2, 33] = byte
    got = c.run(ctx)
    assert np.isnan(got[:, 33]).all()
    rest = [i for i in range(90) if i != 33]
    assert (np.abs(got - y)[:, rest] <= bound[:, rest]).all()


def test_scales_of_all_sizes(ctx):
    """E8M0 from its smallest (a subnormal number) up; E4M3's subnormals, zero and negative scales."""
    c = Case(5, "f16", 2, 512, 64, "e8m0", 32, out="f32")
    c.scales[:, :64] = np.arange(16)[:, None] * 15
    c.scales[0, :64] = 0
    got, (y, bound) = c.run(ctx), c.want()
    assert (np.abs(got - y) <= bound + 2.0**-130).all()
    c = Case(5, "f16", 2, 512, 64, "e4m3", 16, out="f32")
    c.scales[:, :64] = np.arange(32)[:, None] * 8
    c.check(ctx)


def test_no_k(ctx):
    y = torch.full((2, 40), 7.0, device="cuda")
    sbt.matvec_e2m1(ctx, None, 0, 2, None, 40, None, 40, 1, y, 40, 40, 0, dtype="bf16")
    assert (y == 0).all()


def test_offsets_past_32_bits(ctx):
    """Weights, scales and x more than 2^32 elements from their starts."""
    K, N, T = 64, 64, 2
    ldb, ld_s, ld_x = (1 << 27) + 32, (1 << 32) + 16, (1 << 31) + 64
    c = Case(9, "f16", T, K, N, out="f32")
    w, s = torch.zeros(K * ldb // 2, dtype=torch.uint8, device="cuda"), torch.zeros(2 * ld_s, dtype=torch.uint8, device="cuda")
    w.as_strided((K, N // 2), (ldb // 2, 1)).copy_(torch.from_numpy(c.packed))
    s.as_strided((2, N), (ld_s, 1)).copy_(torch.from_numpy(c.scales[:, :N].copy()))
    x = torch.zeros(ld_x + K, dtype=torch.float16, device="cuda")
    xv = x.as_strided((T, K), (ld_x, 1))
    xv.copy_(c.xv)
    y = torch.empty(T, N, device="cuda")
    sbt.matvec_e2m1(ctx, x, ld_x, T, w, ldb, s, ld_s, 2, y, N, N, K)
    want, bound = c.want()
    assert (np.abs(ref.f64(y) - want) <= bound).all()


def test_same_bits_and_the_gemm_agrees(ctx):
    """From run to run the same bits; x of E4M3 values gives the block-scaled GEMM's product."""
    c = Case(8, "f16", 6, 1024, 640, out="f32")
    codes = np.random.default_rng(0).integers(0, 0x78, (6, 1024)).astype(np.uint8)
    c.xv.copy_(torch.from_numpy(ref.code_values(codes, "e4m3")).to(torch.float16))
    first = c.run(ctx)
    assert all(np.array_equal(c.run(ctx), first) for _ in range(3))
    D, A = torch.empty(6, 640, device="cuda"), torch.from_numpy(codes).cuda()
    one = torch.full((6, 32), 127, dtype=torch.uint8, device="cuda")
    need = sbt.gemm_block_scaled_workspace_size(ctx, 6, 640, 1024)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    B, s = torch.from_numpy(c.packed).cuda(), torch.from_numpy(c.scales).cuda()
    sbt.gemm_block_scaled(ctx, A, 1024, B, 640, one, 32, s, 640, 32, D, 640, 6, 640, 1024, workspace=ws,
                          workspace_bytes=need, a_fmt="e4m3", b_fmt="e2m1")
    _, mag = ref.matvec(ref.f64(c.xv), ref.unpack_e2m1(c.packed, 1024, 640, 640), ref.code_values(c.scales, "e8m0"), 32, 1.0)
    assert (np.abs(ref.f64(D) - first) <= 2 * (1024 + 64) * 2.0**-23 * mag).all()


# More columns than there are blocks for: a block goes from tile to tile.  The rows of weights are whole multiples of 16
# bytes, the numbers of columns and the rows of scales are not.
WIDE = [("bf16", "e8m0", 32), ("f16", "e4m3", 16), ("f32", "e4m3", 32), ("bf16", "e8m0", 160)]


@pytest.mark.parametrize("kind,scale,group", WIDE)
@pytest.mark.parametrize("tokens", [1, 9, 35])
@pytest.mark.parametrize("K,N", [(320, 40000), (480, 60001), (1280, 39999)])
def test_many_columns(ctx, K, N, tokens, kind, scale, group):
    pad = -((N + 1) // 2) % 16
    Case(K + tokens, kind, tokens, K, N, scale, group, alpha=0.75, pad=(0, pad, N % 2 * 3, N % 2)).check(ctx)


@pytest.mark.parametrize("tokens", [2, 16])
@pytest.mark.parametrize("K", [32, 64, 96])
def test_many_columns_of_little_k(ctx, K, tokens):
    """Fewer stages than warps: some of them have nothing to add."""
    Case(K, "bf16", tokens, K, 80000, out="f32").check(ctx)


@pytest.mark.parametrize("tokens", [1, 16])
def test_many_columns_twice(ctx, tokens):
    """The order of the sums is fixed."""
    case = Case(3, "bf16", tokens, 1024, 50016, out="f32")
    assert np.array_equal(case.run(ctx), case.run(ctx))
