"""GPU parity of sbt_qk_norm_rope, its gradient and sbt_rope_table with their definitions in 64 bits.

Bounds: an output element is one rounding to the type plus at most D + 16
fp32 roundings of the magnitudes it was summed from (cache_ref returns those);
a weight's gradient, a sum over all rows, one rounding per row more.
"""
import numpy as np
import pytest
import torch

import cache_ref as ref
import scatter_boundary_tile_gb300 as sbt
from gpu_helpers import Canvas

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16", "f16"]
EPS = 1e-6


def bound(y, mag, kind, D):
    return ref.HALF_ULP[kind] * np.abs(y) * 1.01 + ref.TINY[kind] + (D + 16) * 2.0**-23 * mag


class Case:
    def __init__(self, seed, kind, tokens, q_heads, k_heads, D, rot, layout, pad=0, offset=0, n_pos=200, weights=True,
                 amplitude=1.0, bad_pos=True):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.dt, self.T, self.Hq, self.Hk, self.D = kind, ref.TDT[kind], tokens, q_heads, k_heads, D
        self.rot, self.layout, self.n_pos = rot, layout, n_pos
        self.ldh = D + pad
        self.ld = (q_heads + 2 * k_heads) * self.ldh + pad
        rnd = lambda *s: torch.randn(s, generator=g)
        self.buf = torch.full((tokens * self.ld + offset + 8,), float("nan"), dtype=self.dt)
        self.offset = offset
        self.q, self.k, self.v = (self.part(self.buf, 0, q_heads), self.part(self.buf, q_heads, k_heads),
                                  self.part(self.buf, q_heads + k_heads, k_heads))
        for x in (self.q, self.k, self.v):
            x.copy_((rnd(*x.shape) * 1.7).to(self.dt))
        self.gq, self.gk = rnd(tokens, q_heads, D).to(self.dt), rnd(tokens, k_heads, D).to(self.dt)
        self.wq = (1 + 0.2 * rnd(D)).to(self.dt) if weights else None
        self.wk = (1 + 0.2 * rnd(D)).to(self.dt) if weights else None
        self.pos = torch.randint(0, n_pos, (tokens,), generator=g).to(torch.int32)
        if bad_pos and tokens > 3:
            self.pos[1], self.pos[tokens // 2] = -1, n_pos
        self.table = torch.from_numpy(ref.rope_table(n_pos, rot, 10000.0, amplitude=amplitude)).float()

    def part(self, buf, head, heads):
        return buf.as_strided((self.T, heads, self.D), (self.ld, self.ldh, 1), self.offset + head * self.ldh)

    def turn(self):
        self.table_dev = self.table.cuda()
        return sbt.rope(self.table_dev if self.rot else None, self.n_pos, self.rot, self.layout)

    def ref_args(self):
        return EPS, ref.f64(self.table), self.pos.numpy().astype(np.int64), self.rot, self.layout, self.n_pos

    def want(self, x, w):
        return ref.norm_rope(ref.f64(x), None if w is None else ref.f64(w), *self.ref_args())

    def rows(self, canvas, heads):
        if heads == 0:
            return torch.empty((self.T, 0, self.D), dtype=self.dt)
        b = canvas.inner(np.uint8, (self.T, heads, self.D, self.buf.element_size())).copy()
        return torch.from_numpy(b).view(self.dt)[..., 0]

    def cuda(self, x):
        return None if x is None else x.cuda()

    def forward(self, ctx, path="auto", in_place=False):
        b, es = self.buf.cuda(), self.buf.element_size()
        q, k = (b.data_ptr() + (self.offset + h * self.ldh) * es for h in (0, self.Hq))
        if in_place:
            outs, qo, ko, ld, ldh = [b], q, k, self.ld, self.ldh
        else:
            outs = [Canvas(self.T * h * self.D * es) for h in (self.Hq, self.Hk)]
            qo, ko = outs[0].ptr, outs[1].ptr
        wq, wk, pos = self.cuda(self.wq), self.cuda(self.wk), self.pos.cuda()
        ctx.set_path(path)
        sbt.qk_norm_rope(ctx, q, self.ld, self.ldh, k, self.ld, self.ldh, self.T, self.Hq, self.Hk, self.D, pos,
                         self.turn(), qo, self.ld if in_place else self.Hq * self.D, self.ldh if in_place else self.D,
                         k_out=ko, ld_ko=self.ld if in_place else self.Hk * self.D,
                         ld_koh=self.ldh if in_place else self.D, q_weight=wq, k_weight=wk, eps=EPS, dtype=self.kind)
        torch.cuda.synchronize()
        ctx.set_path("auto")
        if in_place:
            back = b.cpu()
            return self.part(back, 0, self.Hq), self.part(back, self.Hq, self.Hk)
        assert all(o.guards_intact() for o in outs)
        return self.rows(outs[0], self.Hq), self.rows(outs[1], self.Hk)

    def check_forward(self, ctx, **kw):
        q, k = self.forward(ctx, **kw)
        for got, x, w in ((q, self.q, self.wq), (k, self.k, self.wk)):
            y, mag = self.want(x, w)
            assert np.all(np.abs(ref.f64(got) - y) <= bound(y, mag, self.kind, self.D))

    def backward(self, ctx, path="auto"):
        b, es = self.buf.cuda(), self.buf.element_size()
        q, k = (b.data_ptr() + (self.offset + h * self.ldh) * es for h in (0, self.Hq))
        D, gq, gk = self.D, self.gq.cuda(), self.gk.cuda()
        dq, dk = Canvas(self.T * self.Hq * D * es), Canvas(self.T * self.Hk * D * es)
        dw = [Canvas(D * 4) if self.wq is not None else None for _ in "qk"]
        n = sbt.qk_norm_rope_backward_workspace_size(ctx, D)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        wq, wk, pos = self.cuda(self.wq), self.cuda(self.wk), self.pos.cuda()
        ctx.set_path(path)
        torch.cuda.synchronize()
        sbt.qk_norm_rope_backward(ctx, gq, self.Hq * D, D, gk, self.Hk * D, D, q, self.ld, self.ldh, k, self.ld,
                                  self.ldh, self.T, self.Hq, self.Hk, D, pos, self.turn(), dq.ptr, self.Hq * D, D,
                                  dk.ptr, self.Hk * D, D, q_weight=wq, k_weight=wk, eps=EPS,
                                  dq_weight=dw[0] and dw[0].ptr, dk_weight=dw[1] and dw[1].ptr, workspace=ws,
                                  workspace_bytes=n, dtype=self.kind)
        torch.cuda.synchronize()
        ctx.set_path("auto")
        assert dq.guards_intact() and dk.guards_intact() and all(x is None or x.guards_intact() for x in dw)
        return self.rows(dq, self.Hq), self.rows(dk, self.Hk), *(None if x is None else x.inner(np.float32, (D,)).copy() for x in dw)

    def check_backward(self, ctx, **kw):
        got = self.backward(ctx, **kw)
        for i, (g, x, w) in enumerate(((self.gq, self.q, self.wq), (self.gk, self.k, self.wk))):
            dx, dw, mx, mw = ref.norm_rope_backward(ref.f64(g), ref.f64(x), None if w is None else ref.f64(w),
                                                    *self.ref_args())
            # dx goes through the norm and the mean over D: twice the roundings of the forward
            assert np.all(np.abs(ref.f64(got[i]) - dx) <= bound(dx, 2 * mx, self.kind, self.D))
            if w is not None:
                assert np.all(np.abs(got[2 + i] - dw) <= (g.shape[0] * g.shape[1] + self.D + 16) * 2.0**-23 * mw + 1e-30)
        return got


SHAPES = [  # D, rot, layout
    (128, 128, "half"), (128, 64, "half"), (128, 64, "interleaved"), (128, 0, "half"), (64, 64, "interleaved"),
    (80, 80, "half"), (80, 40, "interleaved"), (72, 40, "half"), (96, 32, "half"), (256, 256, "half"),
    (512, 512, "interleaved"), (1, 0, "half"), (2, 2, "half"), (33, 22, "interleaved"), (100, 50, "half"),
    (20, 6, "half"), (8, 8, "interleaved"), (16, 16, "half"), (24, 8, "interleaved"), (511, 2, "half")]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,rot,layout", SHAPES)
def test_forward_and_backward(ctx, kind, D, rot, layout):
    c = Case(1, kind, 37, 5, 2, D, rot, layout)
    c.check_forward(ctx)
    c.check_backward(ctx)
    c.check_forward(ctx, path="scalar")
    c.check_backward(ctx, path="scalar")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,q_heads,k_heads", [(1, 1, 1), (1, 32, 8), (3, 7, 1), (700, 12, 3), (5, 4, 0), (5, 0, 4)])
def test_tokens_and_heads(ctx, kind, tokens, q_heads, k_heads):
    c = Case(2, kind, tokens, q_heads, k_heads, 128, 128, "half")
    c.check_forward(ctx)
    c.check_backward(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad,offset", [(8, 8), (4, 4), (1, 0), (0, 1), (3, 5)])
def test_strides_and_alignment(ctx, kind, pad, offset):
    c = Case(3, kind, 19, 4, 2, 64, 32, "half", pad=pad, offset=offset)
    c.check_forward(ctx)
    c.check_backward(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("path", ["auto", "scalar"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place(ctx, kind, path, layout):
    Case(4, kind, 50, 6, 2, 128, 64, layout).check_forward(ctx, path=path, in_place=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("path", ["auto", "scalar"])
def test_without_norm(ctx, kind, path):
    c = Case(5, kind, 40, 4, 2, 64, 64, "half", weights=False, amplitude=1.25)
    c.check_forward(ctx, path=path)
    c.check_backward(ctx, path=path)


@pytest.mark.parametrize("path", ["auto", "scalar"])
def test_gradient_is_the_same_bits_every_run(ctx, path):
    c = Case(6, "bf16", 1500, 8, 2, 128, 128, "half")
    a, b = c.check_backward(ctx, path=path), c.backward(ctx, path=path)
    for x, y in zip(a, b):
        assert np.array_equal(np.asarray(x.view(torch.uint8) if torch.is_tensor(x) else x.view(np.uint8)),
                              np.asarray(y.view(torch.uint8) if torch.is_tensor(y) else y.view(np.uint8)))


@pytest.mark.parametrize("layout,rot", [("half", 24), ("interleaved", 16)])
def test_gradient_against_differences(ctx, layout, rot):
    """The kernel's fp32 gradient along random directions against central differences of the 64-bit forward.

    Step h = 1e-5: truncation h^2 times the third derivative (order 1) and 64-bit rounding 1e-16 / h are
    below 1e-9 of sums of order 10; the kernel's own error is the bound of check_backward."""
    c = Case(7, "f32", 9, 3, 2, 24, rot, layout)
    dq, dk, dwq, dwk = (np.asarray(ref.f64(x) if torch.is_tensor(x) else x, np.float64) for x in c.backward(ctx))
    rng = np.random.default_rng(8)
    for x, w, g, dx, dw in ((c.q, c.wq, c.gq, dq, dwq), (c.k, c.wk, c.gk, dk, dwk)):
        x, w, g = ref.f64(x), ref.f64(w), ref.f64(g)
        f = lambda x, w: (g * ref.norm_rope(x, w, *c.ref_args())[0]).sum()
        mx, mw = ref.norm_rope_backward(g, x, w, *c.ref_args())[2:]
        for _ in range(4):
            vx, vw, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-5
            num = (f(x + h * vx, w + h * vw) - f(x - h * vx, w - h * vw)) / (2 * h)
            got = (dx * vx).sum() + (dw * vw).sum()
            rows = x.shape[0] * x.shape[1]
            tol = (2 * 24 + 32) * 2.0**-23 * (mx * np.abs(vx)).sum() + (rows + 40) * 2.0**-23 * (mw * np.abs(vw)).sum()
            assert abs(num - got) <= tol + 1e-7


@pytest.mark.parametrize("kind", KINDS)
def test_no_tokens_gives_zero_weight_gradients(ctx, kind):
    D = 64
    n = sbt.qk_norm_rope_backward_workspace_size(ctx, D)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    w = torch.ones(D, dtype=ref.TDT[kind], device="cuda")
    dw = torch.full((2, D), 7.0, device="cuda")
    sbt.qk_norm_rope_backward(ctx, w, D, D, w, D, D, w, D, D, w, D, D, 0, 1, 1, D, None, None, w, D, D, w, D, D,
                              q_weight=w, k_weight=w, dq_weight=dw[0], dk_weight=dw[1], workspace=ws,
                              workspace_bytes=n)
    torch.cuda.synchronize()
    assert not dw.any()


# ---------------------------------------------------------------------------- append to the cache

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,rot,layout,pad", [(128, 128, "half", 0), (64, 32, "interleaved", 0), (80, 40, "half", 1),
                                              (33, 10, "half", 0)])
@pytest.mark.parametrize("order", ["nhd", "hnd"])
def test_append(ctx, kind, D, rot, layout, pad, order):
    P, S, mp, n_pages, Hk = 7, 5, 6, 40, 2
    c = Case(9, kind, 60, 4, Hk, D, rot, layout, pad=pad, n_pos=45)
    rng = np.random.default_rng(10)
    place = rng.permutation(S * mp * P)[:60]  # distinct places, some past the row, some on no page
    seq, pos = (place // (mp * P)).astype(np.int32), (place % (mp * P)).astype(np.int32)
    seq[3], seq[4], pos[5], pos[6] = -1, S, -1, mp * P  # none of these reaches the cache
    c.pos = torch.from_numpy(pos)
    table = rng.permutation(n_pages)[:S * mp].reshape(S, mp).astype(np.int32)
    table[2, 1], table[4, 0] = -1, n_pages
    d = D + pad
    ld_slot, ld_head = (Hk * d, d) if order == "nhd" else (d, P * d)
    ld_page = P * Hk * d
    es = c.buf.element_size()
    kc, vc = Canvas(n_pages * ld_page * es), Canvas(n_pages * ld_page * es)
    b, pos_d, seq_d, table_d = c.buf.cuda(), c.pos.cuda(), torch.from_numpy(seq).cuda(), torch.from_numpy(table).cuda()
    at = [b.data_ptr() + h * c.ldh * es for h in (0, 4, 4 + Hk)]
    qo = torch.empty((60, 4, D), dtype=c.dt, device="cuda")
    wq, wk = c.wq.cuda(), c.wk.cuda()
    sbt.qk_norm_rope(ctx, at[0], c.ld, c.ldh, at[1], c.ld, c.ldh, 60, 4, Hk, D, pos_d, c.turn(), qo, 4 * D, D,
                     q_weight=wq, k_weight=wk, eps=EPS, v=at[2], ld_v=c.ld, ld_vh=c.ldh,
                     cache=sbt.kv_cache(kc.ptr, vc.ptr, Hk, D, ld_page, ld_slot, ld_head),
                     map=sbt.page_map(table_d, mp, S, mp, None, n_pages, P), seq=seq_d, dtype=kind)
    torch.cuda.synchronize()
    assert kc.guards_intact() and vc.guards_intact()
    y, mag = c.want(c.q, c.wq)
    assert np.all(np.abs(ref.f64(qo) - y) <= bound(y, mag, kind, D))
    y, mag = c.want(c.k, c.wk)
    idt = np.uint16 if es == 2 else np.uint32
    got_k, got_v = kc.inner(idt, (n_pages * ld_page,)).copy(), vc.inner(idt, (n_pages * ld_page,)).copy()
    want_v = vc.original(idt, (n_pages * ld_page,)).copy()
    touched = np.zeros(n_pages * ld_page, bool)
    vbits = c.v.contiguous().view(torch.int16 if es == 2 else torch.int32).numpy().view(idt)
    tol = bound(y, mag, kind, D)
    kf = ref.f64(torch.from_numpy(got_k.view(np.int16 if es == 2 else np.int32)).view(c.dt))
    for t in range(60):
        s, p = int(seq[t]), int(pos[t])
        if not (0 <= s < S and 0 <= p < mp * P and (rot == 0 or p < c.n_pos)):
            continue
        page = table[s, p // P]
        if not 0 <= page < n_pages:
            continue
        for h in range(Hk):
            o = page * ld_page + (p % P) * ld_slot + h * ld_head
            assert np.all(np.abs(kf[o:o + D] - y[t, h]) <= tol[t, h])
            want_v[o:o + D] = vbits[t, h]
            touched[o:o + D] = True
    assert touched.any()
    assert np.array_equal(got_v, want_v)
    assert np.array_equal(got_k[~touched], kc.original(idt, (n_pages * ld_page,))[~touched])


# ---------------------------------------------------------------------------- table

@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="by_parts", factor=16.0, orig_len=4096, amplitude=1.277),
                                dict(base=500000.0)])
@pytest.mark.parametrize("n_pos,rot", [(1000, 128), (131, 2), (7, 46)])
def test_rope_table(ctx, kw, n_pos, rot):
    """Angles in 64 bits (a few ulps of 10^3 radians at most), then one rounding to fp32."""
    out = Canvas(n_pos * rot * 4)
    sbt.rope_table(ctx, out.ptr, n_pos, rot, **kw)
    torch.cuda.synchronize()
    assert out.guards_intact()
    r = {"orig_len": "orig"}
    args = {r.get(k, k): v for k, v in kw.items()}
    want = ref.rope_table(n_pos, rot, args.pop("base", 10000.0), **args)
    assert np.all(np.abs(out.inner(np.float32, (n_pos, rot // 2, 2)) - want) <= 2.0**-24 * 1.3 + 1e-11)


def test_rope_table_at_a_million(ctx):
    n, rot = 1 << 20, 4
    t = torch.empty((n, 2, 2), device="cuda")
    sbt.rope_table(ctx, t, n, rot)
    want = ref.rope_table(n, rot, 10000.0)[-1000:]
    assert np.abs(ref.f64(t[-1000:]) - want).max() <= 2.0**-24 + 1e-9


def test_refusals(ctx):
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    y, pos, t = torch.empty_like(x), torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros((8, 32, 2), device="cuda")
    cache = sbt.kv_cache(x, x, 2, 64, 128, 128, 64)
    pm = sbt.page_map(pos, 1, 4, 1, None, 1, 1)

    def call(T=4, D=64, rot=64, layout=0, k_out=y, v=None, cache=None, map=None, ld=128, heads=2, eps=1e-6):
        sbt.qk_norm_rope(ctx, x, 128, 64, x, 128, 64, T, 2, heads, D, pos, sbt.rope(t, 8, rot, layout), y, ld, 64,
                         k_out=k_out, ld_ko=128, ld_koh=64, eps=eps, v=v, ld_v=128, ld_vh=64, cache=cache, map=map)

    call()
    before = ctx.launch_count
    call(T=0)
    bad, uns = sbt.SBT_ERR_INVALID_ARG, sbt.SBT_ERR_UNSUPPORTED
    for kw, status in [({"T": -1}, bad), ({"D": 513}, bad), ({"rot": 63}, bad), ({"rot": 66}, bad), ({"layout": 5}, uns),
                       ({"k_out": None}, bad), ({"v": x}, bad), ({"cache": cache}, bad), ({"ld": 60}, bad),
                       ({"cache": cache, "map": pm, "heads": 1}, bad), ({"eps": -1.0}, bad)]:
        with pytest.raises(sbt.SbtError) as e:
            call(**kw)
        assert e.value.status == status, kw
    with pytest.raises(sbt.SbtError) as e:
        sbt.rope_table(ctx, t, 8, 64, scaling="by_parts", factor=2.0)
    assert e.value.status == bad
    with pytest.raises(sbt.SbtError) as e:
        sbt.qk_norm_rope_backward(ctx, x, 128, 64, x, 128, 64, x, 128, 64, x, 128, 64, 4, 2, 2, 64, pos, None, y, 128,
                                  64, y, 128, 64, q_weight=x)
    assert e.value.status == bad
    assert ctx.launch_count == before
