"""GPU parity of sbt_paged_tree_attention with its definition in 64 bits.

Bounds (step_ref.tree_attention_bounds): scores off by D + 3 roundings of their terms, sums over the
visible positions, probabilities of two 16-bit numbers (one where a key-value head has more than 128 rows of
up to 128 elements), one rounding to the type.
"""
import numpy as np
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
import step_ref as ref

pytestmark = pytest.mark.gpu
FILL = 7.5  # what out and lse hold before a call


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32).copy()).cuda()


def random_mask(rng, cu, rows, words, empty=0.1):
    """Any bits: ancestors, later tokens, tokens past the entry's last; some rows without one."""
    m = rng.integers(0, 2**32, (rows, words), dtype=np.uint64).astype(np.uint32)
    m[rng.random(rows) < empty] = 0
    return m.view(np.int32)


class Case:
    """Entries of (new tokens, context) over a pool whose other slots all hold NaN."""

    def __init__(self, seed, kind, sizes, kv=2, group=2, D=64, P=16, order="nhd", masked=True, max_new=None, extra=3,
                 words=None, pad=0, offset=0, scale=None, holes=0.0, std=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.kind, self.dt, self.kv, self.group, self.D, self.P, self.order = kind, ref.TDT[kind], kv, group, D, P, order
        self.n = np.array([n for n, _ in sizes])
        B = len(sizes)
        self.cu = np.concatenate([[0], np.cumsum(np.maximum(self.n, 0))])
        self.rows = int(self.cu[-1]) + extra
        self.max_new = max_new or max(1, int(self.n.max()))
        self.seq = rng.permutation(B + 1)[:B]
        self.lens = np.full(B + 1, -1)
        self.lens[self.seq] = [n + c for n, c in sizes]
        self.max_pages = max(1, -(-int(self.lens.max()) // P))
        need = [-(-max(int(x), 0) // P) for x in self.lens]
        self.n_pages = sum(need) + 2
        perm = rng.permutation(self.n_pages)
        self.table = np.full((B + 1, self.max_pages), -1)
        at = 0
        for s, c in enumerate(need):
            self.table[s, :c] = perm[at:at + c]
            at += c
        self.table[rng.random(self.table.shape) < holes] = self.n_pages + 5
        # the pool: element (page, slot, head, d) at the strides, everything else NaN
        ldh = D + pad
        if order == "nhd":
            self.ld = (P * kv * ldh + pad, kv * ldh, ldh)
        else:
            self.ld = (kv * P * ldh + pad, ldh, P * ldh)
        self.offset = offset
        size = self.n_pages * self.ld[0] + offset + 16
        self.k, self.v = (torch.full((size,), float("nan"), dtype=self.dt) for _ in "kv")
        held = np.zeros((self.n_pages, P), bool)
        for s in range(B + 1):
            for t in range(max(int(self.lens[s]), 0)):
                if self.table[s, t // P] < self.n_pages:
                    held[self.table[s, t // P], t % P] = True
        g = torch.Generator().manual_seed(seed)
        for x in (self.k, self.v):
            val = (torch.randn((self.n_pages, P, kv, D), generator=g) * std).to(self.dt)
            self.view(x).copy_(torch.where(torch.from_numpy(held)[:, :, None, None], val, torch.tensor(float("nan"), dtype=self.dt)))
        self.q = (torch.randn((self.rows, kv * group, D), generator=g) * 1.5).to(self.dt)
        self.words = words or max(1, -(-self.max_new // 32))
        self.mask = random_mask(rng, self.cu, self.rows, self.words) if masked else None
        self.scale = D**-0.5 if scale is None else scale

    def view(self, x):
        lp, ls, lh = self.ld
        return x.as_strided((self.n_pages, self.P, self.kv, self.D), (lp, ls, lh, 1), self.offset)

    def run(self, ctx, q_pad=0, out_pad=0):
        Hq, D, es = self.kv * self.group, self.D, 2
        kd, vd = self.k.cuda(), self.v.cuda()
        cache = sbt.kv_cache(kd.data_ptr() + self.offset * es, vd.data_ptr() + self.offset * es, self.kv, D, *self.ld)
        td, ld, cu, seq = i32(self.table), i32(self.lens), i32(self.cu), i32(self.seq)
        m = sbt.page_map(td, self.max_pages, len(self.lens), self.max_pages, ld, self.n_pages, self.P)
        qb = torch.full((self.rows * (Hq * (D + q_pad) + q_pad) + 8,), float("nan"), dtype=self.dt)
        qv = qb.as_strided((self.rows, Hq, D), (Hq * (D + q_pad) + q_pad, D + q_pad, 1), q_pad)
        qv.copy_(self.q)
        qb = qb.cuda()
        lo = (Hq * (D + out_pad) + out_pad, D + out_pad)
        out = torch.full((self.rows * lo[0] + out_pad + 8,), FILL, dtype=self.dt, device="cuda")
        lse = torch.full((self.rows, Hq), FILL, device="cuda")
        mask = None if self.mask is None else i32(self.mask)
        n = sbt.paged_tree_attention_workspace_size(ctx, self.max_new, Hq, self.kv, D)
        ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        self.call = lambda: sbt.paged_tree_attention(
            ctx, qb.data_ptr() + q_pad * es, lo[0] - out_pad * (Hq + 1) + q_pad * (Hq + 1), D + q_pad, self.rows, cu,
            len(self.n), self.max_new, Hq, cache, m, self.scale, out.data_ptr() + out_pad * es, *lo, mask=mask,
            ld_mask=self.words if mask is not None else 0, lse=lse, seq=seq, workspace=ws, workspace_bytes=n, dtype=self.kind)
        self.keep = (kd, vd, td, ld, cu, seq, qb, mask, ws)
        self.call()
        torch.cuda.synchronize()
        ctx.check_status()
        assert (ws[n:] == 0xFF).all()
        self.out_dev, self.lse_dev = out, lse
        flat = out.cpu()
        ov = flat.as_strided((self.rows, Hq, D), (*lo, 1), out_pad)
        got = ref.f64(ov)
        ov.fill_(FILL)
        assert (flat == FILL).all()  # nothing between the rows
        return got, ref.f64(lse)

    def want(self):
        return ref.tree_attention(ref.f64(self.q), ref.f64(self.view(self.k)), ref.f64(self.view(self.v)), self.table,
                                  self.lens, self.P, self.scale, self.cu, self.max_new, self.mask, self.seq)

    def bounds(self, want):
        return ref.tree_attention_bounds(want, self.kind, self.D, 1 if self.max_new * self.group > 128 and self.D <= 128 else 2)

    def check(self, ctx, **kw):
        got, lse = self.run(ctx, **kw)
        want = self.want()
        ob, sb = self.bounds(want)
        w = want[2]
        assert (got[~w] == FILL).all() and (lse[~w] == FILL).all()
        none = np.isneginf(want[1])
        assert np.array_equal(np.isneginf(lse[w]), none[w]) and (got[w][none[w]] == 0).all()
        err = np.abs(got - want[0])
        assert (err <= ob)[w].all(), (np.argwhere(~(err <= ob) & w[:, None, None])[:5], np.nanmax((err / ob)[w]))
        seen = w[:, None] & ~none
        assert (np.abs(lse - want[1]) <= sb)[seen].all()


KINDS = ["bf16", "f16"]
SIZES = [  # entries of (new tokens, context); heads, group, head size, page size, order
    ([(1, 0)], 1, 1, 64, 16, "nhd"), ([(1, 1)], 1, 1, 64, 1, "nhd"), ([(3, 61)], 1, 2, 64, 16, "nhd"),
    ([(5, 64), (1, 63), (7, 200)], 2, 4, 128, 16, "nhd"), ([(32, 500)], 2, 4, 128, 16, "hnd"),
    ([(33, 100)], 1, 4, 128, 64, "nhd"),                # 132 rows: two tiles of 128
    ([(64, 300), (2, 700), (17, 0)], 2, 8, 128, 32, "hnd"),  # up to 512 rows: planes
    ([(100, 129)], 1, 7, 64, 13, "nhd"), ([(9, 1000), (4, 3)], 3, 5, 80, 24, "nhd"), ([(6, 90)], 2, 3, 96, 16, "hnd"),
    ([(6, 90), (11, 257)], 1, 4, 192, 16, "nhd"), ([(40, 90)], 1, 8, 192, 16, "nhd"), ([(20, 333)], 2, 2, 256, 16, "nhd"),
    ([(40, 150)], 1, 8, 256, 8, "hnd"), ([(8, 2500)], 1, 1, 64, 16, "nhd"), ([(2, 5000)], 4, 16, 128, 64, "nhd"),
    ([(1 + i % 5, 37 * i % 300) for i in range(70)], 2, 2, 64, 16, "nhd"),
    ([(1 + i % 3, i % 90) for i in range(400)], 1, 1, 64, 16, "nhd"),
    ([(300, 10)], 1, 1, 64, 16, "nhd"), ([(12, 100)], 1, 40, 64, 16, "nhd"),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("masked", [True, False])
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_sizes(ctx, size, masked, kind):
    sizes, kv, group, D, P, order = SIZES[size]
    Case(size, kind, sizes, kv, group, D, P, order, masked).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [1, 2, 3, 8, 20, 36, 63, 65, 72, 100, 112, 130, 160, 200, 255])
def test_head_sizes(ctx, D, kind):
    Case(D, kind, [(5, 70), (3, 0), (20, 33)], 2, 3, D, 8).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad,offset", [(1, 0), (2, 1), (4, 0), (4, 2), (8, 4), (8, 8), (0, 3)])
def test_strides_and_addresses(ctx, pad, offset, kind):
    c = Case(pad + offset, kind, [(5, 70), (9, 200)], 2, 4, 64, 16, "hnd" if pad % 2 else "nhd", pad=pad, offset=offset)
    c.check(ctx, q_pad=pad, out_pad=offset)
    Case(3, kind, [(40, 90)], 1, 4, 128, 16, pad=offset, offset=pad).check(ctx, q_pad=offset, out_pad=pad)


@pytest.mark.parametrize("kind", KINDS)
def test_pages_that_are_not_there(ctx, kind):
    Case(1, kind, [(5, 300), (7, 10), (3, 64), (2, 0), (64, 500)], 2, 2, 64, 16, holes=0.3).check(ctx)
    Case(2, kind, [(40, 300), (3, 64)], 1, 4, 128, 16, holes=1.0).check(ctx)  # nobody sees anything


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("masked", [True, False])
def test_lengths_and_entries_that_are_not_legal(ctx, masked, kind):
    c = Case(4, kind, [(3, 50), (6, 20), (0, 9), (2, 30), (4, 4), (5, 6)], 2, 2, 64, 16, masked=masked, max_new=5)
    c.lens[c.seq[3]] = -7           # an empty sequence
    c.lens[c.seq[4]] = 2            # shorter than its new tokens: the first ones' positions do not exist
    c.seq[5] = 99                   # no such sequence
    c.check(ctx)                    # (the second entry has more than max_new tokens and is left out)
    c.lens[c.seq[0]] = 2**31 - 1    # longer than the table
    c.table[c.seq[0], 1:] = -1
    c.check(ctx)
    c.cu = np.array([2, 4, 3, 3, 100, 4, 9])  # backwards and past the end
    c.check(ctx)
    c.cu = np.array([-3, 2, 2, 4, 4, 4, 4])
    c.check(ctx)


@pytest.mark.parametrize("kind", KINDS)
def test_masks_that_leave_rows_empty(ctx, kind):
    c = Case(5, kind, [(40, 0), (5, 0), (3, 70)], 1, 4, 64, 16)
    c.mask[:] = 0
    c.check(ctx)
    c.mask[7, 0] = 1 << 3
    c.check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("words", [1, 3])
def test_masks_of_fewer_and_more_words_than_tokens(ctx, words, kind):
    Case(6, kind, [(50, 20), (3, 5)], 1, 2, 64, 16, words=words).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("where", ["key", "value"])
@pytest.mark.parametrize("sizes,group,D,P", [([(6, 30)], 2, 64, 16), ([(70, 100)], 4, 128, 8), ([(5, 61), (3, 3000)], 2, 100, 16),
                                             ([(9, 60)], 1, 36, 13), ([(9, 60)], 1, 35, 13), ([(70, 2000)], 4, 128, 16)])
def test_infinities_and_nan_among_the_new_tokens(ctx, sizes, group, D, P, where, value, kind):
    """They reach the rows that see their token and no other."""
    c = Case(7, kind, sizes, 1, group, D, P)
    n = int(c.n[0])
    token, s = n // 2, int(c.seq[0])
    pos = int(c.lens[s]) - n + token
    at = (int(c.table[s, pos // P]), pos % P, 0)
    want = c.want()
    clean = c.view(c.v if where == "value" else c.k)[at][1 if D > 1 else 0].item()
    assert np.isfinite(clean)
    c.view(c.v if where == "value" else c.k)[at][1] = value
    sees = np.zeros(c.rows, bool)
    for i in range(n):
        sees[i] = c.mask.view(np.uint32)[i, token // 32] >> (token % 32) & 1
    assert 0 < sees[:n].sum() < n
    got, lse = c.run(ctx)
    ob, sb = c.bounds(want)
    w = want[2] & ~sees
    none = np.isneginf(want[1])
    assert (np.abs(got - want[0]) <= ob)[w].all() and (np.abs(lse - want[1]) <= sb)[w[:, None] & ~none].all()
    if where == "value":
        hit = got[sees][..., 1]
        assert (np.isnan(hit).all() if np.isnan(value) else (np.isnan(hit) | (hit == value)).all()) and not np.isfinite(hit).any()
        other = np.arange(D) != 1
        assert (np.abs(got - want[0]) <= ob)[sees][..., other].all()
    elif np.isnan(value):
        assert np.isnan(got[sees]).all() and np.isnan(lse[sees]).all()
    else:  # a score of plus infinity makes NaN of its row, one of minus infinity counts for nothing
        q = ref.f64(c.q)[sees][..., 1] * value
        assert np.isnan(got[sees][q > 0]).all() and np.isfinite(got[sees][q < 0]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_infinities_in_the_context_and_queries(ctx, kind):
    c = Case(8, kind, [(6, 90), (4, 50)], 1, 2, 64, 16)
    s = int(c.seq[0])
    c.view(c.v)[int(c.table[s, 1]), 3, 0, 5] = float("inf")
    want = c.want()
    got, _ = c.run(ctx)
    assert not np.isfinite(got[:6, :, 5]).any()
    c.q[8, 1, 2] = float("nan")
    got, lse = c.run(ctx)
    ob, _ = c.bounds(want)
    assert np.isnan(got[8, 1]).all() and np.isnan(lse[8, 1])
    assert (np.abs(got - want[0]) <= ob)[[6, 7, 9]].all() and (np.abs(got - want[0]) <= ob)[8, 0].all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-3, 3.0])
def test_scales(ctx, scale, kind):
    Case(9, kind, [(5, 300), (40, 90)], 1, 4, 64, 16, scale=scale).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
def test_scores_that_grow_along_the_line(ctx, kind):
    """The running reference is taken again and again: keys grow from position to position."""
    c = Case(10, kind, [(8, 1500)], 1, 4, 64, 16)
    s = int(c.seq[0])
    for t in range(int(c.lens[s])):
        c.view(c.k)[int(c.table[s, t // 16]), t % 16] *= 0.05 + 4.0 * t / 1500
    c.check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes,kv,group,D", [
    ([(1, c) for c in (62, 63, 64, 127, 128, 511, 640, 641)], 2, 2, 64), ([(32, 20000)], 1, 4, 128), ([(33, 30000)], 1, 4, 64),
    ([(64, 9000), (3, 17), (1, 12345)], 1, 8, 128), ([(7, 5000 - 64 * i) for i in range(30)], 2, 3, 64),
    ([(2, 64 * i) for i in range(300)], 1, 1, 64), ([(3, 3000)], 1, 2, 192), ([(5, 3000), (5, 100)], 2, 2, 256),
])
def test_splits_with_exact_sums(ctx, sizes, kv, group, D, kind):
    """Queries of zero see every position alike: sums of whole numbers that are exact in fp32, so a tile lost or
    counted twice shows in the sum and in the log of the count."""
    c = Case(11, kind, sizes, kv, group, D, 16, masked=False)
    c.q.zero_()
    vv = c.view(c.v)
    vals = torch.from_numpy(c.rng.integers(-8, 9, tuple(vv.shape))).to(c.dt)
    vv.copy_(torch.where(torch.isnan(vv.float()), vv, vals))
    got, lse = c.run(ctx)
    want = c.want()
    w = want[2]
    count = want[3]["count"]
    assert (np.abs(lse - np.log(np.maximum(count, 1))) <= 2.0**-21 * (1 + np.log(np.maximum(count, 1))))[w].all()
    assert (np.abs(got - want[0]) <= (ref.HALF_ULP[kind] * 1.01 + 2.0**-21) * np.abs(want[0]) + 2.0**-24)[w].all()


@pytest.mark.parametrize("kind", KINDS)
def test_one_token_is_paged_attention(ctx, kind):
    c = Case(12, kind, [(1, n) for n in (0, 5, 64, 1000, 333)], 2, 4, 128, 16, masked=False, extra=0)
    got, lse = c.run(ctx)
    kd, vd, td, ld, cu, seq, qb = c.keep[:7]
    cache = sbt.kv_cache(kd, vd, 2, 128, *c.ld)
    m = sbt.page_map(td, c.max_pages, len(c.lens), c.max_pages, ld, c.n_pages, 16)
    out, l2 = torch.empty_like(c.q.cuda()), torch.empty(5, 8, device="cuda")
    n = sbt.paged_attention_workspace_size(ctx, 8, 2, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    sbt.paged_attention(ctx, c.q.cuda(), 1024, 128, 5, 8, cache, m, c.scale, out, 1024, 128, lse=l2, seq=seq, workspace=ws,
                        workspace_bytes=n)
    ob, sb = c.bounds(c.want())
    assert (np.abs(ref.f64(out) - got) <= 2 * ob).all() and (np.abs(ref.f64(l2) - lse) <= 2 * sb).all()


def test_same_bits_and_a_captured_graph(ctx):
    c = Case(13, "bf16", [(32, 3000), (5, 100), (17, 900)], 2, 4, 128, 16)
    c.run(ctx)
    first = c.out_dev.clone(), c.lse_dev.clone()
    for _ in range(3):
        c.out_dev.zero_()
        c.call()
        assert torch.equal(c.out_dev.nan_to_num(), torch.where(first[0] == FILL, 0, first[0]).nan_to_num())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    for _ in range(2):
        c.out_dev.fill_(FILL), c.lse_dev.fill_(FILL)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out_dev, first[0]) and torch.equal(c.lse_dev, first[1])
    ctx.check_status()


def test_offsets_past_32_bits(ctx):
    c = Case(14, "f16", [(5, 100), (3, 20)], 1, 2, 64, 64)
    c.P, spread = 64, (1 << 31) + 64
    used = sorted(set(c.table[c.table >= 0].tolist()))[:4]
    assert c.n_pages <= 6
    big_k, big_v = (torch.zeros(spread * (c.n_pages - 1) + 64 * 64, dtype=torch.float16, device="cuda") for _ in "kv")
    for big, small in ((big_k, c.k), (big_v, c.v)):
        big.as_strided((c.n_pages, 64, 1, 64), (spread, 64, 64, 1)).copy_(c.view(small))
    assert used and c.n_pages * spread > 2**32
    td, ld, cu, seq, q, mask = i32(c.table), i32(c.lens), i32(c.cu), i32(c.seq), c.q.cuda(), i32(c.mask)
    m = sbt.page_map(td, c.max_pages, len(c.lens), c.max_pages, ld, c.n_pages, 64)
    out = torch.full_like(q, FILL)
    n = sbt.paged_tree_attention_workspace_size(ctx, c.max_new, 2, 1, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    sbt.paged_tree_attention(ctx, q, 128, 64, c.rows, cu, 2, c.max_new, 2, sbt.kv_cache(big_k, big_v, 1, 64, spread, 64, 64),
                             m, c.scale, out, 128, 64, mask=mask, ld_mask=c.words, seq=seq, workspace=ws, workspace_bytes=n)
    want = c.want()
    ob, _ = c.bounds(want)
    assert (np.abs(ref.f64(out) - want[0]) <= ob)[want[2]].all()


@pytest.mark.parametrize("sizes", [[(5, 500)], [(40, 3000), (3, 9)]])
def test_wait_runs_out_then_recovers(ctx, sizes):
    """A tile that is never signalled: the waits give up, the status says so, and the same call then works."""
    c = Case(15, "bf16", sizes, 1, 4, 128, 16)
    got, lse = c.run(ctx)
    ctx.set_wait_limit_ns(20_000_000)
    ctx.set_test_hook(True)
    try:
        c.call()
        with pytest.raises(sbt.SbtError) as e:
            ctx.check_status()
        assert e.value.status == sbt.SBT_ERR_DEVICE_TIMEOUT
    finally:
        ctx.set_test_hook(False)
        ctx.set_wait_limit_ns(2_000_000_000)
    again, lse2 = c.run(ctx)
    assert np.array_equal(got, again) and np.array_equal(lse, lse2)
