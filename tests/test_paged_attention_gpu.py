"""GPU parity of sbt_paged_attention with its definition in 64 bits.

Error bounds come from the number of roundings (cache_ref.attention_bounds);
positions that no query may see hold NaN, so that one read of them shows.
"""
import numpy as np
import pytest
import torch

import cache_ref as ref
import scatter_boundary_tile_gb300 as sbt
from gpu_helpers import Canvas

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, seed, kind, lens, q_heads, heads, dim, page_size, order="nhd", pad=0, offset=0, batch=None,
                 max_pages=None, spare=2, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.dt, self.P, self.H, self.D, self.Hq = kind, ref.TDT[kind], page_size, heads, dim, q_heads
        self.lens = np.asarray(lens, np.int32)
        S = len(lens)
        need = [-(-max(int(n), 0) // page_size) for n in lens]
        self.max_pages = max_pages or max(1, max(need))
        self.n_pages = sum(need) + spare
        perm = torch.randperm(self.n_pages, generator=g).numpy().astype(np.int32)
        self.table = np.full((S, self.max_pages + 3), -1, np.int32)
        at = 0
        for s, c in enumerate(need):
            c = min(c, self.max_pages)
            self.table[s, :c] = perm[at:at + c]
            at += c
        # element strides: rows `pad` elements apart beyond the head, the whole `offset` elements into a buffer
        d = dim + pad
        self.ld_slot, self.ld_head = (heads * d, d) if order == "nhd" else (d, page_size * d)
        self.ld_page = page_size * heads * d + pad
        size = self.n_pages * self.ld_page + offset + 8
        mk = lambda: torch.full((size,), float("nan"), dtype=self.dt)
        self.kbuf, self.vbuf = mk(), mk()
        self.offset = offset
        for s in range(S):
            for t in range(min(max(int(lens[s]), 0), self.max_pages * page_size)):
                p = self.table[s, t // page_size]
                at = offset + p * self.ld_page + (t % page_size) * self.ld_slot
                for h in range(heads):
                    o = at + h * self.ld_head
                    self.kbuf[o:o + dim] = torch.randn(dim, generator=g).to(self.dt)
                    self.vbuf[o:o + dim] = torch.randn(dim, generator=g).to(self.dt)
        self.B = batch or S
        self.q = (torch.randn((self.B, q_heads, dim), generator=g) * 1.5).to(self.dt)
        self.scale = scale if scale is not None else 1.0 / np.sqrt(dim)

    def pages(self, buf):
        st = (self.ld_page, self.ld_slot, self.ld_head, 1)
        return ref.f64(buf.as_strided((self.n_pages, self.P, self.H, self.D), st, self.offset))

    def want(self, window=0, seq=None):
        return ref.attention(ref.f64(self.q), self.pages(self.kbuf), self.pages(self.vbuf),
                             self.table[:, :self.max_pages], self.lens, self.P, self.scale, window, seq)

    def run(self, ctx, window=0, seq=None, path="auto", q_pad=0, stream=None):
        es = self.q.element_size()
        dev = "cuda"
        k, v = self.kbuf.to(dev), self.vbuf.to(dev)
        self.dev = [k, v, torch.from_numpy(self.table).to(dev), torch.from_numpy(self.lens).to(dev)]
        q = torch.full((self.B, self.Hq, self.D + q_pad), float("nan"), dtype=self.dt)
        q[..., :self.D] = self.q
        q = q.to(dev)
        ld = self.D + q_pad
        out = Canvas(self.B * self.Hq * ld * es)
        lse = Canvas(self.B * self.Hq * 4)
        sq = None if seq is None else torch.tensor(seq, dtype=torch.int32, device=dev)
        cache = sbt.kv_cache(k.data_ptr() + self.offset * es, v.data_ptr() + self.offset * es, self.H, self.D,
                             self.ld_page, self.ld_slot, self.ld_head)
        pm = sbt.page_map(self.dev[2], self.table.shape[1], len(self.lens), self.max_pages, self.dev[3], self.n_pages,
                          self.P)
        n = sbt.paged_attention_workspace_size(ctx, self.Hq, self.H, self.D)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)  # whatever an earlier call left there
        ctx.set_path(path)
        torch.cuda.synchronize()
        sbt.paged_attention(ctx, q, self.Hq * ld, ld, self.B, self.Hq, cache, pm, self.scale, out.ptr, self.Hq * ld,
                            ld, lse=lse.ptr, window=window, seq=sq, workspace=ws, workspace_bytes=n, dtype=self.kind,
                            stream=stream)
        torch.cuda.synchronize()
        ctx.set_path("auto")
        assert out.guards_intact() and lse.guards_intact()
        o = out.inner(np.uint8, (self.B, self.Hq, ld, es)).copy()
        gap = o[:, :, self.D:]
        assert np.array_equal(gap, out.original(np.uint8, (self.B, self.Hq, ld, es))[:, :, self.D:])
        o = torch.from_numpy(np.ascontiguousarray(o[:, :, :self.D])).view(self.dt)[..., 0]
        return o, lse.inner(np.float32, (self.B, self.Hq)).copy()

    def check(self, ctx, window=0, seq=None, **kw):
        r = self.want(window, seq)
        out, lse = self.run(ctx, window, seq, **kw)
        ob, lb = ref.attention_bounds(r, self.kind, self.D)
        assert np.all(np.abs(ref.f64(out) - r[0]) <= ob)
        empty = np.isinf(r[1])
        assert np.array_equal(np.isneginf(lse), empty)
        assert np.all(np.abs(lse[~empty] - r[1][~empty]) <= lb[~empty])
        return out


KINDS = ["f32", "bf16", "f16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [1, 8, 33, 64, 80, 100, 128, 160, 256])
def test_head_sizes(ctx, kind, dim):
    Case(1, kind, [37, 130, 1, 200], 6, 3, dim, 16).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 16, 17, 40])
def test_query_heads_per_key(ctx, kind, group):
    Case(2, kind, [70, 5, 133], 2 * group, 2, 64, 8).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page_size", [1, 7, 16, 24, 64, 1000])
@pytest.mark.parametrize("order", ["nhd", "hnd"])
def test_pages_that_end_inside_a_tile(ctx, kind, page_size, order):
    Case(3, kind, [1, 15, 16, 17, 63, 64, 65, 129, 300], 4, 2, 64, page_size, order).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
def test_empty_rows(ctx, kind):
    c = Case(4, kind, [0, 5, -3, 0, 70, 0], 4, 2, 64, 16)
    out = c.check(ctx)
    assert not out[0].any() and not out[2].any() and not out[5].any()
    c = Case(5, kind, [0, 0], 4, 2, 64, 16)  # nothing anywhere
    assert not c.check(ctx).any()


@pytest.mark.parametrize("kind", KINDS)
def test_unmapped_pages_are_masked(ctx, kind):
    c = Case(6, kind, [100, 64, 40], 4, 2, 128, 16)
    c.table[0, 2] = -1
    c.table[0, 6] = c.n_pages      # past the pool
    c.table[1, :4] = [-7, 2**31 - 1, -1, -2**31]  # a whole row without a page
    out = c.check(ctx)
    assert not out[1].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 16, 63, 64, 100, 299, 300, 5000])
def test_window(ctx, kind, window):
    Case(7, kind, [300, 1, 64, 101, 0], 4, 2, 64, 24).check(ctx, window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_lengths_past_the_row_are_cut(ctx, kind):
    c = Case(8, kind, [1000, 64], 4, 2, 64, 16, max_pages=4)
    c.check(ctx)


@pytest.mark.parametrize("kind", KINDS)
def test_sequences_by_number(ctx, kind):
    c = Case(9, kind, [40, 90, 17], 4, 2, 64, 16, batch=7)
    c.check(ctx, seq=[2, 0, -1, 1, 1, 3, 0])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad,offset", [(8, 8), (2, 2), (1, 1), (4, 3)])
def test_strides_and_alignment(ctx, kind, pad, offset):
    Case(10, kind, [50, 3, 129], 6, 2, 64, 16, pad=pad, offset=offset).check(ctx, q_pad=pad)
    Case(11, kind, [50, 3, 129], 6, 2, 80, 16, "hnd", pad=pad, offset=offset).check(ctx, q_pad=pad)


@pytest.mark.parametrize("kind", KINDS)
def test_paths_agree_bit_for_bit(ctx, kind):
    c = Case(12, kind, [300, 7, 64, 1025], 8, 2, 128, 16)
    a, la = c.run(ctx)
    b, lb = c.run(ctx, path="scalar")
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and np.array_equal(la, lb)


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences_of_few_tokens(ctx, kind):
    lens = [(i * 7) % 33 for i in range(700)]
    Case(13, kind, lens, 4, 2, 32, 8).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
def test_long_rows_are_split_and_joined(ctx, kind):
    c = Case(14, kind, [9001, 4097], 2, 1, 64, 64)
    a = c.check(ctx)
    b, _ = c.run(ctx)
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # the same bits every run


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,dim,heads", [([40000, 1, 3000], 64, 1),        # few rows of many parts
                                            ([30000] + [5, 0, 40] * 30, 128, 1),  # one of them among many short ones
                                            ([2600] * 40, 96, 3),               # every row cut
                                            ([17000, 9000], 256, 1)])
def test_rows_cut_over_the_whole_gpu(ctx, kind, lens, dim, heads):
    c = Case(21, kind, lens, 3 * heads, heads, dim, 24)
    a = c.check(ctx)
    b, _ = c.run(ctx)
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("kind", KINDS)
def test_large_scores_and_one_dominant_position(ctx, kind):
    c = Case(15, kind, [500, 500], 4, 2, 64, 16, scale=30.0)
    c.check(ctx)


@pytest.mark.parametrize("kind", KINDS)
def test_infinities_and_nan(ctx, kind):
    """Minus infinity everywhere: an empty row.  NaN or plus infinity among the scores: NaN, in that row only."""
    c = Case(16, kind, [20, 20, 20, 20], 2, 1, 16, 16)
    first = lambda s: c.offset + c.table[s, 0] * c.ld_page
    c.q[:] = 0
    c.q[:, :, 0] = 1.0
    for s, x in ((0, float("-inf")), (1, float("nan")), (2, float("inf"))):
        for t in range(20 if s == 0 else 1):
            p = c.table[s, t // 16]
            c.kbuf[c.offset + p * c.ld_page + (t % 16) * c.ld_slot] = x
    out, lse = c.run(ctx)
    assert not out[0].any() and np.all(np.isneginf(lse[0]))
    for s in (1, 2):
        assert bool(torch.isnan(out[s]).all()) and np.all(np.isnan(lse[s]))
    assert bool(torch.isfinite(out[3]).all())


def test_offsets_past_32_bits(ctx):
    """Pages 3 * 2^31 bytes apart: element offsets above 2^32."""
    dim, P = 64, 16
    ld_page = 3 << 30  # elements
    k = torch.zeros(2 * ld_page + 8192, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator().manual_seed(17)
    rows_k, rows_v = (torch.randn((3, P, dim), generator=g).bfloat16() for _ in "kv")
    for p in range(3):
        k[p * ld_page:p * ld_page + P * dim] = rows_k[p].reshape(-1).cuda()
        v[p * ld_page:p * ld_page + P * dim] = rows_v[p].reshape(-1).cuda()
    q = torch.randn((1, 2, dim), generator=g).bfloat16()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([41], dtype=torch.int32, device="cuda")
    out = torch.empty((1, 2, dim), dtype=torch.bfloat16, device="cuda")
    n = sbt.paged_attention_workspace_size(ctx, 2, 1, dim)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    sbt.paged_attention(ctx, q.cuda(), 2 * dim, dim, 1, 2, sbt.kv_cache(k, v, 1, dim, ld_page, dim, dim),
                        sbt.page_map(table, 3, 1, 3, lens, 3, P), 0.125, out, 2 * dim, dim, workspace=ws,
                        workspace_bytes=n)
    r = ref.attention(ref.f64(q), ref.f64(rows_k)[:, :, None], ref.f64(rows_v)[:, :, None],
                      np.array([[2, 0, 1]], np.int32), [41], P, 0.125)
    assert np.all(np.abs(ref.f64(out) - r[0]) <= ref.attention_bounds(r, "bf16", dim)[0])


def test_on_a_side_stream(ctx):
    c = Case(18, "bf16", [900, 33], 8, 2, 128, 16)
    s = torch.cuda.Stream()
    c.check(ctx, stream=s)


def test_refusals(ctx):
    c = Case(19, "bf16", [20], 4, 2, 64, 16)
    c.run(ctx)
    k, v, table, lens = c.dev
    n = sbt.paged_attention_workspace_size(ctx, 4, 2, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    q = c.q.cuda()
    out = torch.empty_like(q)

    def call(dtype=None, heads=2, dim=64, batch=1, q_heads=4, window=0, ws_bytes=n, P=16, ld_table=4, ld_oh=64,
             max_pages=2):
        sbt.paged_attention(ctx, q, 256, 64, batch, q_heads,
                            sbt.kv_cache(k, v, heads, dim, c.ld_page, c.ld_slot, c.ld_head),
                            sbt.page_map(table, ld_table, 1, max_pages, lens, c.n_pages, P), 0.1, out, 256, ld_oh,
                            window=window, workspace=ws, workspace_bytes=ws_bytes, dtype=dtype)

    call()
    before = ctx.launch_count
    call(batch=0)
    for kw, status in [({"dtype": 9}, sbt.SBT_ERR_UNSUPPORTED), ({"heads": 3}, sbt.SBT_ERR_INVALID_ARG),
                       ({"dim": 257}, sbt.SBT_ERR_INVALID_ARG), ({"batch": -1}, sbt.SBT_ERR_INVALID_ARG),
                       ({"window": -1}, sbt.SBT_ERR_INVALID_ARG), ({"ws_bytes": n - 1}, sbt.SBT_ERR_ALIGNMENT),
                       ({"P": 0}, sbt.SBT_ERR_INVALID_ARG), ({"ld_table": 1}, sbt.SBT_ERR_INVALID_ARG),
                       ({"ld_oh": 63}, sbt.SBT_ERR_INVALID_ARG), ({"max_pages": -1}, sbt.SBT_ERR_INVALID_ARG)]:
        with pytest.raises(sbt.SbtError) as e:
            call(**kw)
        assert e.value.status == status, kw
    assert ctx.launch_count == before



@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,dim,group", [([1, 17, 300], 64, 4), ([20000, 3, 2500], 128, 3), ([900] * 40, 80, 9)])
@pytest.mark.parametrize("what", ["key nan", "key inf", "query nan", "value inf", "value nan"])
def test_infinities_and_nan_that_are_visible(ctx, kind, lens, dim, group, what):
    """They reach the rows (or the column, for values) that they belong to, and no others."""
    heads = 2
    c = Case(11, kind, lens, heads * group, heads, dim, 16)
    s, h, d = len(lens) - 1, 1, dim - 1  # sequence, key-value head, element
    rows = np.zeros((c.B, c.Hq), bool)
    x = float(what[-3:])
    t = lens[s] // 2
    at = c.offset + c.table[s, t // 16] * c.ld_page + (t % 16) * c.ld_slot + h * c.ld_head + d
    rows[s, h * group:] = True
    if what.startswith("key"):
        c.q[s, h * group:, d] = 1.0  # scores of plus infinity or NaN
        c.kbuf[at] = x
    elif what.startswith("query"):
        rows[s, h * group:] = False
        rows[s, -1] = True
        c.q[s, -1, d] = x
    want = c.want()  # before the values are touched: what the other columns hold
    if what.startswith("value"):
        c.vbuf[at] = x
    out, lse = c.run(ctx)
    out = ref.f64(out)
    ob, lb = ref.attention_bounds(want, kind, dim)
    cells = np.broadcast_to(rows[..., None], out.shape).copy()
    if what.startswith("value"):
        cells[..., :d] = False
        assert not np.isfinite(out[cells]).any()
        rows[:] = False
    else:
        assert np.isnan(out[cells]).all() and np.isnan(lse[rows]).all()
    assert np.all(np.abs(out - want[0])[~cells] <= ob[~cells])
    assert np.all(np.abs(lse - want[1])[~rows] <= lb[~rows])
