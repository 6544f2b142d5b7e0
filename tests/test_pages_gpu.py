"""GPU parity of the page operators (copy, reserve, fork, free, compact) with a plain model, bit for bit."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import scatter_boundary_tile_gb300 as sbt
from gpu_helpers import Canvas

pytestmark = pytest.mark.gpu


class State:
    """The model and the device side of one page state."""

    def __init__(self, ctx, lens, n_pages, P, max_pages, page_bytes=64, planes=2, seed=0, stride_pad=0, ld_pad=2,
                 offset=0):
        rng = np.random.default_rng(seed)
        self.ctx, self.P, self.n_pages = ctx, P, n_pages
        S = len(lens)
        table = np.full((S, max_pages), -1, np.int32)
        refs = np.zeros(n_pages, np.int32)
        perm, at = rng.permutation(n_pages), 0
        for s, n in enumerate(lens):
            c = -(-max(n, 0) // P)
            table[s, :c] = perm[at:at + c]
            refs[perm[at:at + c]] = 1
            at += c
        sizes = [page_bytes, page_bytes // 2 or 1]  # two pools of different pages
        pools = [rng.integers(0, 256, (planes, n_pages, b), dtype=np.uint8) for b in sizes]
        self.m = ref.Pages(table, np.asarray(lens, np.int32), refs, P, pools)
        self.ld = max_pages + ld_pad
        self.gap = 0x5A5A5A5A
        self.bufs, handles = [], []
        for p in pools:
            b = p.shape[2]
            gs = b + stride_pad
            ps = n_pages * gs + stride_pad
            c = Canvas(planes * ps + offset)
            self.bufs.append((c, b, gs, ps))
            handles.append((c.ptr + offset, planes, ps, gs, b))
        self.offset, self.planes = offset, planes
        self.handles = sbt.page_pools(handles)
        self.push()
        n = sbt.pages_workspace_size(ctx, S, n_pages)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def push(self):
        """The model's state onto the device."""
        t = np.full((self.m.table.shape[0], self.ld), self.gap, np.int32)
        t[:, :self.m.max_pages] = self.m.table
        self.table, self.lens, self.refs = (torch.from_numpy(x.copy()).cuda() for x in (t, self.m.lens, self.m.refs))
        self.map = sbt.page_map(self.table, self.ld, len(self.m.lens), self.m.max_pages, self.lens, self.n_pages,
                                self.P, refs=self.refs)
        for (c, b, gs, ps), p in zip(self.bufs, self.m.pools):
            x = c.buf.cpu().numpy()
            inner = x[c.guard + self.offset:c.guard + c.nbytes]
            for i in range(self.planes):
                for j in range(self.n_pages):
                    inner[i * ps + j * gs:i * ps + j * gs + b] = p[i, j]
            c.buf.copy_(torch.from_numpy(x))
            c._pattern = x.copy()

    def i32(self, x):
        return torch.tensor(list(x), dtype=torch.int32, device="cuda")

    def check(self, table=None, refs=None):
        torch.cuda.synchronize()
        t = (self.table if table is None else table).cpu().numpy()
        assert np.array_equal(t[:, :self.m.max_pages], self.m.table)
        assert (t[:, self.m.max_pages:] == self.gap).all()
        assert np.array_equal(self.lens.cpu().numpy(), self.m.lens)
        assert np.array_equal((self.refs if refs is None else refs).cpu().numpy(), self.m.refs)
        self.check_pools()

    def check_pools(self):
        torch.cuda.synchronize()
        for (c, b, gs, ps), p in zip(self.bufs, self.m.pools):
            want = c._pattern.copy()
            inner = want[c.guard + self.offset:c.guard + c.nbytes]
            for i in range(self.planes):
                for j in range(self.n_pages):
                    inner[i * ps + j * gs:i * ps + j * gs + b] = p[i, j]
            assert np.array_equal(c.buf.cpu().numpy(), want)

    def held_consistent(self):
        """Holders equal the table entries that name a page."""
        count = np.zeros(self.n_pages, np.int32)
        for s in range(len(self.m.lens)):
            for j in range(self.m.held(s)):
                if self.m.ok(self.m.table[s, j]):
                    count[self.m.table[s, j]] += 1
        assert np.array_equal(count, self.m.refs)

    def free(self, seqs, keep=None):
        sbt.pages_free(self.ctx, self.map, self.i32(seqs), len(seqs), keep=None if keep is None else self.i32(keep))
        self.m.free(seqs, keep)

    def reserve(self, target):
        sbt.pages_reserve(self.ctx, self.map, self.handles, self.i32(target), self.ws, self.ws.numel())
        self.m.reserve(target)

    def fork(self, a, b):
        sbt.pages_fork(self.ctx, self.map, self.handles, self.i32(a), self.i32(b), len(a), self.ws, self.ws.numel())
        self.m.fork(a, b)

    def copy(self, a, b):
        sbt.pages_copy(self.ctx, self.handles, self.n_pages, self.i32(a), self.i32(b), len(a))
        self.m.copy(a, b)


@pytest.mark.parametrize("page_bytes,stride_pad,offset", [(64, 0, 0), (65536, 0, 0), (16400, 32, 16), (30, 0, 0),
                                                          (16385, 3, 1), (40, 8, 8), (20000, 4, 4), (2, 0, 0)])
def test_copy(ctx, page_bytes, stride_pad, offset):
    s = State(ctx, [0], 40, 1, 1, page_bytes, 3, stride_pad=stride_pad, offset=offset)
    rng = np.random.default_rng(1)
    perm = rng.permutation(40)
    src, dst = list(perm[:15]) + [-1, 40, 2, 5], list(perm[15:30]) + [perm[30], perm[31], -5, 2**31 - 1]
    s.copy(src, dst)
    s.check_pools()
    s.copy([3], [3])  # onto itself
    s.check_pools()


@pytest.mark.parametrize("P", [1, 5, 16])
def test_a_life_of_sequences(ctx, P):
    """Random reserve, fork, cut and free; after each call the whole state equals the model's."""
    S, mp = 12, 9
    s = State(ctx, [0] * S, 60, P, mp, seed=P)
    rng = np.random.default_rng(P + 100)
    for step in range(30):
        op = step % 4
        if op == 0:
            s.reserve([int(n) + int(rng.integers(0, 3 * P)) * int(rng.integers(0, 2)) for n in s.m.lens])
        elif op == 1:
            n = int(rng.integers(1, S + 1))
            s.fork([int(x) for x in rng.integers(-1, S + 1, n)], [int(x) for x in rng.integers(-1, S + 1, n)])
        elif op == 2:
            n = int(rng.integers(1, S + 3))
            seqs = [int(x) for x in rng.integers(-1, S + 1, n)]
            s.free(seqs, [int(x) for x in rng.integers(-2, mp * P + 2, n)])
        else:
            s.free([int(x) for x in rng.integers(0, S, 2)])
        s.check()
        s.held_consistent()


def test_a_cut_sequence_gets_its_own_page_before_it_grows(ctx):
    """Fork at 40 of 16 a page, cut the child to 20: its page 1 is shared and part full; growing copies it."""
    s = State(ctx, [40, 0, 0], 12, 16, 4)
    s.fork([0, 0], [1, 2])
    s.check()
    s.free([1, 2], [20, 32])
    s.check()
    s.reserve([0, 21, 33])  # 1 needs a copy of page 1, 2 (at a page's end) a new page only
    s.check()
    s.held_consistent()
    assert s.m.table[1, 1] != s.m.table[0, 1] and s.m.table[2, 1] == s.m.table[0, 1]


def test_two_holders_of_a_part_page_grow_together(ctx):
    s = State(ctx, [32, 0], 10, 16, 4)
    s.fork([0], [1])
    s.free([0, 1], [20, 20])
    s.reserve([30, 30])  # both copy; the page they shared is free again
    s.check()
    s.held_consistent()


def test_no_page_left(ctx):
    s = State(ctx, [16, 16, 16, 5], 6, 16, 3)
    s.reserve([17, 33, 17, 16])  # two pages left: sequence 0 takes one, 1 and 2 are refused, 3 needs none
    s.check()
    assert list(s.m.lens) == [17, 16, 16, 16]
    s = State(ctx, [20, 20, 0, 0, 0], 6, 16, 3)
    s.fork([0, 1, 0], [2, 3, 4])  # two pages left for three part-full last pages
    s.check()
    assert list(s.m.lens) == [20, 20, 20, 20, 0]


def test_room_in_the_row(ctx):
    s = State(ctx, [30, 30], 20, 16, 2)
    s.reserve([33, 32])  # the first row is full
    s.check()
    assert list(s.m.lens) == [30, 32]


def test_free_pages_are_found_across_many(ctx):
    """Free pages thinly spread over a pool of several scan steps."""
    n = 20000
    s = State(ctx, [0, 0, 0], n, 4, 200, page_bytes=2, planes=1)
    s.m.refs[:] = 1
    s.m.refs[::97] = 0
    s.push()
    s.reserve([500, 300, 700])
    s.check()
    s.fork([], [])
    s.reserve([800, 800, 800])  # more than are left: served in order
    s.check()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_pages,live", [(1, 1), (7, 0), (7, 7), (50, 20), (3000, 1700), (9001, 64)])
def test_compact(ctx, in_place, n_pages, live):
    rng = np.random.default_rng(live)
    S, P, mp = 6, 3, max(2, -(-live // 6) + 1)
    s = State(ctx, [0] * S, n_pages, P, mp, page_bytes=32, planes=2)
    pages = rng.permutation(n_pages)[:live]
    at = 0
    for q in range(S):
        c = live // S + (1 if q < live % S else 0)
        s.m.table[q, :c] = pages[at:at + c]
        s.m.lens[q] = max(0, c * P - q % P)
        at += c
    s.m.refs[pages] = 1 + pages % 3
    if live > 10:
        s.m.table[0, 0], s.m.table[1, 0] = -1, n_pages + 5  # entries that name no page become -1
        s.m.refs[pages[2]] = 0                              # so does one whose page nobody holds
    s.push()
    page_to = torch.full((n_pages,), -9, dtype=torch.int32, device="cuda")
    n_live = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    if in_place:
        table_out, refs_out = s.table, s.refs
    else:
        table_out, refs_out = s.table.clone(), torch.full_like(s.refs, -9)
    sbt.pages_compact(s.ctx, s.map, s.handles, table_out, s.ld, refs_out, page_to, n_live, s.ws, s.ws.numel())
    table, refs, to, L = s.m.compact()
    torch.cuda.synchronize()
    assert int(n_live) == L
    assert np.array_equal(page_to.cpu().numpy(), to)
    if not in_place:
        s.check()  # the map is as it was
    s.m.table, s.m.refs = table, refs
    s.check(table_out, refs_out)


def test_compact_then_attention_reads_the_same(ctx):
    """Rows of the cache, read through the table before and after packing the pool."""
    s = State(ctx, [33, 70, 5], 40, 8, 12, page_bytes=512, planes=1)
    rows = lambda: [np.concatenate([s.m.pools[0][0, s.m.table[q, j]] for j in range(s.m.held(q))]) for q in range(3)]
    before = rows()
    page_to, n_live = torch.empty_like(s.refs), torch.empty(1, dtype=torch.int32, device="cuda")
    sbt.pages_compact(ctx, s.map, s.handles, s.table, s.ld, s.refs, page_to, n_live, s.ws, s.ws.numel())
    s.m.table, s.m.refs, _, _ = s.m.compact()
    s.check()
    for a, b in zip(before, rows()):
        assert np.array_equal(a, b)


def test_refusals(ctx):
    s = State(ctx, [5, 0], 4, 4, 2)
    i = s.i32([0, 1])
    to, live = torch.empty_like(s.refs), torch.empty(1, dtype=torch.int32, device="cuda")
    before = ctx.launch_count
    bad, aln = sbt.SBT_ERR_INVALID_ARG, sbt.SBT_ERR_ALIGNMENT
    no_refs = sbt.page_map(s.table, s.ld, 2, 2, s.lens, 4, 4)
    n = s.ws.numel()
    overlap = sbt.page_pools([(s.bufs[0][0].ptr, 1, 0, 32, 64)])
    for call, status in [
            (lambda: sbt.pages_copy(ctx, s.handles, 4, i, i, -1), bad),
            (lambda: sbt.pages_copy(ctx, overlap, 4, i, i, 2), bad),
            (lambda: sbt.pages_copy(ctx, sbt.page_pools([]), 4, i, i, 2), bad),
            (lambda: sbt.pages_copy(ctx, s.handles, 4, None, i, 2), bad),
            (lambda: sbt.pages_free(ctx, no_refs, i, 2), bad),
            (lambda: sbt.pages_reserve(ctx, s.map, s.handles, i, s.ws, n - 1), aln),
            (lambda: sbt.pages_reserve(ctx, s.map, s.handles, None, s.ws, n), bad),
            (lambda: sbt.pages_fork(ctx, s.map, s.handles, i, i, 3, s.ws, n), bad),
            (lambda: sbt.pages_compact(ctx, s.map, s.handles, s.table, s.ld + 1, s.refs, to, live, s.ws, n), bad),
            (lambda: sbt.pages_compact(ctx, s.map, s.handles, s.table, s.ld, s.refs, None, live, s.ws, n), bad)]:
        with pytest.raises(sbt.SbtError) as e:
            call()
        assert e.value.status == status
    sbt.pages_copy(ctx, s.handles, 4, i, i, 0)
    sbt.pages_fork(ctx, s.map, s.handles, i, i, 0, s.ws, n)
    sbt.pages_free(ctx, s.map, i, 0)
    assert ctx.launch_count == before
    s.check()
