"""Page operators on lengths that are out of range: below zero they stand for an empty sequence, past the
row for a full one, as the page map says."""
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt

pytestmark = pytest.mark.gpu
P, MP, N = 4, 3, 20  # up to 12 positions a sequence


class Pages:
    def __init__(self, ctx, lens, rows):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.ctx, self.i32, self.S = ctx, i32, len(lens)
        self.table, self.lens, self.refs = i32(rows), i32(lens), i32([0] * N)
        for row in rows:
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
        self.pool = torch.arange(N, dtype=torch.uint8, device="cuda")[:, None].repeat(1, 16).contiguous()
        self.pools = sbt.page_pools([(self.pool, 1, N * 16, 16, 16)])
        self.map = sbt.page_map(self.table, MP, self.S, MP, self.lens, N, P, refs=self.refs)
        self.ws = torch.empty(sbt.pages_workspace_size(ctx, self.S, N), dtype=torch.uint8, device="cuda")

    def fork(self, a, c):
        sbt.pages_fork(self.ctx, self.map, self.pools, self.i32(a), self.i32(c), len(a), self.ws, self.ws.numel())

    def reserve(self, target):
        sbt.pages_reserve(self.ctx, self.map, self.pools, self.i32(target), self.ws, self.ws.numel())


def test_a_child_below_zero_is_empty(ctx):
    s = Pages(ctx, [6, -1, -2**31, 5], [[0, 1, -1], [-1] * 3, [-1] * 3, [2, 3, -1]])
    s.fork([0, 3, 1], [1, 2, 2])  # the third parent is empty
    assert s.lens.tolist() == [6, 6, 5, 5]
    assert s.table.tolist() == [[0, 1, -1], [0, 4, -1], [2, 5, -1], [2, 3, -1]]
    assert s.refs.tolist()[:7] == [2, 1, 2, 1, 1, 1, 0]
    assert s.pool[4:6, 0].tolist() == [1, 3]


def test_growing_starts_at_zero(ctx):
    s = Pages(ctx, [-5, -2**31, -1, 2], [[-1] * 3, [-1] * 3, [-1] * 3, [0, -1, -1]])
    s.reserve([0, -7, 5, 2])  # none of the first two asks for more than the 0 it has
    assert s.lens.tolist() == [-5, -2**31, 5, 2]
    assert s.table.tolist() == [[-1] * 3, [-1] * 3, [1, 2, -1], [0, -1, -1]]


def test_a_length_past_the_row_is_a_full_row(ctx):
    s = Pages(ctx, [500, 0, 2**31 - 1], [[0, 1, 2], [-1] * 3, [3, 4, 5]])
    s.reserve([600, 0, 2**31 - 1])  # no room
    assert s.lens.tolist() == [500, 0, 2**31 - 1] and s.refs.tolist() == [1] * 6 + [0] * (N - 6)
    s.fork([0], [1])
    assert s.table.tolist()[1] == [0, 1, 2] and s.refs.tolist()[:7] == [2, 2, 2, 1, 1, 1, 0]
    sbt.pages_free(ctx, s.map, s.i32([0, 2]), 2, keep=s.i32([5, 2**31 - 1]))
    assert s.table.tolist() == [[0, 1, -1], [0, 1, 2], [3, 4, 5]]
    assert s.refs.tolist()[:7] == [2, 2, 1, 1, 1, 1, 0]
