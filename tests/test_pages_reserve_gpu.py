"""sbt_pages_reserve where what is asked for is far more than the pool holds."""
import numpy as np
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
from test_pages_gpu import State

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [1, 2])
def test_requests_of_many_sequences_far_beyond_the_pool(ctx, seed):
    """3000 sequences (three steps of the prefix sum) ask for some ten times the pool; served in order."""
    S, P, mp = 3000, 4, 7
    s = State(ctx, [0] * S, 900, P, mp, page_bytes=8, planes=1, seed=seed)
    rng = np.random.default_rng(seed)
    s.reserve([int(x) for x in rng.integers(0, mp * P, S) * (rng.random(S) < 0.05)])  # some hold pages already
    s.check()
    held = np.flatnonzero(s.m.lens)
    a, b = held[:40], np.setdiff1d(np.arange(S), held)[:40]
    s.fork([int(x) for x in a], [int(x) for x in b])  # and share part-full ones
    s.check()
    s.free([int(x) for x in held[20:60]], [int(x) for x in s.m.lens[held[20:60]] // 2])
    s.reserve([int(x) for x in rng.integers(0, mp * P + 9, S)])
    s.check()
    s.held_consistent()


def test_requests_that_add_up_to_more_than_32_bits(ctx):
    """2100 sequences of 2^20 pages each: 2.2e9 pages asked of a pool of 50.  The first two fit, no other does.

    The two at the front and the one at the end, where a 32-bit sum would have wrapped, ask for little."""
    S, mp, n_pages = 2100, 1 << 20, 50
    table = torch.full((S, mp), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[7] = 1
    target = torch.full((S,), mp, dtype=torch.int32, device="cuda")
    target[0], target[1], target[S - 1] = 3, 5, 2
    pool = torch.zeros((n_pages, 64), dtype=torch.uint8, device="cuda")
    pm = sbt.page_map(table, mp, S, mp, lens, n_pages, 1, refs=refs)
    n = sbt.pages_workspace_size(ctx, S, n_pages)
    ws = torch.full((n + 4096,), 0x7E, dtype=torch.uint8, device="cuda")
    sbt.pages_reserve(ctx, pm, sbt.page_pools([(pool, 1, n_pages * 64, 64, 64)]), target, ws, n)
    torch.cuda.synchronize()
    assert lens.tolist() == [3, 5] + [0] * (S - 2)
    assert table[0, :4].tolist() == [0, 1, 2, -1] and table[1, :6].tolist() == [3, 4, 5, 6, 8, -1]
    assert int((table >= 0).sum()) == 8
    assert refs.tolist() == [1] * 9 + [0] * (n_pages - 9)
    assert bool((ws[n:] == 0x7E).all())
    lens_before = lens.clone()
    sbt.pages_reserve(ctx, pm, sbt.page_pools([(pool, 1, n_pages * 64, 64, 64)]), target, ws, n)  # and again
    torch.cuda.synchronize()
    assert torch.equal(lens, lens_before) and int((table >= 0).sum()) == 8
