"""Numbers at the top of their 32-bit range, where a counter that steps past them must not wrap."""
import numpy as np
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
from test_pages_gpu import State

pytestmark = pytest.mark.gpu
TOP = 2**31 - 1


@pytest.mark.parametrize("P", [1, 2, 5])
def test_cut_to_more_than_any_sequence_holds(ctx, P):
    """keep = 2^31 - 1 and a little less: nothing is cut."""
    s = State(ctx, [20, 7, 0, 33, 1, 12], 120, P, 40, page_bytes=16, planes=1)
    for keep in (TOP, TOP - 1, TOP - 255, TOP - 256, TOP - 1000):
        s.free([0, 1, 2, 3], [keep, keep - 3, keep, TOP])
        s.check()
    s.free([0, 3, 4], [TOP, 5, 0])
    s.check()
    s.held_consistent()


@pytest.mark.parametrize("P", [1, 2, 5, TOP])
def test_grow_to_more_than_a_row_holds(ctx, P):
    """Targets near 2^31 - 1: refused where the row has no room for them, taken where one page holds them."""
    s = State(ctx, [3, 0, 1, 2], 50, P, 10, page_bytes=16, planes=1)
    s.reserve([TOP, TOP - 1, 2, TOP - 31])
    s.check()
    s.reserve([4, 1, TOP - 40, -(2**31)])
    s.check()
    s.held_consistent()


def test_an_empty_row_of_as_many_elements_as_there_may_be(ctx):
    """2^31 - 1 query heads of one element: the last steps over out and lse pass 2^31."""
    n = TOP
    x = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out = torch.full((n + 65,), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 65,), 3.0, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, lens = i32([[-1]]), i32([0])
    size = sbt.paged_attention_workspace_size(ctx, n, 1, 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    sbt.paged_attention(ctx, x, 0, 0, 1, n, sbt.kv_cache(x, x, 1, 1, 1, 1, 1), sbt.page_map(table, 1, 1, 1, lens, 1, 1),
                        1.0, out, n, 1, lse=lse, workspace=ws, workspace_bytes=size)
    torch.cuda.synchronize()
    assert bool((out[n:] == 3).all()) and bool((lse[n:] == 3).all())
    step = 1 << 28
    for i in range(0, n, step):
        e = min(n, i + step)
        assert not bool(out[i:e].any()) and bool(torch.isneginf(lse[i:e]).all())
