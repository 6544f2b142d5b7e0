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
