"""The workspace of sbt_paged_tree_attention, on the host (no GPU): that of a larger max_new serves every smaller one."""
import ctypes

import pytest

import scatter_boundary_tile_gb300 as sbt
from test_cache_abi import lib  # noqa: F401

SMS = 152


@pytest.mark.parametrize("head_dim", [1, 64, 65, 128, 129, 192, 256])
@pytest.mark.parametrize("group", [1, 4, 7, 130])
def test_a_larger_max_new_never_needs_less(lib, head_dim, group):  # noqa: F811
    ctx = ctypes.create_string_buffer(4096)
    ctypes.cast(ctx, ctypes.POINTER(ctypes.c_int))[1] = SMS  # the stand-in context's number of SMs
    sizes = []
    for max_new in (1, 5, 18, 19, 31, 32, 33, 128, 129, 200, 5000):
        n = ctypes.c_size_t()
        assert lib.sbt_paged_tree_attention_workspace_size(ctx, max_new, 2 * group, 2, head_dim, ctypes.byref(n)) == sbt.SBT_OK
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[0] > 0
