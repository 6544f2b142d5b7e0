"""How much workspace the norm's gradient asks for, on the host (no GPU): the sums for dweight that a call of these
extents can write, and two numbers a row where rows are too wide for registers."""
import ctypes

import pytest

import scatter_boundary_tile_gb300 as sbt
from test_cache_abi import lib  # noqa: F401

SMS = 152


@pytest.fixture(scope="module")
def size(lib):  # noqa: F811
    ctx = ctypes.create_string_buffer(4096)
    ctypes.cast(ctx, ctypes.POINTER(ctypes.c_int))[1] = SMS  # the stand-in context's number of SMs

    def ask(rows, cols):
        n = ctypes.c_size_t()
        assert lib.sbt_add_rms_norm_backward_workspace_size(ctx, rows, cols, ctypes.byref(n)) == sbt.SBT_OK
        return n.value

    return ask


@pytest.mark.parametrize("rows", [1, 5, 4096, 16384, 2**31 - 1])
@pytest.mark.parametrize("cols", [8193, 12288, 16384, 40000, 2**20, 2**24])
def test_wide_rows(size, rows, cols):
    parts = min(rows, max(1, 4 * SMS // -(-cols // 256)))  # runs of rows that are summed side by side
    assert parts * cols * 4 <= size(rows, cols) <= parts * cols * 4 + rows * 8 + 512


@pytest.mark.parametrize("cols,per_sm", [(1, 16), (256, 16), (512, 16), (1024, 8), (4096, 2), (4097, 1), (8192, 1)])
def test_rows_in_registers(size, cols, per_sm):
    """Blocks of cols / 8 threads (cols / 16 with vectors) rounded up to a power of two, 512 threads an SM."""
    rows = 100000
    assert size(rows, cols) <= per_sm * SMS * cols * 4 + rows * 8 * (cols > 4096) + 512


def test_more_rows_never_need_less(size):
    for cols in (64, 1000, 4096, 8192, 16384):
        sizes = [size(rows, cols) for rows in (0, 1, 2, 19, 152, 153, 2432, 2433, 10**6)]
        assert sizes == sorted(sizes) and sizes[0] == 0
