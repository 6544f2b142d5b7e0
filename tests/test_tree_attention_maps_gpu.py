"""sbt_paged_tree_attention with a driver that refuses its tensor maps."""
import ctypes

import pytest

import scatter_boundary_tile_gb300 as sbt
from test_tree_attention_gpu import Case

pytestmark = pytest.mark.gpu


class Head(ctypes.Structure):
    """The first members of a context: what the library asks the driver for tensor maps with is the last."""
    _fields_ = [("device", ctypes.c_int), ("sm_count", ctypes.c_int), ("cc", ctypes.c_int * 2), ("smem", ctypes.c_size_t),
                ("path", ctypes.c_int), ("wait_ns", ctypes.c_uint64), ("status", ctypes.c_void_p), ("encode", ctypes.c_void_p)]


@pytest.mark.parametrize("refused", [1, 2])
def test_a_refused_tensor_map(refused):
    """A driver that refuses the first or the second map: the pages are copied by lanes, as any others are."""
    ctx = sbt.Context(0)
    head = Head.from_address(ctx.handle.value)
    assert head.device == 0 and list(head.cc) == [10, 3] and head.sm_count > 0 and head.encode
    c = Case(30, "bf16", [(5, 300), (9, 70)], 2, 4, 64, 16)
    c.check(ctx)
    got, calls, driver = c.out_dev.clone(), [], head.encode
    real = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_uint64] * 12)
    through = real(driver)

    def encode(*args):
        calls.append(1)
        return 1 if len(calls) == refused else through(*args)

    fake = real(encode)
    head.encode = ctypes.cast(fake, ctypes.c_void_p).value
    try:
        c.check(ctx)
    finally:
        head.encode = driver
    assert len(calls) == refused
    assert (c.out_dev.double() - got.double()).abs().max() <= 2.0**-6 * got.double().abs().max()
    ctx.close()
