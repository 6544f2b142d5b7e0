"""sbt_matvec_e2m1 where a row's magnitudes grow by more than 2^126 within a warp's share of k.

bf16 and fp32 rows enter scaled by a power of two that follows the largest value seen so far; the running sums are
scaled with it.  What was summed before is negligible then (the bound of step 2^-39 of the row's largest), unless it
is an infinity.
"""
import numpy as np
import pytest

import step_ref as ref
from test_matvec_gpu import Case

pytestmark = pytest.mark.gpu
K, N, LATE = 32768, 96, 64  # warps have several stages of k each; LATE: from the second stage of the first warp on


def far_case(kind, tokens, first):
    """Row 1: `first` at k = 5 and zeros beside it, then values of 2^17 to 2^20."""
    c = Case(tokens, kind, tokens, K, N, out="f32")
    rng = np.random.default_rng(1)
    x = ref.f64(c.xv)
    x[1, :LATE] = 0
    x[1, LATE:] = rng.choice([-1, 1], K - LATE) * 2.0 ** rng.integers(17, 21, K - LATE)
    x[1, 5] = first
    c.xv.copy_(ref.torch.from_numpy(x).to(c.xv.dtype))
    c.packed[5] = 0x21  # the weights that meet it are not zero
    return c


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [2, 13])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_infinities_before_large_values(ctx, value, tokens, kind):
    y, bound = far_case(kind, tokens, 0.0).want()
    c = far_case(kind, tokens, value)
    got = c.run(ctx)
    sign = np.sign(ref.E2M1[ref.unpack_e2m1(c.packed, K, N, c.ldb)[5]])
    assert (sign != 0).all()
    assert np.array_equal(got[1], np.full(N, value) if np.isnan(value) else value * sign, equal_nan=True)
    rest = [i for i in range(tokens) if i != 1]
    assert (np.abs(got - y)[rest] <= bound[rest]).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [2, 13])
@pytest.mark.parametrize("first", [2.0**-126, 2.0**-110, 2.0**-100 * 1.5])
def test_tiny_values_before_large_ones(ctx, first, tokens, kind):
    far_case(kind, tokens, first).check(ctx)
