"""sbt_paged_tree_attention with a scale of zero, or next to it, on scores near the end of fp32's range."""
import numpy as np
import pytest
import torch

from test_tree_attention_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, 1e-45, -1e-45])
@pytest.mark.parametrize("sizes", [[(5, 300), (1, 64)], [(40, 90)]])
def test_scales_of_nothing(ctx, sizes, scale):
    """q . k up to 2^127 times the scale is below 2^-21: every visible position counts alike."""
    c = Case(40, "bf16", sizes, 1, 4, 64, 16, scale=scale)
    sign = lambda t: torch.where(t.float() < 0, -1.0, 1.0)
    c.q.copy_(sign(c.q) * 2.0**61)
    k = c.view(c.k)
    k.copy_(torch.where(torch.isnan(k.float()), k.float(), sign(k) * 2.0**60).to(c.dt))
    got, lse = c.run(ctx)
    want = c.want()
    w, x = want[2], want[3]
    none = np.isneginf(want[1])
    # the probabilities are off by 2^-20 and their own rounding (2^-16), the output by half a step of bf16
    bound = (2.0**-16 + 2.0**-19 + (x["count"] + 64) * 2.0**-23)[..., None] * x["absv"] + 2.0**-8 * 1.01 * np.abs(want[0])
    assert (np.abs(got - want[0]) <= bound)[w].all()
    assert (np.abs(lse - want[1]) <= 2.0**-19 * (1 + np.abs(np.where(none, 0, want[1]))))[w & ~none.any(1)].all()
