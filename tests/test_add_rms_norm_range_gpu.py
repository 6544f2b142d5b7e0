"""The norm where a mean of squares leaves fp32's range, in every form of the kernel."""
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
import step_ref as ref
from test_add_rms_norm_sums_gpu import rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("cols", [8, 257, 4096, 5003, 16384, 20480])
def test_squares_past_the_range(ctx, cols, pad, kind):
    """A sum that overflows makes the row zero, a zero root with eps 0 makes NaN of zeros; other rows do not see it."""
    x = torch.ones(4, cols, device="cuda")
    x[1, cols // 2], x[2] = 2.0**100, 0
    ptr, ld, v = rows_of(x, kind, pad)
    h, y = (rows_of(torch.full((4, cols), 7.0, device="cuda"), kind, pad) for _ in "hy")
    sbt.add_rms_norm(ctx, ptr, ld, 4, cols, eps=0.0, h_out=h[0], ld_h=h[1], y=y[0], ld_y=y[1], dtype=kind)
    torch.cuda.synchronize()
    assert torch.equal(h[2], v) and (y[2][[0, 3]] == 1).all()
    assert (y[2][1] == 0).all() and torch.isnan(y[2][2].float()).all()
    sbt.add_rms_norm(ctx, ptr, ld, 4, cols, eps=1e-6, y=y[0], ld_y=y[1], dtype=kind)
    torch.cuda.synchronize()
    assert (y[2][2] == 0).all() and ((y[2][0].double() - 1).abs() <= 1e-6 + ref.HALF_ULP[kind]).all()
