"""The norm's gradient at the widest rows that the calls allow."""
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
import step_ref as ref
from test_add_rms_norm_sums_gpu import backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(3, 2**24), (5, 2**20 + 1)])
def test_gradient_of_the_widest_rows(ctx, rows, cols):
    """The workspace holds what these rows need, not a part for every block of narrow ones."""
    assert sbt.add_rms_norm_backward_workspace_size(ctx, rows, cols) <= 4 * cols + 8 * rows + 512
    h = torch.ones(rows, cols, device="cuda")
    h[:, ::5] = -1
    gy = torch.ones(rows, cols, device="cuda")
    gy[:, 1::2] = 3
    dx, dw = backward(ctx, gy, h, "bf16", 0)
    h, gy = h.double(), gy.double()
    want = gy - h * (gy * h).sum(1, keepdim=True) / cols
    # sums of whole numbers below 2^24 * 3, taken in 256 strands: exact to 2^24, to 2^-24 of themselves past it
    bound = ref.HALF_ULP["bf16"] * 1.01 * want.abs() + 2.0**-20 * (1 + gy)
    assert ((dx - want).abs() <= bound).all()
    assert torch.equal(dw.double(), (gy * h).sum(0))
