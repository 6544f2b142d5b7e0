"""sbt_qk_norm_rope and its gradient where inputs hold infinities, NaN or minus zero: what is not turned
stays apart from every other element, on all paths."""
import numpy as np
import pytest
import torch

import cache_ref as ref
from test_qk_norm_rope_gpu import Case, bound

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16", "f16"]
SHAPES = [(128, 64, "half"), (128, 64, "interleaved"), (128, 0, "half"), (64, 0, "interleaved"), (96, 32, "half"),
          (80, 40, "interleaved"), (72, 40, "half"), (33, 10, "half"), (256, 16, "half")]
BAD = [float("inf"), float("-inf"), float("nan")]


def same(x, y):
    """The same bits, or NaN in both (a store may give NaN another sign and payload)."""
    bits = lambda t: t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)
    return bool(((bits(x) == bits(y)) | (torch.isnan(x) & torch.isnan(y))).all())


@pytest.mark.parametrize("path", ["auto", "scalar"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,rot,layout", SHAPES)
def test_elements_past_the_rotation_pass_unchanged(ctx, kind, D, rot, layout, path):
    """Without a weight an element that is not turned comes out as it went in: infinities, NaN, minus zero, and all others beside them."""
    c = Case(31, kind, 24, 3, 2, D, rot, layout, weights=False, bad_pos=False)
    g = torch.Generator().manual_seed(7)
    for x in (c.q, c.k, c.gq, c.gk):
        for t in range(c.T):
            x[t, t % x.shape[1], rot + int(torch.randint(0, D - rot, (1,), generator=g))] = (BAD + [-0.0])[t % 4]
    for got, x in zip(c.forward(ctx, path=path), (c.q, c.k)):
        assert same(got[..., rot:], x[..., rot:])
        y, mag = c.want(x, None)
        off, tol = np.abs(ref.f64(got[..., :rot]) - y[..., :rot]), bound(y, mag, kind, D)[..., :rot]
        assert np.all(off <= tol)
    for got, g in zip(c.backward(ctx, path=path)[:2], (c.gq, c.gk)):
        assert same(got[..., rot:], g[..., rot:])
        assert bool(torch.isfinite(got[..., :rot]).all())


@pytest.mark.parametrize("path", ["auto", "scalar"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,rot,layout", SHAPES)
def test_an_infinite_element_under_the_norm(ctx, kind, D, rot, layout, path):
    """An infinity makes the row's norm infinite: NaN in its own place (infinity over infinity), 0 in all others."""
    c = Case(32, kind, 24, 3, 2, D, rot, layout, bad_pos=False)
    at = {}
    for n, x in enumerate((c.q, c.k)):
        for t in range(0, c.T, 3):
            at[n, t] = (t % x.shape[1], rot + (7 * t) % (D - rot))
            x[(t, *at[n, t])] = BAD[t % 2]
    for n, (got, x, w) in enumerate(zip(c.forward(ctx, path=path), (c.q, c.k), (c.wq, c.wk))):
        want = np.zeros(got.shape, bool)
        for (m, t), (h, d) in at.items():
            if m == n:
                want[t, h, d] = True
                others = torch.cat([got[t, h, :d], got[t, h, d + 1:]])
                assert not bool(others.any())
        assert np.array_equal(np.isnan(ref.f64(got)), want)


@pytest.mark.parametrize("path", ["auto", "scalar"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,rot,layout", SHAPES)
def test_an_infinite_gradient_reaches_its_own_weight_only(ctx, kind, D, rot, layout, path):
    """dw[d] sums u[d] x[d] r: an infinity in an element that is not turned shows in that element's sum alone."""
    c = Case(33, kind, 24, 3, 2, D, rot, layout, bad_pos=False)
    d = rot + (D - rot) // 3
    rows = []
    clean = [ref.norm_rope_backward(ref.f64(g), ref.f64(x), ref.f64(w), *c.ref_args())
             for g, x, w in ((c.gq, c.q, c.wq), (c.gk, c.k, c.wk))]
    for g in (c.gq, c.gk):
        rows.append((5, g.shape[1] - 1))
        g[5, g.shape[1] - 1, d] = float("inf")
    got = c.backward(ctx, path=path)
    for n, (_, dw, _, mw) in enumerate(clean):
        off = np.abs(got[2 + n] - dw)
        tol = (c.T * (3, 2)[n] + D + 16) * 2.0**-23 * mw + 1e-30
        others = np.arange(D) != d
        assert not np.isfinite(got[2 + n][d]) and np.all(off[others] <= tol[others])
        dx, keep = ref.f64(got[n]), np.ones(got[n].shape[:2], bool)
        keep[rows[n]] = False  # the row's own gradient goes through its mean: nothing of it is finite
        assert np.all(np.abs(dx - clean[n][0])[keep] <= bound(clean[n][0], 2 * clean[n][2], kind, D)[keep])
