"""sbt_paged_tree_attention with the bounds of probabilities of two 16-bit numbers, whatever max_new is; pages of more
positions than a tile, and more entries than a block has threads on planes of 256 rows."""
import numpy as np
import pytest

import step_ref as ref
from test_tree_attention_gpu import KINDS, Case

pytestmark = pytest.mark.gpu


class Exact(Case):
    """Checked with the bounds of probabilities of two 16-bit numbers."""

    def bounds(self, want):
        return ref.tree_attention_bounds(want, self.kind, self.D, 2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("sizes,group,max_new", [
    ([(40, 3), (5, 1)], 4, None), ([(1, 1), (3, 4), (2, 0)], 4, 200), ([(7, 100)], 2, 65), ([(64, 40), (33, 2)], 8, None),
    ([(130, 5)], 1, None)])
def test_probabilities_keep_their_bits(ctx, sizes, group, max_new, D, kind):
    """Few visible positions: values of either sign cancel in the output, whose own rounding is small then."""
    Exact(D + group, kind, sizes, 2, group, D, 16, max_new=max_new).check(ctx)
    Exact(D + group, kind, sizes, 1, group, D, 16, max_new=max_new, masked=False).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
def test_probabilities_that_cancel(ctx, D, kind):
    """Two positions whose values cancel to a thousandth of themselves."""
    c = Exact(3, kind, [(1, 1), (40, 1)], 1, 4, D, 16, masked=False)
    k, v, page = ref.f64(c.view(c.k)), c.view(c.v), int(c.table[int(c.seq[0]), 0])
    ratio = np.exp((k[page, 0, 0] - k[page, 1, 0]) @ ref.f64(c.q)[0, 0] * c.scale)  # of their probabilities
    v[page, 0, 0] = -min(1.0, 1 / ratio)
    v[page, 1, 0] = min(1.0, ratio)
    c.check(ctx)
    out = np.abs(c.want()[0][0, 0]).max()
    assert out <= 2.0**-7 * min(ratio, 1 / ratio)


@pytest.mark.parametrize("kind", KINDS)
def test_the_same_tokens_under_a_larger_max_new(ctx, kind):
    """Rows of 256 share a block then; the answer has as many bits."""
    for max_new in (5, 32, 33, 400):
        Exact(21, kind, [(5, 300), (2, 64), (1, 0)], 2, 4, 128, 16, max_new=max_new).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P", [64, 128, 192, 256])
@pytest.mark.parametrize("order", ["nhd", "hnd"])
def test_pages_of_more_positions_than_a_tile(ctx, order, P, kind):
    Exact(P, kind, [(5, 700), (9, 128), (3, 61), (1, 0)], 2, 4, 64, P, order).check(ctx)
    Exact(P, kind, [(40, 500), (3, 127)], 1, 8, 128, P, order, masked=False).check(ctx)
    Exact(P, kind, [(5, 300), (9, 1000)], 2, 2, 80, P, order, holes=0.3).check(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes,group,max_new", [
    ([(1 + i % 3, i % 90) for i in range(500)], 1, 200), ([(1 + i % 40, i % 70) for i in range(420)], 4, None),
    ([(0 if i % 3 else 2, 5 * i % 300) for i in range(900)], 2, 300)])
def test_many_entries_on_planes_of_256_rows(ctx, sizes, group, max_new, kind):
    Exact(len(sizes), kind, sizes, 1, group, 64, 16, max_new=max_new).check(ctx)
