"""Extents whose products or sums would pass the kernels' counters are refused on the host (no GPU)."""
import pytest

from test_cache_abi import BACK, BAD, CUDA, OK, ROPE, TABLE, ctx, lib  # noqa: F401 (ctx and lib are fixtures)

HEADS = 1 << 30  # q_heads + 2 k_heads at most
CASES = [
    ("sbt_qk_norm_rope", ROPE, {8: HEADS, 9: 0, 22: None, 25: None, 26: None}, CUDA),
    ("sbt_qk_norm_rope", ROPE, {8: HEADS + 1, 9: 0, 22: None, 25: None, 26: None}, BAD),
    ("sbt_qk_norm_rope", ROPE, {8: HEADS - 4, 9: 2}, CUDA),
    ("sbt_qk_norm_rope", ROPE, {8: HEADS - 3, 9: 2}, BAD),
    ("sbt_qk_norm_rope", ROPE, {8: 2**31 - 1, 9: 2}, BAD),
    ("sbt_qk_norm_rope", ROPE, {8: 2**31 - 2, 9: 2**31 - 2, 22: None, 25: None, 26: None}, BAD),
    ("sbt_qk_norm_rope_backward", BACK, {14: HEADS - 4}, CUDA),
    ("sbt_qk_norm_rope_backward", BACK, {14: HEADS - 3}, BAD),
    ("sbt_qk_norm_rope_backward", BACK, {14: 2**31 - 1, 15: 2**31 - 1}, BAD),
    ("sbt_rope_table", TABLE, {1: (1 << 40) - 1, 2: 2}, CUDA),
    ("sbt_rope_table", TABLE, {1: 1 << 39, 2: 1 << 30}, BAD),
    ("sbt_rope_table", TABLE, {1: 1 << 34, 2: 2**31 - 2}, BAD),
    ("sbt_rope_table", TABLE, {1: 1 << 20, 2: 1 << 21}, CUDA),
    ("sbt_rope_table", TABLE, {1: 0, 2: 2**31 - 2}, OK),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_extents(lib, ctx, i):  # noqa: F811
    name, base, change, want = CASES[i]
    args = [change.get(k, a) for k, a in enumerate(base)]
    args = [a() if callable(a) else a for a in args]
    assert getattr(lib, name)(ctx, *args) == want, (name, change, lib.sbt_last_error_message())
