"""Host-side validation of the calls around the attention, before anything touches the device (no GPU).

As in the cache's checks: a zero-filled buffer stands in for the context and addresses are
never dereferenced; with a GPU present the tests do not run.
"""
import pytest

import scatter_boundary_tile_gb300 as sbt
from test_cache_abi import ALN, BAD, BF16, CUDA, F16, F32, OK, UNS, WS, cache, ctx, lib, p, pmap  # noqa: F401

E4M3, E5M2, E8M0, E2M1 = 0, 1, 2, 3


def codes(**kw):
    c = dict(codes=p(20), ld=128, scales=p(21), ld_scale=4, format=E4M3, block=32)
    c.update(kw)
    return sbt.CodeRows(*c.values())


NORM = [BF16, p(0), 128, p(1), 128, 5, 128, p(2), 1e-6, p(3), 128, p(4), 128, codes, None]
BACK = [BF16, p(0), 128, p(1), 128, p(2), 128, 5, 128, p(3), 1e-6, p(4), 128, p(5), *WS, None]
MATVEC = [BF16, p(0), 256, 3, p(1), 64, E8M0, p(2), 64, 8, 1.0, p(3), 64, F32, 64, 256, None]
SLOTS = [pmap, p(7), 3, p(8), p(9), 100, p(10), p(11), p(12), p(13), p(14), None]
PLAN = [p(7), p(8), 3, 50, p(9), p(10), p(11), 2, None]
TREE = [BF16, p(7), 256, 64, 50, p(8), 3, 16, 4, cache, pmap, p(9), 0.125, p(10), 1, p(11), 256, 64, p(12), *WS, None]

CASES = [  # (call, valid arguments, {index: value}, expected status)
    ("sbt_add_rms_norm", NORM, {}, CUDA),
    ("sbt_add_rms_norm", NORM, {0: 7}, UNS),
    ("sbt_add_rms_norm", NORM, {1: None}, BAD),
    ("sbt_add_rms_norm", NORM, {1: p(0, 1)}, ALN),
    ("sbt_add_rms_norm", NORM, {2: -1}, BAD),
    ("sbt_add_rms_norm", NORM, {2: 0}, CUDA),
    ("sbt_add_rms_norm", NORM, {3: None}, CUDA),
    ("sbt_add_rms_norm", NORM, {3: p(1, 1)}, ALN),
    ("sbt_add_rms_norm", NORM, {5: 0}, OK),
    ("sbt_add_rms_norm", NORM, {5: -1}, BAD),
    ("sbt_add_rms_norm", NORM, {5: 1 << 31}, BAD),
    ("sbt_add_rms_norm", NORM, {6: 0}, BAD),
    ("sbt_add_rms_norm", NORM, {6: (1 << 24) + 32}, BAD),
    ("sbt_add_rms_norm", NORM, {6: 120, 13: None}, CUDA),
    ("sbt_add_rms_norm", NORM, {6: 120}, BAD),
    ("sbt_add_rms_norm", NORM, {7: None}, CUDA),
    ("sbt_add_rms_norm", NORM, {7: p(2, 1)}, ALN),
    ("sbt_add_rms_norm", NORM, {8: -1.0}, BAD),
    ("sbt_add_rms_norm", NORM, {9: None}, CUDA),
    ("sbt_add_rms_norm", NORM, {10: 127}, BAD),
    ("sbt_add_rms_norm", NORM, {11: None}, CUDA),
    ("sbt_add_rms_norm", NORM, {11: None, 13: None}, BAD),
    ("sbt_add_rms_norm", NORM, {12: 127}, BAD),
    ("sbt_add_rms_norm", NORM, {11: p(3)}, BAD),
    ("sbt_add_rms_norm", NORM, {9: p(0)}, CUDA),
    ("sbt_add_rms_norm", NORM, {9: p(0), 10: 136}, BAD),
    ("sbt_add_rms_norm", NORM, {11: p(1), 12: 136}, BAD),
    ("sbt_add_rms_norm", NORM, {13: None}, CUDA),
    ("sbt_add_rms_norm", NORM, {13: lambda: codes(format=E2M1)}, UNS),
    ("sbt_add_rms_norm", NORM, {13: lambda: codes(format=E5M2)}, CUDA),
    ("sbt_add_rms_norm", NORM, {13: lambda: codes(block=24)}, BAD),
    ("sbt_add_rms_norm", NORM, {13: lambda: codes(block=0)}, BAD),
    ("sbt_add_rms_norm", NORM, {13: lambda: codes(block=128, ld_scale=1)}, CUDA),
    ("sbt_add_rms_norm", NORM, {13: lambda: codes(ld_scale=3)}, BAD),
    ("sbt_add_rms_norm", NORM, {13: lambda: codes(ld=127)}, BAD),
    ("sbt_add_rms_norm", NORM, {13: lambda: codes(codes=None)}, BAD),
    ("sbt_add_rms_norm", NORM, {13: lambda: codes(scales=None)}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {}, CUDA),
    ("sbt_add_rms_norm_backward", BACK, {0: 9}, UNS),
    ("sbt_add_rms_norm_backward", BACK, {1: None}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {3: None}, CUDA),
    ("sbt_add_rms_norm_backward", BACK, {3: p(1, 1)}, ALN),
    ("sbt_add_rms_norm_backward", BACK, {5: None}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {7: 0}, CUDA),
    ("sbt_add_rms_norm_backward", BACK, {7: 0, 9: None, 13: None}, OK),
    ("sbt_add_rms_norm_backward", BACK, {7: -1}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {8: 0}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {9: None}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {13: None}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {9: None, 13: None}, CUDA),
    ("sbt_add_rms_norm_backward", BACK, {11: None}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {12: 100}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {11: p(0)}, CUDA),
    ("sbt_add_rms_norm_backward", BACK, {11: p(0), 12: 136}, BAD),
    ("sbt_add_rms_norm_backward", BACK, {13: p(5, 2)}, ALN),
    ("sbt_add_rms_norm_backward", BACK, {14: None}, ALN),
    ("sbt_add_rms_norm_backward", BACK, {14: p(64, 16)}, ALN),
    ("sbt_add_rms_norm_backward", BACK, {15: 0}, ALN),
    ("sbt_matvec_e2m1", MATVEC, {}, CUDA),
    ("sbt_matvec_e2m1", MATVEC, {0: 5}, UNS),
    ("sbt_matvec_e2m1", MATVEC, {1: None}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {1: p(0, 1)}, ALN),
    ("sbt_matvec_e2m1", MATVEC, {3: 0}, OK),
    ("sbt_matvec_e2m1", MATVEC, {3: -1}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {3: 65535 * 8 + 1}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {4: None}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {4: p(1, 3)}, CUDA),
    ("sbt_matvec_e2m1", MATVEC, {5: 65}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {5: 62}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {6: E2M1}, UNS),
    ("sbt_matvec_e2m1", MATVEC, {6: E4M3}, CUDA),
    ("sbt_matvec_e2m1", MATVEC, {7: None}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {8: 63}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {8: 63, 9: 1}, CUDA),
    ("sbt_matvec_e2m1", MATVEC, {9: 0}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {9: 7}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {9: 32}, UNS),
    ("sbt_matvec_e2m1", MATVEC, {9: 16}, CUDA),
    ("sbt_matvec_e2m1", MATVEC, {11: None}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {11: p(3, 2)}, ALN),
    ("sbt_matvec_e2m1", MATVEC, {12: 63}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {13: 8}, UNS),
    ("sbt_matvec_e2m1", MATVEC, {14: 0, 5: 0}, OK),
    ("sbt_matvec_e2m1", MATVEC, {14: 1 << 31, 5: 1 << 31, 8: 1 << 31, 12: 1 << 31}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {15: -256}, BAD),
    ("sbt_matvec_e2m1", MATVEC, {15: 0, 1: None, 4: None, 7: None, 9: 0}, CUDA),
    ("sbt_pages_slots", SLOTS, {}, CUDA),
    ("sbt_pages_slots", SLOTS, {0: None}, BAD),
    ("sbt_pages_slots", SLOTS, {0: lambda: pmap(lens=None)}, CUDA),
    ("sbt_pages_slots", SLOTS, {0: lambda: pmap(lens=None), 4: None}, BAD),
    ("sbt_pages_slots", SLOTS, {0: lambda: pmap(n_pages=(1 << 27) + 1)}, BAD),
    ("sbt_pages_slots", SLOTS, {0: lambda: pmap(n_pages=1 << 27)}, CUDA),
    ("sbt_pages_slots", SLOTS, {0: lambda: pmap(n_pages=(1 << 27) + 1), 9: None}, CUDA),
    ("sbt_pages_slots", SLOTS, {1: None}, BAD),
    ("sbt_pages_slots", SLOTS, {1: None, 2: 0}, CUDA),
    ("sbt_pages_slots", SLOTS, {2: -1}, BAD),
    ("sbt_pages_slots", SLOTS, {5: -1}, BAD),
    ("sbt_pages_slots", SLOTS, {5: 0}, CUDA),
    ("sbt_pages_slots", SLOTS, {5: 0, 6: None, 10: None}, OK),
    ("sbt_pages_slots", SLOTS, {6: None, 7: None, 8: None, 9: None, 10: None}, OK),
    *[("sbt_pages_slots", SLOTS, {i: p(7 + i, 2)}, ALN) for i in (1, 3, 4, 6, 7, 8, 9, 10)],
    ("sbt_tree_plan", PLAN, {}, CUDA),
    ("sbt_tree_plan", PLAN, {0: None}, BAD),
    ("sbt_tree_plan", PLAN, {1: None}, BAD),
    ("sbt_tree_plan", PLAN, {0: None, 1: None, 2: 0, 4: None}, CUDA),
    ("sbt_tree_plan", PLAN, {2: -1}, BAD),
    ("sbt_tree_plan", PLAN, {3: -1}, BAD),
    ("sbt_tree_plan", PLAN, {3: 0}, OK),
    ("sbt_tree_plan", PLAN, {4: None}, BAD),
    ("sbt_tree_plan", PLAN, {4: None, 5: None}, CUDA),
    ("sbt_tree_plan", PLAN, {5: None, 6: None}, OK),
    ("sbt_tree_plan", PLAN, {7: 0}, BAD),
    ("sbt_tree_plan", PLAN, {6: None, 7: 0}, CUDA),
    ("sbt_tree_plan", PLAN, {7: (1 << 20) + 1}, BAD),
    *[("sbt_tree_plan", PLAN, {i: p(7 + i, 1)}, ALN) for i in (0, 1, 4, 5, 6)],
    ("sbt_paged_tree_attention", TREE, {}, CUDA),
    ("sbt_paged_tree_attention", TREE, {0: F32}, UNS),
    ("sbt_paged_tree_attention", TREE, {0: F16}, CUDA),
    ("sbt_paged_tree_attention", TREE, {1: None}, BAD),
    ("sbt_paged_tree_attention", TREE, {1: p(7, 1)}, ALN),
    ("sbt_paged_tree_attention", TREE, {2: -1}, BAD),
    ("sbt_paged_tree_attention", TREE, {4: 0}, OK),
    ("sbt_paged_tree_attention", TREE, {4: -1}, BAD),
    ("sbt_paged_tree_attention", TREE, {5: None}, BAD),
    ("sbt_paged_tree_attention", TREE, {5: p(8, 2)}, ALN),
    ("sbt_paged_tree_attention", TREE, {6: 0}, OK),
    ("sbt_paged_tree_attention", TREE, {6: -1}, BAD),
    ("sbt_paged_tree_attention", TREE, {6: 1 << 30}, BAD),
    ("sbt_paged_tree_attention", TREE, {7: 0}, BAD),
    ("sbt_paged_tree_attention", TREE, {7: 1 << 23}, BAD),
    ("sbt_paged_tree_attention", TREE, {7: (1 << 23) - 1}, CUDA),
    ("sbt_paged_tree_attention", TREE, {8: 3}, BAD),
    ("sbt_paged_tree_attention", TREE, {9: None}, BAD),
    ("sbt_paged_tree_attention", TREE, {9: lambda: cache(head_dim=257, ld_slot=600, ld_head=300)}, BAD),
    ("sbt_paged_tree_attention", TREE, {9: lambda: cache(k=p(0, 1))}, ALN),
    ("sbt_paged_tree_attention", TREE, {10: None}, BAD),
    ("sbt_paged_tree_attention", TREE, {10: lambda: pmap(lens=None)}, BAD),
    ("sbt_paged_tree_attention", TREE, {11: p(9, 2)}, ALN),
    ("sbt_paged_tree_attention", TREE, {13: None, 14: 0}, CUDA),
    ("sbt_paged_tree_attention", TREE, {14: 0}, BAD),
    ("sbt_paged_tree_attention", TREE, {13: p(10, 1)}, ALN),
    ("sbt_paged_tree_attention", TREE, {15: None}, BAD),
    ("sbt_paged_tree_attention", TREE, {17: 63}, BAD),
    ("sbt_paged_tree_attention", TREE, {18: None}, CUDA),
    ("sbt_paged_tree_attention", TREE, {18: p(12, 2)}, ALN),
    ("sbt_paged_tree_attention", TREE, {19: None}, ALN),
    ("sbt_paged_tree_attention", TREE, {19: p(64, 8)}, ALN),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_arguments(lib, ctx, i):  # noqa: F811
    name, base, change, want = CASES[i]
    args = [change.get(k, a) for k, a in enumerate(base)]
    args = [a() if callable(a) else a for a in args]
    assert getattr(lib, name)(ctx, *args) == want, (name, change, lib.sbt_last_error_message())
    assert getattr(lib, name)(None, *args) == BAD
