"""Host-side validation of the paged cache's calls, before anything touches the device (no GPU).

As in the other calls' checks: a zero-filled buffer stands in for the context, which is
tested for NULL only, and addresses are never dereferenced; with a GPU present the tests do
not run, so a stand-in context never reaches a device.
"""
import ctypes
import os
import re

import pytest

import scatter_boundary_tile_gb300 as sbt
from scatter_boundary_tile_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16, F16 = 0, 1, 2
X = 1 << 20
OK, BAD, UNS, ALN, CUDA = (sbt.SBT_OK, sbt.SBT_ERR_INVALID_ARG, sbt.SBT_ERR_UNSUPPORTED, sbt.SBT_ERR_ALIGNMENT,
                           sbt.SBT_ERR_CUDA)


def p(k, off=0):
    return X + 4096 * k + off


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("CPU-only check: a stand-in context must never reach a device")
    _build.build()
    return sbt.load_library()


@pytest.fixture(scope="module")
def ctx():
    return ctypes.create_string_buffer(4096)


def cache(**kw):
    c = dict(k=p(0), v=p(1), heads=2, head_dim=64, ld_page=2048, ld_slot=128, ld_head=64)
    c.update(kw)
    return sbt.KvCache(*c.values())


def pmap(**kw):
    m = dict(page_table=p(2), ld_table=4, n_seq=3, max_pages=4, lens=p(3), n_pages=10, page_size=16, refs=p(4))
    m.update(kw)
    return sbt.PageMap(*m.values())


def turn(**kw):
    r = dict(table=p(5), n_pos=32, rot_dim=64, layout=0)
    r.update(kw)
    return sbt.Rope(*r.values())


def pools(n=1, **kw):
    q = dict(base=p(6), n_planes=2, plane_stride=64000, page_stride=4096, page_bytes=4096)
    q.update(kw)
    return (sbt.PagePool * n)(*[sbt.PagePool(*q.values()) for _ in range(n)])


WS = [p(64), 1 << 30]

ATTENTION = [BF16, p(7), 256, 64, 3, 4, cache, pmap, None, 0.125, 0, p(8), 256, 64, p(9), *WS, None]
TABLE = [p(5), 32, 64, 10000.0, 0, 1.0, 0, 1.0, 32.0, 1.0, None]
ROPE = [BF16, p(7), 256, 64, p(8), 128, 64, 3, 4, 2, 64, p(9), turn, p(10), p(11), 1e-6, p(12), 256, 64, p(13), 128,
        64, p(14), 128, 64, cache, pmap, p(15), None]
BACK = [BF16, p(7), 256, 64, p(8), 128, 64, p(9), 256, 64, p(10), 128, 64, 3, 4, 2, 64, p(11), turn, p(12), p(13),
        1e-6, p(14), 256, 64, p(15), 128, 64, p(16), p(17), *WS, None]
COPY = [pools, 1, 10, p(7), p(8), 5, None]
RESERVE = [pmap, pools, 1, p(7), *WS, None]
FORK = [pmap, pools, 1, p(7), p(8), 3, *WS, None]
FREE = [pmap, p(7), p(8), 2, None]
COMPACT = [pmap, pools, 1, p(7), 4, p(8), p(9), p(10), *WS, None]

CASES = [  # (call, valid arguments, {index: value}, expected status)
    ("sbt_paged_attention", ATTENTION, {}, CUDA),
    ("sbt_paged_attention", ATTENTION, {0: 7}, UNS),
    ("sbt_paged_attention", ATTENTION, {1: None}, BAD),
    ("sbt_paged_attention", ATTENTION, {1: p(7, 1)}, ALN),
    ("sbt_paged_attention", ATTENTION, {2: -1}, BAD),
    ("sbt_paged_attention", ATTENTION, {4: 0}, OK),
    ("sbt_paged_attention", ATTENTION, {4: -1}, BAD),
    ("sbt_paged_attention", ATTENTION, {5: 3}, BAD),
    ("sbt_paged_attention", ATTENTION, {6: None}, BAD),
    ("sbt_paged_attention", ATTENTION, {6: lambda: cache(k=None)}, BAD),
    ("sbt_paged_attention", ATTENTION, {6: lambda: cache(v=p(1, 1))}, ALN),
    ("sbt_paged_attention", ATTENTION, {6: lambda: cache(head_dim=257, ld_slot=600, ld_head=300)}, BAD),
    ("sbt_paged_attention", ATTENTION, {6: lambda: cache(ld_slot=63)}, BAD),
    ("sbt_paged_attention", ATTENTION, {6: lambda: cache(ld_head=-64)}, BAD),
    ("sbt_paged_attention", ATTENTION, {6: lambda: cache(heads=0)}, BAD),
    ("sbt_paged_attention", ATTENTION, {7: None}, BAD),
    ("sbt_paged_attention", ATTENTION, {7: lambda: pmap(page_size=0)}, BAD),
    ("sbt_paged_attention", ATTENTION, {7: lambda: pmap(ld_table=3)}, BAD),
    ("sbt_paged_attention", ATTENTION, {7: lambda: pmap(n_seq=-1)}, BAD),
    ("sbt_paged_attention", ATTENTION, {7: lambda: pmap(n_pages=1 << 31)}, BAD),
    ("sbt_paged_attention", ATTENTION, {7: lambda: pmap(lens=None)}, BAD),
    ("sbt_paged_attention", ATTENTION, {7: lambda: pmap(lens=p(3, 2))}, ALN),
    ("sbt_paged_attention", ATTENTION, {7: lambda: pmap(refs=None)}, CUDA),
    ("sbt_paged_attention", ATTENTION, {8: p(5, 2)}, ALN),
    ("sbt_paged_attention", ATTENTION, {10: -1}, BAD),
    ("sbt_paged_attention", ATTENTION, {11: None}, BAD),
    ("sbt_paged_attention", ATTENTION, {13: 63}, BAD),
    ("sbt_paged_attention", ATTENTION, {14: None}, CUDA),
    ("sbt_paged_attention", ATTENTION, {14: p(9, 2)}, ALN),
    ("sbt_paged_attention", ATTENTION, {15: p(64, 16)}, ALN),
    ("sbt_paged_attention", ATTENTION, {15: None}, ALN),
    ("sbt_rope_table", TABLE, {}, CUDA),
    ("sbt_rope_table", TABLE, {1: 0}, OK),
    ("sbt_rope_table", TABLE, {1: -1}, BAD),
    ("sbt_rope_table", TABLE, {2: 63}, BAD),
    ("sbt_rope_table", TABLE, {0: p(5, 4)}, ALN),
    ("sbt_rope_table", TABLE, {3: 0.0}, BAD),
    ("sbt_rope_table", TABLE, {4: 9}, UNS),
    ("sbt_rope_table", TABLE, {5: -1.0}, BAD),
    ("sbt_rope_table", TABLE, {4: 3, 6: 0}, BAD),
    ("sbt_rope_table", TABLE, {4: 3, 6: 4096, 8: 1.0}, BAD),
    ("sbt_rope_table", TABLE, {4: 3, 6: 4096}, CUDA),
    ("sbt_qk_norm_rope", ROPE, {}, CUDA),
    ("sbt_qk_norm_rope", ROPE, {0: 9}, UNS),
    ("sbt_qk_norm_rope", ROPE, {7: 0}, OK),
    ("sbt_qk_norm_rope", ROPE, {7: -1}, BAD),
    ("sbt_qk_norm_rope", ROPE, {1: None}, BAD),
    ("sbt_qk_norm_rope", ROPE, {4: p(8, 1)}, ALN),
    ("sbt_qk_norm_rope", ROPE, {10: 513}, BAD),
    ("sbt_qk_norm_rope", ROPE, {11: None}, BAD),
    ("sbt_qk_norm_rope", ROPE, {12: lambda: turn(rot_dim=66)}, BAD),
    ("sbt_qk_norm_rope", ROPE, {12: lambda: turn(rot_dim=3)}, BAD),
    ("sbt_qk_norm_rope", ROPE, {12: lambda: turn(layout=2)}, UNS),
    ("sbt_qk_norm_rope", ROPE, {12: lambda: turn(table=None)}, BAD),
    ("sbt_qk_norm_rope", ROPE, {12: lambda: turn(table=p(5, 4))}, ALN),
    ("sbt_qk_norm_rope", ROPE, {12: None}, CUDA),
    ("sbt_qk_norm_rope", ROPE, {13: p(10, 1)}, ALN),
    ("sbt_qk_norm_rope", ROPE, {15: -1.0}, BAD),
    ("sbt_qk_norm_rope", ROPE, {16: None}, BAD),
    ("sbt_qk_norm_rope", ROPE, {18: 63}, BAD),
    ("sbt_qk_norm_rope", ROPE, {19: None}, CUDA),
    ("sbt_qk_norm_rope", ROPE, {19: None, 22: None, 25: None}, BAD),
    ("sbt_qk_norm_rope", ROPE, {25: None}, BAD),
    ("sbt_qk_norm_rope", ROPE, {25: lambda: cache(heads=1)}, BAD),
    ("sbt_qk_norm_rope", ROPE, {25: lambda: cache(ld_page=63)}, BAD),
    ("sbt_qk_norm_rope", ROPE, {26: None}, BAD),
    ("sbt_qk_norm_rope", ROPE, {26: lambda: pmap(lens=None, refs=None)}, CUDA),
    ("sbt_qk_norm_rope", ROPE, {27: p(15, 1)}, ALN),
    ("sbt_qk_norm_rope_backward", BACK, {}, CUDA),
    ("sbt_qk_norm_rope_backward", BACK, {0: 5}, UNS),
    ("sbt_qk_norm_rope_backward", BACK, {19: None}, BAD),
    ("sbt_qk_norm_rope_backward", BACK, {28: None}, BAD),
    ("sbt_qk_norm_rope_backward", BACK, {7: None}, BAD),
    ("sbt_qk_norm_rope_backward", BACK, {7: None, 19: None, 28: None}, CUDA),
    ("sbt_qk_norm_rope_backward", BACK, {24: 63}, BAD),
    ("sbt_qk_norm_rope_backward", BACK, {30: p(64, 8)}, ALN),
    ("sbt_qk_norm_rope_backward", BACK, {13: 0}, CUDA),
    ("sbt_qk_norm_rope_backward", BACK, {13: 0, 19: None, 20: None, 28: None, 29: None}, OK),
    ("sbt_pages_copy", COPY, {}, CUDA),
    ("sbt_pages_copy", COPY, {5: 0}, OK),
    ("sbt_pages_copy", COPY, {5: -1}, BAD),
    ("sbt_pages_copy", COPY, {1: 0}, BAD),
    ("sbt_pages_copy", COPY, {0: lambda: pools(65), 1: 65}, BAD),
    ("sbt_pages_copy", COPY, {0: lambda: pools(page_stride=4095)}, BAD),
    ("sbt_pages_copy", COPY, {0: lambda: pools(plane_stride=100)}, BAD),
    ("sbt_pages_copy", COPY, {0: lambda: pools(base=None)}, BAD),
    ("sbt_pages_copy", COPY, {0: lambda: pools(page_bytes=0)}, BAD),
    ("sbt_pages_copy", COPY, {3: p(7, 2)}, ALN),
    ("sbt_pages_copy", COPY, {4: None}, BAD),
    ("sbt_pages_reserve", RESERVE, {}, CUDA),
    ("sbt_pages_reserve", RESERVE, {0: lambda: pmap(refs=None)}, BAD),
    ("sbt_pages_reserve", RESERVE, {0: lambda: pmap(n_seq=0)}, OK),
    ("sbt_pages_reserve", RESERVE, {3: None}, BAD),
    ("sbt_pages_reserve", RESERVE, {5: 8}, ALN),
    ("sbt_pages_fork", FORK, {}, CUDA),
    ("sbt_pages_fork", FORK, {5: 4}, BAD),
    ("sbt_pages_fork", FORK, {5: 0}, OK),
    ("sbt_pages_fork", FORK, {4: p(8, 1)}, ALN),
    ("sbt_pages_free", FREE, {}, CUDA),
    ("sbt_pages_free", FREE, {2: None}, CUDA),
    ("sbt_pages_free", FREE, {1: None}, BAD),
    ("sbt_pages_free", FREE, {3: -1}, BAD),
    ("sbt_pages_free", FREE, {3: 0}, OK),
    ("sbt_pages_compact", COMPACT, {}, CUDA),
    ("sbt_pages_compact", COMPACT, {4: 3}, BAD),
    ("sbt_pages_compact", COMPACT, {3: p(2), 4: 5}, BAD),
    ("sbt_pages_compact", COMPACT, {3: p(2)}, CUDA),
    ("sbt_pages_compact", COMPACT, {5: None}, BAD),
    ("sbt_pages_compact", COMPACT, {7: None}, BAD),
    ("sbt_pages_compact", COMPACT, {6: p(9, 1)}, ALN),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_validation_before_the_device(lib, ctx, i):
    name, base, change, want = CASES[i]
    args = [change.get(k, a) for k, a in enumerate(base)]
    args = [a() if callable(a) else a for a in args]
    assert getattr(lib, name)(ctx, *args) == want, (name, change, lib.sbt_last_error_message())
    assert getattr(lib, name)(None, *args) == BAD


def test_workspace_queries(lib, ctx):
    n = ctypes.c_size_t(0)
    r = ctypes.byref(n)
    assert lib.sbt_paged_attention_workspace_size(ctx, 8, 2, 128, r) == OK
    assert lib.sbt_paged_attention_workspace_size(ctx, 8, 3, 128, r) == BAD
    assert lib.sbt_paged_attention_workspace_size(ctx, 8, 2, 257, r) == BAD
    assert lib.sbt_qk_norm_rope_backward_workspace_size(ctx, 512, r) == OK
    assert lib.sbt_qk_norm_rope_backward_workspace_size(ctx, 0, r) == BAD
    assert lib.sbt_pages_workspace_size(ctx, 5, 100, r) == OK and n.value >= 4 * (2 * 100 + 100)
    assert lib.sbt_pages_workspace_size(ctx, -1, 100, r) == BAD
    assert lib.sbt_pages_workspace_size(ctx, 5, 1 << 31, r) == BAD


def test_structs_and_limits_match_the_header():
    """The binding's struct layouts are the header's, compiled by gcc."""
    import subprocess
    import tempfile
    fields = {"sbt_page_map": (sbt.PageMap, "page_table ld_table n_seq max_pages lens n_pages page_size refs"),
              "sbt_kv_cache": (sbt.KvCache, "k v heads head_dim ld_page ld_slot ld_head"),
              "sbt_rope": (sbt.Rope, "table n_pos rot_dim layout"),
              "sbt_page_pool": (sbt.PagePool, "base n_planes plane_stride page_stride page_bytes")}
    body = "".join(f'printf("%zu", sizeof({t}));' + "".join(f'printf(" %zu", offsetof({t}, {f}));' for f in fs.split())
                   + 'printf("\\n");' for t, (_, fs) in fields.items())
    src = f'#include <stdio.h>\n#include "sbt.h"\nint main(void) {{ {body} printf("%d\\n", SBT_MAX_PAGE_POOLS); return 0; }}\n'
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "a.c"), os.path.join(d, "a")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    for line, (cls, fs) in zip(out, fields.values()):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fs.split()]
    assert int(out[len(fields)]) == sbt.MAX_PAGE_POOLS
    text = open(os.path.join(ROOT, "include", "sbt.h")).read()
    for name, codes in (("SBT_ROPE_", {**{k.upper(): v for k, v in sbt.ROPE_LAYOUTS.items()},
                                       **{k.upper(): v for k, v in sbt.ROPE_SCALINGS.items()}}),):
        for k, v in codes.items():
            assert re.search(rf"\b{name}{k} = {v}\b", text), k
