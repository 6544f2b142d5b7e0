"""sbt_paged_attention: every position counts once, wherever rows are cut and joined.

Scores are whole powers of two apart and values are small whole numbers, so that sums of either are exact
in fp32 and one position lost, doubled or given to another row shows: by 1 / n in the sum (the log-sum-exp
is known to a few 2^-24), by whole steps in the outputs, whose elements each count one stretch of positions.
"""
import numpy as np
import pytest
import torch

import cache_ref as ref
import scatter_boundary_tile_gb300 as sbt

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16", "f16"]
LN2 = float(np.float32(np.log(2)))  # times the fp32 log2(e) this is 1 exactly: a key of -j has the probability 2^-j

ROWS = {  # lengths, head size, key-value heads, query heads of each
    "few rows of many parts": ([40000, 1, 3000], 64, 1, 3),
    "one long row among short ones": ([30000] + [5, 0, 40] * 30, 128, 1, 4),
    "every row cut": ([2600] * 40, 96, 3, 2),
    "two rows": ([17000, 9000], 256, 1, 1),
    "two chunks of query heads": ([20001, 7, 9001, 300], 128, 2, 17),
    "16 query heads": ([131071, 16, 0, 65], 128, 1, 16),
    "more rows than warps": ([(i * 37) % 61 for i in range(700)] + [20000, 0, 3001, 9999], 64, 8, 1),
    "more rows than warps, all of them cut or long": ([1024 + (i * 131) % 700 for i in range(300)], 32, 8, 2),
}


def test_the_scale_is_one():
    assert np.float32(np.float32(LN2) * np.float32(1.4426950408889634)) == 1


@pytest.mark.parametrize("levels", [1, 6])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("window", [0, 1777])
def test_every_position_counts_once(ctx, kind, rows, levels, window):
    """levels = 1: equal scores, lse = log n.  More: the probabilities go up and down in powers of two along the row,
    a part's largest one is another one's smaller one.

    out[d] is (h + 1) times the weight of stretch d (of D) of the positions, over the weight of all.  Both sums
    are exact (below 2^17 times 2^5 whole steps) but for the exponential's own 2^-22; the quotient rounds three
    times and the output once."""
    lens, D, H, group = ROWS[rows]
    dt, S, P = ref.TDT[kind], len(lens), 16
    need = [-(-n // P) for n in lens]
    g = torch.Generator().manual_seed(S + D)
    perm = torch.randperm(sum(need) + 2, generator=g).to(torch.int32)
    table = torch.full((S, max(need)), -1, dtype=torch.int32)
    k = torch.full((len(perm), P, H, D), float("nan"), dtype=dt, device="cuda")
    v = torch.full_like(k, float("nan"))
    want, lse_want = np.zeros((S, H * group, D)), np.full((S, H * group), -np.inf)
    at = 0
    for s, n in enumerate(lens):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
        if n == 0:
            continue
        lo = max(0, n - window) if window else 0
        t = torch.arange(n)
        level = (t // 7 * 5 + t // 900 + s) % levels
        key = torch.zeros(n, H, D)
        key[:, :, 0] = -level[:, None].float()
        value, w = torch.zeros(n, H, D), torch.exp2(-level.double()).numpy()
        w[:lo] = 0
        lse_s = np.log(w.sum())
        for h in range(H):
            part = (t * D // n + 7 * h + s) % D
            value[t, h, part] = h + 1.0
            sums = np.bincount(part.numpy(), weights=w, minlength=D) * (h + 1) / w.sum()
            want[s, h * group:(h + 1) * group], lse_want[s, h * group:(h + 1) * group] = sums, lse_s
        pages = table[s, :need[s]].long().cuda()
        pad = need[s] * P - n
        for dst, src in ((k, key), (v, value)):  # the slots past the length keep their NaN
            x = torch.cat([src, torch.full((pad, H, D), float("nan"))]).view(need[s], P, H, D)
            dst[pages] = x.to(dt).cuda()
    q = torch.zeros(S, H * group, D)
    q[:, :, 0] = 1.0
    q = q.to(dt).cuda()
    out, lse = torch.empty_like(q), torch.empty((S, H * group), device="cuda")
    size = sbt.paged_attention_workspace_size(ctx, H * group, H, D)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    table_d, lens_d = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    sbt.paged_attention(ctx, q, H * group * D, D, S, H * group,
                        sbt.kv_cache(k, v, H, D, P * H * D, H * D, D),
                        sbt.page_map(table_d, max(need), S, max(need), lens_d, len(perm), P), LN2, out,
                        H * group * D, D, lse=lse, window=window, workspace=ws, workspace_bytes=size)
    torch.cuda.synchronize()
    got, lse = ref.f64(out), lse.cpu().numpy()
    empty = np.isneginf(lse_want)
    assert np.array_equal(np.isneginf(lse), empty)
    # log2 and its factor: a few roundings of the value; the exponential's error under the logarithm
    assert np.all(np.abs(lse[~empty] - lse_want[~empty]) <= 2.0**-22 * (2 + np.abs(lse_want[~empty])))
    assert np.all(np.abs(got - want) <= (1.01 * ref.HALF_ULP[kind] + 2.0**-20) * want)
