"""sbt_paged_attention where the probabilities' own precision shows: one dominant position among many
small ones, values next to the type's largest, and the output's error next to one rounding of it.

All sequences read the same pages (a page may stand in any number of tables), so that one small
cache serves one row, rows that are cut, and more rows than the GPU has warps.
"""
import numpy as np
import pytest
import torch

import cache_ref as ref
import scatter_boundary_tile_gb300 as sbt

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16", "f16"]


def attend(ctx, kind, q, k, v, n, batch, scale, page_size=16):
    """q [Hq][D], k and v [>= n][H][D]: `batch` sequences of the same n positions; out and lse of all of them."""
    dt, (Hq, D), H = ref.TDT[kind], q.shape, k.shape[1]
    pages = -(-n // page_size)
    pool = lambda x: torch.cat([x, x.new_zeros(pages * page_size - len(x), H, D)]).to(dt).cuda().contiguous()
    kc, vc = pool(k), pool(v)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(batch, 1).contiguous()
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    qs = q.to(dt).cuda().repeat(batch, 1, 1).contiguous()
    out, lse = torch.empty_like(qs), torch.empty((batch, Hq), device="cuda")
    size = sbt.paged_attention_workspace_size(ctx, Hq, H, D)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    sbt.paged_attention(ctx, qs, Hq * D, D, batch, Hq,
                        sbt.kv_cache(kc, vc, H, D, page_size * H * D, H * D, D),
                        sbt.page_map(table, pages, batch, pages, lens, pages, page_size), scale, out, Hq * D, D,
                        lse=lse, workspace=ws, workspace_bytes=size)
    torch.cuda.synchronize()
    return ref.f64(out), lse.cpu().numpy()


# rows: one (a cluster), a few that are cut, more than the GPU has warps (most of them whole in one warp's range)
@pytest.mark.parametrize("batch", [1, 9, 1100])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bits", [18.0, 20.3, 22.6, 23.5, 25.2, 26.0])
@pytest.mark.parametrize("sink", [0, 2000, 4096])
def test_one_dominant_position_and_many_small_ones(ctx, kind, batch, bits, sink):
    """A position of value 0 and 4096 others of value 1 at 2^-bits of its probability.

    Exact: x / (1 + x) with x = 4096 2^-bits.  Relative error of a small probability: its exponent is off by two
    roundings of `bits`, the exponential by 2^-22, the two 16-bit parts by 2^-16 (bf16) or by 2^-22 and half a
    step of 2^-24 of 2^15 p (fp16); the sums round once per position, l = 1 + x by a share of itself, which is also
    what the log-sum-exp may be off by; the output is rounded once."""
    n, D, H = 4097, 64, 2
    q, k, v = torch.zeros(4, D), torch.zeros(n, H, D), torch.ones(n, H, D)
    q[:, 0], k[:, :, 0] = 1.0, -1.0
    k[sink], v[sink] = 0.0, 0.0
    scale = float(np.float32(bits * np.log(2)))
    x = 4096 * np.exp(-scale)
    want = x / (1 + x)
    out, lse = attend(ctx, kind, q, k, v, n, batch, scale)
    sums = (n + 64) * 2.0**-23
    rel = 2 * bits * 2.0**-23 + 2.0**-22
    lse_off = 2.0**-20 * (1 + np.log1p(x)) + sums + rel * x
    rel += sums + {"f32": 0.0, "bf16": 2.0**-16, "f16": 2.0**-22 + 2.0**-25 / (2.0**15 * 2.0**-bits)}[kind]
    assert np.all(np.abs(out - want) <= (rel + 1.01 * ref.HALF_ULP[kind]) * want + ref.TINY[kind])
    assert np.all(np.abs(lse - np.log1p(x)) <= lse_off)


@pytest.mark.parametrize("batch", [1, 9, 1100])
@pytest.mark.parametrize("over", [0.3, 0.55, 0.8])
def test_values_next_to_the_largest_stay_finite(ctx, batch, over):
    """Every value is fp16's largest number, so that is the average, whatever the probabilities.

    They lie `over` of a step above a number of 11 bits: rounded up, all but one of them would add up to 2^-11 of
    the sum, past the border to infinity, which is 2^-12 above the largest number.  The sums' error, at most
    364 2^-23, and the two parts', 2^-22, are far below that border.  (In bf16 an fp32 sum of such values is
    infinite itself.)"""
    n, D, top = 300, 64, 65504.0
    q, k, v = torch.zeros(4, D), torch.zeros(n, 2, D), torch.full((n, 2, D), top)
    q[:, 0], k[:, :, 0] = 1.0, -1.0
    k[7] = 0.0
    scale = float(np.float32(-np.log(0.5 * (1 + over * 2.0**-10))))
    out, _ = attend(ctx, "f16", q, k, v, n, batch, scale)
    assert np.all(out == top)


@pytest.mark.parametrize("batch", [1, 9, 1100])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("D,H,group,n", [(128, 2, 4, 777), (64, 1, 16, 1500), (100, 2, 1, 400)])
def test_error_is_that_of_one_rounding(ctx, kind, batch, D, H, group, n):
    """Over ordinary inputs the output's error (2-norm) is that of rounding the exact one to the type once.

    What else there is, fp32 scores (2^-22 of values near 10, a few 2^-20 in the exponent) and the two parts
    of the probabilities (2^-16 at most each, of either sign), adds in squares: (2^-17 / 2^-12.8)^2 < 1 % even
    for fp16's smaller rounding."""
    g = torch.Generator().manual_seed(D + n)
    dt = ref.TDT[kind]
    q, k, v = (torch.randn(*s, generator=g).to(dt) for s in ((H * group, D), (n, H, D), (n, H, D)))
    scale = float(np.float32(1.5 / np.sqrt(D)))
    out, _ = attend(ctx, kind, q, k, v, n, batch, scale)
    P = 1
    want, _, _ = ref.attention(ref.f64(q)[None], ref.f64(k)[:, None], ref.f64(v)[:, None],
                               np.arange(n, dtype=np.int32)[None], [n], P, scale)
    once = ref.f64(torch.from_numpy(want).to(dt)) - want
    assert np.linalg.norm(out - want, axis=(1, 2)).max() <= 1.02 * np.linalg.norm(once)
