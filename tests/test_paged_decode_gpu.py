"""The decoding example end to end: what the cache holds and what the last step returned, against 64 bits.

Keys in the pages are the norm and rotation of the projections the tokens had (one bf16 rounding and
D + 16 fp32 roundings), values the projections' own bits, whatever was forked, dropped and packed on the
way; the attention of the last step is compared on the cache's own contents.
"""
import os
import sys

import numpy as np
import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_decode_example(ctx):
    import paged_decode

    layer, tokens, last = paged_decode.run(ctx)
    torch.cuda.synchronize()
    d, hq, hk, P = layer.d, layer.hq, layer.hk, layer.P
    table, lens, refs = layer.pages.cpu().numpy(), layer.lens.cpu().numpy(), layer.refs.cpu().numpy()
    assert [int(n) for n in lens] == [len(tokens[s]) for s in range(layer.n_seq)]
    held = np.zeros(layer.n_pages, np.int64)
    k, v = ref.f64(layer.k), layer.v.cpu()
    rot_table = ref.f64(layer.table)
    for s in range(layer.n_seq):
        n = len(tokens[s])
        pages = table[s, :-(-n // P)]
        np.add.at(held, pages, 1)
        if n == 0:
            continue
        qkv = torch.stack(tokens[s]).cpu().view(n, hq + 2 * hk, d)
        t = np.arange(n)
        y, mag = ref.norm_rope(ref.f64(qkv[:, hq:hq + hk]), ref.f64(layer.k_weight), 1e-6, rot_table, t, d, "half",
                               layer.max_len)
        bound = ref.HALF_ULP["bf16"] * np.abs(y) * 1.01 + ref.TINY["bf16"] + (d + 16) * 2.0**-23 * mag
        assert np.all(np.abs(k[pages[t // P], t % P] - y) <= bound)
        got = v[torch.from_numpy(pages[t // P]).long(), torch.from_numpy(t % P)]
        assert torch.equal(got.view(torch.int16), qkv[:, hq + hk:].contiguous().view(torch.int16))
    assert np.array_equal(held, refs)
    want = ref.attention(ref.f64(last["q"]), k, ref.f64(layer.v), table, lens, P, d**-0.5, seq=last["seqs"])
    assert np.all(np.abs(ref.f64(last["heads"]) - want[0]) <= ref.attention_bounds(want, "bf16", d)[0])
    assert bool(torch.isfinite(last["y"].float()).all())
    ctx.check_status()


def test_a_step_in_a_graph(ctx):
    """Grow, append and attend captured once and replayed: the same bits as the calls made directly."""
    import scatter_boundary_tile_gb300 as sbt
    from paged_decode import PagedLayer

    def state():
        layer = PagedLayer(ctx)
        g = torch.Generator(device="cuda").manual_seed(3)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        layer.grow(i32([20, 33] + [0] * 6))
        seq = i32([0] * 20 + [1] * 33)
        pos = i32(list(range(20)) + list(range(33)))
        layer.append(torch.randn((53, layer.d_model), generator=g, device="cuda").to(torch.bfloat16), seq, pos)
        x = torch.randn((2, layer.d_model), generator=g, device="cuda").to(torch.bfloat16)
        return layer, x, i32([0, 1]), i32([20, 33]), i32([21, 34] + [0] * 6)

    layer, x, seq, pos, target = state()
    layer.grow(target)
    want, _, _, heads = layer.step(x, seq, pos)
    torch.cuda.synchronize()

    layer, x, seq, pos, target = state()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.grow(target)
        out, _, _, h = layer.step(x, seq, pos)
    assert int(layer.lens[0]) == 20  # nothing has run yet
    for _ in range(3):               # the second and third replay find the sequences grown already
        graph.replay()
    torch.cuda.synchronize()
    assert [int(n) for n in layer.lens[:2]] == [21, 34]
    assert torch.equal(h.view(torch.int16), heads.view(torch.int16))
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    ctx.check_status()
