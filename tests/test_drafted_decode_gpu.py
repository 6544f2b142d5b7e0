"""The operators around the attention together, as a layer that verifies drafted trees uses them, and captured in a graph."""
import os
import sys

import numpy as np
import pytest
import torch

import step_ref as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def weights(packed, scales):
    """4-bit weights as numbers."""
    k, n = packed.shape[0], 2 * packed.shape[1]
    s = ref.code_values(scales.cpu().numpy(), "e8m0")
    return ref.E2M1[ref.unpack_e2m1(packed.cpu().numpy(), k, n, n)] * np.repeat(s, 32, 0)


def test_every_step_against_64_bits(ctx):
    import drafted_decode as dd

    layer, records = dd.run(ctx)
    ctx.check_status()
    w = weights(layer.w_in, layer.s_in)
    for i, rec in enumerate(records):
        cu, rows = rec["m"]["cu"].tolist(), rec["q"].shape[0]
        sizes = [37, 5, 90] if i == 0 else [len(dd.TREE)] * 3
        assert cu == np.cumsum([0] + sizes).tolist()
        assert rec["m"]["seq"].tolist() == [s for s in range(3) for _ in range(sizes[s])]
        lens = rec["lens"].tolist()
        assert rec["m"]["positions"].tolist() == [lens[s] - sizes[s] + j for s in range(3) for j in range(sizes[s])]
        # norm and projection: E4M3 codes are off by 2^-4 of a value, bf16 by 2^-8, and so are the sums of their products at most
        _, y = ref.add_rms_norm(ref.f64(rec["x"]), ref.f64(rec["r"]), ref.f64(layer.weight), 1e-6)
        mag = np.abs(y) @ np.abs(w)
        step = (2.0**-4 if i == 0 else 2.0**-8) + 2.0**-8
        top = np.abs(y).max(1, keepdims=True) * np.abs(w).sum(0) * 2.0**-17 if i == 0 else 0  # the codes' smallest step
        assert (np.abs(ref.f64(rec["qkv"]) - y @ w) <= step * mag + top + 2.0**-7 * np.abs(y @ w)).all()
        # attention over what the cache holds
        mask = None if rec["mask"] is None else rec["mask"].cpu().numpy()
        if mask is not None:
            want_mask, want_turned = ref.tree_plan(rec["parents"].cpu().numpy(), cu, rows, mask.shape[1],
                                                   rec["m"]["positions"].cpu().numpy())
            assert np.array_equal(mask.view(np.uint32), want_mask)
            assert np.array_equal(rec["turned"].cpu().numpy(), want_turned)
        want = ref.tree_attention(ref.f64(rec["q"]), ref.f64(rec["pool_k"]), ref.f64(rec["pool_v"]),
                                  rec["pages"].cpu().numpy(), lens, layer.P, layer.d**-0.5, cu, layer.most, mask)
        ob, _ = ref.tree_attention_bounds(want, "bf16", layer.d, 1)  # most * group > 128
        assert (np.abs(ref.f64(rec["heads"]) - want[0]) <= ob).all()
    # the kept paths stand where the next step's tokens continue them
    assert layer.lens.tolist() == [n + 3 * (len(records) - 1) for n in (37, 5, 90)]
    last = records[-1]
    k, pages = layer.k.cpu().float(), layer.pages.tolist()
    for s in range(3):
        base = last["lens"].tolist()[s] - len(dd.TREE)
        for j, token in enumerate(dd.PATH):
            pos = base + j
            assert torch.equal(k[pages[s][pos // layer.P], pos % layer.P],
                               last["k"][s * len(dd.TREE) + token].cpu().float())


def test_a_drafted_step_captured_in_a_graph(ctx):
    import drafted_decode as dd

    layer, records = dd.run(ctx, steps=1)
    n, b = len(dd.TREE), layer.n_seq
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    n_new, parents, capacity = i32([n, 0, n]), i32(dd.TREE * 3 + [-1] * 4), n * b + 4  # padded places and an idle sequence
    x, r = (torch.randn(capacity, layer.d_model, device="cuda").to(torch.bfloat16) for _ in "xr")
    layer.grow(n_new)
    state = [t.clone() for t in (layer.k, layer.v)]

    def step():
        m = layer.slots(n_new, capacity)
        out, h, saw = layer.step(x, r, m, parents=parents)
        return out, h, saw["heads"], m["cu"], m["seq"]

    want = [t.clone() for t in step()]
    assert want[3].tolist() == [0, n, n, 2 * n] and want[4].tolist()[2 * n:] == [-1] * (capacity - 2 * n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t, was in zip((layer.k, layer.v), state):
            t.copy_(was)
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        ctx.check_status()
        assert all(torch.equal(a, w) for a, w in zip(got, want))
