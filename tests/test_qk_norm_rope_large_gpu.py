"""sbt_qk_norm_rope and its gradient at sizes that take several heads per group and several items per ring,
with head counts that those do not divide; and the gradient in place."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import scatter_boundary_tile_gb300 as sbt
from test_qk_norm_rope_gpu import EPS, Case, bound

pytestmark = pytest.mark.gpu
KINDS = ["f32", "bf16", "f16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout,rot", [("half", 128), ("interleaved", 64)])
@pytest.mark.parametrize("in_place", [False, True])
def test_forward_with_several_heads_per_group(ctx, kind, layout, rot, in_place):
    """13 + 3 heads of 3001 tokens: groups of four heads, the last with one, the keys' only one with three."""
    Case(41, kind, 3001, 13, 3, 128, rot, layout).check_forward(ctx, in_place=in_place)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout,rot", [("half", 64), ("interleaved", 128)])
def test_append_with_several_heads_per_group(ctx, kind, layout, rot):
    """The same with keys and values appended: 2999 tokens of one sequence, in shuffled order, pages of 16."""
    T, Hq, Hk, D, P = 2999, 13, 3, 128, 16
    c = Case(42, kind, T, Hq, Hk, D, rot, layout, n_pos=T)
    rng = np.random.default_rng(43)
    pos = rng.permutation(T).astype(np.int32)
    pos[7], pos[2000] = -1, T  # padding: past the table
    c.pos = torch.from_numpy(pos)
    pages = -(-T // P)
    table = rng.permutation(pages + 3)[:pages].astype(np.int32)
    b, es = c.buf.cuda(), c.buf.element_size()
    at = [b.data_ptr() + (c.offset + h * c.ldh) * es for h in (0, Hq, Hq + Hk)]
    dev = lambda x: torch.from_numpy(x).cuda()
    pos_d, table_d, seq = dev(pos), dev(table[None].copy()), torch.zeros(T, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((pages + 3, P, Hk, D), 9.0, dtype=c.dt, device="cuda") for _ in "kv")
    qo = torch.empty((T, Hq, D), dtype=c.dt, device="cuda")
    wq, wk = c.wq.cuda(), c.wk.cuda()
    sbt.qk_norm_rope(ctx, at[0], c.ld, c.ldh, at[1], c.ld, c.ldh, T, Hq, Hk, D, pos_d, c.turn(), qo, Hq * D, D,
                     q_weight=wq, k_weight=wk, eps=EPS, v=at[2], ld_v=c.ld, ld_vh=c.ldh,
                     cache=sbt.kv_cache(kc, vc, Hk, D, P * Hk * D, Hk * D, D),
                     map=sbt.page_map(table_d, pages, 1, pages, None, pages + 3, P), seq=seq, dtype=kind)
    torch.cuda.synchronize()
    y, mag = c.want(c.q, c.wq)
    assert np.all(np.abs(ref.f64(qo) - y) <= bound(y, mag, kind, D))
    y, mag = c.want(c.k, c.wk)
    real = (pos >= 0) & (pos < T)
    page, slot = table[pos[real] // P], pos[real] % P
    got_k, got_v = ref.f64(kc), ref.f64(vc)
    assert np.all(np.abs(got_k[page, slot] - y[real]) <= bound(y, mag, kind, D)[real])
    assert np.array_equal(got_v[page, slot], ref.f64(c.v)[real])
    left = np.ones(got_k.shape[:2], bool)
    left[page, slot] = False
    assert np.all(got_k[left] == 9) and np.all(got_v[left] == 9)


@pytest.mark.parametrize("kind,layout,rot", [("f32", "half", 64), ("bf16", "half", 128), ("f16", "interleaved", 64),
                                             ("bf16", "interleaved", 0)])
def test_gradient_with_several_items_per_group(ctx, kind, layout, rot):
    """13 + 3 heads of 6007 tokens, two heads an item: five items or more for every group of lanes."""
    Case(44, kind, 6007, 13, 3, 128, rot, layout).check_backward(ctx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("path", ["auto", "scalar"])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("tokens,D,rot,layout", [(6007, 128, 128, "half"), (6007, 64, 32, "interleaved"),
                                                 (41, 100, 50, "half"), (1, 128, 64, "half")])
def test_gradient_in_place(ctx, kind, path, weights, tokens, D, rot, layout):
    """dq over gq and dk over gk: the bits of the call with outputs of their own."""
    Hq, Hk = 5, 2
    c = Case(45, kind, tokens, Hq, Hk, D, rot, layout, weights=weights)
    apart = c.backward(ctx, path=path)
    b, es = c.buf.cuda(), c.buf.element_size()
    q, k = (b.data_ptr() + (c.offset + h * c.ldh) * es for h in (0, Hq))
    gq, gk, pos = c.gq.cuda().contiguous(), c.gk.cuda().contiguous(), c.pos.cuda()
    wq, wk = c.cuda(c.wq), c.cuda(c.wk)
    dw = [torch.empty(D, device="cuda") if weights else None for _ in "qk"]
    n = sbt.qk_norm_rope_backward_workspace_size(ctx, D)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    ctx.set_path(path)
    sbt.qk_norm_rope_backward(ctx, gq, Hq * D, D, gk, Hk * D, D, q, c.ld, c.ldh, k, c.ld, c.ldh, tokens, Hq, Hk, D, pos,
                              c.turn(), gq, Hq * D, D, gk, Hk * D, D, q_weight=wq, k_weight=wk, eps=EPS,
                              dq_weight=dw[0], dk_weight=dw[1], workspace=ws, workspace_bytes=n, dtype=kind)
    torch.cuda.synchronize()
    ctx.set_path("auto")
    word = torch.int16 if es == 2 else torch.int32
    for x, y in zip((gq, gk), apart):
        assert torch.equal(x.cpu().view(word), y.contiguous().view(word))
    if weights:
        for x, y in zip(dw, apart[2:]):
            assert np.array_equal(x.cpu().numpy().view(np.int32), y.view(np.int32))
