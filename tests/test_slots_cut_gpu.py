"""Entries that sbt_pages_slots cuts at its capacity, and sbt_paged_tree_attention."""
import numpy as np
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
import step_ref as ref
from test_tree_attention_gpu import FILL, Case, i32

pytestmark = pytest.mark.gpu


def test_an_entry_cut_at_the_capacity(ctx):
    """Slots for fewer tokens than the requests bring: the entry that is cut has no last token, and a sequence number
    that does not exist keeps it out of the attention; the others are as with all of them."""
    c = Case(31, "bf16", [(4, 100), (6, 37), (5, 64)], 2, 4, 64, 16, masked=False, extra=0)
    capacity, Hq = 12, 8
    table, lens, seqs = i32(c.table), i32(c.lens), i32(c.seq)
    m = sbt.page_map(table, c.max_pages, len(c.lens), c.max_pages, lens, c.n_pages, c.P)
    n_new, out = i32(c.n), {k: torch.full((s,), 7, dtype=torch.int32, device="cuda")
                            for k, s in dict(cu=4, positions=capacity, last=3).items()}
    sbt.pages_slots(ctx, m, n_new, 3, capacity, seqs=seqs, **out)
    cut = (out["last"] < 0) & (n_new > 0)
    assert cut.tolist() == [False, False, True] and out["cu"].tolist() == [0, 4, 10, 12]
    first = [int(c.lens[s]) - int(n) for s, n in zip(c.seq, c.n)]
    assert out["positions"].tolist() == [first[b] + j for b, n in ((0, 4), (1, 6), (2, 2)) for j in range(n)]
    attended = torch.where(cut, -1, seqs)
    q, o = c.q[:capacity].cuda(), torch.full((capacity, Hq, 64), FILL, dtype=c.dt, device="cuda")
    lse = torch.full((capacity, Hq), FILL, device="cuda")
    kd, vd = c.k.cuda(), c.v.cuda()
    n = sbt.paged_tree_attention_workspace_size(ctx, 6, Hq, 2, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    sbt.paged_tree_attention(ctx, q, Hq * 64, 64, capacity, out["cu"], 3, 6, Hq, sbt.kv_cache(kd, vd, 2, 64, *c.ld), m, c.scale,
                             o, Hq * 64, 64, lse=lse, seq=attended, workspace=ws, workspace_bytes=n)
    want = c.want()
    ob, sb = c.bounds(want)
    assert (np.abs(ref.f64(o)[:10] - want[0][:10]) <= ob[:10]).all() and (np.abs(ref.f64(lse)[:10] - want[1][:10]) <= sb[:10]).all()
    assert (o[10:] == 0).all() and torch.isneginf(lse[10:]).all()
