"""GPU parity of sbt_pages_slots and sbt_tree_plan with plain loops, integer for integer."""
import numpy as np
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt
import step_ref as ref

pytestmark = pytest.mark.gpu
GAP = 0x5A5A5A5A


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32).copy()).cuda()


def guarded(n):
    return torch.full((n + 8,), GAP, dtype=torch.int32, device="cuda")


def run_slots(ctx, n_new, capacity, table, lens, page_size, n_pages, seqs=None, start=None, ld_pad=3,
              outs=("cu", "seq", "positions", "slots", "last")):
    S, max_pages = table.shape
    t = np.full((S, max_pages + ld_pad), GAP, np.int32)
    t[:, :max_pages] = table
    td, ld, keep = i32(t), None if lens is None else i32(lens), [i32(n_new), None if seqs is None else i32(seqs),
                                                              None if start is None else i32(start)]
    m = sbt.page_map(td, max_pages + ld_pad, S, max_pages, ld, n_pages, page_size)
    B = len(n_new)
    size = dict(cu=B + 1, seq=capacity, positions=capacity, slots=capacity, last=B)
    out = {k: guarded(size[k]) for k in outs}
    sbt.pages_slots(ctx, m, keep[0], B, capacity, seqs=keep[1], start=keep[2], **out)
    torch.cuda.synchronize()
    want = dict(zip(("cu", "seq", "positions", "slots", "last"),
                    ref.pages_slots(n_new, seqs, start, lens, table, page_size, n_pages, capacity)))
    for k in outs:
        got = out[k].cpu().numpy()
        assert (got[size[k]:] == GAP).all(), k
        assert np.array_equal(got[:size[k]], np.asarray(want[k], np.int64)), k
    return want


def a_table(rng, S, max_pages, n_pages):
    return rng.integers(-2, n_pages + 2, (S, max_pages)).astype(np.int32)


@pytest.mark.parametrize("P", [1, 7, 16, 64])
@pytest.mark.parametrize("B,most", [(1, 1), (1, 3000), (3, 0), (5, 40), (64, 1), (256, 3), (1000, 4), (1024, 1), (1025, 2),
                                    (3000, 1), (40, 300), (5000, 2)])
def test_slots(ctx, B, most, P):
    rng = np.random.default_rng(B * 7 + most)
    S, max_pages, n_pages = B + 2, 30, 500
    n_new = rng.integers(0, most + 1, B)
    lens = rng.integers(0, max_pages * P + 40, S)
    seqs = rng.permutation(S)[:B]
    total = int(n_new.sum())
    for capacity in {total, total + 1, total + 1500, total // 2, 0}:
        run_slots(ctx, n_new, capacity, a_table(rng, S, max_pages, n_pages), lens, P, n_pages, seqs=seqs)


def test_counts_below_zero_sequences_out_of_range_and_short_lengths(ctx):
    rng = np.random.default_rng(0)
    table = a_table(rng, 4, 3, 20)
    run_slots(ctx, [3, -5, 2, 0, 4, 100, 1], 130, table, [5, -3, 2**31 - 1, 40], 16, 20, seqs=[0, 1, -1, 2, 4, 3, 1])


def test_given_starts(ctx):
    rng = np.random.default_rng(1)
    table = a_table(rng, 6, 5, 30)
    run_slots(ctx, [4, 3, 5, 9, 2, 3], 30, table, None, 8, 30, start=[0, -2, 38, 1000, 2**31 - 2, -2**31])


@pytest.mark.parametrize("outs", [("cu",), ("last",), ("seq",), ("positions", "last"), ("slots",), ()])
def test_outputs_left_out(ctx, outs):
    rng = np.random.default_rng(2)
    run_slots(ctx, [3, 0, 5], 12, a_table(rng, 3, 4, 9), [20, 4, 9], 8, 9, outs=outs)


def test_empty_batch_pads(ctx):
    rng = np.random.default_rng(3)
    run_slots(ctx, [], 700, a_table(rng, 2, 2, 9), [3, 4], 8, 9)


def test_sums_past_32_bits_and_slots_at_the_end_of_the_range(ctx):
    table = np.array([[2**27 - 1, 0]] * 3, np.int32)
    run_slots(ctx, [2, 2**31 - 1, 2**31 - 1], 40, table, [16, 5, 6], 16, 2**27)
    run_slots(ctx, [2**31 - 1] * 5, 64, table, None, 16, 2**27, seqs=[0, 1, 2, 0, 1], start=[3, 0, 0, 0, 0])


@pytest.mark.parametrize("words", [1, 2, 5])
@pytest.mark.parametrize("sizes", [[1], [5], [32], [33, 1, 64], [0, 7, 0, 40, 3], [100, 300], [1] * 700])
def test_tree_plan(ctx, sizes, words):
    rng = np.random.default_rng(len(sizes) + words)
    cu = np.concatenate([[0], np.cumsum(sizes)])
    rows = int(cu[-1]) + 5
    parents = np.full(rows, 77, np.int64)
    for b, n in enumerate(sizes):
        for i in range(n):
            # mostly earlier tokens; also the sequence itself, the token itself and later ones
            parents[cu[b] + i] = rng.integers(-2, i) if rng.random() < 0.9 else rng.integers(i, i + 5)
    positions = rng.integers(-1, 1000, rows)
    mask, turned = guarded(rows * (words + 1)).view(-1), guarded(rows)
    for with_mask, with_turned in ((1, 1), (1, 0), (0, 1)):
        mask.fill_(GAP), turned.fill_(GAP)
        sbt.tree_plan(ctx, i32(parents), i32(cu), len(sizes), rows, mask=mask if with_mask else None, ld_mask=words,
                      positions=i32(positions) if with_turned else None, turned=turned if with_turned else None)
        torch.cuda.synchronize()
        m, t = ref.tree_plan(parents, cu, rows, words, positions)
        if with_mask:
            got = mask.cpu().numpy()
            assert np.array_equal(got[:rows * words].view(np.uint32).reshape(rows, words), m)
            assert (got[rows * words:] == GAP).all()
        if with_turned:
            assert np.array_equal(turned.cpu().numpy()[:rows], t) and (turned.cpu().numpy()[rows:] == GAP).all()


def test_tree_plan_of_a_deep_chain(ctx):
    n = 3000
    cu, parents = [0, n], np.arange(n) - 1
    mask, turned = guarded(n * 94), guarded(n)
    sbt.tree_plan(ctx, i32(parents), i32(cu), 1, n, mask=mask, ld_mask=94, positions=i32(np.arange(n) + 9), turned=turned)
    m, t = ref.tree_plan(parents, cu, n, 94, np.arange(n) + 9)
    assert np.array_equal(mask.cpu().numpy()[:n * 94].view(np.uint32).reshape(n, 94), m)
    assert np.array_equal(turned.cpu().numpy()[:n], t)
