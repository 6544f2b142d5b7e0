"""The operators around the attention on streams of their own, in captured graphs that share a workspace, and side by side.

Every result is compared bit for bit with the same call alone: the order of their sums is fixed.
"""
import numpy as np
import pytest
import torch

import scatter_boundary_tile_gb300 as sbt

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Ops:
    """One call of each operator; `new` takes fresh workspaces."""

    def __init__(self, ctx, seed, rows=300, cols=1024, kind=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(kind)
        byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device="cuda")
        self.ctx, self.rows, self.cols = ctx, rows, cols
        self.x, self.r, self.w, self.gy = rnd(rows, cols), rnd(rows, cols), rnd(cols), rnd(rows, cols)
        self.packed, self.scales = byte(cols, 320), torch.randint(120, 130, (cols // 32, 640), generator=g,
                                                                  dtype=torch.uint8, device="cuda")
        self.wide, self.wide_scales = byte(64, 20000), torch.randint(120, 130, (2, 40000), generator=g, dtype=torch.uint8,
                                                                     device="cuda")
        # 3 sequences, pages of 16 in any order; 5, 0 and 9 new tokens
        self.hq, self.hk, self.d, self.P = 8, 2, 64, 16
        self.pages = torch.randperm(72, generator=g, device="cuda").int().view(3, 24)
        self.lens, self.n_new = i32([380, 200, 77]), i32([5, 0, 9])
        self.k, self.v = rnd(72, self.P, self.hk, self.d), rnd(72, self.P, self.hk, self.d)
        self.q, self.parents = rnd(16, self.hq, self.d), i32([-1, 0, 0, 1, 1] + [-1, 0, 1, 2, 0, 4, -1, 6, 7] + [-1, -1])
        self.map = sbt.page_map(self.pages, 24, 3, 24, self.lens, 72, self.P)
        self.cache = sbt.kv_cache(self.k, self.v, self.hk, self.d, self.P * self.hk * self.d, self.hk * self.d, self.d)
        u8 = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        self.norm_ws = u8(sbt.add_rms_norm_backward_workspace_size(ctx, rows, cols))
        self.tree_ws = u8(sbt.paged_tree_attention_workspace_size(ctx, 9, self.hq, self.hk, self.d))
        i = lambda n: torch.full((n,), 7, dtype=torch.int32, device="cuda")
        self.cu, self.seq, self.positions, self.turned, self.mask = i(4), i(16), i(16), i(16), i(16)
        e = lambda *s, t=kind: torch.zeros(s, dtype=t, device="cuda")
        self.h, self.y, self.dx, self.dw = e(rows, cols), e(rows, cols), e(rows, cols), e(cols, t=torch.float32)
        self.codes, self.code_scales = e(rows, cols, t=torch.uint8), e(rows, cols // 32, t=torch.uint8)
        self.few, self.many, self.out = e(4, 640), e(13, 40000), e(16, self.hq, self.d)
        self.lse = e(16, self.hq, t=torch.float32)

    def outputs(self):
        return [self.cu, self.seq, self.positions, self.turned, self.mask, self.h, self.y, self.dx, self.dw, self.codes,
                self.code_scales, self.few, self.many, self.out, self.lse]

    def run(self, stream=None):
        c, n, ctx, on = self.cols, self.rows, self.ctx, dict(stream=stream)
        sbt.pages_slots(ctx, self.map, self.n_new, 3, 16, cu=self.cu, seq=self.seq, positions=self.positions, **on)
        sbt.tree_plan(ctx, self.parents, self.cu, 3, 16, positions=self.positions, turned=self.turned, mask=self.mask,
                      ld_mask=1, **on)
        sbt.paged_tree_attention(ctx, self.q, self.hq * self.d, self.d, 16, self.cu, 3, 9, self.hq, self.cache, self.map, 0.125,
                                 self.out, self.hq * self.d, self.d, mask=self.mask, ld_mask=1, lse=self.lse,
                                 workspace=self.tree_ws, workspace_bytes=self.tree_ws.numel(), **on)
        sbt.add_rms_norm(ctx, self.x, c, n, c, weight=self.w, r=self.r, ld_r=c, h_out=self.h, ld_h=c, y=self.y, ld_y=c,
                         codes=sbt.code_rows(self.codes, c, self.code_scales, c // 32, block=32), **on)
        sbt.add_rms_norm_backward(ctx, self.gy, c, self.h, c, n, c, self.dx, c, weight=self.w, dweight=self.dw,
                                  workspace=self.norm_ws, workspace_bytes=self.norm_ws.numel(), **on)
        sbt.matvec_e2m1(ctx, self.y, c, 4, self.packed, 640, self.scales, 640, c // 32, self.few, 640, 640, c, **on)
        sbt.matvec_e2m1(ctx, self.y, c, 13, self.wide, 40000, self.wide_scales, 40000, 2, self.many, 40000, 40000, 64, **on)


@pytest.fixture(scope="module")
def alone(sbt_ctx):
    """Two sets of inputs and what each gives alone."""
    both = []
    for seed in (1, 2):
        ops = Ops(sbt_ctx, seed)
        ops.run()
        torch.cuda.synchronize()
        sbt_ctx.check_status()
        both.append((ops, [t.clone() for t in ops.outputs()]))
    return both


def same(ops, want):
    for i, (a, b) in enumerate(zip(ops.outputs(), want)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


def clear(ops):
    for t in ops.outputs():
        t.view(torch.uint8).fill_(0x55)


def test_rows_of_no_sequence_are_not_written(alone):
    ops, want = alone[0]
    assert want[0].tolist() == [0, 5, 5, 14] and want[1].tolist()[14:] == [-1, -1]
    clear(ops)
    ops.run()
    torch.cuda.synchronize()
    for t in (ops.out, ops.lse):
        assert (t[14:].reshape(-1).view(torch.uint8) == 0x55).all()
    ops.out[14:], ops.lse[14:], ops.turned[14:], ops.mask[14:] = want[13][14:], want[14][14:], want[3][14:], want[4][14:]
    same(ops, want)


def test_two_streams_at_once(alone, ctx):
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for stream, (ops, _) in zip(streams, alone):
            ops.run(stream=stream)
    torch.cuda.synchronize()
    ctx.check_status()
    for ops, want in alone:
        same(ops, want)


def test_two_graphs_that_share_their_workspaces(alone, ctx):
    (a, want_a), (b, want_b) = alone
    kept = b.tree_ws, b.norm_ws
    b.tree_ws, b.norm_ws = a.tree_ws, a.norm_ws
    try:
        graphs = []
        for ops in (a, b):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                ops.run()
        for order in ((0, 1), (1, 0), (0, 0, 1)):
            a.tree_ws.fill_(0xFF), a.norm_ws.fill_(0xFF)  # nothing is read from an earlier call
            for i in order:
                graphs[i].replay()
            torch.cuda.synchronize()
            ctx.check_status()
            same(a, want_a), same(b, want_b)
    finally:
        b.tree_ws, b.norm_ws = kept


def test_a_call_behind_one_that_writes_its_inputs(alone, ctx):
    """The kernels start before the one ahead has ended; what that one writes has to be seen."""
    ops, want = alone[0]
    inputs = [ops.x, ops.q, ops.k, ops.v, ops.gy, ops.packed, ops.wide_scales, ops.pages, ops.lens, ops.n_new, ops.parents]
    held = [t.clone() for t in inputs]
    for _ in range(5):
        for t in inputs:
            t.zero_()
        for t, was in zip(inputs, held):
            t.copy_(was)
        ops.run()
    torch.cuda.synchronize()
    same(ops, want)


def test_the_same_sequence_twice(ctx, alone):
    """Two entries on one sequence read the same cache; each gets its own rows."""
    ops, _ = alone[0]
    seqs, out = i32([2, 0, 2]), torch.zeros_like(ops.out)
    cu = i32([0, 4, 9, 13])
    q = ops.q.clone()
    q[9:13] = q[:4]
    sbt.paged_tree_attention(ctx, q, ops.hq * ops.d, ops.d, 16, cu, 3, 5, ops.hq, ops.cache, ops.map, 0.125, out,
                             ops.hq * ops.d, ops.d, seq=seqs, workspace=ops.tree_ws, workspace_bytes=ops.tree_ws.numel())
    torch.cuda.synchronize()
    close = (out[9:13].double() - out[:4].double()).abs().max()  # cut at different places: one rounding apart
    assert close <= 2.0**-7 * out[:4].double().abs().max() and out[:13].abs().sum(-1).min() > 0 and not out[13:].any()


def test_offsets_past_32_bits(ctx):
    """Rows of x, codes and weights whose strides put them past 2^32 elements."""
    rows, cols, ld = 3, 256, 2**31 + 64
    big = torch.zeros(ld * (rows - 1) + cols, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(rows, cols, device="cuda").to(torch.bfloat16)
    view = big.as_strided((rows, cols), (ld, 1))
    view.copy_(x)
    want, got = torch.empty_like(x), torch.empty_like(x)
    sbt.add_rms_norm(ctx, x, cols, rows, cols, y=want, ld_y=cols)
    sbt.add_rms_norm(ctx, big, ld, rows, cols, y=got, ld_y=cols)
    assert torch.equal(got, want)
    sbt.add_rms_norm(ctx, x, cols, rows, cols, y=big, ld_y=ld)
    assert torch.equal(view, want)
    dx, far = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(max(sbt.add_rms_norm_backward_workspace_size(ctx, rows, cols), 256), dtype=torch.uint8, device="cuda")
    sbt.add_rms_norm_backward(ctx, want, cols, x, cols, rows, cols, dx, cols, workspace=ws, workspace_bytes=ws.numel())
    view.copy_(x)
    sbt.add_rms_norm_backward(ctx, want, cols, big, ld, rows, cols, far, cols, workspace=ws, workspace_bytes=ws.numel())
    assert torch.equal(far, dx)
    # rows of 4-bit weights 2^27 bytes apart
    K, ldb = 64, 2**28
    raw = big.view(torch.uint8)
    packed = torch.randint(0, 256, (K, 64), dtype=torch.uint8, device="cuda")
    raw.as_strided((K, 64), (ldb // 2, 1)).copy_(packed)
    scales, y0, y1 = torch.full((2, 128), 127, dtype=torch.uint8, device="cuda"), *(torch.empty(3, 128, device="cuda") for _ in "ab")
    sbt.matvec_e2m1(ctx, x, cols, 3, packed, 128, scales, 128, 2, y0, 128, 128, K)
    sbt.matvec_e2m1(ctx, x, cols, 3, raw, ldb, scales, 128, 2, y1, 128, 128, K)
    assert torch.equal(y0, y1)
    del big, raw, view
    torch.cuda.empty_cache()
