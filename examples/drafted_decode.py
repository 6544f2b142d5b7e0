"""One attention layer with 4-bit weights that verifies trees of drafted tokens, every step through the library.

    python examples/drafted_decode.py

Prompts are read in one step: slot maps from the requests' lengths, the residual norm to 8-bit codes, the block-scaled
GEMM over 4-bit weights, norm and rotation of queries and keys, append to the pages, attention of all new tokens.  Then
each step appends a small tree of drafted tokens per sequence (the norm's 16-bit output and matrix-vector products over
the same weights), attends with the trees' masks, keeps one path of each tree and gives the other tokens' places back.
The output projection reads the attention's 16-bit numbers, of which no call makes codes, so it is a matrix-vector
product in both kinds of step (for a prompt it passes over the weights once per 16 tokens).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scatter_boundary_tile_gb300 as sbt  # noqa: E402

BLOCK = 32  # columns per scale of the codes, and weights per scale


class DraftedLayer:
    """Weights, cache and page state of one layer; `n_seq` sequences of up to `max_len` tokens, up to `most` new ones a step."""

    def __init__(self, ctx, d_model=256, q_heads=8, kv_heads=2, dim=64, page_size=16, n_seq=3, max_len=256, n_pages=60,
                 most=200, seed=0):
        self.ctx, self.d_model, self.hq, self.hk, self.d = ctx, d_model, q_heads, kv_heads, dim
        self.P, self.n_seq, self.n_pages, self.most = page_size, n_seq, n_pages, most
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.width = (q_heads + 2 * kv_heads) * dim
        bytes_of = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device="cuda")
        scales = lambda k, n: torch.randint(119, 122, (k // BLOCK, n), generator=g, dtype=torch.uint8, device="cuda")
        self.w_in, self.s_in = bytes_of(d_model, self.width // 2), scales(d_model, self.width)
        self.w_out, self.s_out = bytes_of(q_heads * dim, d_model // 2), scales(q_heads * dim, d_model)
        rnd = lambda n: (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)
        self.weight, self.q_weight, self.k_weight = rnd(d_model), rnd(dim), rnd(dim)
        self.table = torch.empty((max_len, dim // 2, 2), device="cuda")
        sbt.rope_table(ctx, self.table, max_len, dim)
        self.rope = sbt.rope(self.table, max_len, dim)
        self.k, self.v = (torch.zeros((n_pages, page_size, kv_heads, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.max_pages = -(-max_len // page_size)
        self.pages = torch.full((n_seq, self.max_pages), -1, **i32)
        self.lens, self.refs = torch.zeros(n_seq, **i32), torch.zeros(n_pages, **i32)
        self.map = sbt.page_map(self.pages, self.max_pages, n_seq, self.max_pages, self.lens, n_pages, page_size,
                                refs=self.refs)
        self.cache = sbt.kv_cache(self.k, self.v, kv_heads, dim, page_size * kv_heads * dim, kv_heads * dim, dim)
        size = page_size * kv_heads * dim * 2
        self.pools = sbt.page_pools([(x, 1, n_pages * size, size, size) for x in (self.k, self.v)])
        u8 = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        self.page_ws = u8(sbt.pages_workspace_size(ctx, n_seq, n_pages))
        self.attn_ws = u8(sbt.paged_tree_attention_workspace_size(ctx, most, q_heads, kv_heads, dim))
        self.gemm_ws = u8(max(sbt.gemm_block_scaled_workspace_size(ctx, most * n_seq, n, k)
                              for k, n in ((d_model, self.width), (q_heads * dim, d_model))))

    def empty(self, *shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def grow(self, n_new):
        """Pages for n_new more tokens of each sequence (int32 [n_seq])."""
        sbt.pages_reserve(self.ctx, self.map, self.pools, self.lens + n_new, self.page_ws, self.page_ws.numel())

    def slots(self, n_new, capacity):
        """What the step's calls read about its tokens; places past the last token hold -1."""
        i32 = lambda n: self.empty(n, dtype=torch.int32)
        m = dict(cu=i32(self.n_seq + 1), seq=i32(capacity), positions=i32(capacity), slots=i32(capacity),
                 last=i32(self.n_seq))
        sbt.pages_slots(self.ctx, self.map, n_new, self.n_seq, capacity, **m)
        return m

    def project(self, x, w, s, codes=None):
        """x (or its codes and scales) times the 4-bit weights."""
        rows, k, n = x.shape[0], w.shape[0], 2 * w.shape[1]
        if codes is None:
            y = self.empty(rows, n)
            sbt.matvec_e2m1(self.ctx, x, k, rows, w, n, s, n, k // BLOCK, y, n, n, k)
            return y
        y = self.empty(rows, n, dtype=torch.float32)
        sbt.gemm_block_scaled(self.ctx, codes[0], k, w, n, codes[1], k // BLOCK, s, n, k // BLOCK, y, n, rows, n, k,
                              workspace=self.gemm_ws, workspace_bytes=self.gemm_ws.numel(), a_fmt="e4m3", b_fmt="e2m1")
        return y.to(torch.bfloat16)

    def norm(self, x, r, coded):
        """The residual stream x + r and its norm, as codes for the GEMM or as numbers for the matrix-vector product."""
        rows, c = x.shape
        h, ld = torch.empty_like(x), dict(ld_r=c, ld_h=c)
        if coded:
            codes = self.empty(rows, c, dtype=torch.uint8), self.empty(rows, c // BLOCK, dtype=torch.uint8)
            sbt.add_rms_norm(self.ctx, x, c, rows, c, weight=self.weight, r=r, h_out=h, **ld,
                             codes=sbt.code_rows(codes[0], c, codes[1], c // BLOCK, block=BLOCK))
            return h, x, codes
        y = torch.empty_like(x)
        sbt.add_rms_norm(self.ctx, x, c, rows, c, weight=self.weight, r=r, h_out=h, **ld, y=y, ld_y=c)
        return h, y, None

    def step(self, x, r, m, parents=None, coded=False, most=None):
        """New tokens of all sequences, in the order of their slots: rows x of the layer's input, r of the residual stream.

        `most`: no sequence has more new tokens (the layer's own limit where it is not given); the attention shares its
        blocks out by it, and the masks are as wide."""
        most = most or self.most
        rows, hq, hk, d = x.shape[0], self.hq, self.hk, self.d
        h, y, codes = self.norm(x, r, coded)
        qkv = self.project(y, self.w_in, self.s_in, codes)
        turned, mask, words = m["positions"], None, 0
        if parents is not None:  # a token's place in its tree turns it, its place in the cache is its own
            turned, words = self.empty(rows, dtype=torch.int32), -(-most // 32)
            mask = self.empty(rows, words, dtype=torch.int32)
            sbt.tree_plan(self.ctx, parents, m["cu"], self.n_seq, rows, mask=mask, ld_mask=words,
                          positions=m["positions"], turned=turned)
        at = lambda head: qkv.data_ptr() + head * d * 2
        q, k, ld = self.empty(rows, hq, d), self.empty(rows, hk, d), self.width
        sbt.qk_norm_rope(self.ctx, at(0), ld, d, at(hq), ld, d, rows, hq, hk, d, turned, self.rope, q, hq * d, d, k_out=k,
                         ld_ko=hk * d, ld_koh=d, q_weight=self.q_weight, k_weight=self.k_weight, dtype="bf16")
        sbt.qk_norm_rope(self.ctx, None, 0, 0, k, hk * d, d, rows, 0, hk, d, m["positions"], None, None, 0, 0,
                         v=at(hq + hk), ld_v=ld, ld_vh=d, cache=self.cache, map=self.map, seq=m["seq"], dtype="bf16")
        heads = torch.zeros_like(q)
        sbt.paged_tree_attention(self.ctx, q, hq * d, d, rows, m["cu"], self.n_seq, most, hq, self.cache, self.map,
                                 d**-0.5, heads, hq * d, d, mask=mask, ld_mask=words, workspace=self.attn_ws,
                                 workspace_bytes=self.attn_ws.numel())
        out = self.project(heads.view(rows, -1), self.w_out, self.s_out)
        return out, h, dict(q=q, k=k, qkv=qkv, heads=heads, mask=mask, turned=turned, out=out, h=h)

    def record(self, saw, m, x, r, parents=None):
        """What a step read and computed, and the cache as it was then."""
        held = dict(lens=self.lens, pages=self.pages, pool_k=self.k, pool_v=self.v)
        return dict(saw, m=m, x=x, r=r, parents=parents, **{k: v.clone() for k, v in held.items()})

    def accept(self, m, rows, to, keep):
        """Keys and values of the tokens `rows` move to the slots of the tokens `to`; sequences are cut to `keep`."""
        n, width = rows.numel(), self.hk * self.d
        total = self.n_pages * self.P
        src, dst = m["slots"][rows], m["slots"][to]
        for pool in (self.k, self.v):
            held = self.empty(n, width)
            sbt.gather_rows(self.ctx, pool, total, width, width, src, n, held, width, width)
            sbt.scatter_rows_masked(self.ctx, pool, total, width, width, dst, n, held, width, width)
        sbt.pages_free(self.ctx, self.map, torch.arange(self.n_seq, dtype=torch.int32, device="cuda"), self.n_seq, keep=keep)


TREE = [-1, 0, 0, 1, 2, 2, 5]           # parents of a drafted tree's tokens
PATH = [0, 2, 5]                        # the path that is kept


def run(ctx, steps=4, seed=1, log=None):
    """Prompts, then drafted trees; returns the layer and what the steps computed."""
    layer = DraftedLayer(ctx)
    g = torch.Generator(device="cuda").manual_seed(seed)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rnd = lambda rows: torch.randn((rows, layer.d_model), generator=g, device="cuda").to(torch.bfloat16)
    prompt = [37, 5, 90]
    n_new = i32(prompt)
    layer.grow(n_new)
    m = layer.slots(n_new, sum(prompt))
    x, r = rnd(sum(prompt)), rnd(sum(prompt))
    _, _, saw = layer.step(x, r, m, coded=True, most=max(prompt))
    records = [layer.record(saw, m, x, r)]
    n, b = len(TREE), layer.n_seq
    n_new, parents = i32([n] * b), i32(TREE * b)
    for step in range(steps):
        base = layer.lens.clone()
        layer.grow(n_new)
        m = layer.slots(n_new, n * b)
        x, r = rnd(n * b), rnd(n * b)
        _, _, saw = layer.step(x, r, m, parents=parents, most=n)
        records.append(layer.record(saw, m, x, r, parents))
        rows = torch.tensor([n * i + j for i in range(b) for j in PATH], device="cuda")
        to = torch.tensor([n * i + j for i in range(b) for j in range(len(PATH))], device="cuda")
        layer.accept(m, rows, to, base + len(PATH))
        if log:
            log(f"step {step}: lengths {layer.lens.tolist()}, pages held {int((layer.refs > 0).sum())}")
    return layer, records


if __name__ == "__main__":
    context = sbt.Context(0)
    run(context, log=print)
    context.check_status()
