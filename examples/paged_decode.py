"""One attention layer decoding with a paged key-value cache, every step through the library.

    python examples/paged_decode.py

A layer of random weights reads its prompts (projection, norm and rotation of queries and
keys, append to the pages), then decodes: each step grows the sequences, appends one token
of each and attends over the cache.  Half way every sequence is forked into a second
continuation; near the end some are dropped and the pool is packed.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scatter_boundary_tile_gb300 as sbt  # noqa: E402


class PagedLayer:
    """Weights, cache and page state of one layer; `n_seq` sequence slots of up to `max_len` tokens."""

    def __init__(self, ctx, d_model=512, q_heads=8, kv_heads=2, dim=64, page_size=16, n_seq=8, max_len=512,
                 n_pages=200, seed=0):
        self.ctx, self.d_model, self.hq, self.hk, self.d = ctx, d_model, q_heads, kv_heads, dim
        self.P, self.n_seq, self.max_len, self.n_pages = page_size, n_seq, max_len, n_pages
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        rnd = lambda *s, scale=1.0: (torch.randn(s, generator=g, device="cuda") * scale).to(torch.bfloat16)
        self.width = (q_heads + 2 * kv_heads) * dim
        self.w_in = rnd(d_model, self.width, scale=d_model**-0.5)
        self.w_out = rnd(q_heads * dim, d_model, scale=(q_heads * dim)**-0.5)
        self.q_weight, self.k_weight = 1 + rnd(dim, scale=0.1), 1 + rnd(dim, scale=0.1)
        # rotations for contexts four times as long as the 128 tokens the layer pretends to be trained on
        self.table = torch.empty((max_len, dim // 2, 2), device="cuda")
        sbt.rope_table(ctx, self.table, max_len, dim, scaling="by_parts", factor=4.0, orig_len=128)
        self.rope = sbt.rope(self.table, max_len, dim, "half")
        # cache and page state
        self.k, self.v = (torch.zeros((n_pages, page_size, kv_heads, dim), **bf) for _ in "kv")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.max_pages = -(-max_len // page_size)
        self.pages = torch.full((n_seq, self.max_pages), -1, **i32)
        self.lens, self.refs = torch.zeros(n_seq, **i32), torch.zeros(n_pages, **i32)
        self.page_to, self.n_live = torch.empty(n_pages, **i32), torch.empty(1, **i32)
        self.map = sbt.page_map(self.pages, self.max_pages, n_seq, self.max_pages, self.lens, n_pages, page_size,
                                refs=self.refs)
        self.cache = sbt.kv_cache(self.k, self.v, kv_heads, dim, page_size * kv_heads * dim, kv_heads * dim, dim)
        size = page_size * kv_heads * dim * 2
        self.pools = sbt.page_pools([(x, 1, n_pages * size, size, size) for x in (self.k, self.v)])
        self.page_ws = torch.empty(sbt.pages_workspace_size(ctx, n_seq, n_pages), dtype=torch.uint8, device="cuda")
        n = sbt.paged_attention_workspace_size(ctx, q_heads, kv_heads, dim)
        self.attn_ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def matmul(self, x, w):
        out = torch.empty((x.shape[0], w.shape[1]), dtype=torch.bfloat16, device="cuda")
        (m, k), n = x.shape, w.shape[1]
        need = sbt.gemm_bounded_workspace_size(self.ctx, m, n, k, k, n)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        sbt.gemm_bounded(self.ctx, x, k, w, n, out, n, m, n, k, ws, need)
        return out

    def grow(self, target):
        """Pages for the tokens to come; target: int32 [n_seq] lengths."""
        sbt.pages_reserve(self.ctx, self.map, self.pools, target, self.page_ws, self.page_ws.numel())

    def append(self, x, seq, pos):
        """Project tokens x, norm and rotate their queries and keys, write keys and values to their pages."""
        qkv, d, t = self.matmul(x, self.w_in), self.d, x.shape[0]
        q = torch.empty((t, self.hq, d), dtype=torch.bfloat16, device="cuda")
        at = lambda head: qkv.data_ptr() + head * d * 2
        sbt.qk_norm_rope(self.ctx, at(0), self.width, d, at(self.hq), self.width, d, t, self.hq, self.hk, d, pos,
                         self.rope, q, self.hq * d, d, q_weight=self.q_weight, k_weight=self.k_weight,
                         v=at(self.hq + self.hk), ld_v=self.width, ld_vh=d, cache=self.cache, map=self.map, seq=seq,
                         dtype="bf16")
        return q, qkv

    def attend(self, q, seq):
        """One new token of each sequence in `seq` over its cache."""
        out = torch.empty_like(q)
        ld = self.hq * self.d
        sbt.paged_attention(self.ctx, q, ld, self.d, q.shape[0], self.hq, self.cache, self.map, self.d**-0.5, out, ld,
                            self.d, seq=seq, workspace=self.attn_ws, workspace_bytes=self.attn_ws.numel())
        return out

    def step(self, x, seq, pos):
        q, qkv = self.append(x, seq, pos)
        heads = self.attend(q, seq)
        return self.matmul(heads.view(x.shape[0], -1), self.w_out), q, qkv, heads

    def fork(self, parents, children):
        sbt.pages_fork(self.ctx, self.map, self.pools, parents, children, parents.numel(), self.page_ws,
                       self.page_ws.numel())

    def drop(self, seqs):
        sbt.pages_free(self.ctx, self.map, seqs, seqs.numel())

    def pack(self):
        sbt.pages_compact(self.ctx, self.map, self.pools, self.pages, self.max_pages, self.refs, self.page_to,
                          self.n_live, self.page_ws, self.page_ws.numel())


def run(ctx, steps=12, seed=1, log=None):
    """Prompts, decoding with a fork, a drop and a packing on the way; returns the layer and what happened.

    The record lists, per sequence slot, the packed projections of its tokens, and the last step's
    sequences, queries and attention outputs."""
    layer = PagedLayer(ctx)
    g = torch.Generator(device="cuda").manual_seed(seed)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tokens = {s: [] for s in range(layer.n_seq)}
    live = [0, 1, 2]
    prompt = [37, 5, 64]
    target = [0] * layer.n_seq
    for s, n in zip(live, prompt):
        target[s] = n
    layer.grow(i32(target))
    x = torch.randn((sum(prompt), layer.d_model), generator=g, device="cuda").to(torch.bfloat16)
    seq = [s for s, n in zip(live, prompt) for _ in range(n)]
    pos = [i for n in prompt for i in range(n)]
    _, qkv = layer.append(x, i32(seq), i32(pos))
    for i, s in enumerate(seq):
        tokens[s].append(qkv[i])
    last = None
    for step in range(steps):
        if step == steps // 2:  # a second continuation of each
            layer.fork(i32(live), i32([s + 3 for s in live]))
            for s in list(live):
                tokens[s + 3] = list(tokens[s])
            live += [s + 3 for s in live]
        if step == steps - 2:   # two of them end; what is left is packed to the front of the pool
            layer.drop(i32([1, 3]))
            tokens[1], tokens[3] = [], []
            live = [s for s in live if s not in (1, 3)]
            layer.pack()
        for s in range(layer.n_seq):
            target[s] = len(tokens[s]) + 1 if s in live else 0
        layer.grow(i32(target))
        x = torch.randn((len(live), layer.d_model), generator=g, device="cuda").to(torch.bfloat16)
        y, q, qkv, heads = layer.step(x, i32(live), i32([len(tokens[s]) for s in live]))
        for i, s in enumerate(live):
            tokens[s].append(qkv[i])
        last = dict(seqs=list(live), q=q, heads=heads, y=y)
        if log:
            log(f"step {step:2d}: sequences {live}, lengths {layer.lens.tolist()}, pages held {int((layer.refs > 0).sum())}")
    return layer, tokens, last


if __name__ == "__main__":
    context = sbt.Context(0)
    run(context, log=print)
    context.check_status()
