"""Cases of the paged-cache operators: what is timed, on which inputs, and what the answer is.

Three operators that a decoding step runs together:

  attention   one new token per sequence attends over its paged key-value cache
  norm_rope   per-head RMS norm of queries and keys with the position rotation in the same pass;
              forward with the keys and values appended to the cache's pages, or backward
  pages       copying pages, compacting the pool, and one step of a beam search
              (free, truncate, grow, fork)

`run` computes the plain form (elementary torch operations in 32 bits) where `own` is false, and
calls the library where it is true.  `exact` computes the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROPE_BASE = 10000.0
EPS = 1e-6


def cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one user's chat turn on a small model: latency of the smallest decode call
        dict(name="attention_one_sequence_f16", op="attention", dtype="f16", batch=1, max_len=777, equal=True,
             q_heads=16, kv_heads=4, dim=64, page_size=16, order="nhd", window=0),
        # a serving batch: 64 sequences of 64 to 4096 tokens, 8 key-value heads of depth 128
        dict(name="attention_ragged_batch_bf16", op="attention", dtype="bf16", batch=64, max_len=4096, equal=False,
             q_heads=32, kv_heads=8, dim=128, page_size=16, order="nhd", window=0),
        # two long documents: few rows, a long axis
        dict(name="attention_long_context_bf16", op="attention", dtype="bf16", batch=2, max_len=131071, equal=True,
             q_heads=64, kv_heads=8, dim=128, page_size=64, order="hnd", window=0),
        # a full server: the largest read of the cache, 16 queries on each key
        dict(name="attention_full_server_f16", op="attention", dtype="f16", batch=128, max_len=8192, equal=False,
             q_heads=128, kv_heads=8, dim=128, page_size=32, order="nhd", window=0),
        # 32-bit cache, head sizes and pages that are no power of two, a sliding window
        dict(name="attention_odd_sizes_f32", op="attention", dtype="f32", batch=17, max_len=1501, equal=False,
             q_heads=15, kv_heads=5, dim=80, page_size=24, order="nhd", window=1000),
        # one decoding step of a batch: 64 new tokens, one for each sequence
        dict(name="norm_rope_append_decode_bf16", op="norm_rope", dtype="bf16", tokens=64, sequences=64, start=900,
             q_heads=32, kv_heads=8, dim=128, rot=128, layout="half", page_size=16),
        # prefill of eleven prompts, rotation of half of the head, interleaved pairs
        dict(name="norm_rope_append_prefill_f16", op="norm_rope", dtype="f16", tokens=30011, sequences=11, start=0,
             q_heads=32, kv_heads=8, dim=128, rot=64, layout="interleaved", page_size=32),
        # training: gradients of 16384 tokens
        dict(name="norm_rope_backward_bf16", op="norm_rope_backward", dtype="bf16", tokens=16384, q_heads=32,
             kv_heads=8, dim=128, rot=128, layout="half"),
        # training in 32 bits with odd sizes
        dict(name="norm_rope_backward_odd_f32", op="norm_rope_backward", dtype="f32", tokens=1021, q_heads=15,
             kv_heads=5, dim=80, rot=40, layout="interleaved"),
        # one step of a beam search: drop the old beams, grow the parents, fork them again
        dict(name="pages_beam_step", op="pages_step", parents=16, beams=3, max_len=1000, grow=33, page_size=16,
             n_pages=2048, page_bytes=16 * 8 * 128 * 2, planes=2),
        # pages of all layers moved at once (a swapped or migrated set of sequences)
        dict(name="pages_copy_layers", op="pages_copy", n_pages=2200, pairs=1000, page_bytes=16 * 8 * 128 * 2,
             planes=8),
        # the pool packed to its front after many sequences ended
        dict(name="pages_compact_pool", op="pages_compact", n_pages=2047, live=1200, moved=500, sequences=40,
             page_size=16, page_bytes=16 * 8 * 128 * 2, planes=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "norm_rope", "norm_rope_backward", "pages_step", "pages_copy",
                     "pages_compact"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    es = 4 if dtype == "f32" else 2
    if op == "attention":
        dim = rng.choice([32, 64, 72, 80, 96, 100, 112, 128, 128, 160, 192, 256])
        kv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16, 32])
        batch = _log_int(rng, 1, 128)
        top = min(131072, int(2e9 / (batch * kv * dim * es * 2)))
        max_len = _log_int(rng, 1, top)
        window = rng.choice([0, 0, 0, rng.randint(1, max_len)])
        return dict(op=op, dtype=dtype, batch=batch, max_len=max_len, equal=rng.random() < 0.3, q_heads=kv * group,
                    kv_heads=kv, dim=dim, page_size=rng.choice([1, 8, 13, 16, 16, 24, 32, 64, 128]),
                    order=rng.choice(["nhd", "hnd"]), window=window)
    if op in ("norm_rope", "norm_rope_backward"):
        dim = rng.choice([32, 64, 72, 80, 96, 100, 128, 128, 192, 256])
        kv = rng.choice([1, 2, 4, 5, 8, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 8])
        top = min(32768, int(5e8 / ((heads + 2 * kv) * dim * es * 2)))
        rot = rng.choice([dim, dim, dim // 2 // 2 * 2, 16, 0])
        case = dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, top), q_heads=heads, kv_heads=kv, dim=dim, rot=rot,
                    layout=rng.choice(["half", "interleaved"]))
        if op == "norm_rope":
            case.update(sequences=rng.randint(1, min(64, case["tokens"])), start=rng.randint(0, 500),
                        page_size=rng.choice([1, 8, 13, 16, 32, 64]))
        return case
    page_bytes = rng.choice([16, 32, 64]) * rng.choice([1, 2, 4, 8]) * rng.choice([64, 80, 128]) * 2
    planes = rng.choice([1, 2, 3, 8])
    if op == "pages_copy":
        pairs = _log_int(rng, 1, min(1000, int(5e8 / (page_bytes * planes))))
        return dict(op=op, n_pages=2 * pairs + rng.randint(0, 200), pairs=pairs, page_bytes=page_bytes, planes=planes)
    if op == "pages_step":
        parents, beams = rng.randint(1, 32), rng.randint(1, 4)
        page_size = rng.choice([1, 8, 13, 16, 32])
        max_len, grow = _log_int(rng, 1, 1000), rng.randint(0, 100)
        need = parents * (cdiv(max_len + grow, page_size) + beams)
        page_bytes = min(page_bytes, int(1e9 / (need * planes)) // 16 * 16)
        return dict(op=op, parents=parents, beams=beams, max_len=max_len, grow=grow, page_size=page_size,
                    n_pages=need + rng.randint(0, 300), page_bytes=max(page_bytes, 16), planes=planes)
    n_pages = _log_int(rng, 16, min(2047, int(1e9 / (page_bytes * planes))))
    live = rng.randint(1, n_pages - 1)
    return dict(op=op, n_pages=n_pages, live=live, moved=rng.randint(0, min(live, n_pages - live, 500)),
                sequences=rng.randint(1, 50), page_size=rng.choice([1, 16, 24]), page_bytes=page_bytes, planes=planes)


# ----------------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, dtype, gen, scale=1.0):
    """N(0, scale^2) in slabs, so that the 32-bit draws of a large pool do not pile up."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device="cuda") * scale
    return out


def _lengths(batch, max_len, equal):
    """A fixed set of lengths (the seed only shuffles it): all equal, or evenly spread up to max_len."""
    if equal:
        return [max_len] * batch
    return [max(1, max_len * (i + 1) // batch) for i in range(batch)]


def _permutation(n, gen):
    return torch.randperm(n, generator=gen, device="cuda").to(torch.int32)


def _fill_table(lens, page_size, n_pages, max_pages, gen):
    """Each sequence's pages, drawn without repeats from the pool; -1 past its end."""
    need = (lens + page_size - 1) // page_size
    start = torch.cumsum(need, 0) - need
    j = torch.arange(max_pages, device="cuda")
    perm = _permutation(n_pages, gen)
    pick = (start[:, None] + j[None, :]).clamp(max=n_pages - 1)
    return torch.where(j[None, :] < need[:, None], perm[pick.long()], -1).to(torch.int32).contiguous()


def _rope_table(n_pos, rot):
    """cos and sin of every position and frequency, from 64-bit angles."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * ROPE_BASE ** (-2.0 * i / max(rot, 1))
    return torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()


def _attention_inputs(case, seed):
    gen, dt = _generator(seed), TYPES[case["dtype"]]
    b, p, h, d = case["batch"], case["page_size"], case["kv_heads"], case["dim"]
    lens = torch.tensor(_lengths(b, case["max_len"], case["equal"]), device="cuda")
    lens = lens[_permutation(b, gen).long()]
    max_pages = cdiv(case["max_len"], p)
    n_pages = sum(cdiv(n, p) for n in _lengths(b, case["max_len"], case["equal"])) + 3
    table = _fill_table(lens, p, n_pages, max_pages, gen)
    shape = (n_pages, p, h, d) if case["order"] == "nhd" else (n_pages, h, p, d)
    return dict(case=case, q=_normal((b, case["q_heads"], d), dt, gen, 1.5), k=_normal(shape, dt, gen),
                v=_normal(shape, dt, gen), lens=lens.to(torch.int32), table=table, n_pages=n_pages,
                max_pages=max_pages, scale=1.0 / math.sqrt(d))


def _norm_rope_inputs(case, seed):
    gen, dt = _generator(seed), TYPES[case["dtype"]]
    t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    qkv = _normal((t, (hq + 2 * hk) * d), dt, gen, 1.7)  # the packed projection a layer makes
    state = dict(case=case, qkv=qkv, q=qkv[:, :hq * d].view(t, hq, d),
                 k=qkv[:, hq * d:(hq + hk) * d].view(t, hk, d), v=qkv[:, (hq + hk) * d:].view(t, hk, d),
                 wq=(1 + _normal((d,), torch.float32, gen, 0.2)).to(dt),
                 wk=(1 + _normal((d,), torch.float32, gen, 0.2)).to(dt))
    if case["op"] == "norm_rope_backward":
        n_pos = 4096
        state["pos"] = (torch.arange(t, device="cuda") % n_pos).to(torch.int32)
        state["gq"], state["gk"] = _normal((t, hq, d), dt, gen), _normal((t, hk, d), dt, gen)
    else:
        # the tokens of sequence s continue it from position `start` (plus a few, differing by sequence)
        s, p = case["sequences"], case["page_size"]
        count = [t // s + (1 if i < t % s else 0) for i in range(s)]
        first = [case["start"] + 7 * i % 61 if case["start"] else 0 for i in range(s)]
        state["seq"] = torch.tensor([i for i in range(s) for _ in range(count[i])], device="cuda").to(torch.int32)
        state["pos"] = torch.tensor([first[i] + j for i in range(s) for j in range(count[i])],
                                    device="cuda").to(torch.int32)
        ends = [first[i] + count[i] for i in range(s)]
        n_pos, max_pages = max(ends), cdiv(max(ends), p)
        n_pages = sum(cdiv(e, p) for e in ends) + 3
        state["lens"] = torch.tensor(ends, device="cuda").to(torch.int32)
        state["table"] = _fill_table(state["lens"].long(), p, n_pages, max_pages, gen)
        state["k_cache"] = _normal((n_pages, p, hk, d), dt, gen)
        state["v_cache"] = _normal((n_pages, p, hk, d), dt, gen)
        state["n_pages"], state["max_pages"] = n_pages, max_pages
    state["rope"] = _rope_table(n_pos, case["rot"]) if case["rot"] else None
    state["n_pos"] = n_pos
    return state


def _pool(case, gen):
    """Pages of K and V (two allocations), `planes` layers each, as 16-bit words."""
    shape = (case["planes"], case["n_pages"], case["page_bytes"] // 2)
    words = lambda: torch.randint(-32768, 32767, shape, dtype=torch.int16, device="cuda", generator=gen)
    return [words(), words()]


def _pages_inputs(case, seed):
    gen = _generator(seed)
    state = dict(case=case, pools=_pool(case, gen))
    n = case["n_pages"]
    if case["op"] == "pages_copy":
        perm = _permutation(n, gen)
        state["src"], state["dst"] = perm[:case["pairs"]].clone(), perm[case["pairs"]:2 * case["pairs"]].clone()
    elif case["op"] == "pages_compact":
        live, moved, p, s = case["live"], case["moved"], case["page_size"], case["sequences"]
        refs = torch.zeros(n, dtype=torch.int32, device="cuda")
        pages = torch.cat([_permutation(live, gen)[:live - moved], live + _permutation(n - live, gen)[:moved]])
        pages = pages[_permutation(live, gen).long()]
        # the live pages dealt out to the sequences; the last page of each may be part full
        count = [live // s + (1 if i < live % s else 0) for i in range(s)]
        state["lens"] = torch.tensor([max(0, c * p - (i * 5) % p) for i, c in enumerate(count)],
                                     device="cuda").to(torch.int32)
        max_pages = max(count) + 2
        table = torch.full((s, max_pages), -1, dtype=torch.int32)
        host, at = pages.cpu(), 0
        for i, c in enumerate(count):
            table[i, :c] = host[at:at + c]
            at += c
        refs[pages.long()] = 1 + (pages % 3 == 0).to(torch.int32)  # some are held outside the tables too
        state.update(table=table.cuda(), refs=refs, max_pages=max_pages, table_out=torch.full_like(table, -1).cuda(),
                     refs_out=torch.zeros_like(refs), page_to=torch.zeros_like(refs),
                     n_live=torch.zeros(1, dtype=torch.int32, device="cuda"))
    else:
        # parents hold max_len (or less) tokens; each step grows them by `grow` and forks each `beams` times
        s, b, p = case["parents"], case["beams"], case["page_size"]
        base = [max(1, case["max_len"] - (i * 37) % max(1, case["max_len"] // 2)) for i in range(s)]
        max_pages = cdiv(case["max_len"] + case["grow"], p)
        lens = torch.zeros(s * (1 + b), dtype=torch.int64, device="cuda")
        lens[:s] = torch.tensor(base, device="cuda")
        table = _fill_table(lens, p, n, max_pages, gen)
        refs = torch.zeros(n, dtype=torch.int32, device="cuda")
        refs[table[table >= 0].long()] = 1
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        state.update(table=table, refs=refs, lens=lens.to(torch.int32), max_pages=max_pages,
                     parents=i32(list(range(s))), keep=i32(base),
                     target=i32([n + case["grow"] for n in base] + [0] * (s * b)),
                     fork_from=i32([i for i in range(s) for _ in range(b)]), fork_to=i32(list(range(s, s * (1 + b)))))
    return state


def _inputs(case, seed):
    make = {"attention": _attention_inputs, "norm_rope": _norm_rope_inputs, "norm_rope_backward": _norm_rope_inputs}
    return make.get(case["op"], _pages_inputs)(case, seed)


def prepare(case, seed):
    state = _inputs(case, seed)
    if case["op"] == "pages_step":
        _plain_pages_step(state)  # the state a running search is in: beams of the last step in place
    if own:
        _prepare_own(state)
    return state


# ------------------------------------------------------------------------------ plain forms

def _plain_attention(s):
    c = s["case"]
    b, p, h, d, hq = c["batch"], c["page_size"], c["kv_heads"], c["dim"], c["q_heads"]
    page = s["table"].clamp(min=0).long()

    def rows(pool):  # [batch][kv_heads][positions][dim]
        x = pool[page].float()
        x = x.permute(0, 3, 1, 2, 4) if c["order"] == "nhd" else x.permute(0, 2, 1, 3, 4)
        return x.reshape(b, h, s["max_pages"] * p, d)

    q = s["q"].float().view(b, h, hq // h, d)
    score = (q @ rows(s["k"]).transpose(2, 3)) * s["scale"]
    at = torch.arange(s["max_pages"] * p, device="cuda")
    n = s["lens"].long()[:, None]
    seen = (at < n) & ((at >= n - c["window"]) if c["window"] else (at >= 0))
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - top)
    total = weight.sum(-1, keepdim=True)
    out = (weight @ rows(s["v"])) / total
    return {"out": out.reshape(b, hq, d).to(s["q"].dtype), "lse": (top + total.log()).reshape(b, hq)}


def _turn(x, cos, sin, rot, layout, back=False):
    """The pairs of the first `rot` elements turned by their angles (back: by minus them)."""
    if rot == 0:
        return x
    sin = -sin if back else sin
    y, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _angles(s):
    if s["rope"] is None:
        return None, None
    row = s["rope"][s["pos"].long()][:, None]
    return row[..., 0], row[..., 1]


def _plain_norm_rope(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        return _turn(x, cos, sin, c["rot"], c["layout"]).to(s["qkv"].dtype)

    pos, p = s["pos"].long(), c["page_size"]
    page = s["table"][s["seq"].long(), pos // p].long()
    s["k_cache"][page, pos % p] = one(s["k"], s["wk"])
    s["v_cache"][page, pos % p] = s["v"]
    return {"q": one(s["q"], s["wq"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_norm_rope_backward(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(g, x, w):
        g, x, w = _turn(g.float(), cos, sin, c["rot"], c["layout"], back=True), x.float(), w.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        gw = g * w
        dx = r * (gw - x * (r * r) * (gw * x).mean(-1, keepdim=True))
        return dx.to(s["qkv"].dtype), (g * x * r).sum((0, 1))

    dq, dwq = one(s["gq"], s["q"], s["wq"])
    dk, dwk = one(s["gk"], s["k"], s["wk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _free_list(refs):
    """The free pages in ascending order, the others after them."""
    return torch.argsort((refs > 0).to(torch.int8), stable=True).to(torch.int32)


def _plain_free(s, rows, keep):
    p = s["case"]["page_size"]
    rows = rows.long()
    j = torch.arange(s["max_pages"], device="cuda")[None, :]
    table, n = s["table"][rows], s["lens"][rows]
    gone = (j >= cdiv_t(keep, p)[:, None]) & (j < cdiv_t(n, p)[:, None]) & (table >= 0)
    s["refs"].index_add_(0, table.clamp(min=0).flatten().long(), -gone.flatten().to(torch.int32))
    s["table"][rows] = torch.where(gone, -1, table).to(torch.int32)
    s["lens"][rows] = torch.minimum(n, keep)


def cdiv_t(x, p):
    return (x + (p - 1)) // p


def _plain_grow(s, target):
    p = s["case"]["page_size"]
    j = torch.arange(s["max_pages"], device="cuda")[None, :]
    have, want = cdiv_t(s["lens"], p), cdiv_t(torch.maximum(s["lens"], target), p)
    need = want - have
    start = torch.cumsum(need, 0) - need
    free = _free_list(s["refs"])
    new = (j >= have[:, None]) & (j < want[:, None])
    pick = free[(start[:, None] + j - have[:, None]).clamp(0, free.numel() - 1).long()]
    s["refs"].index_add_(0, torch.where(new, pick, 0).flatten().long(), new.flatten().to(torch.int32))
    s["table"].copy_(torch.where(new, pick, s["table"]))
    s["lens"].copy_(torch.maximum(s["lens"], target))


def _plain_fork(s):
    p = s["case"]["page_size"]
    a, b = s["fork_from"].long(), s["fork_to"].long()
    n = s["lens"][a]
    j = torch.arange(s["max_pages"], device="cuda")[None, :]
    part = (n % p != 0)
    free = _free_list(s["refs"])
    rank = torch.cumsum(part, 0) - part.long()
    old = s["table"][a]
    tail_at = (n // p).clamp(max=s["max_pages"] - 1).long()[:, None]
    tail_old = old.gather(1, tail_at)[:, 0]
    tail_new = torch.where(part, free[rank], tail_old)
    full = (j < (n // p)[:, None])
    row = torch.where(full, old, -1)
    row = torch.where((j == (n // p)[:, None]) & part[:, None], tail_new[:, None], row).to(torch.int32)
    s["refs"].index_add_(0, row.clamp(min=0).flatten().long(), (row >= 0).flatten().to(torch.int32))
    s["table"][b] = row
    s["lens"][b] = n
    src, dst = torch.where(part, tail_old, 0).long(), torch.where(part, tail_new, 0).long()
    for pool in s["pools"]:
        pool[:, dst] = pool[:, src]


def _plain_pages_step(s):
    _plain_free(s, s["fork_to"], torch.zeros_like(s["fork_to"]))
    _plain_free(s, s["parents"], s["keep"])
    _plain_grow(s, s["target"])
    _plain_fork(s)
    return {"table": s["table"], "refs": s["refs"], "lens": s["lens"], "pools": s["pools"]}


def _plain_pages_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for pool in s["pools"]:
        pool[:, dst] = pool[:, src]
    return s["pools"]


def _plain_pages_compact(s):
    c = s["case"]
    live = s["refs"] > 0
    n_live = live.sum()
    i = torch.arange(c["n_pages"], device="cuda")
    src = (live & (i >= n_live)).nonzero()[:, 0]        # live pages past the end, ascending
    dst = (~live & (i < n_live)).nonzero()[:, 0]        # as many holes before it
    s["page_to"].copy_(torch.where(live, i, -1))
    s["page_to"][src] = dst.to(torch.int32)
    s["refs_out"].copy_(torch.where(live & (i < n_live), s["refs"], 0))
    s["refs_out"][dst] = s["refs"][src]
    for pool in s["pools"]:
        pool[:, dst] = pool[:, src]
    j = torch.arange(s["max_pages"], device="cuda")[None, :]
    used = j < cdiv_t(s["lens"], c["page_size"])[:, None]
    s["table_out"].copy_(torch.where(used & (s["table"] >= 0), s["page_to"][s["table"].clamp(min=0).long()], -1))
    s["n_live"].copy_(n_live)
    return {"pools": s["pools"], "table": s["table_out"], "refs": s["refs_out"], "page_to": s["page_to"],
            "n_live": s["n_live"]}


# ---------------------------------------------------------------------- the library's calls

def _prepare_own(s):
    import scatter_boundary_tile_gb300 as sbt

    c = s["case"]
    s["sbt"], s["ctx"] = sbt, sbt.Context(0)
    workspace = 0
    if c["op"] in ("attention", "norm_rope"):
        p, h, d = c["page_size"], c["kv_heads"], c["dim"]
        s["map"] = sbt.page_map(s["table"], s["max_pages"], s["table"].shape[0], s["max_pages"], s["lens"],
                                s["n_pages"], p)
    if c["op"] == "attention":
        slot, head = (h * d, d) if c["order"] == "nhd" else (d, p * d)
        s["cache"] = sbt.kv_cache(s["k"], s["v"], h, d, p * h * d, slot, head)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        workspace = sbt.paged_attention_workspace_size(s["ctx"], c["q_heads"], h, d)
    elif c["op"].startswith("norm_rope"):
        s["turn"] = sbt.rope(s["rope"], s["n_pos"], c["rot"], c["layout"])
        if c["op"] == "norm_rope":
            s["cache"] = sbt.kv_cache(s["k_cache"], s["v_cache"], h, d, p * h * d, h * d, d)
            s["q_out"] = torch.empty(s["q"].shape, dtype=s["qkv"].dtype, device="cuda")
        else:
            s["dq"], s["dk"] = torch.empty_like(s["gq"]), torch.empty_like(s["gk"])
            s["dwq"], s["dwk"] = (torch.empty(c["dim"], dtype=torch.float32, device="cuda") for _ in "qk")
            workspace = sbt.qk_norm_rope_backward_workspace_size(s["ctx"], c["dim"])
    else:
        n, size = c["n_pages"], c["page_bytes"]
        s["handles"] = sbt.page_pools([(pool, c["planes"], n * size, size, size) for pool in s["pools"]])
        if c["op"] != "pages_copy":
            s["map"] = sbt.page_map(s["table"], s["max_pages"], s["table"].shape[0], s["max_pages"], s["lens"], n,
                                    c["page_size"], refs=s["refs"])
            workspace = sbt.pages_workspace_size(s["ctx"], s["table"].shape[0], n)
    s["workspace"] = torch.empty(max(workspace, 256), dtype=torch.uint8, device="cuda")
    s["workspace_bytes"] = workspace


def _own_attention(s):
    c, d = s["case"], s["case"]["dim"]
    s["sbt"].paged_attention(s["ctx"], s["q"], c["q_heads"] * d, d, c["batch"], c["q_heads"], s["cache"], s["map"],
                             s["scale"], s["out"], c["q_heads"] * d, d, lse=s["lse"], window=c["window"],
                             workspace=s["workspace"], workspace_bytes=s["workspace_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_norm_rope(s):
    c, d, ld = s["case"], s["case"]["dim"], s["qkv"].shape[1]
    s["sbt"].qk_norm_rope(s["ctx"], s["q"], ld, d, s["k"], ld, d, c["tokens"], c["q_heads"], c["kv_heads"], d,
                          s["pos"], s["turn"], s["q_out"], c["q_heads"] * d, d, q_weight=s["wq"], k_weight=s["wk"],
                          eps=EPS, v=s["v"], ld_v=ld, ld_vh=d, cache=s["cache"], map=s["map"], seq=s["seq"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_norm_rope_backward(s):
    c, d, ld = s["case"], s["case"]["dim"], s["qkv"].shape[1]
    hq, hk = c["q_heads"] * d, c["kv_heads"] * d
    s["sbt"].qk_norm_rope_backward(s["ctx"], s["gq"], hq, d, s["gk"], hk, d, s["q"], ld, d, s["k"], ld, d,
                                   c["tokens"], c["q_heads"], c["kv_heads"], d, s["pos"], s["turn"], s["dq"], hq, d,
                                   s["dk"], hk, d, q_weight=s["wq"], k_weight=s["wk"], eps=EPS, dq_weight=s["dwq"],
                                   dk_weight=s["dwk"], workspace=s["workspace"],
                                   workspace_bytes=s["workspace_bytes"])
    return {"dq": s["dq"], "dk": s["dk"], "dwq": s["dwq"], "dwk": s["dwk"]}


def _own_pages_step(s):
    sbt, ctx, m, ws = s["sbt"], s["ctx"], s["map"], (s["workspace"], s["workspace_bytes"])
    sbt.pages_free(ctx, m, s["fork_to"], s["fork_to"].numel())
    sbt.pages_free(ctx, m, s["parents"], s["parents"].numel(), keep=s["keep"])
    sbt.pages_reserve(ctx, m, s["handles"], s["target"], *ws)
    sbt.pages_fork(ctx, m, s["handles"], s["fork_from"], s["fork_to"], s["fork_to"].numel(), *ws)
    return {"table": s["table"], "refs": s["refs"], "lens": s["lens"], "pools": s["pools"]}


def _own_pages_copy(s):
    s["sbt"].pages_copy(s["ctx"], s["handles"], s["case"]["n_pages"], s["src"], s["dst"], s["src"].numel())
    return s["pools"]


def _own_pages_compact(s):
    s["sbt"].pages_compact(s["ctx"], s["map"], s["handles"], s["table_out"], s["max_pages"], s["refs_out"],
                           s["page_to"], s["n_live"], s["workspace"], s["workspace_bytes"])
    return {"pools": s["pools"], "table": s["table_out"], "refs": s["refs_out"], "page_to": s["page_to"],
            "n_live": s["n_live"]}


def run(state):
    op = state["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](state)


# ---------------------------------------------------------------------------- work and exact

def work(case):
    c, op = case, case["op"]
    es = 4 if c.get("dtype") == "f32" else 2
    if op == "attention":
        lens = _lengths(c["batch"], c["max_len"], c["equal"])
        seen = sum(min(n, c["window"]) if c["window"] else n for n in lens)
        pages = sum(cdiv(n, c["page_size"]) for n in lens)
        return {"bytes": 2 * seen * c["kv_heads"] * c["dim"] * es + 2 * c["batch"] * c["q_heads"] * c["dim"] * es
                + 4 * (pages + c["batch"] + c["batch"] * c["q_heads"]),
                "flops": 4 * seen * c["q_heads"] * c["dim"]}
    if op.startswith("norm_rope"):
        heads = c["q_heads"] + c["kv_heads"]
        row = c["tokens"] * c["dim"] * es
        if op == "norm_rope":  # q, k and v in, q and the cache's rows out
            return {"bytes": 2 * row * (heads + c["kv_heads"]) + c["tokens"] * 8,
                    "flops": c["tokens"] * heads * (4 * c["dim"] + 3 * c["rot"])}
        return {"bytes": 3 * row * heads + c["tokens"] * 4,
                "flops": c["tokens"] * heads * (11 * c["dim"] + 3 * c["rot"])}
    page = 2 * c["planes"] * c["page_bytes"]  # K and V
    if op == "pages_copy":
        return {"bytes": c["pairs"] * (2 * page + 8), "flops": 0}
    if op == "pages_compact":
        return {"bytes": c["moved"] * 2 * page + c["n_pages"] * 12 + c["live"] * 8, "flops": 0}
    forks = c["parents"] * c["beams"]
    entries = forks * cdiv(c["max_len"] + c["grow"], c["page_size"])
    return {"bytes": forks * 2 * page + entries * 16 + c["n_pages"] * 8, "flops": 0}


def _exact_attention(s):
    c, d = s["case"], s["case"]["dim"]
    p, hk, g = c["page_size"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros((c["batch"], c["q_heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["batch"], c["q_heads"]), dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] else 0
        pos = torch.arange(lo, n, device="cuda")
        page, slot = s["table"][i, pos // p].long(), pos % p
        for h in range(hk):
            at = (page, slot, h) if c["order"] == "nhd" else (page, h, slot)
            k, v = s["k"][at].double(), s["v"][at].double()
            q = s["q"][i, h * g:(h + 1) * g].double()
            score = torch.einsum("gd,nd->gn", q, k) * s["scale"]
            lse[i, h * g:(h + 1) * g] = torch.logsumexp(score, 1)
            out[i, h * g:(h + 1) * g] = torch.softmax(score, 1) @ v
    return {"out": out, "lse": lse}


def _exact_turn(x, s, sign):
    """x rotated as a matrix product of 2 x 2 blocks, pair by pair (sign -1: the transposed blocks)."""
    rot, half = s["case"]["rot"], s["case"]["rot"] // 2
    out = x.clone()
    for i in range(half):
        a, b = (i, i + half) if s["case"]["layout"] == "half" else (2 * i, 2 * i + 1)
        cos = s["rope"][s["pos"].long(), i, 0].double()[:, None]
        sin = sign * s["rope"][s["pos"].long(), i, 1].double()[:, None]
        out[:, :, a] = x[:, :, a] * cos - x[:, :, b] * sin
        out[:, :, b] = x[:, :, a] * sin + x[:, :, b] * cos
    return out


def _exact_norm_rope(s):
    c, d = s["case"], s["case"]["dim"]

    def one(x, w):
        x = x.double()
        return _exact_turn(x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double(), s, 1)

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    pos = s["pos"].long()
    flat = s["table"][s["seq"].long(), pos // c["page_size"]].long() * c["page_size"] + pos % c["page_size"]
    k_cache.view(-1, c["kv_heads"], d).index_copy_(0, flat, one(s["k"], s["wk"]))
    v_cache.view(-1, c["kv_heads"], d).index_copy_(0, flat, s["v"].double())
    return {"q": one(s["q"], s["wq"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_norm_rope_backward(s):
    d = s["case"]["dim"]

    def one(g, x, w):
        u = _exact_turn(g.double(), s, -1)       # the gradient before the rotation
        x, w = x.double(), w.double()
        norm = ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt()
        n = x / norm                             # the normalised row; d n / d x = (I - n n^T / d) / norm
        uw = u * w
        return (uw - n * ((uw * n).sum(-1, keepdim=True) / d)) / norm, torch.einsum("thd,thd->d", u, n)

    dq, dwq = one(s["gq"], s["q"], s["wq"])
    dk, dwk = one(s["gk"], s["k"], s["wk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def exact(case, seed):
    """The definition in 64 bits; None for the page operators, whose outputs are whole numbers."""
    op = case["op"]
    if op.startswith("pages"):
        return None
    return globals()["_exact_" + op](_inputs(case, seed))
