"""Cases of a decoding step's operators around the paged cache: what is timed, on which inputs, and what the answer is.

  norm           root-mean-square norm with the residual's addition; out come the sum and the normed rows, or the
                 normed rows as 8-bit codes with a power-of-two scale per block (the block-scaled GEMM's A operand)
  norm_backward  its gradient, the weight's included
  matvec         a few tokens times a matrix of 4-bit weights with group scales (the block-scaled GEMM's B operand)
  slots          from the number of new tokens of each request: prefix sums, and every token's sequence, position
                 and slot in the paged cache
  tree           trees of drafted tokens, one tree per request: from the tokens' parents their masks and positions,
                 and their attention over the paged cache, which holds the context and the drafted tokens

`run` computes the plain form (elementary torch operations in 32 bits) where `own` is false, and calls the library
where it is true.  `exact` computes the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"e4m3": (torch.float8_e4m3fn, 448.0, -6, 3), "e5m2": (torch.float8_e5m2, 57344.0, -14, 2)}
LEAST_SCALE = -124  # exponent of the smallest scale of a block
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
EPS = 1e-6


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one user's token in a layer's residual stream: latency of the smallest call
        dict(name="norm_one_token_bf16", op="norm", dtype="bf16", rows=1, cols=4096, codes="", block=0),
        # a mixed batch on a width that no vector divides
        dict(name="norm_odd_width_f16", op="norm", dtype="f16", rows=333, cols=5003, codes="", block=0),
        # prompts whose projections run in 8 bits: codes and scales for the block-scaled GEMM
        dict(name="norm_codes_prompts_bf16", op="norm", dtype="bf16", rows=16384, cols=8192, codes="e4m3", block=32),
        # training: gradients of 16384 tokens
        dict(name="norm_backward_bf16", op="norm_backward", dtype="bf16", rows=16384, cols=4096),
        # training in 32 bits with odd sizes
        dict(name="norm_backward_odd_f32", op="norm_backward", dtype="f32", rows=1021, cols=1537),
        # one token through an output projection: the smallest product of a decoding step
        dict(name="matvec_one_token_bf16", op="matvec", dtype="bf16", out="bf16", tokens=1, k=4096, n=4096,
             scale="e8m0", group=32),
        # five users' tokens through a feed-forward layer, scales per 16 weights
        dict(name="matvec_feed_forward_f16", op="matvec", dtype="f16", out="f16", tokens=5, k=8192, n=28672,
             scale="e4m3", group=16),
        # logits of a batch: the widest product, an odd number of columns, 32 bits out
        dict(name="matvec_vocabulary_bf16", op="matvec", dtype="bf16", out="f32", tokens=16, k=4096, n=131071,
             scale="e8m0", group=32),
        # one decoding step of a batch: a new token for each of 256 requests
        dict(name="slots_decode", op="slots", batch=256, most=1, page_size=16, held=4096, spare=0),
        # prompts of up to 16384 tokens read at once, padded to a fixed capacity
        dict(name="slots_prompts", op="slots", batch=64, most=16384, page_size=64, held=0, spare=1000),
        # one user's 32 drafted tokens over a long context
        dict(name="tree_one_user_bf16", op="tree", dtype="bf16", batch=1, drafted=32, context=16384, equal=True,
             q_heads=32, kv_heads=8, dim=128, page_size=16, order="nhd"),
        # a serving batch: trees of 1 to 64 tokens over contexts of up to 8192, eight queries on each key
        dict(name="tree_batch_f16", op="tree", dtype="f16", batch=48, drafted=64, context=8191, equal=False,
             q_heads=64, kv_heads=8, dim=128, page_size=32, order="hnd"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "matvec", "matvec", "slots", "tree", "tree"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    es = 4 if dtype == "f32" else 2
    if op in ("norm", "norm_backward"):
        codes = rng.choice(["", "", "e4m3", "e5m2"]) if op == "norm" else ""
        block = rng.choice([16, 32, 32, 64, 128]) if codes else 0
        cols = _log_int(rng, 64, 16384)
        unit = block or rng.choice([1, 8, 64, 64])
        cols = max(unit, cols // unit * unit)
        rows = _log_int(rng, 1, min(65536, int(1.2e8 / cols * 2 / es)))
        case = dict(op=op, dtype=dtype, rows=rows, cols=cols)
        return dict(case, codes=codes, block=block) if op == "norm" else case
    if op == "matvec":
        scale, group = rng.choice([("e8m0", 32), ("e8m0", 32), ("e4m3", 16), ("e4m3", 16), ("e8m0", 128), ("e4m3", 64)])
        k = max(1, _log_int(rng, 64, 16384) // group) * group
        n = _log_int(rng, 64, min(131071, int(4e8 / k)))
        if rng.random() < 0.6:
            n = max(64, n // 64 * 64)
        return dict(op=op, dtype=dtype, out=rng.choice([dtype, "f32"]), tokens=rng.randint(1, 16), k=k, n=n,
                    scale=scale, group=group)
    if op == "tree":
        kv, group = rng.choice([1, 2, 3, 4, 5, 8, 8]), rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 8, 16])
        dim = rng.choice([32, 64, 64, 72, 80, 96, 100, 112, 128, 128, 128, 160, 192, 256])
        batch, drafted = _log_int(rng, 1, 64), _log_int(rng, 1, 100)
        top = min(32768, int(1.2e9 / (batch * drafted * kv * group)), int(1e9 / (batch * kv * dim * 4)))
        return dict(op=op, dtype=rng.choice(["bf16", "f16"]), batch=batch, drafted=drafted,
                    context=_log_int(rng, 1, max(1, top)), equal=rng.random() < 0.3, q_heads=kv * group, kv_heads=kv,
                    dim=dim, page_size=rng.choice([1, 8, 13, 16, 16, 24, 32, 64, 128]),
                    order=rng.choice(["nhd", "hnd"]))
    batch = _log_int(rng, 1, 1024)
    most = rng.choice([1, 1, 8, _log_int(rng, 1, min(16384, int(1e6 / batch)))])
    return dict(op=op, batch=batch, most=most, page_size=rng.choice([1, 8, 13, 16, 24, 32, 64, 128]),
                held=rng.choice([0, _log_int(rng, 1, 4096)]), spare=rng.randint(0, 2000))


# ----------------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, dtype, gen, scale=1.0):
    """N(0, scale^2) in slabs, so that the 32-bit draws of a large array do not pile up."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=gen, device="cuda") * scale
    return out


def _norm_inputs(case, seed):
    gen, dt, shape = _generator(seed), TYPES[case["dtype"]], (case["rows"], case["cols"])
    weight = (1 + _normal((case["cols"],), torch.float32, gen, 0.2)).to(dt)
    if case["op"] == "norm_backward":
        return dict(case=case, h=_normal(shape, dt, gen, 2.5), gy=_normal(shape, dt, gen, 0.02),
                    gh=_normal(shape, dt, gen, 0.02), weight=weight)
    # a residual stream is several times as large as what a layer adds to it, with a few large channels
    r = _normal(shape, dt, gen, 2.5)
    r[:, ::97] *= 8
    return dict(case=case, x=_normal(shape, dt, gen, 0.7), r=r, weight=weight)


def _power(e):
    """2^e of integers, exactly (normal range)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _least_power(top, largest):
    """The smallest e with top <= largest * 2^e (0 where top is 0)."""
    m, p = torch.frexp(top)
    m_largest, p_largest = math.frexp(largest)
    return torch.where(top > 0, p - p_largest + (m > m_largest).int(), 0)


def _matvec_inputs(case, seed):
    """Weights N(0, k^-1) rounded to E2M1 by groups along k; two columns per byte, the even one in the low nibble."""
    gen, dt = _generator(seed), TYPES[case["dtype"]]
    k, n, group = case["k"], case["n"], case["group"]
    ld = n + n % 2
    packed = torch.empty((k, ld // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((k // group, n), dtype=torch.uint8, device="cuda")
    alpha = 1.0 if case["scale"] == "e8m0" else 1.7 / (64 * k**0.5)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 26) // (n * group))
    for g0 in range(0, k // group, step):
        g = min(step, k // group - g0)
        w = torch.randn((g, group, n), generator=gen, device="cuda") * k**-0.5
        top = w.abs().amax(1)
        if case["scale"] == "e8m0":
            e = _least_power(top, 6.0)
            s, byte = _power(e), (e + 127).to(torch.uint8)
        else:
            s8 = (top / (6.0 * alpha)).clamp(2.0**-6, 448.0).to(torch.float8_e4m3fn)
            s, byte = s8.float() * alpha, s8.view(torch.uint8)
        code = torch.bucketize(w.abs() / s[:, None], edges).to(torch.uint8) | ((w < 0).to(torch.uint8) << 3)
        code = torch.nn.functional.pad(code.view(g * group, n), (0, ld - n))
        packed[g0 * group:(g0 + g) * group] = code[:, 0::2] | (code[:, 1::2] << 4)
        scales[g0:g0 + g] = byte
    x = _normal((case["tokens"], k), dt, gen)
    x[:, ::101] *= 12  # a few large channels
    return dict(case=case, x=x, packed=packed, scales=scales, ld=ld, alpha=alpha)


def _slots_sizes(case):
    """A fixed set of counts (the seed shuffles it) and the capacity they are padded to."""
    b, most = case["batch"], case["most"]
    counts = [max(1, most * (i + 1) // b) for i in range(b)]
    return counts, sum(counts) + case["spare"]


def _slots_inputs(case, seed):
    gen, b, p = _generator(seed), case["batch"], case["page_size"]
    counts, capacity = _slots_sizes(case)
    perm = torch.randperm(b, generator=gen, device="cuda")
    n_new = torch.tensor(counts, device="cuda")[perm]
    held = (torch.arange(b, device="cuda") * 7919 + 13) % max(1, case["held"]) if case["held"] else torch.zeros_like(n_new)
    n_seq = b + 3
    seqs = torch.randperm(n_seq, generator=gen, device="cuda")[:b]  # which sequences the requests belong to
    lens = torch.zeros(n_seq, dtype=torch.int64, device="cuda")
    lens[seqs] = held + n_new
    most = max(1, case["held"]) + case["most"]
    max_pages = -(-most // p)
    need = (lens + p - 1) // p
    n_pages = int(sum(counts) + b * max(1, case["held"])) // p + 2 * b + 3
    start = torch.cumsum(need, 0) - need
    j = torch.arange(max_pages, device="cuda")
    order = torch.randperm(n_pages, generator=gen, device="cuda")
    pick = order[(start[:, None] + j).clamp(max=n_pages - 1)]
    table = torch.where(j < need[:, None], pick, -1).to(torch.int32).contiguous()
    i32 = lambda t: t.to(torch.int32).contiguous()
    return dict(case=case, n_new=i32(n_new), seqs=i32(seqs), lens=i32(lens), table=table, capacity=capacity,
                n_pages=n_pages, max_pages=max_pages)


def _tree_sizes(case):
    """(drafted tokens, context) of each request: a fixed set, which the seed shuffles."""
    b = case["batch"]
    if case["equal"]:
        return [(case["drafted"], case["context"])] * b
    return [(max(1, case["drafted"] * (i + 1) // b), case["context"] * ((i * 29) % b + 1) // b) for i in range(b)]


def _tree_inputs(case, seed):
    gen, dt, b = _generator(seed), TYPES[case["dtype"]], case["batch"]
    p, h, d, hq = case["page_size"], case["kv_heads"], case["dim"], case["q_heads"]
    sizes = torch.tensor(_tree_sizes(case), device="cuda")[torch.randperm(b, generator=gen, device="cuda")]
    n, lens = sizes[:, 0], sizes.sum(1)
    rows = sum(t for t, _ in _tree_sizes(case))
    cu = torch.nn.functional.pad(torch.cumsum(n, 0), (1, 0))
    entry = torch.repeat_interleave(torch.arange(b, device="cuda"), n)
    i = torch.arange(rows, device="cuda") - cu[entry]
    # a parent is one of the eight tokens before, or the context's last token (-1)
    parents = (i - 1 - (torch.rand(rows, generator=gen, device="cuda") ** 2 * 8).long()).clamp(min=-1)
    positions = (lens - n)[entry] + i
    max_pages = -(-max(t + c for t, c in _tree_sizes(case)) // p)
    n_pages = sum(-(-(t + c) // p) for t, c in _tree_sizes(case)) + 3
    need = (lens + p - 1) // p
    start = torch.cumsum(need, 0) - need
    j = torch.arange(max_pages, device="cuda")
    order = torch.randperm(n_pages, generator=gen, device="cuda")
    table = torch.where(j < need[:, None], order[(start[:, None] + j).clamp(max=n_pages - 1)], -1)
    shape = (n_pages, p, h, d) if case["order"] == "nhd" else (n_pages, h, p, d)
    i32 = lambda t: t.to(torch.int32).contiguous()
    return dict(case=case, q=_normal((rows, hq, d), dt, gen, 1.5), k=_normal(shape, dt, gen),
                v=_normal(shape, dt, gen), parents=i32(parents), cu=i32(cu), positions=i32(positions),
                lens=i32(lens), table=i32(table), n_pages=n_pages, max_pages=max_pages, rows=rows,
                words=-(-case["drafted"] // 32), scale=1.0 / math.sqrt(d))


def _inputs(case, seed):
    make = {"norm": _norm_inputs, "norm_backward": _norm_inputs, "matvec": _matvec_inputs, "slots": _slots_inputs,
            "tree": _tree_inputs}
    return make[case["op"]](case, seed)


def prepare(case, seed):
    state = _inputs(case, seed)
    if own:
        _prepare_own(state)
    return state


# ------------------------------------------------------------------------------ plain forms

def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    h = s["x"].float() + s["r"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if not c["codes"]:
        return {"h": h.to(dt), "y": y.to(dt)}
    kind, largest, _, _ = CODES[c["codes"]]
    y = y.view(c["rows"], c["cols"] // c["block"], c["block"])
    e = _least_power(y.abs().amax(-1), largest).clamp(min=LEAST_SCALE)
    codes = (y * _power(-e)[..., None]).to(kind)
    return {"h": h.to(dt), "codes": codes.view(c["rows"], c["cols"]),
            "scales": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}


def _plain_norm_backward(s):
    h, gy, w = s["h"].float(), s["gy"].float(), s["weight"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    gw = gy * w
    dx = s["gh"].float() + r * (gw - h * (r * r) * (gw * h).mean(-1, keepdim=True))
    return {"dx": dx.to(s["h"].dtype), "dweight": (gy * h * r).sum(0)}


def _scale_values(s, dtype):
    if s["case"]["scale"] == "e8m0":
        return torch.pow(torch.tensor(2.0, dtype=dtype, device="cuda"), s["scales"].to(dtype) - 127)
    return s["scales"].view(torch.float8_e4m3fn).to(dtype)


def _plain_matvec(s):
    c = s["case"]
    values = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")
    codes = torch.stack([s["packed"] & 15, s["packed"] >> 4], -1).view(c["k"], s["ld"])[:, :c["n"]]
    w = values[codes.int()].view(-1, c["group"], c["n"])
    w = (w * _scale_values(s, torch.float32)[:, None]).view(c["k"], c["n"])
    return {"y": (s["x"].float() @ w * s["alpha"]).to(TYPES[c["out"]])}


def _plain_slots(s):
    p = s["case"]["page_size"]
    n, seqs = s["n_new"].long(), s["seqs"].long()
    end = torch.cumsum(n, 0)
    at = torch.arange(s["capacity"], device="cuda")
    entry = torch.searchsorted(end, at, right=True)
    real = entry < n.numel()
    entry = entry.clamp(max=n.numel() - 1)
    seq = seqs[entry]
    pos = (s["lens"][seqs].long() - end)[entry] + at
    pos = torch.where(real, pos, 0)
    slot = s["table"][seq, pos // p].long() * p + pos % p
    pad = lambda v: torch.where(real, v, -1).to(torch.int32)
    return {"cu": torch.nn.functional.pad(end, (1, 0)).to(torch.int32), "seq": pad(seq), "positions": pad(pos),
            "slots": pad(slot), "last": (end - 1).to(torch.int32)}


def _plain_tree(s):
    c = s["case"]
    b, p, h, d, hq, most = c["batch"], c["page_size"], c["kv_heads"], c["dim"], c["q_heads"], c["drafted"]
    cu, lens, width = s["cu"].long(), s["lens"].long(), 32 * s["words"]
    row = torch.arange(s["rows"], device="cuda")
    entry = torch.searchsorted(cu[1:], row, right=True)
    i = row - cu[entry]
    # ancestors: the closure of "is the parent of or the token itself", squared until paths of any length are in it
    parents = torch.full((b, width), -1, device="cuda")
    parents[entry, i] = s["parents"].long()
    j = torch.arange(width, device="cuda")
    sees = ((parents[:, :, None] == j) | (j[:, None] == j)).float()
    for _ in range(max(1, (most - 1).bit_length())):
        sees = ((sees @ sees) > 0).float()
    seen = sees[entry, i] > 0                                                 # [rows][width]
    bits = (seen.view(-1, s["words"], 32).long() << torch.arange(32, device="cuda")).sum(-1)
    mask = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    turned = s["positions"].long() - i + seen.sum(-1) - 1

    page = s["table"].clamp(min=0).long()

    def keys(pool):  # [batch][kv_heads][positions][dim]
        x = pool[page].float()
        x = x.permute(0, 3, 1, 2, 4) if c["order"] == "nhd" else x.permute(0, 2, 1, 3, 4)
        return x.reshape(b, h, s["max_pages"] * p, d)

    g = hq // h
    q = torch.zeros((b, most, hq, d), device="cuda")
    q[entry, i] = s["q"].float()
    q = q.view(b, most, h, g, d).permute(0, 2, 1, 3, 4).reshape(b, h, most * g, d)
    score = (q @ keys(s["k"]).transpose(2, 3)).view(b, h, most, g, -1) * s["scale"]
    at = torch.arange(s["max_pages"] * p, device="cuda")
    new = at - (lens - (cu[1:] - cu[:-1]))[:, None]                           # which drafted token a position holds
    own_row = sees[:, :most].gather(2, new.clamp(0, width - 1)[:, None].expand(b, most, -1)) > 0
    visible = (new < 0)[:, None] | (own_row & (at < lens[:, None])[:, None])  # [batch][most][positions]
    score.masked_fill_(~visible[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight.view(b, h, most * g, -1) @ keys(s["v"])).view(b, h, most, g, d) / total
    out = out.permute(0, 2, 1, 3, 4).reshape(b, most, hq, d)[entry, i]
    lse = (top + total.log()).view(b, h, most, g).permute(0, 2, 1, 3).reshape(b, most, hq)[entry, i]
    return {"mask": mask, "turned": turned.to(torch.int32), "out": out.to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------------- the library's calls

def _prepare_own(s):
    import scatter_boundary_tile_gb300 as sbt

    c = s["case"]
    s["sbt"], s["ctx"] = sbt, sbt.Context(0)
    workspace = 0
    if c["op"] == "norm":
        s["h"] = torch.empty_like(s["x"])
        if c["codes"]:
            s["codes"] = torch.empty(s["x"].shape, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty((c["rows"], c["cols"] // c["block"]), dtype=torch.uint8, device="cuda")
            s["code_rows"] = sbt.code_rows(s["codes"], c["cols"], s["scales"], c["cols"] // c["block"],
                                           fmt=c["codes"], block=c["block"])
        else:
            s["y"] = torch.empty_like(s["x"])
    elif c["op"] == "norm_backward":
        s["dx"] = torch.empty_like(s["h"])
        s["dweight"] = torch.empty(c["cols"], dtype=torch.float32, device="cuda")
        workspace = sbt.add_rms_norm_backward_workspace_size(s["ctx"], c["rows"], c["cols"])
    elif c["op"] == "matvec":
        s["y"] = torch.empty((c["tokens"], c["n"]), dtype=TYPES[c["out"]], device="cuda")
    elif c["op"] == "tree":
        p, h, d = c["page_size"], c["kv_heads"], c["dim"]
        slot, head = (h * d, d) if c["order"] == "nhd" else (d, p * d)
        s["map"] = sbt.page_map(s["table"], s["max_pages"], c["batch"], s["max_pages"], s["lens"], s["n_pages"], p)
        s["cache"] = sbt.kv_cache(s["k"], s["v"], h, d, p * h * d, slot, head)
        s["mask"] = torch.empty((s["rows"], s["words"]), dtype=torch.int32, device="cuda")
        s["turned"] = torch.empty(s["rows"], dtype=torch.int32, device="cuda")
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        workspace = sbt.paged_tree_attention_workspace_size(s["ctx"], c["drafted"], c["q_heads"], h, d)
    else:
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
        s["map"] = sbt.page_map(s["table"], s["max_pages"], s["table"].shape[0], s["max_pages"], s["lens"],
                                s["n_pages"], c["page_size"])
        s["out"] = {"cu": i32(c["batch"] + 1), "seq": i32(s["capacity"]), "positions": i32(s["capacity"]),
                    "slots": i32(s["capacity"]), "last": i32(c["batch"])}
    s["workspace"] = torch.empty(max(workspace, 256), dtype=torch.uint8, device="cuda")
    s["workspace_bytes"] = workspace


def _own_norm(s):
    c, ld = s["case"], s["case"]["cols"]
    if c["codes"]:
        s["sbt"].add_rms_norm(s["ctx"], s["x"], ld, c["rows"], ld, weight=s["weight"], eps=EPS, r=s["r"], ld_r=ld,
                              h_out=s["h"], ld_h=ld, codes=s["code_rows"])
        return {"h": s["h"], "codes": s["codes"].view(CODES[c["codes"]][0]),
                "scales": s["scales"].view(torch.float8_e8m0fnu)}
    s["sbt"].add_rms_norm(s["ctx"], s["x"], ld, c["rows"], ld, weight=s["weight"], eps=EPS, r=s["r"], ld_r=ld,
                          h_out=s["h"], ld_h=ld, y=s["y"], ld_y=ld)
    return {"h": s["h"], "y": s["y"]}


def _own_norm_backward(s):
    c, ld = s["case"], s["case"]["cols"]
    s["sbt"].add_rms_norm_backward(s["ctx"], s["gy"], ld, s["h"], ld, c["rows"], ld, s["dx"], ld, gh=s["gh"], ld_gh=ld,
                                   weight=s["weight"], eps=EPS, dweight=s["dweight"], workspace=s["workspace"],
                                   workspace_bytes=s["workspace_bytes"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_matvec(s):
    c = s["case"]
    s["sbt"].matvec_e2m1(s["ctx"], s["x"], c["k"], c["tokens"], s["packed"], s["ld"], s["scales"], c["n"],
                         c["k"] // c["group"], s["y"], c["n"], c["n"], c["k"], s_fmt=c["scale"], alpha=s["alpha"])
    return {"y": s["y"]}


def _own_slots(s):
    s["sbt"].pages_slots(s["ctx"], s["map"], s["n_new"], s["case"]["batch"], s["capacity"], seqs=s["seqs"], **s["out"])
    return s["out"]


def _own_tree(s):
    c, d, ld = s["case"], s["case"]["dim"], s["case"]["q_heads"] * s["case"]["dim"]
    s["sbt"].tree_plan(s["ctx"], s["parents"], s["cu"], c["batch"], s["rows"], mask=s["mask"], ld_mask=s["words"],
                       positions=s["positions"], turned=s["turned"])
    s["sbt"].paged_tree_attention(s["ctx"], s["q"], ld, d, s["rows"], s["cu"], c["batch"], c["drafted"], c["q_heads"],
                                  s["cache"], s["map"], s["scale"], s["out"], ld, d, mask=s["mask"],
                                  ld_mask=s["words"], lse=s["lse"], workspace=s["workspace"],
                                  workspace_bytes=s["workspace_bytes"])
    return {"mask": s["mask"], "turned": s["turned"], "out": s["out"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](state)


# ---------------------------------------------------------------------------- work and exact

def work(case):
    c, op = case, case["op"]
    es = 4 if c.get("dtype") == "f32" else 2
    if op == "norm":
        size = c["rows"] * c["cols"]
        out = size * (1 + 1 / c["block"]) if c["codes"] else size * es
        return {"bytes": 3 * size * es + out + c["cols"] * es, "flops": size * (8 if c["codes"] else 5)}
    if op == "norm_backward":
        size = c["rows"] * c["cols"]
        return {"bytes": 4 * size * es + c["cols"] * (es + 4), "flops": 12 * size}
    if op == "matvec":
        out = 4 if c["out"] == "f32" else 2
        return {"bytes": c["k"] * c["n"] / 2 + c["k"] // c["group"] * c["n"] + c["tokens"] * (c["k"] * es + c["n"] * out),
                "flops": 2 * c["tokens"] * c["k"] * c["n"]}
    if op == "tree":
        sizes, hq, d = _tree_sizes(c), c["q_heads"], c["dim"]
        held, rows = sum(n + ctx for n, ctx in sizes), sum(n for n, _ in sizes)
        pairs = sum(n * ctx + n * (n + 1) // 2 for n, ctx in sizes)  # at most: a chain sees all that came before
        return {"bytes": 2 * held * c["kv_heads"] * d * es + 2 * rows * hq * d * es
                + 4 * (rows * (hq + 3 + -(-c["drafted"] // 32)) + held // c["page_size"] + 2 * c["batch"]),
                "flops": 4 * pairs * hq * d}
    counts, capacity = _slots_sizes(c)
    pages = sum(-(-n // c["page_size"]) for n in counts)
    return {"bytes": 12 * capacity + 4 * pages + 20 * c["batch"], "flops": 0}


def _on_grid(v, least, bits):
    """v rounded to the nearest number with `bits` fraction bits, exponents from `least` up, ties to even."""
    _, p = torch.frexp(v)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), ((p - 1).clamp(min=least) - bits).double())
    return torch.round(v / step) * step


def _exact_norm(s):
    c = s["case"]
    h = s["x"].double() + s["r"].double()
    y = h / ((h ** 2).sum(-1, keepdim=True) / c["cols"] + EPS).sqrt() * s["weight"].double()
    if not c["codes"]:
        return {"h": h, "y": y}
    _, largest, least, bits = CODES[c["codes"]]
    y = y.view(c["rows"], -1, c["block"])
    top = y.abs().amax(-1)
    e = torch.ceil(torch.log2(top / largest))
    e = torch.where(top == 0, 0, e)
    e = e + (top > largest * 2 ** e).double() - (top <= largest * 2 ** (e - 1)).double() * (top > 0)
    scale = 2 ** e.clamp(min=LEAST_SCALE)
    return {"h": h, "codes": _on_grid(y / scale[..., None], least, bits).view(c["rows"], c["cols"]), "scales": scale}


def _exact_norm_backward(s):
    h, gy, w, cols = s["h"].double(), s["gy"].double(), s["weight"].double(), s["case"]["cols"]
    norm = ((h ** 2).sum(-1, keepdim=True) / cols + EPS).sqrt()
    n = h / norm                                  # the normed row; d n / d h = (I - n n^T / cols) / norm
    gn = gy * w
    dx = s["gh"].double() + (gn - n * ((gn * n).sum(-1, keepdim=True) / cols)) / norm
    return {"dx": dx, "dweight": (gy * n).sum(0)}


def _exact_matvec(s):
    c = s["case"]
    x, scale = s["x"].double(), _scale_values(s, torch.float64)
    values = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    y = torch.empty((c["tokens"], c["n"]), dtype=torch.float64, device="cuda")
    step = max(2, (1 << 25) // c["k"] // 2 * 2)
    for n0 in range(0, c["n"], step):
        n1 = min(c["n"], n0 + step)
        column = torch.arange(n0, n1, device="cuda")
        code = (s["packed"][:, n0 // 2:(n1 + 1) // 2].repeat_interleave(2, 1)[:, :n1 - n0] >> (4 * (column % 2))).int() & 15
        w = values[code & 7] * (1 - 2 * (code >> 3)) * scale[:, n0:n1].repeat_interleave(c["group"], 0)
        y[:, n0:n1] = x @ w * s["alpha"]
    return {"y": y}


def _exact_tree(s):
    c, d = s["case"], s["case"]["dim"]
    p, hk, g = c["page_size"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros((s["rows"], c["q_heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["rows"], c["q_heads"]), dtype=torch.float64, device="cuda")
    cu, parents = s["cu"].tolist(), s["parents"].tolist()
    for b, length in enumerate(s["lens"].tolist()):
        n = cu[b + 1] - cu[b]
        sees = torch.zeros((n, length), dtype=torch.bool)
        for i in range(n):
            parent = parents[cu[b] + i]
            sees[i] = sees[parent] if parent >= 0 else torch.arange(length) < length - n
            sees[i, length - n + i] = True
        sees = sees.cuda().repeat_interleave(g, 0)
        pos = torch.arange(length, device="cuda")
        page, slot = s["table"][b, pos // p].long(), pos % p
        for h in range(hk):
            at = (page, slot, h) if c["order"] == "nhd" else (page, h, slot)
            q = s["q"][cu[b]:cu[b + 1], h * g:(h + 1) * g].double().reshape(n * g, d)
            score = torch.where(sees, (q @ s["k"][at].double().T) * s["scale"], -math.inf)
            lse[cu[b]:cu[b + 1], h * g:(h + 1) * g] = torch.logsumexp(score, 1).view(n, g)
            out[cu[b]:cu[b + 1], h * g:(h + 1) * g] = (torch.softmax(score, 1) @ s["v"][at].double()).view(n, g, d)
    return {"mask": None, "turned": None, "out": out, "lse": lse}


def exact(case, seed):
    """The definition in 64 bits; None for the slots, which are whole numbers."""
    if case["op"] == "slots":
        return None
    return globals()["_exact_" + case["op"]](_inputs(case, seed))
