"""Plain 64-bit references of the paged cache's operators (numpy and torch on the CPU).

Each is its definition written out, one loop per sequence, token or page; the
tests compare the library with them and pin them to closed forms.
"""
import numpy as np
import torch

TDT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0**-24, "bf16": 2.0**-8, "f16": 2.0**-11}  # relative rounding of one store
TINY = {"f32": 2.0**-149, "bf16": 2.0**-134, "f16": 2.0**-25}   # and its absolute part, among subnormals


def f64(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------------------- attention

def visible(n, window, page_size, row, n_pages):
    """Positions a query sees: inside the length and the window, on a page of the pool."""
    lo = max(0, n - window) if window else 0
    t = np.arange(lo, max(n, 0))
    page = row[t // page_size]
    return t[(page >= 0) & (page < n_pages)]


def attention(q, k, v, table, lens, page_size, scale, window=0, seq=None):
    """q [B][Hq][D]; k, v [n_pages][page_size][H][D] (any strides), all float64.

    Returns out, lse, and for the error bound: mean |v| under the probabilities,
    the largest sum of |q k| scale over the visible positions, their number."""
    B, Hq, D = q.shape
    n_pages, _, H, _ = k.shape
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    absv, mag, count = np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, Hq))
    vmax = np.zeros((B, Hq))
    for b in range(B):
        s = b if seq is None else int(seq[b])
        if not 0 <= s < len(lens):
            continue
        n = min(max(int(lens[s]), 0), table.shape[1] * page_size)
        t = visible(n, window, page_size, table[s], n_pages)
        if t.size == 0:
            continue
        kk, vv = k[table[s][t // page_size], t % page_size], v[table[s][t // page_size], t % page_size]
        for h in range(Hq):
            g = h // (Hq // H)
            x = kk[:, g] @ q[b, h] * scale
            if np.all(x == -np.inf):
                continue
            m = x.max()
            e = np.exp(x - m)
            out[b, h] = e @ vv[:, g] / e.sum()
            lse[b, h] = m + np.log(e.sum())
            absv[b, h] = e @ np.abs(vv[:, g]) / e.sum()
            mag[b, h] = (np.abs(kk[:, g]) @ np.abs(q[b, h])).max() * abs(scale)
            vmax[b, h] = np.abs(vv[:, g]).max()
            count[b, h] = t.size
    return out, lse, dict(absv=absv, mag=mag, count=count, vmax=vmax)


def attention_bounds(ref, kind, D):
    """Error bounds of out and lse.

    A score is off by at most D + 3 roundings of terms no larger than `mag`; in
    the exponent that is a relative error of the probability, twice (numerator
    and sum).  The sums over n positions round n times more.  The probabilities
    enter the second product with 16 (bf16) or 11 (fp16) bits, fp16 ones below
    its normal range with an absolute error of 2^-25."""
    out, lse, x = ref
    score = (D + 3) * 2.0**-23 * x["mag"]
    rel = 2 * score + (x["count"] + 64) * 2.0**-23 + {"f32": 0.0, "bf16": 2.0**-16, "f16": 2.0**-11}[kind]
    o = rel[..., None] * x["absv"] + HALF_ULP[kind] * np.abs(out) * 1.01 + TINY[kind]
    if kind == "f16":
        o = o + (x["count"] * 2.0**-25 * x["vmax"])[..., None]
    with np.errstate(invalid="ignore"):
        s = score + (x["count"] + 64) * 2.0**-23 + 2.0**-20 * (1 + np.where(np.isfinite(lse), np.abs(lse), 0))
    return o, s


# ---------------------------------------------------------------------------- norm and rotation

def pairs(rot, layout):
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def rotate(x, table, pos, rot, layout, sign=1.0):
    """x [T][H][D]; table [n_pos][rot/2][2]; positions in range."""
    y = x.copy()
    if rot:
        a, b = pairs(rot, layout)
        c, s = table[pos][:, None, :, 0], sign * table[pos][:, None, :, 1]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def is_real(pos, rot, n_pos):
    return (pos >= 0) & ((pos < n_pos) if rot else True)


def norm_rope(x, w, eps, table, pos, rot, layout, n_pos):
    """Rows of padding tokens are zero.  Also returns the magnitude each output element was summed from."""
    real = is_real(pos, rot, n_pos)
    p = np.where(real, pos, 0) if n_pos else np.zeros_like(pos)
    n = x if w is None else x / np.sqrt((x**2).mean(-1, keepdims=True) + eps) * w
    y = rotate(n, table, p, rot, layout)
    mag = np.abs(n).copy()
    if rot:
        a, b = pairs(rot, layout)
        amp = np.abs(table[p]).max(-1)[:, None]
        m = (np.abs(n[..., a]) + np.abs(n[..., b])) * amp
        mag[..., a] = mag[..., b] = m
    return np.where(real[:, None, None], y, 0.0), np.where(real[:, None, None], mag, 0.0)


def norm_rope_backward(g, x, w, eps, table, pos, rot, layout, n_pos):
    """dx, dw and the magnitudes that the terms of either summed from."""
    real = is_real(pos, rot, n_pos)
    p = np.where(real, pos, 0) if n_pos else np.zeros_like(pos)
    u = rotate(g, table, p, rot, layout, -1.0)
    au = np.abs(u)
    if rot:
        a, b = pairs(rot, layout)
        amp = np.abs(table[p]).max(-1)[:, None]
        au[..., a] = au[..., b] = (np.abs(g[..., a]) + np.abs(g[..., b])) * amp
    z = real[:, None, None]
    if w is None:
        return np.where(z, u, 0.0), None, np.where(z, au, 0.0), None
    r = 1.0 / np.sqrt((x**2).mean(-1, keepdims=True) + eps)
    uw = u * w
    dx = r * (uw - x * r**2 * (uw * x).mean(-1, keepdims=True))
    mx = r * (au * np.abs(w) + np.abs(x) * r**2 * (au * np.abs(w * x)).mean(-1, keepdims=True))
    dw = np.where(z, u * x * r, 0.0).sum((0, 1))
    mw = np.where(z, au * np.abs(x) * r, 0.0).sum((0, 1))
    return np.where(z, dx, 0.0), dw, np.where(z, mx, 0.0), mw


def rope_table(n_pos, rot, base, scaling="none", factor=1.0, orig=0, low=1.0, high=32.0, amplitude=1.0):
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2 * i / max(rot, 1))
    if scaling == "linear":
        f = f / factor
    elif scaling == "ntk":
        f = (base * factor ** (rot / (rot - 2))) ** (-2 * i / rot) if rot > 2 else f
    elif scaling == "by_parts":
        g = np.clip((orig * f / (2 * np.pi) - low) / (high - low), 0, 1)
        f = (1 - g) * f / factor + g * f
    a = np.arange(n_pos, dtype=np.float64)[:, None] * f
    return amplitude * np.stack([np.cos(a), np.sin(a)], -1)


# ---------------------------------------------------------------------------- pages

class Pages:
    """The page state as plain Python: table, lengths, holders and the pools' pages."""

    def __init__(self, table, lens, refs, page_size, pools):
        self.table, self.lens, self.refs = table.copy(), lens.copy(), refs.copy()
        self.P, self.pools = page_size, [p.copy() for p in pools]  # pools: [planes][n_pages][bytes]

    @property
    def max_pages(self):
        return self.table.shape[1]

    def ok(self, p):
        return 0 <= p < len(self.refs)

    def pages(self, n):
        return max(0, -(-int(n) // self.P))

    def held(self, s):
        return min(self.pages(self.lens[s]), self.max_pages)

    def free_pages(self):
        return [p for p in range(len(self.refs)) if self.refs[p] <= 0]

    def copy(self, src, dst):
        old = [p.copy() for p in self.pools]
        for s, d in zip(src, dst):
            if self.ok(s) and self.ok(d):
                for new, o in zip(self.pools, old):
                    new[:, d] = o[:, s]

    def free(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            if not 0 <= s < len(self.lens):
                continue
            k = 0 if keep is None else max(0, int(keep[i]))
            for j in range(self.pages(k), self.held(s)):
                p = self.table[s, j]
                if self.ok(p):
                    self.refs[p] -= 1
                self.table[s, j] = -1
            self.lens[s] = min(self.lens[s], k)

    def reserve(self, target):
        free, at, old_refs, moves = self.free_pages(), 0, self.refs.copy(), []
        for s in range(len(self.lens)):
            n, t = int(self.lens[s]), int(target[s])
            if t <= n or self.pages(t) > self.max_pages:
                continue
            first = self.pages(n)
            own = n > 0 and n % self.P != 0 and self.ok(self.table[s, first - 1]) and \
                old_refs[self.table[s, first - 1]] > 1
            need = self.pages(t) - first + own
            if need and at + need > len(free):
                at += need
                continue
            for i in range(need):
                p, j = free[at + i], first - own + i
                if own and i == 0:
                    moves.append((self.table[s, j], p))
                    self.refs[self.table[s, j]] -= 1
                self.table[s, j] = p
                self.refs[p] = 1
            at += need
            self.lens[s] = t
        self.copy(*zip(*moves)) if moves else None

    def fork(self, src, dst):
        before, free, at, taken, moves = self.lens.copy(), self.free_pages(), 0, set(), []
        S = len(before)
        for a, c in zip(src, dst):
            if not (0 <= a < S and 0 <= c < S) or a == c or before[a] <= 0 or before[c] != 0 or c in taken:
                continue
            taken.add(c)
            n = int(before[a])
            last = self.pages(n) - 1
            part = n % self.P != 0 and last < self.max_pages and self.ok(self.table[a, last])
            if part:
                at += 1
                if at > len(free):
                    continue
            for j in range(min(self.pages(n), self.max_pages)):
                p = self.table[a, j]
                if part and j == last:
                    moves.append((p, free[at - 1]))
                    p = free[at - 1]
                    self.refs[p] = 1
                elif self.ok(p):
                    self.refs[p] += 1
                self.table[c, j] = p
            self.lens[c] = n
        self.copy(*zip(*moves)) if moves else None

    def compact(self):
        """(table, refs, page_to, n_live): the pool's pages move, the map stays."""
        n = len(self.refs)
        live = [p for p in range(n) if self.refs[p] > 0]
        L = len(live)
        holes = [p for p in range(L) if self.refs[p] <= 0]
        movers = [p for p in live if p >= L]
        to = np.full(n, -1, np.int32)
        to[live] = live
        to[movers] = holes
        refs = np.zeros(n, np.int32)
        for p in live:
            refs[to[p]] = self.refs[p]
        table = self.table.copy()
        for s in range(len(self.lens)):
            for j in range(self.held(s)):
                p = self.table[s, j]
                table[s, j] = to[p] if self.ok(p) else -1
        self.copy(movers, holes)
        return table, refs, to, L
