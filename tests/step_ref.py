"""Plain 64-bit references of a decoding step's operators around the attention (numpy on the CPU).

Each is its definition written out, one loop per token, row or block; the
tests compare the library with them and pin them to closed forms.
"""
import numpy as np
import torch

from cache_ref import HALF_ULP, TDT, TINY, f64  # noqa: F401 (shared with the tests)

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6] + [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
CODES = {"e4m3": (torch.float8_e4m3fn, 448.0, 2.0**-9), "e5m2": (torch.float8_e5m2, 57344.0, 2.0**-16)}
LEAST_SCALE = -124


def code_values(raw, fmt):
    """Values of 8-bit codes (E4M3, E5M2 or E8M0 bytes) in float64."""
    raw = np.asarray(raw, np.uint8)
    if fmt == "e8m0":
        v = np.ldexp(1.0, raw.astype(np.int64) - 127)
        return np.where(raw == 255, np.nan, v)
    return torch.from_numpy(raw.copy()).view(CODES[fmt][0]).float().double().numpy()


# ---------------------------------------------------------------------------- norm

def add_rms_norm(x, r, w, eps):
    """h, y in float64."""
    h = x if r is None else x + r
    y = h / np.sqrt((h**2).mean(-1, keepdims=True) + eps)
    return h, y if w is None else y * w


def scale_exponents(y, fmt, block):
    """Exponent of every block's scale; None stands for NaN."""
    largest = CODES[fmt][1]
    out = np.empty((y.shape[0], y.shape[1] // block), object)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            top = np.abs(y[i, j * block:(j + 1) * block]).max()
            if not np.isfinite(top):
                out[i, j] = None
                continue
            e = 0
            if top > 0:
                e = LEAST_SCALE
                while top > largest * 2.0**e:
                    e += 1
            out[i, j] = e
    return out


def add_rms_norm_backward(gy, gh, h, w, eps):
    """dx, dweight in float64, by the normed row n: d n / d h = (I - n n^T / C) / norm."""
    norm = np.sqrt((h**2).mean(-1, keepdims=True) + eps)
    n = h / norm
    g = gy if w is None else gy * w
    dx = (g - n * (g * n).mean(-1, keepdims=True)) / norm
    return dx + (0 if gh is None else gh), (gy * n).sum(0)


# ---------------------------------------------------------------------------- 4-bit products

def unpack_e2m1(packed, K, N, ld):
    """Codes [K][N] of packed rows (`ld` codes each, two a byte, the even one low)."""
    b = np.asarray(packed, np.uint8).reshape(-1)
    i = np.arange(K)[:, None] * ld + np.arange(N)[None, :]
    return (b[i // 2] >> (4 * (i % 2))) & 15


def matvec(x, codes, scales, group, alpha):
    """y [T][N], and the magnitude its sums were made of; x, scales float64, codes [K][N]."""
    w = E2M1[codes] * np.repeat(scales, group, 0)
    with np.errstate(invalid="ignore", over="ignore"):
        return alpha * (x @ w), abs(alpha) * (np.abs(x) @ np.abs(w))


# ---------------------------------------------------------------------------- slots and trees

def pages_slots(n_new, seqs, start, lens, table, page_size, n_pages, capacity):
    """cu, seq, positions, slots, last as lists of ints."""
    n_seq, max_pages = table.shape
    cu, seq, positions, slots, last = [0], [], [], [], []
    total = 0
    for b, n in enumerate(n_new):
        n = max(int(n), 0)
        s = b if seqs is None else int(seqs[b])
        ok = 0 <= s < n_seq
        first = 0
        if ok:
            held = min(max(int(lens[s]), 0), max_pages * page_size) if start is None else 0
            first = held - n if start is None else int(start[b])
        for i in range(min(n, max(0, capacity - total))):
            at, slot = first + i, -1
            if not ok or at < 0 or at >= 2**31:
                at = -1
            elif at // page_size < max_pages:
                page = int(table[s, at // page_size])
                if 0 <= page < n_pages:
                    slot = page * page_size + at % page_size
            seq.append(s if ok else -1)
            positions.append(at)
            slots.append(slot)
        total += n
        cu.append(min(total, capacity))
        last.append(total - 1 if n and total <= capacity else -1)
    pad = [-1] * (capacity - len(seq))
    return cu, seq + pad, positions + pad, slots + pad, last


def tree_plan(parents, cu, rows, words, positions):
    """mask [rows][words] and turned [rows]."""
    mask, turned = np.zeros((rows, words), np.uint32), np.full(rows, -1, np.int64)
    for b in range(len(cu) - 1):
        for row in range(cu[b], min(cu[b + 1], rows)):
            i = j = row - cu[b]
            depth = 0
            while True:
                if j // 32 < words:
                    mask[row, j // 32] |= np.uint32(1 << (j % 32))
                up = int(parents[cu[b] + j])
                if not 0 <= up < j:
                    break
                j, depth = up, depth + 1
            if positions[row] >= 0:
                turned[row] = positions[row] - i + depth
    return mask, turned


# ---------------------------------------------------------------------------- attention of several new tokens

def visible(i, n, length, mask_row):
    """bool [length]: what token i of n sees of the positions; mask_row: its int32 words, or None for a chain."""
    t = np.arange(length)
    j = t - (length - n)
    if mask_row is None:
        return j <= i
    words = np.asarray(mask_row).view(np.uint32)
    bit = np.zeros(length, bool)
    inside = (j >= 0) & (j < min(n, 32 * len(words)))
    bit[inside] = words[j[inside] // 32] >> (j[inside] % 32).astype(np.uint32) & 1
    return (j < 0) | bit


def tree_attention(q, k, v, table, lens, page_size, scale, cu, max_new, mask=None, seq=None):
    """q [rows][Hq][D]; k, v [n_pages][page_size][H][D], float64.

    Returns out, lse, the rows that are written, and for the error bound what cache_ref.attention returns."""
    rows, Hq, D = q.shape
    n_pages, _, H, _ = k.shape
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    x = dict(absv=np.zeros((rows, Hq, D)), mag=np.zeros((rows, Hq)), count=np.zeros((rows, Hq)), vmax=np.zeros((rows, Hq)))
    written = np.zeros(rows, bool)
    for b in range(len(cu) - 1):
        n = int(cu[b + 1]) - int(cu[b])
        if n <= 0 or n > max_new or cu[b] < 0 or cu[b + 1] > rows:
            continue
        written[cu[b]:cu[b + 1]] = True
        s = b if seq is None else int(seq[b])
        if not 0 <= s < len(lens):
            continue
        length = min(max(int(lens[s]), 0), table.shape[1] * page_size)
        t = np.arange(length)
        page = table[s, t // page_size]
        held = (page >= 0) & (page < n_pages)
        kk = np.where(held[:, None, None], k[np.where(held, page, 0), t % page_size], 0)
        vv = np.where(held[:, None, None], v[np.where(held, page, 0), t % page_size], 0)
        for i in range(n):
            row = cu[b] + i
            sees = held & visible(i, n, length, None if mask is None else mask[row])
            if not sees.any():
                continue
            for h in range(Hq):
                g = h // (Hq // H)
                with np.errstate(invalid="ignore", over="ignore"):
                    score = kk[sees, g] @ q[row, h] * scale
                    m = score.max()
                    if m == -np.inf:
                        continue
                    e = np.exp(score - m)
                    out[row, h] = e @ vv[sees, g] / e.sum()
                    lse[row, h] = m + np.log(e.sum())
                    x["absv"][row, h] = e @ np.abs(vv[sees, g]) / e.sum()
                x["mag"][row, h] = (np.abs(kk[sees, g]) @ np.abs(q[row, h])).max() * abs(scale)
                x["vmax"][row, h] = np.abs(vv[sees, g]).max()
                x["count"][row, h] = sees.sum()
    return out, lse, written, x


def tree_attention_bounds(ref, kind, D, terms=2):
    """As cache_ref.attention_bounds.  Probabilities of two 16-bit numbers have 16 (bf16) or 22 (fp16) bits, those of one
    are off by half a step (2^-8, 2^-11 of themselves); fp16 ones have steps of 2^-33 of the row's largest at least."""
    out, lse, _, x = ref
    score = (D + 3) * 2.0**-23 * x["mag"]
    p = {"bf16": 2.0**-16, "f16": 2.0**-21}[kind] if terms == 2 else HALF_ULP[kind]
    rel = 2 * score + (x["count"] + 64) * 2.0**-23 + p
    o = rel[..., None] * x["absv"] + HALF_ULP[kind] * np.abs(out) * 1.01 + TINY[kind]
    if kind == "f16":
        o = o + (x["count"] * 2.0**-34 * x["vmax"])[..., None]
    s = score + (x["count"] + 64) * 2.0**-23 + 2.0**-20 * (1 + np.where(np.isfinite(lse), np.abs(lse), 0))
    return o, s
