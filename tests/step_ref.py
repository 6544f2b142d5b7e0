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
