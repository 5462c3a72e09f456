"""Float64 oracle of the serving operators (test infrastructure only).

Plain NumPy, written from the definitions in include/ssa.h, one token, row and
page at a time; it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

E_MIN, E_MAX = -40, 120


def rotate(x, freq, positions, layout="half", mscale=1.0):
    """x [T, h, d] float64 with its first 2*len(freq) dims rotated."""
    x = np.array(x, dtype=np.float64)
    n = len(freq)
    for t, pos in enumerate(positions):
        for i in range(n):
            c, s = mscale * np.cos(float(pos) * freq[i]), mscale * np.sin(float(pos) * freq[i])
            u, v = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
            a, b = x[t, :, u].copy(), x[t, :, v].copy()
            x[t, :, u], x[t, :, v] = a * c - b * s, b * c + a * s
    return x


def norm(x, w=None, eps=1e-6):
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if w is None else y * np.asarray(w, dtype=np.float64)


# ---------------------------------------------------------------- e4m3

def e4m3_values():
    """The 256 codes' values (NaN at 0x7F and 0xFF)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def to_e4m3(x):
    """Codes of x rounded to nearest, ties to the even code; infinities and
    larger values to +-448, NaN to the NaN code."""
    x = np.asarray(x, dtype=np.float64)
    grid = e4m3_values()[:127]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(grid, np.where(np.isnan(a), 0, a), side="left")
    lo = np.maximum(hi - 1, 0)
    dh, dl = grid[hi] - a, a - grid[lo]
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.isnan(x), 127, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def exponent(x):
    """The least e with |x| <= 448 * 2^e for the finite x, clamped."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    a = a[np.isfinite(a)]
    top = a.max() if a.size else 0.0
    e = E_MIN
    while e < E_MAX and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(x, new_start, cached, table, page, codes, scale):
    """x [T, h, d] float64 appended to codes [n_pages, h, page, d] and scale
    [n_pages, h]; returns the new arrays and the number of tokens left out."""
    codes, scale, bad = codes.copy(), scale.copy(), 0
    val = e4m3_values()
    for s in range(len(cached)):
        rows = range(new_start[s], new_start[s + 1])
        if cached[s] < 0:
            bad += len(rows)
            continue
        by_page = {}
        for o, r in enumerate(rows):
            pos = int(cached[s]) + o
            by_page.setdefault(pos // page, []).append((pos % page, r))
        for pi, items in by_page.items():
            pid = table[s][pi] if pi < len(table[s]) else -1
            if pid < 0 or pid >= codes.shape[0]:
                bad += len(items)
                continue
            first = min(sl for sl, _ in items)
            for h in range(codes.shape[1]):
                e = exponent([x[r, h] for _, r in items])
                if first > 0:
                    old = int(round(np.log2(float(scale[pid, h]))))
                    if e > old:
                        codes[pid, h, :first] = to_e4m3(val[codes[pid, h, :first]] * 2.0 ** (old - e))
                    e = max(e, old)
                for sl, r in items:
                    codes[pid, h, sl] = to_e4m3(x[r, h] * 2.0 ** -e)
                scale[pid, h] = 2.0 ** e
    return codes, scale, bad


# ---------------------------------------------------------------- attention

def attend(q, k, v, scale):
    """One row: (o, lse) of softmax(scale q.k) over the given keys."""
    if len(k) == 0:
        return np.zeros(v.shape[-1]), -np.inf
    s = scale * (k @ q)
    m = s.max()
    p = np.exp(s - m)
    return p @ v / p.sum(), m + np.log(p.sum())


def used_blocks(row, pos, page):
    """The block_idx entries that count: fully visible and larger than every
    earlier in-range entry; and how many are skipped."""
    used, top, skipped = [], -1, 0
    for c in row:
        if c >= 0 and (c + 1) * page - 1 <= pos:
            if c > top:
                used.append(int(c))
            else:
                skipped += 1
            top = max(top, c)
        elif c != -1:
            skipped += 1
    return used, skipped


def cache_attention(q, table, kv_len, page, codes_k, codes_v, scale_k, scale_v, scale, block_idx=None, window=0):
    """q [n, n_q, h_q, d]; returns (o, lse)."""
    n, n_q, h_q, d = q.shape
    n_pages, h_kv = scale_k.shape
    G = h_q // h_kv
    val = e4m3_values()
    o = np.zeros((n, n_q, h_q, d))
    lse = np.full((n, n_q, h_q), -np.inf)
    for s in range(n):
        L = min(max(int(kv_len[s]), 0), table.shape[1] * page)
        for i in range(n_q):
            pos = L - n_q + i
            for h in range(h_kv):
                if block_idx is None:
                    keys = list(range(pos + 1))
                else:
                    used, _ = used_blocks(block_idx[s, i, h], pos, page)
                    keys = sorted({j for c in used for j in range(c * page, (c + 1) * page)}
                                  | set(range(max(pos - window + 1, 0), pos + 1)))
                keys = [j for j in keys if 0 <= table[s][j // page] < n_pages]
                pid = np.array([table[s][j // page] for j in keys], dtype=int)
                sl = np.array([j % page for j in keys], dtype=int)
                kk = val[codes_k[pid, h, sl]] * scale_k[pid, h].astype(np.float64)[:, None]
                vv = val[codes_v[pid, h, sl]] * scale_v[pid, h].astype(np.float64)[:, None]
                for g in range(G):
                    o[s, i, h * G + g], lse[s, i, h * G + g] = attend(q[s, i, h * G + g], kk, vv, scale)
    return o, lse


def prompt_attention(q, k, v, q_start, kv_start, scale):
    """Packed causal attention; rows outside every sequence are NaN."""
    T, h_q, d = q.shape
    G = h_q // k.shape[1]
    o, lse = np.full((T, h_q, d), np.nan), np.full((T, h_q), np.nan)
    for s in range(len(q_start) - 1):
        q0, q1, k0, k1 = q_start[s], q_start[s + 1], kv_start[s], kv_start[s + 1]
        for r in range(q0, q1):
            n = max(r - q0 + (k1 - k0) - (q1 - q0) + 1, 0)
            for h in range(h_q):
                o[r, h], lse[r, h] = attend(q[r, h], k[k0:k0 + n, h // G], v[k0:k0 + n, h // G], scale)
    return o, lse
