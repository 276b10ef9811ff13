"""Oracle for the rotary positions and the paged 4-bit key/value cache: plain
numpy in 64 bits, written from the formulas.

TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no code
with ``gguf_block_quant_gq_amd``. Pinned by ``tests/test_oracle_kv4.py``.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def norm(x, w, eps):
    """x_c w_c / sqrt(mean_c x_c^2 + eps) over the last axis, in 64 bits."""
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * np.asarray(w, np.float64)


def rope(x, pos, freqs, interleaved=False, mscale=1.0, w=None, eps=1e-6):
    """Heads x [tokens, heads, head_dim] normed (w given) and rotated to pos."""
    y = np.array(x, np.float64) if w is None else norm(x, w, eps)
    half = len(freqs)
    angle = np.asarray(pos, np.float64)[:, None] * np.asarray(freqs, np.float32).astype(np.float64)
    m = float(np.float32(mscale))
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        c, s = np.cos(angle[:, p])[:, None], np.sin(angle[:, p])[:, None]
        u, v = y[..., i].copy(), y[..., j].copy()
        y[..., i], y[..., j] = m * (u * c - v * s), m * (v * c + u * s)
    return y


def scale_of(a):
    """The scale of a block whose value of largest magnitude is a."""
    if np.isnan(a):
        return np.nan
    d = -a / 8.0
    if d == 0.0:
        return 0.0
    if abs(d) > 8160.0:
        return np.copysign(8160.0, d)
    step = max(2.0 ** (np.frexp(d)[1] - 8), 2.0 ** -24)   # 8 significant bits
    return float(np.clip(np.rint(d / step) * step, -8160.0, 8160.0))


def quantise(x):
    """(d [..., blocks], codes 0..15 [..., channels]) of x [..., channels]."""
    x = np.asarray(x, np.float64)
    b = x.reshape(-1, BLOCK)
    d = np.empty(len(b))
    codes = np.full(b.shape, 8, np.uint8)
    for r, row in enumerate(b):
        bad = np.flatnonzero(np.isnan(row))
        a = row[bad[0]] if len(bad) else row[np.argmax(np.abs(row))]   # the first of equals
        d[r] = scale_of(a)
        if d[r] != 0.0 and not np.isnan(d[r]):
            codes[r] = np.clip(np.rint(row / d[r]), -8, 7) + 8
    return d.reshape(*x.shape[:-1], -1), codes.reshape(x.shape)


def values(d, codes):
    return (codes.astype(np.float64) - 8.0) * np.repeat(d, BLOCK, -1)


def nibble(c):
    """Where channel c of eight sits in its dword."""
    return (c >> 1) + 4 * (c & 1)


def page_bytes(page_tokens, n_kv, hd):
    return page_tokens * n_kv * (hd + hd // 8)


def _part(page_tokens, hd, head, kv):
    return (2 * head + kv) * page_tokens * (hd // 2 + hd // 16)


def store(pages, page, slot, P, hd, head, kv, x):
    """One head's key (kv = 0) or value (1) into a page (pages: uint8 [n, bytes])."""
    d, codes = quantise(x)
    at = _part(P, hd, head, kv)
    for wd in range(hd // 8):
        word = 0
        for c in range(8):
            word |= int(codes[8 * wd + c]) << (4 * nibble(c))
        o = at + slot * (hd // 2) + 4 * wd
        pages[page, o: o + 4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
    for blk in range(hd // BLOCK):
        o = at + P * hd // 2 + 2 * (blk * P + slot)
        pages[page, o: o + 2] = np.frombuffer(np.float16(d[blk]).tobytes(), np.uint8)


def load(pages, page, slot, P, hd, head, kv):
    """The held values of one head's key or value, in 64 bits."""
    at = _part(P, hd, head, kv)
    words = np.frombuffer(pages[page, at + slot * (hd // 2): at + (slot + 1) * (hd // 2)].tobytes(), "<u4")
    codes = np.array([[(int(wd) >> (4 * nibble(c))) & 15 for c in range(8)] for wd in words]).reshape(-1)
    d = [np.frombuffer(pages[page, at + P * hd // 2 + 2 * (b * P + slot):][:2].tobytes(), "<f2")[0]
         for b in range(hd // BLOCK)]
    return values(np.array(d, np.float64), codes)


def rows(q_start, lens, n_tok):
    """(sequence, position) of every row, None where it has none."""
    n_seq = len(lens)
    if q_start is None:
        q_start = np.arange(n_seq + 1)
    out = [None] * n_tok
    for b in range(n_seq):
        lo, hi = int(q_start[b]), int(q_start[b + 1])
        for t in range(lo, hi):
            out[t] = (b, int(lens[b]) - (hi - lo) + t - lo)
    return out


def unpack(pages, P, n_kv, hd):
    """load() of every slot at once: [pages, P, n_kv, 2, hd]."""
    n = len(pages)
    parts = pages.reshape(n, n_kv, 2, -1)
    words = np.ascontiguousarray(parts[..., : P * hd // 2]).view("<u4").reshape(n, n_kv, 2, P, hd // 8)
    codes = np.stack([(words >> np.uint32(4 * nibble(c))) & 15 for c in range(8)], -1).reshape(n, n_kv, 2, P, hd)
    d = np.ascontiguousarray(parts[..., P * hd // 2:]).view("<f2").reshape(n, n_kv, 2, hd // BLOCK, P)
    return values(np.swapaxes(d, -1, -2).astype(np.float64), codes).transpose(0, 3, 1, 2, 4)


def sequence(pages, table, b, n, P, n_kv, hd):
    """K and V [n, n_kv, hd] of sequence b's first n tokens; NaN where the
    page number is not one."""
    kv = np.full((2, n, n_kv, hd), np.nan)
    for i in range(-(-n // P)):
        page, m = int(table[b, i]), min(P, n - i * P)
        if 0 <= page < len(pages):
            x = unpack(pages[page: page + 1], P, n_kv, hd)[0, :m]
            kv[:, i * P: i * P + m] = x.transpose(2, 0, 1, 3)
    return kv[0], kv[1]


def attention(q, pos, length, K, V, scale, causal=True, window=0):
    """One row's heads q [heads, hd] at position pos over K, V [length, n_kv,
    hd]: (out, sum_j w_j |v_j| / sum_j w_j, largest sum_c |q_c k_c| scale)."""
    q = np.asarray(q, np.float64)
    heads, hd = q.shape
    out, mag, big = np.zeros((heads, hd)), np.zeros((heads, hd)), np.zeros(heads)
    hi = min(length, pos + 1) if causal else length
    lo = max(0, pos + 1 - window) if window > 0 else 0
    if hi <= lo:
        return out, mag, big
    for h in range(heads):
        g = h // (heads // K.shape[1])
        k, v = K[lo:hi, g], V[lo:hi, g]
        s = scale * (k @ q[h])
        w = np.exp(s - s.max())
        w /= w.sum()
        out[h], mag[h] = w @ v, w @ np.abs(v)
        big[h] = abs(scale) * (np.abs(k) @ np.abs(q[h])).max()
    return out, mag, big
