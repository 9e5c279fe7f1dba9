"""The history cache and its attention in fp64 (TEST INFRASTRUCTURE ONLY; only
the tests may import this module).

The cache holds MX-quantised keys and values (oracle/mx.py's E4M3 format) in
pages; what is computed over it is block attention's rule for events that
are added to a history (include/ba.h, ba_cache and the calls after it):
slots by page table, page means, pages selected by mean key, and attention of
new rows (chains, trees, candidates). Everything is evaluated row by row and
slot by slot from that text. Pins: tests/test_oracle_cache.py.
"""
from __future__ import annotations

import numpy as np

from oracle import mx as MX


def e4m3_values(codes):
    """E4M3 codes (uint8) as numbers, from sign, exponent and mantissa fields."""
    c = np.asarray(codes).astype(np.int64)
    ef, m = (c >> 3) & 15, c & 7
    v = np.where(ef > 0, (1 + m / 8.0) * np.exp2(ef - 7.0), m / 8.0 * 2.0 ** -6)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def dequantize(codes, scales):
    """Rows [..., D] of codes with scale codes [..., D / 32] as numbers."""
    return e4m3_values(codes) * np.repeat(np.exp2(scales.astype(np.float64) - 127), 32, axis=-1)


def quantize(x):
    """(element values [..., D], scale exponents [..., D / 32]) of finite rows."""
    el, sc = MX.quantize(x, "e4m3")
    return el.reshape(np.shape(x)), np.log2(sc[..., 0]).astype(np.int64)


class Cache:
    """Dequantised pools and page table."""

    def __init__(self, k, v, k_scales, v_scales, page_table):
        self.k, self.v = dequantize(k, k_scales), dequantize(v, v_scales)   # [pages, heads, size, D]
        self.table = np.asarray(page_table)
        self.size = k.shape[2]

    def slot(self, b, p):
        """(page, row) of slot p of sequence b, or None where it has none."""
        if p < 0 or p // self.size >= self.table.shape[1]:
            return None
        page = int(self.table[b, p // self.size])
        return (page, p % self.size) if 0 <= page < self.k.shape[0] else None


def window_start(pos, block, window):
    return max(0, pos // block - (window - 1)) * block


def bit(words, i):
    """Bit i of a row of int32 / uint32 words (False past its end)."""
    return i // 32 < len(words) and bool((int(words[i // 32]) >> (i % 32)) & 1)


def visible(cache, b, h, n, t, length, pos, block, window, tree=None, mask=None):
    """Slots that row t (of n rows at positions pos) of sequence b sees for key/value head h.
    tree: words [n, w] or None; mask: words [n, heads, w] or None."""
    if pos[t] < 0:
        return []
    ws = window_start(pos[t], block, window)
    seen = [p for p in range(min(length, pos[t] + 1))
            if p >= ws or (mask is not None and bit(mask[t][h], p // cache.size))]
    seen += [length + j for j in range(n)
             if ws <= pos[j] <= pos[t] and (j <= t if tree is None else bit(tree[t], j))]
    return [p for p in seen if cache.slot(b, p) is not None]


def attend(cache, q, q_offsets, lens, block, window, positions=None, tree=None, mask=None):
    """(out [rows, heads, D], lse [heads, rows], spread [rows, heads, D], reach [heads, rows]): spread is
    sum p |v|, reach the largest sum_d |q_d k_d| / sqrt(D) over a row's slots (for error bounds)."""
    rows, heads, D = q.shape
    kv_heads = cache.k.shape[1]
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach = np.full((heads, rows), -np.inf), np.zeros((heads, rows))
    for b in range(len(lens)):
        lo, hi = int(q_offsets[b]), int(q_offsets[b + 1])
        n, length = hi - lo, max(int(lens[b]), 0)
        pos = [length + t for t in range(n)] if positions is None else [int(x) for x in positions[lo:hi]]
        for t in range(n):
            for h in range(kv_heads):
                seen = visible(cache, b, h, n, t, length, pos, block, window,
                               None if tree is None else tree[lo:hi], None if mask is None else mask[lo:hi])
                if not seen:
                    continue
                at = [cache.slot(b, p) for p in seen]
                pages, at = [x[0] for x in at], [x[1] for x in at]
                k, v = cache.k[pages, h, at], cache.v[pages, h, at]
                for x in range(h * heads // kv_heads, (h + 1) * heads // kv_heads):
                    s = k @ q[lo + t, x] / np.sqrt(D)
                    top = np.max(s)
                    p = np.exp(s - top)
                    lse[x, lo + t] = top + np.log(np.sum(p))
                    p /= np.sum(p)
                    out[lo + t, x], spread[lo + t, x] = p @ v, p @ np.abs(v)
                    reach[x, lo + t] = np.max(np.abs(k) @ np.abs(q[lo + t, x])) / np.sqrt(D)
    return out, lse, spread, reach


def summarize(cache, starts, ends, into):
    """Mean keys of the full pages that hold a slot in [start, end), written into `into`."""
    for b in range(len(starts)):
        for c in range(cache.table.shape[1]):
            full = (c + 1) * cache.size <= ends[b]
            touched = (c + 1) * cache.size > max(int(starts[b]), 0)
            where = cache.slot(b, c * cache.size)
            if full and touched and where is not None:
                into[where[0]] = cache.k[where[0]].mean(axis=1)
    return into


def select(cache, q, q_offsets, lens, summaries, block, window, topk, positions=None):
    """Selected pages as truth values [rows, heads, max_pages]."""
    rows, heads, _ = q.shape
    kv_heads, P = cache.k.shape[1], cache.table.shape[1]
    got = np.zeros((rows, kv_heads, P), dtype=bool)
    for b in range(len(lens)):
        for row in range(int(q_offsets[b]), int(q_offsets[b + 1])):
            length = max(int(lens[b]), 0)
            pos = length + row - int(q_offsets[b]) if positions is None else int(positions[row])
            if pos < 0:
                continue
            ws = window_start(pos, block, window)
            cand = [c for c in range(P) if c * cache.size < ws and (c + 1) * cache.size <= length
                    and cache.slot(b, c * cache.size) is not None]
            for h in range(kv_heads):
                g = heads // kv_heads
                qs = q[row, h * g:(h + 1) * g].sum(axis=0)
                score = {c: float(qs @ summaries[cache.slot(b, c * cache.size)[0], h]) for c in cand}
                order = sorted(cand, key=lambda c: (np.isnan(score[c]), -score[c] if score[c] == score[c] else 0.0, c))
                got[row, h, order[:topk]] = True
    return got


def words(bits):
    """Truth values [..., n] as int32 words [..., ceil(n / 32)]."""
    n = bits.shape[-1]
    pad = np.concatenate([bits, np.zeros(bits.shape[:-1] + (-n % 32,), dtype=bool)], axis=-1)
    w = (pad.reshape(pad.shape[:-1] + (-1, 32)).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(axis=-1)
    return w.astype(np.uint32).view(np.int32)
