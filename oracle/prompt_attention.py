"""Attention of many query rows per sequence, and the write path into the
cache, restated in float64.

Prompt rows (cs2680 Lecture 10, §10.3, step three, for more than one query):
row i of a sequence's n packed rows is the token at position p = ctx - n + i
and sees positions 0 .. p of the cache, read through the block table. Draft
rows see the whole context in the cache and, of their own sequence's packed
drafts, those whose mask bit is set. Either way

    x_j = scale * <q, k_j>,   o = sum_j exp(x_j - max x) v_j / sum_j exp(x_j - max x)

over the seen tokens only; a row that sees nothing gives zeros.

Beside the result each function returns, for error bounds, the weighted sum
of absolute values  a = sum_j softmax(x)_j |v_j|  and, per row, the largest
sum of absolute products  e = max_j scale * sum_d |q_d k_jd|.
"""
from __future__ import annotations

import numpy as np

from .paged_attention import gather_tokens, widen_bf16


def _rows(q, keys, values, seen, scale):
    """q [n, D], keys / values [t, D], seen [n, t] -> (o, a [n, D], e [n])."""
    n, d = q.shape
    o, a, e = np.zeros((n, d)), np.zeros((n, d)), np.zeros(n)
    for i in range(n):
        j = np.flatnonzero(seen[i])
        if j.size == 0:
            continue
        x = scale * (keys[j] @ q[i])
        w = np.exp(x - x.max())
        w /= w.sum()
        with np.errstate(invalid="ignore"):
            o[i] = w @ values[j]
            a[i] = w @ np.abs(values[j])
        e[i] = scale * (np.abs(keys[j]) @ np.abs(q[i])).max()
    return o, a, e


def _attend(q, k_cache, v_cache, tables, ctx, starts, scale, drafts=None):
    T, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    out, absum, spread = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    qf = widen_bf16(q)
    for s in range(len(ctx)):
        lo, hi, c = int(starts[s]), int(starts[s + 1]), int(ctx[s])
        n = hi - lo
        if n == 0:
            continue
        if drafts is None:
            seen = np.arange(c)[None, :] <= (c - n + np.arange(n))[:, None]
        else:
            bits = [int(m) for m in drafts[2][lo:hi]]
            tree = np.array([[bool(b >> j & 1) for j in range(n)] for b in bits])
            seen = np.concatenate([np.ones((n, c), dtype=bool), tree], axis=1)
        for g in range(Hkv):
            keys = gather_tokens(k_cache, tables[s], c, g)
            values = gather_tokens(v_cache, tables[s], c, g)
            if drafts is not None:
                keys = np.concatenate([keys, widen_bf16(drafts[0][lo:hi, g])])
                values = np.concatenate([values, widen_bf16(drafts[1][lo:hi, g])])
            for h in range(g * G, (g + 1) * G):
                out[lo:hi, h], absum[lo:hi, h], spread[lo:hi, h] = _rows(qf[lo:hi, h], keys, values, seen, scale)
    return out, absum, spread


def prompt_attention(q, k_cache, v_cache, block_tables, context_lens, query_starts, scale):
    """bf16 bit patterns in; float64 (out, a [T, Hq, D], e [T, Hq])."""
    return _attend(q, k_cache, v_cache, block_tables, context_lens, query_starts, scale)


def tree_attention(q, k_draft, v_draft, masks, k_cache, v_cache, block_tables, context_lens, query_starts, scale):
    return _attend(q, k_cache, v_cache, block_tables, context_lens, query_starts, scale, (k_draft, v_draft, masks))


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """x: bits [T, H, D]; weight: bits [D] or None; cos_sin fp32 [P, R]."""
    y = widen_bf16(x)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * widen_bf16(weight)
    if cos_sin is None:
        return y
    half = cos_sin.shape[1] // 2
    cos = cos_sin[positions, :half].astype(np.float64)[:, None, :]
    sin = cos_sin[positions, half:].astype(np.float64)[:, None, :]
    out = y.copy()
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = y[..., first], y[..., second]
    out[..., first] = a * cos - b * sin
    out[..., second] = a * sin + b * cos
    return out
