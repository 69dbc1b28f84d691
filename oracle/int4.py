"""A cache held in 4 bits, restated.

Per group of G of a row's 128 values, in fp32 with one rounding per step:
    lo, hi = least and greatest value, held to +-65504
    m = fp16(lo), s = fp16((hi - lo) / 15)
    c = rint((x - m) / s), held to 0 .. 15 (0 where s is 0)
and the row stands for s c + m. A NaN makes its group's s and m NaN.

pack() lays a block's rows out in bytes: slabs of 16 tokens (8 where the block has
no more), in each the KV heads, in each of these units of 8 tokens, each
    key codes    word 4 c + w of a token's 16: dims 32 w + 8 c .. + 7
    value codes  16-bit piece (r, t / 2, w, t % 2): dims 32 w + 4 r .. + 3
    keys' (s, m) by token and group, values' s by group and token, values' m.
"""
from __future__ import annotations

import numpy as np

DIM = 128
HALF_MAX = np.float32(65504.0)


def quantise(x, group_dims: int):
    """x fp32 [..., 128] -> (codes uint8 [..., 128], s, m float16 [..., 128 / G])."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], DIM // group_dims, group_dims)
    nan = np.isnan(g).any(axis=-1)
    lo = np.clip(g.min(axis=-1), -HALF_MAX, HALF_MAX)
    hi = np.clip(g.max(axis=-1), -HALF_MAX, HALF_MAX)
    with np.errstate(all="ignore"):
        m = lo.astype(np.float16)
        s = ((hi - lo) / np.float32(15)).astype(np.float16)
        t = g - m.astype(np.float32)[..., None]
        c = np.rint(t / s.astype(np.float32)[..., None])
        c = np.where((s > 0)[..., None], np.clip(c, 0, 15), 0)
    c = np.where(nan[..., None], 0, c)
    s, m = np.where(nan, np.float16(np.nan), s), np.where(nan, np.float16(np.nan), m)
    return c.astype(np.uint8).reshape(x.shape), s, m


def values(codes, s, m):
    """float64 rows that the codes stand for."""
    g = codes.reshape(*codes.shape[:-1], s.shape[-1], -1).astype(np.float64)
    return (s.astype(np.float64)[..., None] * g + m.astype(np.float64)[..., None]).reshape(codes.shape)


def pack(k, v):
    """k, v: (codes, s, m) of rows [..., heads, tokens, 128] -> bytes [..., slabs, heads,
    slab tokens / 8 * unit]."""
    slab = min(16, k[0].shape[-2])
    by_slab = lambda x: np.moveaxis(x.reshape(*x.shape[:-2], -1, slab, x.shape[-1]), -3, -4)
    return _pack_rows([by_slab(x) for x in k], [by_slab(x) for x in v])


def _pack_rows(k, v):
    """Rows [..., tokens, 128] of one head -> bytes [..., tokens / 8 * unit]."""
    (kc, ks, km), (vc, vs, vm) = k, v
    lead, tokens, groups = kc.shape[:-2], kc.shape[-2], ks.shape[-1]
    u = tokens // 8

    def words(codes, bits):
        """Codes [..., n] of 4 bits into little-endian words of `bits`, lowest first."""
        n = bits // 4
        c = codes.reshape(*codes.shape[:-1], -1, n).astype(np.uint32)
        w = (c << (4 * np.arange(n, dtype=np.uint32))).sum(axis=-1, dtype=np.uint32)
        return w.astype({32: "<u4", 16: "<u2"}[bits])

    kw = words(kc, 32).reshape(*lead, u, 8, 4, 4)           # token, w, c
    kw = np.ascontiguousarray(np.swapaxes(kw, -1, -2)).reshape(*lead, u, -1)
    vw = words(vc, 16).reshape(*lead, u, 4, 2, 4, 8)        # t / 2, t % 2, w, r
    vw = np.ascontiguousarray(np.moveaxis(vw, (-1, -4, -2, -3), (-4, -3, -2, -1))).reshape(*lead, u, -1)
    kp = np.stack([ks, km], axis=-1).reshape(*lead, u, -1)  # token, group, (s, m)
    by_group = lambda p: np.ascontiguousarray(np.swapaxes(p.reshape(*lead, u, 8, groups), -1, -2)).reshape(*lead, u, -1)
    parts = [kw, vw, kp.astype("<f2"), by_group(vs).astype("<f2"), by_group(vm).astype("<f2")]
    return np.concatenate([np.ascontiguousarray(p).view(np.uint8) for p in parts], axis=-1).reshape(*lead, -1)


def decode(q, k, v, tables, ctx, scale):
    """Decode attention over such a cache. q float64 [B, Hq, 128]; k, v: (codes, s,
    m) of the pool's rows [blocks, Hkv, block tokens, 128]. Returns float64 (out,
    a, e): a = sum_j softmax(x)_j (s c + |m|)_j, the size of the values' terms,
    and e [B, Hq] = max_j |scale| * sum_d |q_d| (s c + |m|)_jd, that of the keys'."""
    B, Hq, _ = q.shape
    Hkv, bt = k[0].shape[1:3]
    G = Hq // Hkv
    out, a, e = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Hq))
    for b in range(B):
        n = int(ctx[b])
        if n <= 0:
            continue
        t = np.arange(n)
        at = np.asarray(tables[b])[t // bt]
        for g in range(Hkv):
            rows = [[x[at, g, t % bt] for x in kv] for kv in (k, v)]
            key, val = (values(*r) for r in rows)
            ksz, vsz = (values(c, s, np.abs(m)) for c, s, m in rows)
            h = slice(g * G, (g + 1) * G)
            x = scale * (q[b, h] @ key.T)
            with np.errstate(invalid="ignore"):
                w = np.exp(x - x.max(axis=-1, keepdims=True))
                w /= w.sum(axis=-1, keepdims=True)
                out[b, h], a[b, h] = w @ val, w @ vsz
                e[b, h] = (abs(scale) * (np.abs(q[b, h]) @ ksz.T)).max(axis=-1)
    return out, a, e
