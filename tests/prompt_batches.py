"""Packed batches over a paged cache, and the error bounds of their results."""
import numpy as np

from workloads import randn_bf16

NAN = np.uint16(0x7FC0)


class Batch:
    """new[s] packed query rows on held[s] tokens in the cache; every slot of
    the pool that holds no token of the batch is NaN."""

    def __init__(self, seed, new, held, hq, hkv, bt, first_row=0, rows_behind=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.held, self.hq, self.hkv, self.bt = new, held, hq, hkv, bt
        self.scale = 1.0 / np.sqrt(128.0)
        blocks = [-(-c // bt) for c in held]
        self.width = max(1, max(blocks))
        nb = sum(blocks) + 3
        order = rng.permutation(nb).astype(np.int32)
        self.k = np.full((nb, hkv, bt, 128), NAN, np.uint16)
        self.v = np.full((nb, hkv, bt, 128), NAN, np.uint16)
        self.tables = np.full((len(held), self.width), -1, np.int32)
        at = 0
        for s, c in enumerate(held):
            row = order[at : at + blocks[s]]
            self.tables[s, : blocks[s]] = row
            at += blocks[s]
            t = np.arange(c)
            self.k[row[t // bt], :, t % bt] = randn_bf16(rng, (c, hkv, 128))
            self.v[row[t // bt], :, t % bt] = randn_bf16(rng, (c, hkv, 128))
        self.starts = (first_row + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        self.ctx = np.array(held, np.int32)
        T = int(self.starts[-1]) + rows_behind
        q = randn_bf16(rng, (T, hq, 128))
        if spread != 1.0:
            q = bits_of(floats(q) * np.float32(spread))
        self.q = q
        self.kd = randn_bf16(rng, (T, hkv, 128))
        self.vd = randn_bf16(rng, (T, hkv, 128))
        self.masks = np.zeros(T, np.int64)
        for s, n in enumerate(new):
            rows = []
            for i in range(n):
                p = int(rng.integers(-1, i)) if i else -1
                rows.append((rows[p] if p >= 0 else 0) | (1 << i & (1 << 64) - 1))
            self.masks[self.starts[s] : self.starts[s + 1]] = [r - (1 << 64) if r >> 63 else r for r in rows]

    def slot(self, s, position):
        return self.tables[s, position // self.bt], position % self.bt


def floats(bits):
    return (bits.astype(np.uint32) << np.uint32(16)).view(np.float32)


def bits_of(x):
    from workloads.gen import bf16_bits
    return bf16_bits(np.ascontiguousarray(x, np.float32))


def bound(ref):
    """Largest error of a bf16 result against the float64 (out, a, e):
    - the result's rounding, half a step: 2^-8 |o|;
    - each weight rounded to bf16 before the product with the values, half a
      step of each term: 2^-8 a;
    - fp32 scores of 128 products: off by at most 128 * 2^-24 e, which the
      exponential turns into the same relative error of a weight, in the
      numerator and in the sum: 2 * 2^-17 e a;
    - the exponential, the sums and the joins of partial results in fp32: a
      few 2^-22 for each of at most some thousand terms, within 2^-10 a."""
    out, a, e = ref
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -16 * e[..., None]) * a
