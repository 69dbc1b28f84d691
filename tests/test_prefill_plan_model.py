"""The work partition of prompt and tree attention as arithmetic, on the host.

The kernel lays the batch's items -- up to two query tiles of one (sequence,
KV head) against their key tiles -- end to end by cost and cuts the line into
one range per CTA; a cut near an item's end, or in a short item, moves to an
end, any other splits the item's key tiles. Every CTA finds its two ends from
the prefix sum with float estimates that it corrects, walks its range, and the
join enumerates the pieces of a split item from the item's place alone. This
model restates those steps and checks them: every key tile of every item is in
exactly one piece, the estimates give the plain search's item, and the join
sees the pieces that the walks made."""
import math

import numpy as np
import pytest

KEYS, COST_TWO, SNAP, WHOLE, MIN_RANGE = 128, 8, 8 * 256, 8 * 768, 8 * 256
F = np.float32


class Line:
    def __init__(self, lens, hkv, group, tree, one, grid):
        """lens: (query rows, context) of each sequence."""
        self.lens, self.hkv, self.tree, self.grid = lens, hkv, tree, grid
        self.tpt = 128 // group
        self.tokens = self.tpt if one else 2 * self.tpt
        self.cost_one = 8 if tree else 6
        self.cost_item = 8 * 200 if tree else 8 * 290
        self.full_cost = self.cost_one if one else COST_TWO
        self.total = hkv * sum(self.head(s) for s in range(len(lens)))
        ranges = min(grid, max(self.total // MIN_RANGE, 1))
        self.chunk = int(F(F(np.nextafter(F(self.total), F(np.inf)) / F(ranges)) * F(1.000001))) + 1

    def cost(self, s):
        n, ctx = self.lens[s]
        keys = ctx + KEYS if self.tree else max(ctx - n, 0)
        b = 0 if self.tree else self.full_cost * self.tokens // 2
        rest = n % self.tokens
        last = ((COST_TWO if rest > self.tpt else self.cost_one) * (keys if self.tree else ctx) + self.cost_item) if rest else 0
        return self.full_cost * keys + self.cost_item + b, b, last

    def first(self, s, i):
        a, b, _ = self.cost(s)
        return i * (a + b * i)

    def head(self, s):
        return self.first(s, self.lens[s][0] // self.tokens) + self.cost(s)[2]

    def items(self, s):
        return -(-self.lens[s][0] // self.tokens)

    def item(self, s, i):
        """(cost, key tiles for the cut)."""
        n, ctx = self.lens[s]
        full = n // self.tokens
        c = self.first(s, i + 1) - self.first(s, i) if i < full else self.cost(s)[2]
        kend = ctx if self.tree else max(ctx - n + min((i + 1) * self.tokens, n), 0)
        return c, max(-(-kend // KEYS) + (1 if self.tree else 0), 1)

    def cut_tile(self, off, cost, nt):
        if off <= SNAP or (cost <= WHOLE and 2 * off < cost):
            return 0
        if cost - off <= SNAP or cost <= WHOLE:
            return nt
        return min(max(int(F(F(F(off) / F(cost)) * F(nt)) + F(0.5)), 0), nt)

    def cut(self, x):
        """The kernel's search: (sequence, head, item, tile, item start), or None behind the line."""
        at = 0
        for s in range(len(self.lens)):
            hc = self.head(s)
            if x >= at + hc * self.hkv:
                at += hc * self.hkv
                continue
            off = x - at
            h = min(int(F(off) / F(hc)), self.hkv - 1)
            off -= hc * h
            if off < 0:
                off, h = off + hc, h - 1
            elif off >= hc:
                off, h = off - hc, h + 1
            assert 0 <= off < hc and 0 <= h < self.hkv  # one correction is enough
            a, b, _ = self.cost(s)
            i = min(int(F(2) * F(off) / F(F(a) + F(math.sqrt(F(F(a) * F(a) + F(4) * F(b) * F(off)))))), self.items(s) - 1)
            steps = 0
            while self.first(s, i) > off:
                i, steps = i - 1, steps + 1
            while i < self.items(s) - 1 and self.first(s, i + 1) <= off:
                i, steps = i + 1, steps + 1
            assert steps <= 2  # the estimate is near
            start = x - off + self.first(s, i)
            c, nt = self.item(s, i)
            assert 0 <= x - start < c
            return s, h, i, self.cut_tile(x - start, c, nt), start
        return None

    def pieces(self, b):
        """CTA b's walk: (sequence, head, item, first tile, end tile)."""
        lo, hi = self.cut(self.chunk * b), self.cut(self.chunk * (b + 1))
        if lo is None:
            return []
        out = []
        for s in range(lo[0], len(self.lens)):
            for h in range(lo[1] if s == lo[0] else 0, self.hkv):
                for i in range(lo[2] if (s, h) == lo[:2] else 0, self.items(s)):
                    key = (s, h, i)
                    ta = lo[3] if key == lo[:3] else 0
                    nt = self.item(s, i)[1]
                    if ta >= nt:
                        continue
                    if hi is not None and key > hi[:3]:
                        return out
                    tb = hi[3] if hi is not None and key == hi[:3] else nt
                    if tb <= ta:
                        return out
                    out.append((s, h, i, ta, tb))
        return out

    def joined(self, c0):
        """The ranges and tiles the join enumerates for the item whose first piece CTA c0 has, if its end cuts one."""
        hi = self.cut(self.chunk * (c0 + 1))
        if hi is None:
            return None
        s, h, i, t, start = hi
        c, nt = self.item(s, i)
        if not 0 < t < nt:
            return None
        x0 = self.chunk * c0
        if not (x0 <= start or self.cut_tile(x0 - start, c, nt) == 0):
            return None
        got, at, r = [], 0, c0
        while at < nt:
            end = self.chunk * (r + 1) - start
            e = nt if end >= c else self.cut_tile(end, c, nt)
            if e > at:
                got.append((r, at, e))
            at, r = max(at, e), r + 1
        return (s, h, i), got


def _lens(rng, n, tree, most, ctx):
    out = []
    for _ in range(n):
        c = int(np.exp(rng.uniform(0, np.log(ctx))))
        q = int(rng.integers(0, min(most, 64) + 1)) if tree else int(rng.integers(0, min(c, most) + 1))
        out.append((q, c))
    return out


CASES = [
    # lens, hkv, group, tree, one, grid
    ([(37, 37)], 8, 4, False, False, 152),
    ([(16411, 16411)], 8, 8, False, False, 152),
    ([(0, 5), (0, 0)], 4, 1, False, False, 152),
    ([(5, 200000), (1, 1), (0, 7), (64, 3)], 2, 8, True, True, 152),
    ([(60, 131072)], 1, 8, True, False, 152),
    ([(1, 1 + s % 5) for s in range(500)], 1, 2, False, True, 152),
    ([(33, 30), (700, 700), (1, 9000)], 3, 3, False, False, 7),
    ([(1500, 26003), (700, 9001), (0, 17), (300, 300)], 8, 8, False, False, 3 * 152),  # three ranges a CTA
]
for k in range(12):
    r = np.random.default_rng(k)
    tree = bool(k & 1)
    CASES.append((_lens(r, int(r.integers(1, 40)), tree, 1500, 40000), int(r.choice([1, 2, 8])), int(r.choice([1, 4, 5, 7, 8])),
                  tree, bool(k & 2), int(r.choice([1, 13, 152]))))


@pytest.mark.parametrize("case", range(len(CASES)))
def test_every_key_tile_in_one_piece_and_the_join_sees_them_all(case):
    line = Line(*CASES[case])
    assert line.chunk * line.grid >= line.total
    seen, of = {}, {}
    for b in range(line.grid):
        for s, h, i, ta, tb in line.pieces(b):
            assert seen.get((s, h, i), 0) == ta  # in order, without a gap
            seen[(s, h, i)] = tb
            of.setdefault((s, h, i), []).append((b, ta, tb))
    want = {(s, h, i): line.item(s, i)[1] for s in range(len(line.lens)) for h in range(line.hkv) for i in range(line.items(s))}
    assert seen == want
    joins = {}
    for b in range(line.grid):
        j = line.joined(b)
        if j is not None:
            assert j[0] not in joins
            joins[j[0]] = j[1]
    assert joins == {k: p for k, p in of.items() if len(p) > 1}


def ring_entry(two, pos, count):
    if two or pos == 0 or pos == 2 * count - 1:
        return bool(pos & 1), pos >> 1
    return (False, (pos >> 1) + 1) if pos & 1 else (True, (pos >> 1) - 1)


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("count", range(1, 12))
def test_ring_order_is_the_order_of_use(two, count):
    """The loader's order of a piece's tiles, and the places at which the
    issuer and the cleaning warps look for them."""
    order = [ring_entry(two, pos, count) for pos in range(2 * count)]
    assert sorted(order) == [(v, j) for v in (False, True) for j in range(count)]
    for j in range(count):
        assert order[2 * j if two else max(2 * j - 1, 0)] == (False, j)
        assert order[2 * j + 1 if two or j == count - 1 else 2 * j + 2] == (True, j)
    # the issuer's steps: first S of each stream, then P V of a tile with S of the stream's next one
    uses = []
    cnt = [count, count] if two else [(count + 1) // 2, count // 2]
    for turn in range(-2, 2 * max(cnt)):
        stream, i = turn & 1, turn >> 1
        j = i if two else 2 * i + stream
        if 0 <= i < cnt[stream]:
            uses.append((True, j))
        if i + 1 < cnt[stream]:
            uses.append((False, j + (1 if two else 2)))
    firsts = list(dict.fromkeys(uses))
    assert firsts == order


def test_item_division_is_exact():
    """n / tokens by a multiplication with ceil(2^36 / tokens), for every size of
    an item and row counts up to the limit."""
    rng = np.random.default_rng(1)
    for group in range(1, 9):
        for tokens in {128 // group, 2 * (128 // group)}:
            magic = ((1 << 36) + tokens - 1) // tokens
            ns = [0, 1, tokens - 1, tokens, tokens + 1, (1 << 28) - 1] + rng.integers(0, 1 << 28, size=3000).tolist()
            ns += [k * tokens + d for k in rng.integers(1, (1 << 28) // tokens, size=2000).tolist() for d in (-1, 0)]
            for n in ns:
                assert (n * magic) >> 36 == n // tokens
                assert n * magic < 1 << 64
