"""The rules by which the host and the device decide alike about a call of
prompt or tree attention, and the model's constants against the kernel's.

The host launches no join where no item can be cut, going by the keys that the
tables hold; the device cuts items by their cost. So an item may cost no more
than the keys that the tables hold, whatever its rows -- those of a chunk that is
longer than its context (an error of the caller's, whose other rows are
computed) among them."""
import ctypes
import os
import re
import subprocess

import pytest

from tests import test_prefill_plan_model as model

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_49_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


KERNEL = _source("pkv_prefill_kernel.cuh")


def _number(pattern):
    """The value of a product of whole numbers in the kernel's source."""
    found = re.findall(pattern, KERNEL)
    assert len(found) == 1, (pattern, found)
    value = 1
    for f in found[0].split("*"):
        value *= int(f)
    return value


def test_the_models_constants_are_the_kernels():
    assert model.COST_TWO == _number(r"constexpr int kCostTwo = ([\d* ]+);")
    assert model.SNAP == _number(r"constexpr int kSnap = ([\d* ]+);")
    assert model.WHOLE == _number(r"constexpr int kWhole = ([\d* ]+);")
    assert model.MIN_RANGE == _number(r"constexpr int kMinRange = ([\d* ]+);")
    assert model.KEYS == _number(r"constexpr int kKeys = ([\d* ]+);")
    for tree in (True, False):
        line = Line([(1, 1)], 1, 1, tree, False, 1)
        one = r"cost_one\(bool tree\) \{ return tree \? (?:[\d* ]+) : ([\d* ]+); \}"
        item = r"cost_item\(bool tree\) \{ return tree \? (?:[\d* ]+) : ([\d* ]+); \}"
        if tree:
            one, item = (x.replace("(?:", "(").replace(": ([", ": (?:[") for x in (one, item))
        assert line.cost_one == _number(one) and line.cost_item == _number(item)


class Line(model.Line):
    """The work line with the price of a chunk longer than its context: every
    item as if it saw the whole of it."""

    def cost(self, s):
        n, ctx = self.lens[s]
        if self.tree or n <= ctx:
            return super().cost(s)
        rest = n % self.tokens
        last = ((model.COST_TWO if rest > self.tpt else self.cost_one) * ctx + self.cost_item) if rest else 0
        return self.full_cost * ctx + self.cost_item, 0, last


def _joins(line, capacity):
    """The host's rule: whether the join is launched, by the keys of a table."""
    most = capacity + (model.KEYS if line.tree else 0)
    return model.COST_TWO * most + line.cost_item > model.WHOLE


def _split(line):
    """{item: pieces} of the items that the walks of all ranges cut."""
    pieces = {}
    for b in range(line.grid):
        for s, h, i, ta, tb in line.pieces(b):
            pieces.setdefault((s, h, i), []).append((b, ta, tb))
    return {k: p for k, p in pieces.items() if len(p) > 1}


# (query rows, context) of each sequence, KV heads, group, blocks of a table row, tokens of a block
LONGER = [
    ([(600, 448)], 8, 4, 28, 16),
    ([(2000, 448)], 8, 4, 28, 16),
    ([(700, 256)], 8, 8, 16, 16),
    ([(900, 0), (40, 30)], 2, 1, 4, 8),
    ([(5, 400), (5000, 448), (1, 448)], 8, 8, 7, 64),
    ([(5000, 1), (300, 300)], 1, 8, 40, 8),
]


@pytest.mark.parametrize("lens,hkv,group,width,bt", LONGER)
@pytest.mark.parametrize("one", [False, True])
@pytest.mark.parametrize("grid", [7, 152])
def test_no_item_is_cut_where_no_join_is_launched(lens, hkv, group, width, bt, one, grid):
    line = Line(lens, hkv, group, False, one, grid)
    if not _joins(line, width * bt):
        assert not _split(line)
    for s in range(len(lens)):
        for i in range(line.items(s)):
            assert line.item(s, i)[0] <= model.COST_TWO * width * bt + line.cost_item


def test_the_price_that_was_too_high_is_seen():
    """With each item priced by its rows, these were cut and never joined."""
    for lens, hkv, group, width, bt in LONGER[:3]:
        line = model.Line(lens, hkv, group, False, False, 152)
        assert not _joins(line, width * bt) and _split(line)


@pytest.mark.parametrize("case", range(len(LONGER)))
@pytest.mark.parametrize("grid", [13, 152])
def test_chunks_longer_than_their_context_are_partitioned(case, grid):
    """Every key tile in one piece, and the join sees the pieces of every cut item."""
    lens, hkv, group, _, _ = LONGER[case]
    lens = lens + [(3, 20000), (400, 9000), (9000, 7000)]
    line = Line(lens, hkv, group, False, False, grid)
    seen, of = {}, {}
    for b in range(line.grid):
        for s, h, i, ta, tb in line.pieces(b):
            assert seen.get((s, h, i), 0) == ta
            seen[(s, h, i)] = tb
            of.setdefault((s, h, i), []).append((b, ta, tb))
    assert seen == {(s, h, i): line.item(s, i)[1] for s in range(len(lens)) for h in range(hkv) for i in range(line.items(s))}
    joins = {}
    for b in range(line.grid):
        j = line.joined(b)
        if j is not None:
            joins[j[0]] = j[1]
    assert joins == {k: p for k, p in of.items() if len(p) > 1}


@pytest.mark.parametrize("tree,lens,width,bt", [
    (False, [(s % 40, 40 + s) for s in range(400)], 32, 16),
    (True, [(s % 65, s) for s in range(400)], 28, 16),
    (True, [(64, 440)] * 200, 55, 8),
])
def test_ordinary_batches_on_short_tables_are_never_cut(tree, lens, width, bt):
    for one in (False, True):
        line = Line(lens, 4, 4, tree, one, 152)
        if not _joins(line, width * bt):
            assert not _split(line)


def _cut_out(start, end):
    at = KERNEL.index(start)
    return KERNEL[at : KERNEL.index(end, at) + len(end)]


@pytest.fixture(scope="module")
def priced(tmp_path_factory):
    """The kernel's own pricing and cut, compiled for the host."""
    where = tmp_path_factory.mktemp("prices")
    parts = [
        "#include <algorithm>\nusing std::max; using std::min;\n"
        "#define __device__\n#define __host__\n#define __forceinline__ inline\n"
        "static float __ll2float_rn(long long x) { return static_cast<float>(x); }\n",
        _cut_out("constexpr int kKeys =", ";"), _cut_out("constexpr int kCostTwo", "kMinRange = 8 * 256;"),
        _cut_out("struct Seq {", "};"), _cut_out("template <bool kOne>\n__device__ __forceinline__ int item_tokens", "}"),
        _cut_out("struct Cost {", "\n};"),
        _cut_out("template <bool kTree, bool kOne>\n__device__ __forceinline__ Cost cost_of", "\n}\n"),
        _cut_out("__device__ __forceinline__ int cut_tile", "\n}\n"),
        """
template <bool kTree, bool kOne>
static void price(const Seq& q, int tpt, long long* out) {
    const Cost c = cost_of<kTree, kOne>(q, tpt);
    out[0] = c.a, out[1] = c.b, out[2] = c.last;
}
extern "C" void price(int tree, int one, int n, int ctx, int tpt, long long* out) {
    const int tokens = one ? tpt : 2 * tpt;
    const Seq q = {n, ctx, 0, n / tokens, n % tokens};
    tree ? one ? price<true, true>(q, tpt, out) : price<true, false>(q, tpt, out)
         : one ? price<false, true>(q, tpt, out) : price<false, false>(q, tpt, out);
}
extern "C" int cut(long long off, long long cost, int tiles) { return cut_tile(off, cost, tiles); }
"""]
    src, lib = where / "price.cpp", where / "price.so"
    src.write_text("\n".join(parts))
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    return ctypes.CDLL(str(lib))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("one", [False, True])
def test_the_model_prices_items_as_the_kernel_does(priced, tree, one):
    lens = [(n, ctx) for n in (1, 5, 31, 64, 128, 129, 700, 5000) for ctx in (0, 1, 30, 128, 448, 5000, 70001)]
    out = (ctypes.c_longlong * 3)()
    for group in range(1, 9):
        line = Line(lens, 1, group, tree, one, 152)
        for s, (n, ctx) in enumerate(lens):
            priced.price(tree, one, n, ctx, line.tpt, out)
            a, b, last = line.cost(s)
            assert (out[0], out[2]) == (a, last), (n, ctx, group)
            assert out[1] == b
    for off in range(0, 20000, 331):
        for cost, tiles in ((6000, 4), (6145, 4), (9000, 7), (20011, 19)):
            got = priced.cut(ctypes.c_longlong(off), ctypes.c_longlong(cost), tiles)
            assert got == line.cut_tile(off, cost, tiles)
