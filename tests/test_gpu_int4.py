"""The 4-bit cache's kernels against the oracle: bytes and loaded pages exactly,
attention within bounds that count its roundings."""
import numpy as np
import pytest
import torch

from oracle import int4
from oracle.paged_attention import widen_bf16
from workloads import randn_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tests.conftest import build_native
    build_native()
    import paged_kv_cache_49_gb300 as m
    return m


def _f32(bits):
    return (bits.astype(np.uint32) << np.uint32(16)).view(np.float32)


def _rows(rng, shape, offset=1.0):
    """bf16 bits of values whose channels differ in mean."""
    x = torch.from_numpy(widen_bf16(randn_bf16(rng, shape)) + offset * rng.standard_normal(shape[1:]))
    return x.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _dev(pkv, bits):
    return pkv.bf16_from_bits(bits).cuda()


def _bf16(x):
    """float64 -> the bits of its rounding to fp32, then to bf16."""
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


class Pool:
    """A cache whose slots have all been written, and what it holds."""

    def __init__(self, pkv, rng, blocks, hkv, bt, gd, k=None, v=None):
        self.cache = pkv.Int4Cache(blocks, hkv, bt, gd)
        shape = (blocks * bt, hkv, 128)
        self.k_bits, self.v_bits = (_rows(rng, shape, o) if x is None else x for x, o in ((k, 1.0), (v, 0.0)))
        self.slots = rng.permutation(blocks * bt)
        err = pkv.new_error_word()
        pkv.append_int4(_dev(pkv, self.k_bits), _dev(pkv, self.v_bits), torch.from_numpy(self.slots).cuda(), self.cache, err)
        assert pkv.read_device_error(err) == 0
        self.k, self.v = (self._paged(b, blocks, hkv, bt, gd) for b in (self.k_bits, self.v_bits))

    def _paged(self, bits, blocks, hkv, bt, gd):
        rows = np.empty((blocks * bt, hkv, 128), np.float32)
        rows[self.slots] = _f32(bits)
        return int4.quantise(rows.reshape(blocks, bt, hkv, 128).swapaxes(1, 2), gd)


# ---- append, load, copy -------------------------------------------------------


@pytest.mark.parametrize("gd", [32, 64, 128])
@pytest.mark.parametrize("bt", [8, 16, 32, 64])
def test_every_byte_of_a_pool(pkv, bt, gd):
    pool = Pool(pkv, np.random.default_rng(bt + gd), 5, 3, bt, gd)
    assert np.array_equal(pool.cache.data.cpu().numpy(), int4.pack(pool.k, pool.v))


@pytest.mark.parametrize("T,hkv,bt,gd", [(1, 1, 8, 128), (1, 8, 16, 64), (3, 1, 16, 32), (37, 2, 32, 64), (100, 5, 64, 128),
                                         (513, 8, 16, 64)])
def test_append_views_padding_and_neighbours(pkv, T, hkv, bt, gd):
    """Views of a fused projection; padding rows; bytes of other slots stay."""
    rng = np.random.default_rng(T)
    blocks = T // bt + 2
    kb, vb = _rows(rng, (T, hkv, 128)), _rows(rng, (T, hkv, 128))
    fused = torch.zeros((T, 3 * hkv, 128), dtype=torch.bfloat16, device="cuda")
    fused[:, hkv:2 * hkv], fused[:, 2 * hkv:] = _dev(pkv, kb), _dev(pkv, vb)
    slots = rng.permutation(blocks * bt)[:T]
    slots[::5] = -1 - np.arange(len(slots[::5]))
    cache = pkv.Int4Cache(blocks, hkv, bt, gd)
    before = rng.integers(0, 256, size=cache.data.shape, dtype=np.uint8)
    cache.data.copy_(torch.from_numpy(before))
    err = pkv.new_error_word()
    pkv.append_int4(fused[:, hkv:2 * hkv], fused[:, 2 * hkv:], torch.from_numpy(slots).cuda(), cache, err)
    assert pkv.read_device_error(err) == 0
    # what pack() makes of the new rows where they are, the old bytes elsewhere
    kept = slots >= 0
    marks, want = np.zeros(before.shape, np.uint8), before.copy()
    for name, fill in (("marks", True), ("rows", False)):
        parts = []
        for bits in (kb, vb):
            rows = np.zeros((blocks * bt, hkv, 128), np.float32)
            rows[slots[kept]] = _f32(bits)[kept]
            c, s, m = int4.quantise(rows.reshape(blocks, bt, hkv, 128).swapaxes(1, 2), gd)
            if fill:
                live = np.zeros(blocks * bt, bool)
                live[slots[kept]] = True
                live = live.reshape(blocks, 1, bt, 1)
                c = np.broadcast_to(np.where(live, 15, 0), c.shape).astype(np.uint8)
                ones = np.array(0xFFFF, np.uint16).view(np.float16)
                s = m = np.broadcast_to(np.where(live, ones, np.float16(0)), s.shape)
            parts.append((c, s, m))
        if fill:
            marks = int4.pack(*parts)
        else:
            want = np.where(marks == 0xFF, int4.pack(*parts), before)
    assert np.array_equal(cache.data.cpu().numpy(), want)


def test_append_edge_values(pkv):
    """Zeros, constants, infinities, NaN, tiny and huge ranges, exact halves."""
    x = np.zeros((16, 1, 128), np.float32)
    x[1] = 2.5
    x[2, 0, ::2] = np.inf
    x[3] = -np.inf
    x[4, 0, 5] = np.nan
    x[5, 0, 3] = 2.0 ** -30
    x[6, 0, 0], x[6, 0, 1] = -0.9375, 0.9375
    x[6, 0, 2:18] = -0.9375 + (np.arange(16) + 0.5) / 8
    x[7] = np.float32(3.0e38) * np.sign(np.arange(128) % 3 - 1.0)
    x[8] = np.arange(128) * np.float32(2.0 ** -24)
    x[9] = np.linspace(-1, 1, 128)
    x[10] = -np.linspace(0, 7, 128) ** 3
    x[11] = np.nan
    x[12, 0, :] = 65280.0
    x[12, 0, 64:] = -65280.0
    x[13] = 2.0 ** -14 * np.arange(128)
    x[14] = -0.0
    x[15, 0, 100] = -np.nan
    bits = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    for gd in (32, 64, 128):
        cache = pkv.Int4Cache(2, 1, 8, gd)
        pkv.append_int4(_dev(pkv, bits), _dev(pkv, bits[::-1].copy()), torch.arange(16, device="cuda"), cache)
        rows = [int4.quantise(_f32(b).reshape(2, 8, 1, 128).swapaxes(1, 2), gd) for b in (bits, bits[::-1])]
        got, want = cache.data.cpu().numpy(), int4.pack(*rows)
        params = np.r_[1024:got.shape[-1]]  # a NaN has many forms
        g, w = (a[..., params].copy().view(np.float16) for a in (got, want))
        assert np.array_equal(g, w, equal_nan=True)
        assert np.array_equal(got[..., :1024], want[..., :1024])


def test_codes_of_quotients_near_a_half(pkv):
    """Groups of few bf16 steps far from zero (scales from a thousandth to 1/30 of the
    values and less), groups that step by halves of their scale, wide ones: bytes exactly."""
    rng = np.random.default_rng(77)
    n, gd = 16384, 64
    kinds = np.arange(n) % 4
    steps = rng.integers(1, 64, n)[:, None]
    few = 128.0 + rng.integers(0, 96, (n, 1)) + rng.integers(0, 64, (n, gd)) % (steps + 1)  # of 256 steps up to 256
    halves = rng.integers(0, 31, (n, gd)) * 0.5
    halves[:, 0], halves[:, 1] = 0, 15  # a scale of one: every other value on a half
    wide = rng.standard_normal((n, gd)) * 2.0 ** rng.integers(-6, 6, (n, gd))
    values = np.choose(kinds[:, None], [few, halves, wide, -few]) * 2.0 ** rng.integers(-10, 8, (n, 1))
    x = torch.from_numpy(values.reshape(2, n // 16, 4, 128)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    pool = Pool(pkv, rng, n // 16 // 16, 4, 16, gd, x[0], x[1])
    assert np.array_equal(pool.cache.data.cpu().numpy(), int4.pack(pool.k, pool.v))


@pytest.mark.parametrize("gd", [32, 64, 128])
@pytest.mark.parametrize("bt", [8, 16, 32, 64])
def test_load_is_the_values_rounded_once(pkv, bt, gd):
    rng = np.random.default_rng(3)
    pool = Pool(pkv, rng, 7, 3, bt, gd)
    pairs = np.array([[6, 0], [0, 4], [3, 1], [3, 2]], np.int32)
    k, v = (torch.full((6, 3, bt, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = pkv.new_error_word()
    pkv.load_int4(pool.cache, torch.from_numpy(pairs).cuda(), k, v, err)
    assert pkv.read_device_error(err) == 0
    for got, held in ((k, pool.k), (v, pool.v)):
        got, want = pkv.bits_from_bf16(got), _bf16(int4.values(*held))
        assert np.array_equal(got[pairs[:, 1]], want[pairs[:, 0]])
        assert (_f32(got[[3, 5]]) == 7.0).all()


def test_load_and_copy_of_nothing_and_of_bad_pairs(pkv):
    rng = np.random.default_rng(4)
    pool = Pool(pkv, rng, 4, 2, 16, 64)
    k, v = (torch.full((3, 2, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    none = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    before = pool.cache.data.clone()
    pkv.load_int4(pool.cache, none, k, v)
    pkv.block_copy_int4(pool.cache, none)
    err = pkv.new_error_word()
    for bad in ([[0, 3]], [[4, 0]], [[-1, 0]], [[0, -2]]):
        pkv.load_int4(pool.cache, torch.tensor(bad, dtype=torch.int32, device="cuda"), k, v, err)
        assert pkv.read_device_error(err) == pkv.DEVERR_BLOCK_ID
    for bad in ([[0, 4]], [[4, 0]], [[-1, 0]], [[0, -2]]):
        pkv.block_copy_int4(pool.cache, torch.tensor(bad, dtype=torch.int32, device="cuda"), err)
        assert pkv.read_device_error(err) == pkv.DEVERR_BLOCK_ID
    assert (k == 7).all() and (v == 7).all() and torch.equal(before, pool.cache.data)
    # a bad slot, among good ones
    rows = _dev(pkv, _rows(rng, (3, 2, 128)))
    pkv.append_int4(rows, rows, torch.tensor([5, 64, -1], device="cuda"), pool.cache, err)
    assert pkv.read_device_error(err) == pkv.DEVERR_SLOT
    assert torch.equal(before[1:], pool.cache.data[1:]) and not torch.equal(before[0], pool.cache.data[0])


@pytest.mark.parametrize("bt,gd,hkv", [(8, 128, 1), (16, 64, 8), (64, 32, 3)])
def test_copies_of_blocks(pkv, bt, gd, hkv):
    rng = np.random.default_rng(5)
    cache = pkv.Int4Cache(9, hkv, bt, gd)
    before = rng.integers(0, 256, size=cache.data.shape, dtype=np.uint8)
    cache.data.copy_(torch.from_numpy(before))
    pkv.block_copy_int4(cache, torch.tensor([[0, 8], [0, 3], [5, 1]], dtype=torch.int32, device="cuda"))
    before[[8, 3, 1]] = before[[0, 0, 5]]
    assert np.array_equal(cache.data.cpu().numpy(), before)


# ---- decode attention ---------------------------------------------------------


def _near(got, want, a, e, n):
    """bf16 out against float64. In turn: the output's rounding, 2^-8 of it; the
    weights' rounding to fp16 (2^-11, in the values' sum and in the denominator)
    and that of weight times scale (2^-11): 3 * 2^-11 of a; a score off by 2^-17
    of the size of its terms e (128 products and the groups' sums in fp32), which
    moves weight and denominator alike: 2 * 2^-17 e a; exp2 and the fp32 sums:
    2^-14 a; weights below fp16's range, 2^-24 each at most: n 2^-24 of the
    largest value, which a / 2^-24 bounds where it counts -- n 2^-20 max a."""
    big = a.max(axis=-1, keepdims=True)
    tol = 2.0 ** -8 * np.abs(want) + a * (3 * 2.0 ** -11 + 2.0 ** -16 * e[..., None] + 2.0 ** -14)
    tol += np.asarray(n, float)[:, None, None] * 2.0 ** -20 * big
    g = _f32(got).astype(np.float64)
    assert np.isfinite(g).all() and (np.abs(g - want) <= tol).all(), (np.abs(g - want) - tol).max()


def _batch(rng, lens, blocks, bt):
    """Tables over a shuffled pool; unused entries are bad ids, never read."""
    per = [-(-n // bt) for n in lens]
    order = rng.permutation(blocks)
    width = max(max(per), 1) + 1
    tables = np.full((len(lens), width), -7, np.int32)
    at = 0
    for i, n in enumerate(per):
        tables[i, :n] = order[at:at + n]
        at += n
    assert at <= blocks
    return tables


def _poison(pool, tables, lens, bt):
    """NaN scales and full codes behind every context and in unused blocks."""
    d = pool.cache.data
    blocks, hkv = d.shape[0], d.shape[2]
    live = np.zeros((blocks, bt), bool)
    for row, n in zip(tables, lens):
        t = np.arange(n)
        live[row[t // bt], t % bt] = True
    live = np.broadcast_to(live[:, None], (blocks, hkv, bt))
    c = np.where(live[..., None], 15, 0).astype(np.uint8).repeat(128, axis=-1)
    ones = np.array(0xFFFF, np.uint16).view(np.float16)
    p = np.where(live[..., None], ones, np.float16(0)).repeat(pool.k[1].shape[-1], axis=-1)
    keep = torch.from_numpy(int4.pack((c, p, p), (c, p, p)) == 0xFF).cuda()
    d.copy_(torch.where(keep, d, torch.full_like(d, 0xFF)))


def _decode(pkv, rng, lens, hq, hkv, bt=16, gd=64, num_ctas=0, q_scale=1.0, scale=128 ** -0.5, poison=True, pool=None, ws=None):
    blocks = sum(-(-n // bt) for n in lens) + 3
    pool = pool or Pool(pkv, rng, blocks, hkv, bt, gd)
    tables = _batch(rng, lens, blocks, bt)
    if poison:
        _poison(pool, tables, lens, bt)
    q = torch.from_numpy(q_scale * rng.standard_normal((len(lens), hq, 128))).to(torch.bfloat16)
    ws = ws or pkv.AttentionWorkspace(len(lens), hkv)
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    args = (q.cuda(), pool.cache, torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), scale)
    got = pkv.attn_decode_int4(*args, out=out, workspace=ws, num_ctas=num_ctas)
    assert got.data_ptr() == out.data_ptr() and ws.read_error() == 0
    want, a, e = int4.decode(q.double().numpy(), pool.k, pool.v, tables, lens, scale)
    _near(pkv.bits_from_bf16(got), want, a, e, lens)
    return args, ws, got


@pytest.mark.parametrize("gd", [32, 64, 128])
@pytest.mark.parametrize("bt", [8, 16, 32, 64])
def test_ragged_lengths(pkv, bt, gd):
    lens = [1, 0, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 129, 255, 257, 700]
    _decode(pkv, np.random.default_rng(bt * gd), lens, 8, 2, bt, gd)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (8, 1), (5, 5), (14, 2), (24, 4), (32, 8), (64, 8), (16, 16)])
def test_head_layouts(pkv, hq, hkv):
    _decode(pkv, np.random.default_rng(hq), [1, 77, 300, 0, 513], hq, hkv)


@pytest.mark.parametrize("gd", [32, 64, 128])
@pytest.mark.parametrize("bt", [8, 32, 64])
@pytest.mark.parametrize("hkv", [1, 6, 8, 12])
def test_heads_blocks_and_groups_together(pkv, hkv, bt, gd):
    """Runs of one, two and four heads (one warp, two, all of a head), of one run
    and of several a sequence, cut at a few places."""
    _decode(pkv, np.random.default_rng(hkv + bt + gd), [1, 200, 65, 0, 130, 23], 2 * hkv, hkv, bt, gd, num_ctas=5)


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7, 64, 151, 152, 300, 304])
def test_every_grid(pkv, num_ctas):
    """Pieces of all kinds: a context cut among many CTAs, CTAs of many contexts.
    (Grids that the workspace has no room for are refused.)"""
    _decode(pkv, np.random.default_rng(num_ctas), [1500, 3, 0, 40, 4097, 16], 8, 2, num_ctas=num_ctas)


def test_one_long_context(pkv):
    _decode(pkv, np.random.default_rng(8), [40001], 8, 1)


def test_many_short_contexts(pkv):
    rng = np.random.default_rng(9)
    _decode(pkv, rng, rng.integers(0, 41, size=1000).tolist(), 4, 1, bt=8)


def test_the_largest_batch(pkv):
    rng = np.random.default_rng(10)
    _decode(pkv, rng, rng.integers(0, 20, size=4096).tolist(), 2, 1)


@pytest.mark.parametrize("q_scale", [2.0 ** -30, 2.0 ** -9, 30.0, 2.0 ** 17])
def test_queries_of_any_size(pkv, q_scale):
    """Scores of the usual size: what the queries gain the scale gives back."""
    _decode(pkv, np.random.default_rng(11), [50, 300], 8, 2, q_scale=q_scale, scale=128 ** -0.5 / q_scale)


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.6])
def test_scales(pkv, scale):
    _decode(pkv, np.random.default_rng(12), [50, 1000], 8, 2, scale=scale)


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -6, 300.0, 5000.0])
def test_values_of_any_size(pkv, size):
    """Small and large values: their scales span most of fp16."""
    rng = np.random.default_rng(13)
    v = (size * rng.standard_normal((25 * 16, 2, 128))).astype(np.float32)
    v[::3] *= np.float32(1 / 64)
    v = torch.from_numpy(v).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    _decode(pkv, rng, [300, 33], 8, 2, pool=Pool(pkv, rng, 25, 2, 16, 64, v=v))


def _attend(pkv, pool, tables, lens, q, scale, **kw):
    """(out float64, the oracle's) of q float64, which bf16 holds."""
    ws = pkv.AttentionWorkspace(len(lens), pool.cache.num_kv_heads)
    got = pkv.attn_decode_int4(torch.from_numpy(q).to(torch.bfloat16).cuda(), pool.cache, torch.from_numpy(tables).cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, workspace=ws, **kw)
    assert ws.read_error() == 0
    return _f32(pkv.bits_from_bf16(got)).astype(np.float64), int4.decode(q, pool.k, pool.v, tables, lens, scale)


def _bf16_rows(x):
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("size", [1.0, 60000.0])
def test_scores_of_any_size(pkv, size, sign):
    """Scores from 2^15 to 2^34, a factor of 1.4 at a time, so far apart that each row
    is one token's value: no weight leaves fp16 where fp32 scores are 16 apart. What
    may differ: the output's rounding, 2^-8 of it, and that of weight times scale,
    2^-11 of the value's terms."""
    rng = np.random.default_rng(24)
    lens = [40, 333]
    v = size * np.clip(rng.standard_normal((30 * 16, 2, 128)), -1.05, 1.05)
    pool = Pool(pkv, rng, 30, 2, 16, 64, v=_bf16_rows(v).view(torch.int16).numpy().view(np.uint16))
    tables = _batch(rng, lens, 30, 16)
    q = _bf16_rows(rng.standard_normal((2, 16, 128))).double().numpy()
    for step in range(38):
        scale = sign * 2.0 ** (10 + step / 2)
        got, (want, a, e) = _attend(pkv, pool, tables, lens, q, scale)
        # rows whose two best scores differ by less than fp32's rounding of their terms could be either's
        clear = np.ones(want.shape[:2], bool)
        for b, n in enumerate(lens):
            t = np.arange(n)
            for h in range(16):
                key = int4.values(*(x[tables[b][t // 16], h // 8, t % 16] for x in pool.k))
                best = np.sort(scale * (key @ q[b, h]))[-2:]
                clear[b, h] = best[1] - best[0] > 2.0 ** -16 * abs(e).max() + 20
        assert clear.mean() > 0.9
        assert np.isfinite(got).all(), (scale, np.isnan(got).any(axis=-1))
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * a)[clear].all(), scale


def _dropped(scale):
    """What fp16 drops of a weight (of 1 at most) times a value's scale, given the largest
    scale up to a factor of 2: 2^-25 of products that are held times 2^10, and times
    2^11 more where all scales are below 2^-6; times 2^2 where they reach 32."""
    return 2.0 ** -46 if scale < 2.0 ** -7 else 2.0 ** -35 if scale < 16 else 2.0 ** -27


@pytest.mark.parametrize("gd", [32, 64, 128])
@pytest.mark.parametrize("top", [2.0 ** -16, 2.0 ** -13, 2.0 ** -8, 1.0])
def test_many_small_weights_beside_a_large_one(pkv, top, gd):
    """One token of weight 1 and 2^15 of 2^-15, all in one warp's piece, with values up
    to `top`: half of the output is theirs, weight times scale far below 2^-14."""
    rng = np.random.default_rng(25)
    n, hkv = 1 + (1 << 15), 4
    blocks = -(-n // 64)
    k, v = np.zeros((blocks * 64, hkv, 128), np.float32), np.zeros((blocks * 64, hkv, 128), np.float32)
    v[:] = top * (np.arange(128) * 37 % 128) / 127
    bits = lambda x: _bf16_rows(x).view(torch.int16).numpy().view(np.uint16)
    at = 7001  # the token of weight 1: value zero
    pool = Pool(pkv, rng, blocks, hkv, 64, gd, bits(k), bits(v))
    tables = np.arange(blocks, dtype=np.int32)[None]
    key = np.zeros((1, hkv, 128), np.float32)
    key[:, :, 0] = 1.0
    kb, vb = _bf16_rows(key), _bf16_rows(0 * key)
    pkv.append_int4(kb.cuda(), vb.cuda(), torch.tensor([at], device="cuda"), pool.cache)
    for held, x in ((pool.k, kb), (pool.v, vb)):
        for dst, src in zip(held, int4.quantise(x.float().numpy(), gd)):
            dst[at // 64, :, at % 64] = src[0]
    q = np.zeros((1, 2 * hkv, 128))
    q[:, ::2, 0], q[:, 1::2, 0] = 8.0, 16.0  # (and of 2^-30)
    got, (want, a, e) = _attend(pkv, pool, tables, [n], q, 15 * np.log(2) / 8, num_ctas=1)
    # roundings as in _near(), and what fp16 drops: of n weights 2^-25 of 2^10 each, times
    # value and output; of n products as _dropped() says, times codes up to 15.
    tol = 2.0 ** -8 * np.abs(want) + a * (3 * 2.0 ** -11 + 2.0 ** -16 * e[..., None] + 2.0 ** -14)
    tol += n * (15 * _dropped(top / 15) + 2.0 ** -34 * top)
    assert want[0, 0].max() > 0.45 * top and (np.abs(got - want) <= tol).all(), (np.abs(got - want) - tol).max() / top


@pytest.mark.parametrize("num_ctas", [0, 1])
@pytest.mark.parametrize("growing", [True, False])
def test_values_that_grow_along_a_context(pkv, growing, num_ctas):
    """Tiles whose values' scales rise or fall from 2^-19 to 2^12 along a context of
    equal weights, so that what the sums are held in units of changes on the way."""
    rng = np.random.default_rng(26)
    n = 4001
    blocks = -(-n // 16) + 3
    tables = _batch(rng, [n], blocks, 16)
    v = np.clip(rng.standard_normal((blocks * 16, 2, 128)), -1, 1).astype(np.float32)
    size = 2.0 ** (-19 + 34 * np.arange(n) / n)
    slot = tables[0][np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
    pool = Pool(pkv, rng, blocks, 2, 16, 64)
    v[:n] *= (size if growing else size[::-1])[:, None, None].astype(np.float32)
    k0, v0 = torch.zeros((n, 2, 128)).to(torch.bfloat16), _bf16_rows(v[:n])
    pkv.append_int4(k0.cuda(), v0.cuda(), torch.from_numpy(slot).cuda(), pool.cache)
    for held, x in ((pool.k, k0), (pool.v, v0)):
        for dst, src in zip(held, int4.quantise(x.float().numpy(), 64)):
            dst[slot // 16, :, slot % 16] = src
    q = _bf16_rows(rng.standard_normal((1, 8, 128))).double().numpy()
    for m in (n, 16, 100, 1000, 3000):  # (growing: of the small ones alone)
        got, (want, a, e) = _attend(pkv, pool, tables, [m], q, 0.1, num_ctas=num_ctas)
        tol = 2.0 ** -8 * np.abs(want) + a * (3 * 2.0 ** -11 + 2.0 ** -14)
        big = (size if growing else size[::-1])[:m].max()
        tol += 15 * _dropped(big / 7.5)  # of m products, each of weight 1 / m
        assert (np.abs(got - want) <= tol).all(), (m, (np.abs(got - want) - tol).max())


@pytest.mark.parametrize("lens,hq,hkv,num_ctas", [([40_001], 8, 1, 0), ([40_001], 8, 1, 512), ([131_072], 16, 4, 0),
                                                  ([4097, 0, 1500], 8, 2, 7), ([4097, 0, 1500], 8, 2, 64),
                                                  ([4097, 0, 1500], 8, 2, 152), ([4097, 0, 1500], 8, 2, 304)])
def test_no_stretch_of_a_context_is_lost(pkv, lens, hq, hkv, num_ctas):
    """Each of the values' dims stands for a stretch of the context: a result that leaves
    out, or counts twice, 1/300 of it is far from the bounds."""
    rng = np.random.default_rng(27)
    bt, gd = 16, 64
    blocks = sum(-(-n // bt) for n in lens) + 3
    pool = Pool(pkv, rng, blocks, hkv, bt, gd)
    tables = _batch(rng, lens, blocks, bt)
    slots, rows = [], []
    for b, n in enumerate(lens):
        t = np.arange(n)
        slots.append(tables[b][t // bt].astype(np.int64) * bt + t % bt)
        rows.append(0.2 * rng.random((n, hkv, 128)))
        rows[b][t, :, t * 128 // max(n, 1)] += 3.0
    slots, v = np.concatenate(slots), _bf16_rows(np.concatenate(rows))
    order = np.argsort(pool.slots)
    k_bits = pool.k_bits[order][slots]
    pkv.append_int4(_dev(pkv, k_bits), v.cuda(), torch.from_numpy(slots).cuda(), pool.cache)
    for dst, src in zip(pool.v, int4.quantise(v.float().numpy(), gd)):
        dst[slots // bt, :, slots % bt] = src
    q = _bf16_rows(0.3 * rng.standard_normal((len(lens), hq, 128))).double().numpy()
    got, (want, a, e) = _attend(pkv, pool, tables, lens, q, 0.09, num_ctas=num_ctas)
    # roundings as in _near(), and what fp16 drops of n weights and products
    most, span = float(pool.v[1].max()), float(np.abs(v.float().numpy()).max())
    tol = 2.0 ** -8 * np.abs(want) + a * (3 * 2.0 ** -11 + 2.0 ** -16 * e[..., None] + 2.0 ** -14)
    tol += np.array(lens)[:, None, None] * (15 * _dropped(most) + 2.0 ** -34 * span)
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) - tol).max()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        t = np.arange(n)
        at = tables[b][t // bt]
        for lo in (0, n // 2, n - n // 300):
            lost = (t >= lo) & (t < lo + n // 300)
            for times in (0.0, 2.0):  # left out, counted twice
                worst = 0.0
                for g in range(hkv):
                    key, val = (int4.values(*(x[at, g, t % bt] for x in kv)) for kv in (pool.k, pool.v))
                    h = slice(g * hq // hkv, (g + 1) * hq // hkv)
                    x = 0.09 * (q[b, h] @ key.T)
                    w = np.exp(x - x.max(axis=-1, keepdims=True)) * np.where(lost, times, 1.0)
                    wrong = w @ val / w.sum(axis=-1, keepdims=True)
                    worst = max(worst, (np.abs(wrong - want[b, h]) / tol[b, h]).max())
                assert worst > 5, (b, lo, times, worst)


@pytest.mark.parametrize("gd", [32, 64, 128])
@pytest.mark.parametrize("lens,hkv", [([131_072], 4), ([131_072], 1), ([60_000, 50_001], 2)])
def test_sums_of_long_pieces(pkv, lens, hkv, gd):
    """A whole context in one piece, of values about zero whose codes and minima are two
    large sums: the error over all outputs is that of independent roundings."""
    rng = np.random.default_rng(31)
    blocks = sum(-(-n // 64) for n in lens)
    pool = Pool(pkv, rng, blocks, hkv, 64, gd)
    tables = _batch(rng, lens, blocks, 64)
    q = _bf16_rows(rng.standard_normal((len(lens), 2 * hkv, 128))).double().numpy()
    got, (want, a, e) = _attend(pkv, pool, tables, lens, q, 0.05, num_ctas=1)
    # bf16: 2^-8 of an output at most, evenly spread. Weights, and their products with the
    # scales, in fp16: 2^-11 at most each, of terms whose squares' sum is that of n equal ones
    # times at most max p / mean p; three such roundings. What the matrix unit cuts off of an
    # fp32 sum: half a step of 2^-24 of it each time, over 8 turns of 4 tiles at most 32
    # times, the sum being half of its last value on average.
    for b, n in enumerate(lens):
        t = np.arange(n)
        spread = 0.0
        for g in range(hkv):
            key = int4.values(*(x[tables[b][t // 64], g, t % 64] for x in pool.k))
            x = 0.05 * (q[b, 2 * g:2 * g + 2] @ key.T)
            w = np.exp(x - x.max(axis=-1, keepdims=True))
            w /= w.sum(axis=-1, keepdims=True)
            spread = max(spread, np.sqrt((w ** 2).sum(axis=-1)).max())
        rms = lambda x: np.sqrt((x ** 2).mean())
        size = np.abs(a[b]).max()
        bound = np.hypot(2.0 ** -8 / 3 ** 0.5 * rms(want[b]), 3 * 2.0 ** -11 / 3 ** 0.5 * spread * size) + 32 * 2.0 ** -26 * size
        assert rms(got[b] - want[b]) <= bound, (rms(got[b] - want[b]), bound, rms(want[b]))


def test_nan_where_it_is_seen(pkv):
    """A NaN in a key reaches its heads, one in a group of a value those dims."""
    rng = np.random.default_rng(14)
    blocks, lens = 8, [60, 60]
    k, v = _rows(rng, (blocks * 16, 2, 128)), _rows(rng, (blocks * 16, 2, 128))
    pool = Pool(pkv, rng, blocks, 2, 16, 64, k, v)
    tables = _batch(rng, lens, blocks, 16)
    slot = lambda s, t: int(tables[s, t // 16]) * 16 + t % 16
    at = {int(x): i for i, x in enumerate(pool.slots)}
    k[at[slot(0, 59)], 1, 5] = 0x7FC0
    v[at[slot(1, 3)], 0, 70] = 0x7FC0
    pkv.append_int4(_dev(pkv, k), _dev(pkv, v), torch.from_numpy(pool.slots).cuda(), pool.cache)
    q = torch.from_numpy(rng.standard_normal((2, 8, 128))).to(torch.bfloat16).cuda()
    out = pkv.attn_decode_int4(q, pool.cache, torch.from_numpy(tables).cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1).isnan().cpu()
    assert out[0, 4:].all() and not out[0, :4].any()
    assert out[1, :4, 64:].all() and not out[1, :4, :64].any() and not out[1, 4:].any()


def test_bad_blocks_and_contexts_are_reported(pkv):
    rng = np.random.default_rng(15)
    pool = Pool(pkv, rng, 6, 2, 16, 64)
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    ws = pkv.AttentionWorkspace(2, 2)
    for bad in (6, -1, 1 << 30, -(1 << 31)):
        tables = torch.tensor([[0, bad], [1, 2]], dtype=torch.int32, device="cuda")
        pkv.attn_decode_int4(q, pool.cache, tables, torch.tensor([32, 32], dtype=torch.int32, device="cuda"), 0.1, workspace=ws)
        assert ws.read_error() == pkv.DEVERR_BLOCK_ID
    tables = torch.tensor([[0, 3], [1, 2]], dtype=torch.int32, device="cuda")
    pkv.attn_decode_int4(q, pool.cache, tables, torch.tensor([33, -5], dtype=torch.int32, device="cuda"), 0.1, workspace=ws)
    assert ws.read_error() == pkv.DEVERR_CONTEXT
    out = pkv.attn_decode_int4(q, pool.cache, tables, torch.tensor([0, -5], dtype=torch.int32, device="cuda"), 0.1, workspace=ws)
    assert ws.read_error() == 0 and not out.any()


def test_one_workspace_for_both_caches(pkv):
    """bf16 and 4-bit calls of different batches take turns on one workspace."""
    rng = np.random.default_rng(16)
    args, ws, first = _decode(pkv, rng, [900, 20, 333], 8, 2, num_ctas=100)
    first = first.clone()
    k = torch.randn((90, 2, 16, 128), device="cuda").to(torch.bfloat16)
    tables = torch.arange(90, dtype=torch.int32, device="cuda").view(3, 30)
    ctx = torch.tensor([480, 1, 77], dtype=torch.int32, device="cuda")
    other = pkv.attn_decode(args[0], k, k, tables, ctx, 0.1, workspace=ws).clone()
    for grid in (100, 1, 37):
        got = pkv.attn_decode_int4(*args, workspace=ws, num_ctas=grid)
        assert torch.equal(other, pkv.attn_decode(args[0], k, k, tables, ctx, 0.1, workspace=ws))
        if grid == 100:
            assert torch.equal(first, got)
    assert ws.read_error() == 0


def test_repeats_are_equal_to_the_bit(pkv):
    args, ws, first = _decode(pkv, np.random.default_rng(17), [5000, 64, 1, 900], 16, 2)
    first = first.clone()
    for _ in range(20):
        assert torch.equal(first, pkv.attn_decode_int4(*args, workspace=ws))


def test_streams_and_graphs(pkv):
    """Append and attention on a side stream, then captured; two graphs that share
    a workspace replayed in turn with new inputs."""
    rng = np.random.default_rng(18)
    args, ws, first = _decode(pkv, rng, [500, 70], 8, 2)
    q, cache, tables, ctx, scale = args
    first = first.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(first)
    for stream in (side, side.cuda_stream):
        pkv.attn_decode_int4(*args, out=out, workspace=ws, stream=stream)
        side.synchronize()
        assert torch.equal(out, first)
        out.zero_()
    rows = torch.randn((2, 2, 128), device="cuda").to(torch.bfloat16)
    t = tables.cpu().tolist()
    slots = torch.tensor([t[0][500 // 16] * 16 + 500 % 16, t[1][70 // 16] * 16 + 70 % 16], device="cuda")
    outs = [torch.zeros_like(first) for _ in range(2)]
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.append_int4(rows, rows, slots, cache)
            pkv.attn_decode_int4(q, cache, tables, ctx, scale, out=o, workspace=ws)
        graphs.append(g)
    ctx += 1
    for i in range(6):
        rows.copy_(torch.randn((2, 2, 128), device="cuda"))
        graphs[i % 2].replay()
        pkv.append_int4(rows, rows, slots, cache)
        assert torch.equal(outs[i % 2], pkv.attn_decode_int4(q, cache, tables, ctx, scale))
    assert ws.read_error() == 0


def test_calls_in_turn_without_a_wait(pkv):
    """Appends, loads, copies and attention, each launched while the one before may
    still run, read and write the same pages: a token at a time, the results of
    every call kept, against the same calls one by one."""
    rng = np.random.default_rng(21)
    n, hkv, bt = 48, 4, 16
    kb, vb = _rows(rng, (n, 300, hkv, 128)), _rows(rng, (n, 300, hkv, 128))
    k, v = _dev(pkv, kb), _dev(pkv, vb)
    q = torch.randn((n, 2, 16, 128), device="cuda").to(torch.bfloat16)
    slots = torch.arange(300, device="cuda")
    pairs = torch.tensor([[i, i + 1] for i in range(19)], dtype=torch.int32, device="cuda")
    copies = torch.tensor([[0, 20], [7, 21]], dtype=torch.int32, device="cuda")
    tables = torch.stack([torch.arange(19), 21 - torch.arange(19)]).int().cuda()
    ctx = torch.tensor([300, 290], dtype=torch.int32, device="cuda")

    def run(wait):
        cache, ws = pkv.Int4Cache(22, hkv, bt, 64), pkv.AttentionWorkspace(2, hkv)
        loaded = torch.zeros((n, 2, 20, hkv, bt, 128), dtype=torch.bfloat16, device="cuda")
        outs = torch.zeros_like(q)
        torch.cuda.synchronize()
        for i in range(n):
            for call in (lambda: pkv.append_int4(k[i], v[i], slots, cache), lambda: pkv.load_int4(cache, pairs, *loaded[i]),
                         lambda: pkv.block_copy_int4(cache, copies),
                         lambda: pkv.attn_decode_int4(q[i], cache, tables, ctx, 0.09, out=outs[i], workspace=ws)):
                call()
                if wait:
                    torch.cuda.synchronize()
        assert ws.read_error() == 0
        return loaded, outs

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_captured_behind_two_streams(pkv):
    """Every call captured where two streams meet: what they wrote is there."""
    rng = np.random.default_rng(22)
    args, ws, _ = _decode(pkv, rng, [500, 70], 8, 2, poison=False)
    q, cache, tables, ctx, scale = args
    kv = [torch.zeros((64, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    given = [torch.randn_like(t) for t in kv]
    slots = torch.arange(64, device="cuda")
    pairs = torch.tensor([[i, i] for i in range(4)], dtype=torch.int32, device="cuda")
    pools = [torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lens, out = torch.zeros_like(ctx), torch.zeros_like(q)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        kv[0].copy_(given[0])
        with torch.cuda.stream(side):
            kv[1].copy_(given[1])
            lens.copy_(ctx)
        main.wait_stream(side)
        pkv.append_int4(*kv, slots, cache)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            pkv.load_int4(cache, pairs, *pools)
        pkv.attn_decode_int4(q, cache, tables, lens, scale, out=out, workspace=ws)
        main.wait_stream(side)
    for _ in range(3):
        for t in given:
            t.copy_(torch.randn_like(t))
        g.replay()
        pkv.append_int4(*given, slots, cache)
        assert torch.equal(out, pkv.attn_decode_int4(*args))
        again = [torch.zeros_like(p) for p in pools]
        pkv.load_int4(cache, pairs, *again)
        for a, b in zip(pools, again):
            assert torch.equal(a, b)
            a.zero_()
        out.zero_()
        lens.zero_()
    assert ws.read_error() == 0


def test_two_calls_at_once(pkv):
    """On two streams, each with a workspace of its own, over one cache."""
    rng = np.random.default_rng(23)
    args, ws, first = _decode(pkv, rng, [3000, 64, 1, 900, 2000], 8, 2)
    first, other = first.clone(), pkv.AttentionWorkspace(5, 2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(first) for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for st, w, o in zip(streams, (ws, other), outs):
            pkv.attn_decode_int4(*args, out=o[i], workspace=w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(first, x) for o in outs for x in o) and ws.read_error() == other.read_error() == 0


def test_a_pool_past_four_gigabytes(pkv):
    """Offsets beyond 32 bits: blocks at both ends of a pool of 5.4 GB."""
    rng = np.random.default_rng(19)
    blocks = 300_000
    cache = pkv.Int4Cache(blocks, 8, 16, 64)
    ids = [blocks - 1, 0, 233_017, 240_000]
    kb, vb = _rows(rng, (64, 8, 128)), _rows(rng, (64, 8, 128))
    slots = np.concatenate([np.arange(16) + 16 * b for b in ids[:2] + ids[3:] + ids[2:3]])
    pkv.append_int4(_dev(pkv, kb), _dev(pkv, vb), torch.from_numpy(slots).cuda(), cache)
    pkv.block_copy_int4(cache, torch.tensor([[ids[0], 250_001]], dtype=torch.int32, device="cuda"))
    held = [int4.quantise(_f32(b).reshape(4, 16, 8, 128).swapaxes(1, 2), 64) for b in (kb, vb)]
    k, v = (torch.empty((2, 8, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.load_int4(cache, torch.tensor([[250_001, 1], [ids[2], 0]], dtype=torch.int32, device="cuda"), k, v)
    for got, h in ((k, held[0]), (v, held[1])):
        assert np.array_equal(pkv.bits_from_bf16(got), _bf16(int4.values(*h))[[3, 0]])
    q = torch.from_numpy(rng.standard_normal((1, 32, 128))).to(torch.bfloat16)
    lens = [61]
    got = pkv.attn_decode_int4(q.cuda(), cache, torch.tensor([[250_001, 0, 240_000, 233_017]], dtype=torch.int32, device="cuda"),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1)
    want, a, e = int4.decode(q.double().numpy(), *held, [[0, 1, 2, 3]], lens, 0.1)
    _near(pkv.bits_from_bf16(got), want, a, e, lens)


def test_grids_and_workspaces_at_their_limits(pkv):
    """512 CTAs and no more; as many as the bytes hold, fewer where the call may choose,
    and a share at least."""
    from paged_kv_cache_49_gb300 import _native as nat
    rng = np.random.default_rng(28)
    lens = [700, 0, 333]
    pool = Pool(pkv, rng, 70, 4, 16, 64)
    (q, cache, tables, ctx, scale), _, _ = _decode(pkv, rng, lens, 8, 4, pool=pool)
    oracle = int4.decode(q.double().cpu().numpy(), pool.k, pool.v, tables.cpu().numpy(), lens, scale)
    fixed, share = pkv.AttentionWorkspace.fixed_bytes(), 2 * 8 * 132 * 4  # (8 query rows a run)
    space = torch.zeros(fixed + 512 * share + 256, dtype=torch.uint8, device="cuda")
    at = -(-space.data_ptr() // 256) * 256

    def call(num_ctas, nbytes):
        out = torch.full_like(q, 9.0)
        st = nat.lib.pkv_attn_decode_int4(q.data_ptr(), cache.data.data_ptr(), tables.data_ptr(), tables.shape[1], ctx.data_ptr(), 3,
                                          8, 4, 128, cache.num_blocks, 16, 64, scale, num_ctas, at, nbytes, out.data_ptr(),
                                          torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert not space[at - space.data_ptr():][:256].any()  # the error word
        return st, out

    for num_ctas, shares in ((512, 512), (3, 3), (0, 3), (0, 1), (1, 1), (0, 512)):
        st, out = call(num_ctas, fixed + shares * share)
        assert st == nat.PKV_OK
        _near(pkv.bits_from_bf16(out), *oracle, lens)
    for num_ctas, nbytes in ((513, fixed + 512 * share), (4, fixed + 3 * share), (4, fixed + 4 * share - 1), (0, fixed + share - 1),
                             (1, fixed), (0, 0)):
        st, out = call(num_ctas, nbytes)
        assert st == nat.PKV_EINVAL and (out == 9).all()


def test_room_for_4_bit_calls_is_taken_by_them_alone(pkv):
    """A workspace has the bf16 calls' bytes until its first call over a 4-bit cache;
    what was captured before goes on in the bytes that it had, errors are read of both."""
    from paged_kv_cache_49_gb300 import _native as nat
    rng = np.random.default_rng(29)
    small = nat.lib.pkv_attn_workspace_size(3, 2) + 256
    large = max(small, nat.lib.pkv_attn_int4_workspace_size() + 256)
    args, _, want = _decode(pkv, rng, [900, 20, 333], 8, 2)
    want = want.clone()
    k = torch.randn((90, 2, 16, 128), device="cuda").to(torch.bfloat16)
    tables = torch.arange(90, dtype=torch.int32, device="cuda").view(3, 30)
    ctx = torch.tensor([480, 1, 77], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(want)
    ws = pkv.AttentionWorkspace(3, 2)
    bf16 = lambda **kw: pkv.attn_decode(args[0], k, k, tables, ctx, 0.1, workspace=ws, **kw)
    first = bf16().clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bf16(out=out)
    assert ws.buffer.numel() == small
    bad = ctx.clone()
    ctx[0] = 481  # past the table
    bf16()
    ctx.copy_(bad)
    assert torch.equal(want, pkv.attn_decode_int4(*args, workspace=ws)) and ws.buffer.numel() == large
    bad_tables = args[2].clone()
    bad_tables[1, 0] = -1
    pkv.attn_decode_int4(args[0], args[1], bad_tables, *args[3:], workspace=ws)
    assert ws.read_error() == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK_ID and ws.read_error() == 0
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, first) and torch.equal(bf16(), first)
        assert torch.equal(want, pkv.attn_decode_int4(*args, workspace=ws))
    # made with room: the same results, captured by the first call too
    ws = pkv.AttentionWorkspace(3, 2, int4=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.attn_decode_int4(*args, out=out, workspace=ws)
    out.zero_()
    g.replay()
    assert ws.buffer.numel() == large and torch.equal(out, want) and torch.equal(bf16(), first)
    # made without, and captured by the first call: in the bytes at hand, so of another
    # cut (two results off by 2^-8 of up to 1 and by 2^-9 of their terms each: under 0.02)
    ws = pkv.AttentionWorkspace(3, 2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.attn_decode_int4(*args, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert ws.buffer.numel() == small and (out.float() - want.float()).abs().max() < 0.02 and torch.equal(bf16(), first)
    assert torch.equal(want, pkv.attn_decode_int4(*args, workspace=ws)) and ws.buffer.numel() == large
    out.zero_()
    g.replay()
    assert (out.float() - want.float()).abs().max() < 0.02 and ws.read_error() == 0
    assert small <= 256 + nat.lib.pkv_attn_workspace_size(3, 2) < large


def test_engines_take_room_for_their_cache_alone(pkv):
    """Of 16 and of 4 bits: the workspaces of steps and of captured steps."""
    from paged_kv_cache_49_gb300 import _native as nat
    for bits in (16, 4):
        eng = pkv.PagedKVEngine(20, 8, 2, cache_bits=bits)
        seq = eng.bm.admit(20, 8)
        zeros = np.zeros((1, 8, 128), np.uint16)
        step = eng.prepare_step([seq], zeros, zeros[:, :2], zeros[:, :2])
        graphed = pkv.GraphedDecoder(eng, 1, 4, 0.1)
        want = nat.lib.pkv_attn_workspace_size(1, 2)
        if bits == 4:
            want = max(want, nat.lib.pkv_attn_int4_workspace_size())
        for ws in (step.workspace, graphed.buckets[1].ws):
            assert ws.buffer.numel() == want + 256


@pytest.mark.parametrize("hkv,stop_tiles", [(4, 0), (4, 5), (4, 14), (1, 3)])
def test_wait_runs_out_and_the_next_call_is_exact(pkv, hkv, stop_tiles):
    """CTA 0's tiles from stop_tiles on never come: the call ends after a second, with the
    error set, and the same calls as before give the same results."""
    from paged_kv_cache_49_gb300 import _native as nat
    rng = np.random.default_rng(30)
    args, ws, want = _decode(pkv, rng, [1500, 300, 45], 2 * hkv, hkv, num_ctas=4)
    want = want.clone()
    q, cache, tables, ctx, scale = args
    out, stream = torch.zeros_like(q), torch.cuda.current_stream().cuda_stream
    call = lambda stop: nat.lib.pkv_attn_decode_int4_wait_test(
        q.data_ptr(), cache.data.data_ptr(), tables.data_ptr(), tables.shape[1], ctx.data_ptr(), 3, 2 * hkv, hkv, 128, cache.num_blocks,
        16, 64, scale, 4, ws.ptr, ws.for_int4(stream), out.data_ptr(), stop, stream)
    assert call(-1) == nat.PKV_EINVAL
    assert call(stop_tiles) == nat.PKV_OK
    torch.cuda.synchronize()  # returns: the wait gave up instead of hanging
    assert ws.read_error(clear=False) == pkv.DEVERR_TIMEOUT
    nat.lib.pkv_attn_workspace_init(ws.ptr, ws.fixed_bytes(), stream)
    for _ in range(2):
        assert torch.equal(want, pkv.attn_decode_int4(*args, workspace=ws, num_ctas=4)) and ws.read_error() == 0
    rows = _dev(pkv, _rows(rng, (5, hkv, 128)))
    new = pkv.Int4Cache(2, hkv)
    pkv.append_int4(rows, rows, torch.arange(5, device="cuda"), new)
    k, v = (torch.zeros((2, hkv, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pkv.load_int4(new, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), k, v)
    assert torch.equal(k, v) and k[1, :, :5].any() and not k[0].any() and not k[1, :, 5:].any()


def test_refusals_on_the_gpu(pkv):
    c = pkv.Int4Cache(4, 2)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")
    i32, i64 = torch.int32, torch.int64
    ok = dict(k=z(3, 2, 128), v=z(3, 2, 128), slots=z(3, dtype=i64))
    for bad in (dict(k=z(3, 2, 128, dtype=torch.float16)), dict(k=z(2, 2, 128)), dict(v=z(3, 4, 128)[:, ::2]), dict(v=z(3, 256)),
                dict(slots=z(3, dtype=i32)), dict(slots=z(4, dtype=i64)), dict(k=ok["k"].cpu()),
                dict(k=z(3, 1, 128).expand(3, 2, 128))):
        a = {**ok, **bad}
        with pytest.raises(ValueError):
            pkv.append_int4(a["k"], a["v"], a["slots"], c)
    with pytest.raises(pkv.PkvError):  # the rows of a broadcast tensor overlap: their stride is zero
        pkv.append_int4(z(1, 2, 128).expand(3, 2, 128), ok["v"], ok["slots"], c)
    for k, v, p in ((z(4, 2, 8, 128), z(4, 2, 8, 128), z(1, 2, dtype=i32)), (z(4, 2, 16, 128), z(5, 2, 16, 128), z(1, 2, dtype=i32)),
                    (z(4, 2, 16, 128), z(4, 2, 16, 128), z(1, 2, dtype=i64)), (z(4, 2, 16, 128), z(4, 2, 16, 128), z(3, dtype=i32))):
        with pytest.raises(ValueError):
            pkv.load_int4(c, p, k, v)
    ok = dict(q=z(2, 4, 128), tables=z(2, 3, dtype=i32), ctx=z(2, dtype=i32), out=None)
    for bad in (dict(q=z(2, 4, 64)), dict(q=z(2, 128)), dict(tables=z(3, 3, dtype=i32)), dict(ctx=z(2, dtype=i64)),
                dict(ctx=z(3, dtype=i32)), dict(out=z(2, 3, 128)), dict(out=z(2, 4, 128, dtype=torch.float32))):
        a = {**ok, **bad}
        with pytest.raises(ValueError):
            pkv.attn_decode_int4(a["q"], c, a["tables"], a["ctx"], 0.1, out=a["out"])
    for bad in (dict(q=z(2, 3, 128)), dict(q=z(2, 18, 128))):
        a = {**ok, **bad}
        with pytest.raises(pkv.PkvError):
            pkv.attn_decode_int4(a["q"], c, a["tables"], a["ctx"], 0.1)
    with pytest.raises(pkv.PkvError):
        pkv.attn_decode_int4(ok["q"], c, ok["tables"], ok["ctx"], float("nan"))
    with pytest.raises(pkv.PkvError):  # more CTAs than the workspace has room for
        pkv.attn_decode_int4(ok["q"], c, ok["tables"], ok["ctx"], 0.1, num_ctas=2048)
