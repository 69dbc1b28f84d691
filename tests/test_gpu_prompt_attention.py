"""Prompt and draft-tree attention over the cache against the oracle."""
import numpy as np
import pytest
import torch

from oracle import prompt_attention as po
from tests.prompt_batches import NAN, Batch, bits_of, bound, floats

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tests.conftest import build_native
    build_native()
    import paged_kv_cache_49_gb300 as m
    return m


def _dev(pkv, b, tree):
    d = {n: pkv.bf16_from_bits(getattr(b, n)).cuda() for n in ("q", "k", "v")}
    d.update(tables=torch.from_numpy(b.tables).cuda(), ctx=torch.from_numpy(b.ctx).cuda(),
             starts=torch.from_numpy(b.starts).cuda())
    if tree:
        d.update(kd=pkv.bf16_from_bits(b.kd).cuda(), vd=pkv.bf16_from_bits(b.vd).cuda(),
                 masks=torch.from_numpy(b.masks).cuda())
    return d


def _call(pkv, d, scale, **kw):
    if "kd" in d:
        return pkv.attn_tree(d["q"], d["kd"], d["vd"], d["masks"], d["k"], d["v"], d["tables"], d["ctx"], d["starts"],
                             scale, **kw)
    return pkv.attn_prefill(d["q"], d["k"], d["v"], d["tables"], d["ctx"], d["starts"], scale, **kw)


def _ref(b, tree):
    if tree:
        return po.tree_attention(b.q, b.kd, b.vd, b.masks, b.k, b.v, b.tables, b.ctx, b.starts, b.scale)
    return po.prompt_attention(b.q, b.k, b.v, b.tables, b.ctx, b.starts, b.scale)


def _check(got, ref, rows=slice(None)):
    g = got.float().cpu().numpy().astype(np.float64)[rows]
    out, tol = ref[0][rows], bound(ref)[rows]
    finite = np.isfinite(out)
    assert np.array_equal(np.isfinite(g), finite)
    err = np.abs(np.where(finite, g - np.where(finite, out, 0.0), 0.0))
    worst = (err - np.where(finite, tol, 0.0)).max() if err.size else 0.0
    assert worst <= 0.0, f"error {err.max()}, over its bound by {worst}"


def _run(pkv, b, tree, **kw):
    d = _dev(pkv, b, tree)
    ws = pkv.PrefillWorkspace()
    out = torch.full_like(d["q"], 7.0)
    _call(pkv, d, b.scale, out=out, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert ws.read_error() == 0
    lo, hi = int(b.starts[0]), int(b.starts[-1])
    assert (out[:lo] == 7.0).all() and (out[hi:] == 7.0).all()  # rows of no sequence
    _check(out, _ref(b, tree), slice(lo, hi))
    return out, d


HEADS = [(32, 8), (8, 8), (16, 8), (64, 8), (8, 1), (6, 2), (5, 1), (12, 2), (7, 1)]


@pytest.mark.parametrize("hq,hkv", HEADS)
def test_prompts_of_many_lengths(pkv, hq, hkv):
    """Whole prompts, chunks on cached contexts, single rows, none at all."""
    new = [1, 0, 37, 128, 129, 255, 5, 16, 300, 1]
    held = [1, 9, 37, 192, 130, 755, 2005, 16, 300, 517]
    _run(pkv, Batch(hq * 100 + hkv, new, held, hq, hkv, 16, first_row=3, rows_behind=2), tree=False)


@pytest.mark.parametrize("hq,hkv", HEADS)
def test_trees_of_many_sizes(pkv, hq, hkv):
    new = [1, 0, 7, 64, 63, 16, 2, 33, 5, 64]
    held = [0, 9, 37, 128, 0, 127, 2005, 129, 1, 300]
    _run(pkv, Batch(hq * 100 + hkv + 1, new, held, hq, hkv, 16, first_row=2, rows_behind=3), tree=True)


@pytest.mark.parametrize("bt", [8, 32, 64])
@pytest.mark.parametrize("tree", [False, True])
def test_block_sizes(pkv, bt, tree):
    new = [1, 64, 17, 40, 3]
    held = [65, 64, 177, 1000, 7]
    _run(pkv, Batch(bt, new, held, 16, 4, bt), tree=tree)


@pytest.mark.parametrize("tree,new,held", [
    (False, [5], [40001]), (False, [130], [9001]), (True, [9], [70003]), (True, [64, 1], [20000, 33333]),
    (False, [1] * 5, [1, 8191, 8192, 8193, 3]), (False, [700], [700]),
])
def test_few_rows_on_long_contexts(pkv, tree, new, held):
    """The keys of a row are split and joined."""
    _run(pkv, Batch(len(new) + new[0], new, held, 8, 2, 16), tree=tree)


@pytest.mark.parametrize("tree,new,held,hq,hkv", [
    (True, [60], [17003], 7, 1),                         # a tile of 126 rows and a short one, all in many pieces
    (True, [64], [30001], 24, 3),                        # items of fewer pieces
    (False, [40, 3], [20011, 40], 10, 2),
    (False, [3] + [2] * 159, [50021] + [300] * 159, 8, 1),  # as many items as CTAs, one of them long
    (True, [3] + [2] * 159, [50021] + [300] * 159, 8, 1),
])
def test_items_in_many_pieces(pkv, tree, new, held, hq, hkv):
    """The warps of the join share the pieces of a row."""
    _run(pkv, Batch(hq + new[0], new, held, hq, hkv, 16, first_row=1, rows_behind=1), tree=tree)


@pytest.mark.parametrize("new,held", [([1500, 700, 0, 300], [26003, 9001, 17, 300]), ([2500], [26000])])
def test_chunks_whose_contexts_exceed_the_l2_cache(pkv, new, held):
    """Ranges in several rounds; some rows of each sequence, as decode rows of the oracle."""
    b = Batch(new[0], new, held, 64, 8, 16, first_row=2, rows_behind=3)
    d = _dev(pkv, b, False)
    ws = pkv.PrefillWorkspace()
    out = torch.full_like(d["q"], 7.0)
    _call(pkv, d, b.scale, out=out, workspace=ws)
    again = torch.full_like(d["q"], 5.0)
    _call(pkv, d, b.scale, out=again, workspace=ws)
    assert ws.read_error() == 0
    lo, hi = int(b.starts[0]), int(b.starts[-1])
    assert (out[:lo] == 7.0).all() and (out[hi:] == 7.0).all()
    assert torch.equal(out[lo:hi], again[lo:hi])
    assert torch.isfinite(out.float()).all()
    rows, seqs, ctx = [], [], []
    for s, n in enumerate(new):
        for i in sorted({0, 1, 31, 32, n // 3, n // 2, n - 33, n - 2, n - 1} if n else ()):
            rows.append(int(b.starts[s]) + i)
            seqs.append(s)
            ctx.append(held[s] - n + i + 1)
    ref = po.prompt_attention(b.q[rows], b.k, b.v, b.tables[seqs], np.array(ctx, np.int32),
                              np.arange(len(rows) + 1, dtype=np.int32), b.scale)
    _check(out[rows], ref)


def test_many_sequences(pkv):
    rng = np.random.default_rng(5)
    held = [int(x) for x in rng.integers(1, 60, size=700)]
    new = [int(rng.integers(0, c + 1)) if rng.random() < 0.7 else 0 for c in held]
    _run(pkv, Batch(9, new, held, 4, 1, 8), tree=False)
    _run(pkv, Batch(10, [min(n, 64) for n in new], held, 4, 1, 8), tree=True)


def test_the_most_sequences(pkv):
    new, held = [1] * 4096, [1 + s % 5 for s in range(4096)]
    _run(pkv, Batch(11, new, held, 2, 1, 8), tree=False)
    _run(pkv, Batch(12, new, held, 2, 1, 8), tree=True)


@pytest.mark.parametrize("tree", [False, True])
def test_peaked_and_growing_scores(pkv, tree):
    """Scores of tens whose maximum keeps growing along the context: the
    running maximum is raised again and again."""
    b = Batch(13, [40, 64], [900, 700], 8, 2, 16, spread=12.0)
    for s, c in enumerate(b.held):
        t = np.arange(c)
        row = b.tables[s][t // b.bt]
        ramp = (0.2 + 1.8 * t / c).astype(np.float32)[:, None, None]
        b.k[row, :, t % b.bt] = bits_of(floats(b.k[row, :, t % b.bt]) * ramp)
    _run(pkv, b, tree)


@pytest.mark.parametrize("value", [0x7FC0, 0x7F80, 0xFF80])
def test_non_finite_tokens_reach_only_the_rows_that_see_them(pkv, value):
    """A prompt's last tokens hold NaN or infinities: earlier rows do not see
    them, later ones do."""
    b = Batch(14, [200, 37], [300, 37], 8, 2, 16)
    for s, position in ((0, 290), (0, 150), (1, 20)):
        blk, r = b.slot(s, position)
        b.v[blk, 1, r, 5] = value
    blk, r = b.slot(0, 299)
    b.v[blk, 0, r, :] = value
    b.k[blk, 0, r, :] = NAN
    got, _ = _run(pkv, b, tree=False)
    g = got.float().cpu().numpy()
    first = 300 - 200
    assert np.isfinite(g[:200, :4][: 299 - first]).all() and not np.isfinite(g[200 - 1, :4]).any()
    assert np.isfinite(g[: 150 - first, 4:]).all() and not np.isfinite(g[150 - first, 4:, 5]).any()


def test_non_finite_drafts_reach_only_the_rows_that_see_them(pkv):
    b = Batch(15, [6, 33], [100, 128], 8, 2, 16)
    b.vd[2, 0] = NAN
    b.kd[2, 0] = NAN
    b.vd[6 + 30, 1, 100:] = 0x7F80
    b.masks[:6] = [0b1, 0b11, 0b101, 0b1001, 0b10101, 0b100000]
    got, _ = _run(pkv, b, tree=True)
    g = got.float().cpu().numpy()
    assert [bool(np.isnan(g[i, 0]).all()) for i in range(6)] == [False, False, True, False, True, False]


def test_rows_that_see_nothing_give_zeros(pkv):
    b = Batch(16, [4, 3], [0, 0], 8, 2, 16)
    b.masks[:] = [0, 1 << 40, 0b10, 0, 0b111, 0, -(1 << 63)]  # bits past the drafts do not count
    got, _ = _run(pkv, b, tree=True)
    g = got.float().cpu().numpy()
    assert (g[[0, 1, 3, 5, 6]] == 0).all() and (g[[2, 4]] != 0).any()
    c = Batch(17, [9], [64], 8, 2, 16)
    c.masks[:] = 0  # the context alone
    _run(pkv, c, tree=True)


def test_extreme_scores(pkv):
    """Equal scores, a zero scale, and scores that underflow against the largest."""
    b = Batch(18, [40], [400], 8, 2, 16)
    b.k[...] = np.where(b.k == NAN, NAN, np.uint16(0))
    _run(pkv, b, tree=False)
    c = Batch(19, [40], [400], 8, 2, 16)
    c.scale = 0.0
    _run(pkv, c, tree=False)
    d = Batch(20, [40], [400], 8, 2, 16)
    d.scale = 30.0
    _run(pkv, d, tree=True)


@pytest.mark.parametrize("tree", [False, True])
def test_bad_tables_and_lengths_set_their_bits(pkv, tree):
    """Nothing is read or written outside its buffer; the good sequence is exact."""
    b = Batch(21, [20, 33, 7], [100, 133, 7], 8, 2, 16)
    ref = _ref(b, tree)
    ws = pkv.PrefillWorkspace()

    def run(d):
        out = torch.full_like(d["q"], 7.0)
        _call(pkv, d, b.scale, out=out, workspace=ws)
        torch.cuda.synchronize()
        return out, ws.read_error()

    d = _dev(pkv, b, tree)
    d["tables"][1, 3], d["tables"][1, 4] = b.k.shape[0], -5
    out, err = run(d)
    assert err == pkv.DEVERR_BLOCK_ID
    _check(out, ref, slice(0, 20))
    _check(out, ref, slice(53, 60))

    d = _dev(pkv, b, tree)
    d["ctx"][1] = 16 * b.width + 1
    out, err = run(d)
    assert err & pkv.DEVERR_CONTEXT
    _check(out, ref, slice(0, 20))

    d = _dev(pkv, b, tree)
    d["starts"][3] = 61  # past the rows of q
    out, err = run(d)
    assert err & pkv.DEVERR_QUERY
    _check(out, ref, slice(0, 53))

    d = _dev(pkv, b, tree)
    d["starts"][2] = -4  # sequence 1 ends before it starts
    out, err = run(d)
    assert err & pkv.DEVERR_QUERY
    if not tree:
        d = _dev(pkv, b, tree)
        d["ctx"][1] = 30  # 33 rows on 30 tokens: three rows before position 0
        out, err = run(d)
        assert err == pkv.DEVERR_CONTEXT and (out[20:23] == 0).all()
        _check(out, ref, slice(0, 20))


def test_a_tree_over_the_limit(pkv):
    b = Batch(22, [70, 5], [40, 50], 8, 2, 16)
    d = _dev(pkv, b, True)
    ws = pkv.PrefillWorkspace()
    out = torch.full_like(d["q"], 7.0)
    _call(pkv, d, b.scale, out=out, workspace=ws)
    assert ws.read_error() == pkv.DEVERR_QUERY
    assert (out[64:70] == 7.0).all()
    _check(out, _ref(b, True), slice(70, 75))


@pytest.mark.parametrize("tree", [False, True])
def test_repeats_graphs_streams_and_a_shared_workspace(pkv, tree):
    """Bit-identical on every path; captured calls of two shapes replay on one
    workspace; lengths changed between replays are read anew."""
    a = Batch(23, [50, 64, 1], [3000, 64, 700], 8, 2, 16)
    b = Batch(24, [9], [12000], 16, 2, 16)
    da, db = _dev(pkv, a, tree), _dev(pkv, b, tree)
    ws = pkv.PrefillWorkspace()
    ref_a, ref_b = _call(pkv, da, a.scale, workspace=ws).clone(), _call(pkv, db, b.scale, workspace=ws).clone()
    _check(ref_a, _ref(a, tree))
    _check(ref_b, _ref(b, tree))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = _call(pkv, da, a.scale, stream=side)
    side.synchronize()
    assert torch.equal(on_side, ref_a)
    raw = _call(pkv, da, a.scale, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(raw, ref_a)
    out_a, out_b = torch.zeros_like(ref_a), torch.zeros_like(ref_b)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        _call(pkv, da, a.scale, out=out_a, workspace=ws)
    with torch.cuda.graph(gb):
        _call(pkv, db, b.scale, out=out_b, workspace=ws)
    for _ in range(3):
        out_a.zero_(), out_b.zero_()
        ga.replay(), gb.replay(), ga.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_a, ref_a) and torch.equal(out_b, ref_b)
    da["ctx"][0] = 2900
    want = _call(pkv, da, a.scale, workspace=ws).clone()
    ga.replay()
    torch.cuda.synchronize()
    assert torch.equal(out_a, want) and not torch.equal(want, ref_a)
    assert ws.read_error() == 0


def test_calls_on_two_streams_at_once(pkv):
    """Two calls whose kernels may run side by side, each with its workspace."""
    a = Batch(28, [300, 40], [4000, 900], 8, 2, 16)
    b = Batch(29, [64, 33, 5], [9000, 64, 700], 8, 2, 16)
    da, db = _dev(pkv, a, False), _dev(pkv, b, True)
    ra, rb = _call(pkv, da, a.scale).clone(), _call(pkv, db, b.scale).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [pkv.PrefillWorkspace(), pkv.PrefillWorkspace()]
    outs = [torch.zeros_like(ra), torch.zeros_like(rb)]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s, w, o, x in zip((da, db), streams, spaces, outs, (a, b)):
            _call(pkv, d, x.scale, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ra) and torch.equal(outs[1], rb)
    assert spaces[0].read_error() == 0 and spaces[1].read_error() == 0


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one device")
def test_another_device_than_the_current_one(pkv):
    b = Batch(30, [9, 64], [500, 64], 8, 2, 16)
    for tree in (False, True):
        d = {k: t.to("cuda:1") for k, t in _dev(pkv, b, tree).items()}
        out = _call(pkv, d, b.scale)
        torch.cuda.synchronize("cuda:1")
        _check(out, _ref(b, tree))


def test_a_single_draft_is_a_decode_step(pkv):
    """One draft that sees itself: decode attention once it has been appended."""
    held = [1, 16, 203, 700]
    b = Batch(25, [1] * 4, held, 32, 8, 16)
    tree, d = _run(pkv, b, tree=True)
    c = Batch(25, [1] * 4, [h + 1 for h in held], 32, 8, 16)
    dc = _dev(pkv, c, False)
    slots = []
    for s, h in enumerate(held):
        t = np.arange(h)
        src, dst = b.tables[s][t // 16], c.tables[s][t // 16]
        dc["k"][torch.from_numpy(dst).long(), :, torch.from_numpy(t % 16)] = d["k"][torch.from_numpy(src).long(), :, torch.from_numpy(t % 16)]
        dc["v"][torch.from_numpy(dst).long(), :, torch.from_numpy(t % 16)] = d["v"][torch.from_numpy(src).long(), :, torch.from_numpy(t % 16)]
        slots.append(int(c.tables[s][h // 16]) * 16 + h % 16)
    pkv.append(d["kd"], d["vd"], torch.tensor(slots, device="cuda"), dc["k"], dc["v"])
    _check(pkv.attn_decode(d["q"], dc["k"], dc["v"], dc["tables"], dc["ctx"], b.scale), _ref(b, True))
    _check(_call(pkv, {**dc, "q": d["q"]}, b.scale), _ref(b, True))


def test_no_rows(pkv):
    b = Batch(26, [0, 0], [10, 0], 8, 2, 16)
    for tree in (False, True):
        d = _dev(pkv, b, tree)
        assert _call(pkv, d, b.scale).shape == (0, 8, 128)
    c = Batch(27, [0, 0], [10, 0], 8, 2, 16, rows_behind=5)
    _run(pkv, c, tree=False)
    _run(pkv, c, tree=True)
