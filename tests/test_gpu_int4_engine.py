"""An engine whose cache is held in 4 bits, and beam search over either cache:
prompts in chunks, decode steps (captured ones too), drafted trees and their
acceptance, hypotheses that share and copy pages -- each against the oracle on
what the cache holds, or on the tokens themselves."""
import numpy as np
import pytest
import torch

from oracle import int4
from oracle import paged_attention as pa
from oracle import prompt_attention as po
from tests.prompt_batches import bound
from workloads import randn_bf16

pytestmark = pytest.mark.gpu

HQ, HKV, D = 16, 4, 128
SCALE = 1.0 / np.sqrt(D)


@pytest.fixture(scope="module")
def pkv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tests.conftest import build_native
    build_native()
    import paged_kv_cache_49_gb300 as m
    return m


def _f32(bits):
    return (bits.astype(np.uint32) << np.uint32(16)).view(np.float32)


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _close(got, ref):
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(g).all() and (np.abs(g - ref[0]) <= bound(ref)).all(), np.abs(g - ref[0]).max()


def _pages(pkv, eng):
    """Every page as bf16 bits."""
    n = eng.num_blocks
    k, v = (torch.empty((n, HKV, eng.block_tokens, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    pkv.load_int4(eng.cache, torch.stack([ids, ids], dim=1), k, v)
    return pkv.bits_from_bf16(k), pkv.bits_from_bf16(v)


def _held(bits, gd):
    """What a 4-bit cache gives back of rows, as bf16 bits."""
    return _bf16(int4.values(*int4.quantise(_f32(bits), gd)))


def _projections(pkv, rng, T, fused=True):
    bits = [randn_bf16(rng, (T, h, D)) for h in (HQ, HKV, HKV)]
    if not fused:
        return bits, [pkv.bf16_from_bits(b).cuda() for b in bits]
    fused = torch.cat([pkv.bf16_from_bits(b).reshape(T, -1) for b in bits], dim=1).cuda()
    at = np.cumsum([0, HQ * D, HKV * D, HKV * D])
    return bits, [fused[:, at[i]:at[i + 1]].view(T, h, D) for i, h in enumerate((HQ, HKV, HKV))]


def _decode_error(got, q, kc, vc, tables, ctx):
    """Against pages rounded to bf16: values off by 2^-9 of up to 4, weights by the
    keys' rounding, scores of size 1: all under the 2e-2 that decode steps keep."""
    return np.abs(got.float().cpu().numpy() - pa.paged_decode_attention(q, kc, vc, tables, ctx, SCALE)).max()


@pytest.mark.parametrize("bt,gd,side_stream,with_rope", [(16, 64, False, True), (8, 32, True, True), (64, 128, False, False)])
def test_prompts_drafts_and_decode(pkv, bt, gd, side_stream, with_rope):
    rng = np.random.default_rng(bt)
    prompts = [70, 1, 200, 33]
    eng = pkv.PagedKVEngine(80, HQ, HKV, D, block_tokens=bt, cache_bits=4, group_dims=gd)
    assert eng.k_cache is None and eng.cache.data.shape[0] == 80
    eng.cache.data.fill_(255)
    ids = [eng.bm.admit(n, 12) for n in prompts]
    table = pkv.rope_table(1000, D)
    rope = pkv.RopeSpec(table, None, pkv.bf16_from_bits(randn_bf16(rng, (D,))).cuda(), 1e-5) if with_rope else None
    ws = pkv.PrefillWorkspace()
    stream = torch.cuda.Stream() if side_stream else None

    def turned(q, k, positions):
        if rope is None:
            return pkv.bits_from_bf16(q), pkv.bits_from_bf16(k)
        pool = torch.empty((1, HKV, bt, D), dtype=torch.bfloat16, device="cuda")
        k_out = torch.empty((k.shape[0], HKV, D), dtype=torch.bfloat16, device="cuda")
        q = pkv.qk_norm_rope_append(q, k, k, table, positions, torch.full_like(positions, -1, dtype=torch.int64), pool, pool.clone(),
                                    k_weight=rope.k_weight, eps=1e-5, k_out=k_out)
        return pkv.bits_from_bf16(q), pkv.bits_from_bf16(k_out)

    done = [0] * 4
    for part in (0, 1):
        counts = [n // 3 if part == 0 else n - n // 3 for n in prompts]
        pb = eng.prepare_prefill(ids, counts, done)
        bits, (q, k, v) = _projections(pkv, rng, sum(counts), with_rope)
        torch.cuda.synchronize()
        out = eng.run_prefill(pb, q, k, v, SCALE, ws, rope, stream=stream)
        torch.cuda.synchronize()
        done = [d + c for d, c in zip(done, counts)]
        qb, kb = turned(q, k, pb.positions)
        kc, vc = _pages(pkv, eng)
        slots = pb.slots.cpu().numpy()
        assert np.array_equal(kc[slots // bt, :, slots % bt], _held(kb, gd))
        assert np.array_equal(vc[slots // bt, :, slots % bt], _held(bits[2], gd))
        _close(out, po.prompt_attention(qb, kc, vc, pb.tables.cpu().numpy(), np.array(done), pb.starts.cpu().numpy(), SCALE))

    def decode():
        bits = [randn_bf16(rng, (4, h, D)) for h in (HQ, HKV, HKV)]
        sb = eng.prepare_step(ids, *bits)
        got = eng.run_step(sb, SCALE)
        torch.cuda.synchronize()
        assert _decode_error(got, bits[0], *_pages(pkv, eng), sb.tables.cpu().numpy(), sb.ctx.cpu().numpy()) <= 2e-2
        assert eng.read_errors(sb) == 0 and eng.cascade_for(sb, 0) is None

    decode()
    parents = [[-1, 0, 0, 1, -1], [-1], [], [-1, 0, 1, 2, 3, 0]]
    before = eng.cache.data.clone()
    db = eng.prepare_drafts(ids, parents)
    bits, (q, k, v) = _projections(pkv, rng, sum(len(p) for p in parents), with_rope)
    torch.cuda.synchronize()
    out, kd = eng.run_drafts(db, q, k, v, SCALE, ws, rope, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(before, eng.cache.data)
    qb, kb = turned(q, k, db.positions)
    assert np.array_equal(pkv.bits_from_bf16(kd), kb)
    kc, vc = _pages(pkv, eng)
    _close(out, po.tree_attention(qb, kb, bits[2], db.masks.cpu().numpy(), kc, vc, db.tables.cpu().numpy(), db.ctx.cpu().numpy(),
                                  db.starts.cpu().numpy(), SCALE))
    slots = eng.accept_drafts(db, [[0, 1, 3], [0], [], [0, 5]], kd, v, stream=stream)
    torch.cuda.synchronize()
    kc, vc = _pages(pkv, eng)
    for i, s in enumerate(slots):
        if s >= 0:
            assert np.array_equal(kc[s // bt, :, s % bt], _held(kb[i], gd))
            assert np.array_equal(vc[s // bt, :, s % bt], _held(bits[2][i], gd))
    decode()
    assert ws.read_error() == 0 and pkv.read_device_error(eng.error) == 0


def test_forked_sequences_and_loaded_pools(pkv):
    """append_tokens, write_positions and copies on write of 4-bit blocks."""
    rng = np.random.default_rng(1)
    eng = pkv.PagedKVEngine(30, HQ, HKV, D, cache_bits=4)
    kb, vb = (randn_bf16(rng, (30, HKV, 16, D)) for _ in range(2))
    eng.load_pool(kb[:20], vb[:20])
    eng.load_pool(kb[20:], vb[20:], 20)
    kc, vc = _pages(pkv, eng)
    assert np.array_equal(kc, _held(kb, 64)) and np.array_equal(vc, _held(vb, 64))
    a = eng.bm.admit(20, 20)
    pk, pv = (randn_bf16(rng, (20, HKV, D)) for _ in range(2))
    eng.write_positions(a, 0, pkv.bf16_from_bits(pk).cuda(), pkv.bf16_from_bits(pv).cuda())
    ids = [a] + eng.bm.fork(a, 2)
    nk, nv = (randn_bf16(rng, (3, HKV, D)) for _ in range(2))
    slots, pairs = eng.append_tokens(ids, pkv.bf16_from_bits(nk).cuda(), pkv.bf16_from_bits(nv).cuda())
    assert len(pairs) == 2
    kc, vc = _pages(pkv, eng)
    for i, s in enumerate(ids):
        t = np.array(eng.bm.table(s))
        at = np.arange(21)
        for got, old, new in ((kc, pk, nk), (vc, pv, nv)):
            assert np.array_equal(got[t[at // 16], :, at % 16], _held(np.concatenate([old, new[i:i + 1]]), 64))


def test_captured_steps(pkv):
    rng = np.random.default_rng(2)
    eng = pkv.PagedKVEngine(60, HQ, HKV, D, cache_bits=4)
    ids = [eng.bm.admit(n, 20) for n in (40, 5, 90)]
    for s, n in zip(ids, (40, 5, 90)):
        k, v = (pkv.bf16_from_bits(randn_bf16(rng, (n, HKV, D))).cuda() for _ in range(2))
        eng.write_positions(s, 0, k, v)
    ids.append(eng.bm.fork(ids[0], 1)[0])
    dec = pkv.GraphedDecoder(eng, 8, 8, SCALE)
    for _ in range(4):
        bits = [randn_bf16(rng, (len(ids), h, D)) for h in (HQ, HKV, HKV)]
        out, slots, pairs = dec.step_bits(ids, *bits)
        torch.cuda.synchronize()
        tables, ctx = eng.bm.batch_tables(ids, 8)
        assert _decode_error(out, bits[0], *_pages(pkv, eng), tables.numpy(), ctx.numpy()) <= 2e-2
        ids = ids[1:]
    assert pkv.read_device_error(eng.error) == 0


def test_what_a_4_bit_engine_refuses(pkv):
    for bad in (dict(cache_bits=8), dict(cache_bits=4, head_dim=64), dict(cache_bits=4, group_dims=16)):
        with pytest.raises(ValueError):
            pkv.PagedKVEngine(4, HQ, HKV, **bad)
    eng = pkv.PagedKVEngine(4, HQ, HKV, cache_bits=4)
    with pytest.raises(ValueError):
        pkv.HostStep(eng, 1, 1)
    with pytest.raises(ValueError):
        eng.run_step_cascade(None, SCALE, None)


# ---- beam search ----------------------------------------------------------------


@pytest.mark.parametrize("incremental", [False, True])
@pytest.mark.parametrize("bits,bt", [(16, 16), (4, 16), (4, 8), (16, 32)])
def test_a_beam_search_attends_its_own_tokens(pkv, bits, bt, incremental):
    """Hypotheses that share pages and part: each step's attention of each is that
    of its own tokens, whose keys and values are functions of the token."""
    rng = np.random.default_rng(bits + bt)
    vocab, beams, steps, eos = 97, 3, 14, 5
    keys, values = (randn_bf16(rng, (vocab, HKV, D)) for _ in range(2))
    kept = [_held(x, 64) if bits == 4 else x for x in (keys, values)]
    eng = pkv.PagedKVEngine(60, HQ, HKV, D, block_tokens=bt, incremental=incremental, cache_bits=bits)
    prompts = [rng.integers(0, vocab, size=n) for n in (21, 8)]
    ids = []
    for p in prompts:
        ids.append(eng.bm.admit(len(p), steps))
        eng.write_positions(ids[-1], 0, *(pkv.bf16_from_bits(x[p]).cuda() for x in (keys, values)))
    search = pkv.BeamSearch(eng, ids, beams, vocab, steps, eos)
    assert search.live == [0, 3] and len(search.seq_ids) == 6
    total = np.full((2, beams), -np.inf)
    total[:, 0] = 0
    ends = 0
    for step in range(steps):
        logits = torch.from_numpy(2 * rng.standard_normal((6, vocab))).to(torch.bfloat16).cuda()
        tokens = search.step(logits)
        hyps = search.histories()
        flat = [h for g in hyps for h in g]
        assert all(len(h) == step + 1 or h[-1] == eos for h in flat)
        assert tokens.flatten().tolist() == [h[-1] for h in flat] and len({tuple(h) for h in hyps[0]}) == beams
        assert search.live == [i for i, h in enumerate(flat) if h[-1] != eos]
        ends += len(flat) - len(search.live)
        total = search.now.scores.cpu().numpy()
        assert (np.diff(total, axis=1) <= 0).all() and np.isfinite(total).all()
        if not search.live:
            break
        live = [search.seq_ids[i] for i in search.live]
        new = [flat[i][-1] for i in search.live]
        q = randn_bf16(rng, (len(live), HQ, D))
        sb = eng.prepare_step(live, q, keys[new], values[new])
        out = eng.run_step(sb, SCALE)
        torch.cuda.synchronize()
        assert eng.read_errors(sb) == 0
        for j, i in enumerate(search.live):
            seen = np.concatenate([prompts[i // beams], flat[i]]).astype(int)
            assert eng.bm.context_len(live[j]) == len(seen)
            pool = [x[seen].swapaxes(0, 1)[None] for x in kept]  # one block of the whole context
            want = pa.paged_decode_attention(q[j:j + 1], *pool, np.zeros((1, 1), int), [len(seen)], SCALE)
            assert np.abs(out[j].float().cpu().numpy() - want[0]).max() <= 2e-2
    assert eng.bm.stats()["cow_copies"] > 0
    search.free()
    assert eng.bm.stats()["free"] == 60


def test_a_search_without_pages_leaves_all_as_it_was(pkv):
    eng = pkv.PagedKVEngine(7, HQ, HKV, D)
    a, b = eng.bm.admit(20, 10), eng.bm.admit(16, 16)
    was = eng.bm.stats()
    with pytest.raises(pkv.PoolExhausted):
        pkv.BeamSearch(eng, [a, b], 6, 50, 4)
    assert eng.bm.stats() == was
    for bad in (([], 2, 50, 4), ([a], 0, 50, 4), ([a], 2, 50, 0)):
        with pytest.raises(ValueError):
            pkv.BeamSearch(eng, *bad)
