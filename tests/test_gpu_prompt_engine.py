"""A prompt's and drafted tokens' way through an engine: chunked prefill with
norms and rotation, decode steps, a verification step, the accepted path's
append, and decode again -- each stage against the oracle on the cache's own
content."""
import numpy as np
import pytest
import torch

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


def _close(got, ref):
    g = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(g).all() and (np.abs(g - ref[0]) <= bound(ref)).all(), np.abs(g - ref[0]).max()


def _projections(pkv, rng, T):
    bits = [randn_bf16(rng, (T, h, D)) for h in (HQ, HKV, HKV)]
    fused = torch.cat([pkv.bf16_from_bits(b).reshape(T, -1) for b in bits], dim=1).cuda()
    at = np.cumsum([0, HQ * D, HKV * D, HKV * D])
    return bits, [fused[:, at[i] : at[i + 1]].view(T, h, D) for i, h in enumerate((HQ, HKV, HKV))]


def _cache(pkv, eng):
    return pkv.bits_from_bf16(eng.k_cache), pkv.bits_from_bf16(eng.v_cache)


def _near(bits, want):
    g = (bits.astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)
    assert (np.abs(g - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(want).max(axis=-1, keepdims=True)).all()


@pytest.mark.parametrize("bt,side_stream", [(16, False), (8, True), (32, False)])
def test_prompts_drafts_and_decode_through_an_engine(pkv, bt, side_stream):
    rng = np.random.default_rng(bt)
    prompts = [70, 1, 200, 33]
    eng = pkv.PagedKVEngine(80, HQ, HKV, D, block_tokens=bt)
    eng.k_cache.fill_(float("nan"))
    eng.v_cache.fill_(float("nan"))
    ids = [eng.bm.admit(n, 12) for n in prompts]
    wq, wk = randn_bf16(rng, (D,)), randn_bf16(rng, (D,))
    table = pkv.rope_table(1000, D)
    rope = pkv.RopeSpec(table, pkv.bf16_from_bits(wq).cuda(), pkv.bf16_from_bits(wk).cuda(), 1e-5)
    cs = table.cpu().numpy()
    ws = pkv.PrefillWorkspace()
    stream = torch.cuda.Stream() if side_stream else None

    def settle():
        torch.cuda.synchronize()

    # two chunks: the first part of each prompt, then the rest
    done = [0] * 4
    for part in (0, 1):
        counts = [n // 3 if part == 0 else n - n // 3 for n in prompts]
        pb = eng.prepare_prefill(ids, counts, done)
        bits, (q, k, v) = _projections(pkv, rng, sum(counts))
        settle()
        out = eng.run_prefill(pb, q, k, v, SCALE, ws, rope, stream=stream)
        settle()
        done = [d + c for d, c in zip(done, counts)]
        positions = pb.positions.cpu().numpy()
        kc, vc = _cache(pkv, eng)
        slots = pb.slots.cpu().numpy()
        _near(kc[slots // bt, :, slots % bt], po.norm_rope(bits[1], wk, 1e-5, cs, positions, False))
        assert np.array_equal(vc[slots // bt, :, slots % bt], bits[2])
        turned = pkv.qk_norm_rope_append(q, k, v, table, pb.positions, torch.full_like(pb.slots, -1), eng.k_cache, eng.v_cache,
                                         q_weight=rope.q_weight, k_weight=rope.k_weight, eps=1e-5)
        _close(out, po.prompt_attention(pkv.bits_from_bf16(turned), kc, vc, pb.tables.cpu().numpy(), np.array(done),
                                        pb.starts.cpu().numpy(), SCALE))

    def decode():
        bits = [randn_bf16(rng, (4, h, D)) for h in (HQ, HKV, HKV)]
        sb = eng.prepare_step(ids, *bits)
        got = eng.run_step(sb, SCALE)
        settle()
        kc, vc = _cache(pkv, eng)
        want = pa.paged_decode_attention(bits[0], kc, vc, sb.tables.cpu().numpy(), sb.ctx.cpu().numpy(), SCALE)
        assert np.abs(got.float().cpu().numpy() - want).max() <= 2e-2
        assert eng.read_errors(sb) == 0

    decode()
    # drafted trees, one sequence without drafts
    parents = [[-1, 0, 0, 1, -1], [-1], [], [-1, 0, 1, 2, 3, 0]]
    before = _cache(pkv, eng)
    db = eng.prepare_drafts(ids, parents)
    T = sum(len(p) for p in parents)
    bits, (q, k, v) = _projections(pkv, rng, T)
    settle()
    out, kd = eng.run_drafts(db, q, k, v, SCALE, ws, rope, stream=stream)
    settle()
    kc, vc = _cache(pkv, eng)
    assert np.array_equal(kc, before[0]) and np.array_equal(vc, before[1])
    assert db.positions.cpu().tolist() == [71, 72, 72, 73, 71, 2, 34, 35, 36, 37, 38, 35]
    turned = pkv.qk_norm_rope_append(q, k, v, table, db.positions, db.slots, eng.k_cache, eng.v_cache,
                                     q_weight=rope.q_weight, k_weight=rope.k_weight, eps=1e-5)
    _close(out, po.tree_attention(pkv.bits_from_bf16(turned), pkv.bits_from_bf16(kd), bits[2], db.masks.cpu().numpy(), kc, vc,
                                  db.tables.cpu().numpy(), db.ctx.cpu().numpy(), db.starts.cpu().numpy(), SCALE))
    # accept a path of each
    paths = [[0, 1, 3], [0], [], [0, 5]]
    slots = eng.accept_drafts(db, paths, kd, v, stream=stream)
    settle()
    assert [i for i, s in enumerate(slots) if s >= 0] == [0, 1, 3, 5, 6, 11]
    kc, vc = _cache(pkv, eng)
    for i, s in enumerate(slots):
        if s >= 0:
            assert np.array_equal(kc[s // bt, :, s % bt], pkv.bits_from_bf16(kd)[i])
            assert np.array_equal(vc[s // bt, :, s % bt], bits[2][i])
    assert [eng.bm.context_len(s) for s in ids] == [74, 3, 201, 36]
    decode()
    assert ws.read_error() == 0 and pkv.read_device_error(eng.error) == 0


def test_a_refused_token_leaves_the_drafts_before_it_appended(pkv):
    eng = pkv.PagedKVEngine(8, HQ, HKV, D)
    sid = eng.bm.admit(14, 3)  # two pages reserved: positions up to 31
    eng.k_cache.zero_(), eng.v_cache.zero_()
    db = eng.prepare_drafts([sid], [list(range(-1, 19))])
    k = torch.randn(20, HKV, D, device="cuda").bfloat16()
    with pytest.raises(pkv.ReservationExceeded):
        eng.accept_drafts(db, [list(range(20))], k, k)
    taken = eng.bm.context_len(sid) - 14
    assert 0 < taken < 20
    for i in range(taken):
        s = eng.bm.slots(sid, 14 + i, 1)[0]
        assert torch.equal(eng.k_cache[s // 16, :, s % 16], k[i])
    for bad in ([[0, 0]], [[20]], [[-1]], []):
        with pytest.raises(ValueError):
            eng.accept_drafts(db, bad, k, k)
    assert eng.bm.context_len(sid) == 14 + taken


def test_prefill_of_a_shared_prefix_and_without_rotation(pkv):
    """The rest of a prompt whose first blocks are another request's, cached."""
    rng = np.random.default_rng(3)
    eng = pkv.PagedKVEngine(40, HQ, HKV, D, prefix_cache=True)
    ws = pkv.PrefillWorkspace()
    tokens = rng.integers(0, 1000, size=100).tolist()
    a = eng.bm.admit(100, 5, tokens=tokens)
    for sid, n in ((a, 100), (None, 0)):
        if sid is None:
            sid = eng.bm.admit(110, 5, tokens=tokens + list(range(10)))
            n = 110 - 16 * eng.bm.reused[sid]
            assert n == 110 - 96
        pb = eng.prepare_prefill([sid], [n])
        bits = [randn_bf16(rng, (n, h, D)) for h in (HQ, HKV, HKV)]
        q, k, v = (pkv.bf16_from_bits(b).cuda() for b in bits)
        out = eng.run_prefill(pb, q, k, v, SCALE, ws)
        torch.cuda.synchronize()
        kc, vc = _cache(pkv, eng)
        _close(out, po.prompt_attention(bits[0], kc, vc, pb.tables.cpu().numpy(), pb.ctx.cpu().numpy(),
                                        pb.starts.cpu().numpy(), SCALE))
    assert ws.read_error() == 0
