"""Host side of prompt attention, draft trees and the fused write: refusals,
tree masks, the rotary table, and pins of their oracle (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import paged_attention as pa
from oracle import prompt_attention as po
from tests.prompt_batches import Batch, bits_of, floats


@pytest.fixture(scope="module")
def nat():
    from tests.conftest import build_native
    build_native()
    import paged_kv_cache_49_gb300._native as n
    return n


P = 4096  # stands for an aligned, non-null pointer: refused calls read nothing


def _prefill(nat, **kw):
    a = dict(q=P, k=P, v=P, tables=P, width=4, ctx=P, starts=P, seqs=2, tokens=5, hq=8, hkv=2, d=128, nb=10, bt=16,
             scale=0.1, ws=P, wsb=1 << 30, out=P)
    a.update(kw)
    return nat.lib.pkv_attn_prefill(a["q"], a["k"], a["v"], a["tables"], a["width"], a["ctx"], a["starts"], a["seqs"],
                                    a["tokens"], a["hq"], a["hkv"], a["d"], a["nb"], a["bt"], a["scale"], a["ws"],
                                    a["wsb"], a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), "EINVAL"), (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(tables=None), "EINVAL"),
    (dict(ctx=None), "EINVAL"), (dict(starts=None), "EINVAL"), (dict(ws=None), "EINVAL"), (dict(out=None), "EINVAL"),
    (dict(q=P + 8), "EINVAL"), (dict(out=P + 2), "EINVAL"), (dict(ws=P + 128), "EINVAL"), (dict(wsb=255), "EINVAL"),
    (dict(tokens=-1), "EINVAL"), (dict(seqs=0), "EINVAL"), (dict(hq=0), "EINVAL"), (dict(width=0), "EINVAL"),
    (dict(scale=float("nan")), "EINVAL"), (dict(scale=-0.5), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
    (dict(seqs=4097), "EUNSUPPORTED"), (dict(d=64), "EUNSUPPORTED"), (dict(hq=9), "EUNSUPPORTED"),
    (dict(hq=18), "EUNSUPPORTED"), (dict(bt=12), "EUNSUPPORTED"), (dict(nb=1 << 27), "ERANGE"),
    (dict(width=1 << 30), "ERANGE"), (dict(tokens=1 << 28), "ERANGE"),
    (dict(tokens=1 << 27, hq=16), "ERANGE"), (dict(tokens=0, q=None, out=None), "OK"),
])
def test_prefill_refusals(nat, kw, status):
    assert _prefill(nat, **kw) == getattr(nat, "PKV_" + status)


@pytest.mark.parametrize("kw,status", [
    (dict(kd=None), "EINVAL"), (dict(vd=None), "EINVAL"), (dict(masks=None), "EINVAL"), (dict(kd=P + 4), "EINVAL"),
    (dict(hq=18), "EUNSUPPORTED"), (dict(tokens=0), "OK"),
])
def test_tree_refusals(nat, kw, status):
    a = dict(kd=P, vd=P, masks=P, hq=8, tokens=5)
    a.update(kw)
    assert nat.lib.pkv_attn_tree(P, a["kd"], a["vd"], a["masks"], P, P, P, 4, P, P, 2, a["tokens"], a["hq"], 2, 128, 10,
                                 16, 0.1, P, 1 << 30, P, None) == getattr(nat, "PKV_" + status)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(slots=None), "EINVAL"), (dict(qo=None), "EINVAL"),
    (dict(table=None), "EINVAL"), (dict(pos=None), "EINVAL"), (dict(mp=0), "EINVAL"), (dict(qs=8 * 128 - 8), "EINVAL"),
    (dict(ks=2 * 128 + 4), "EINVAL"), (dict(vs=0), "EINVAL"), (dict(q=P + 2), "EINVAL"), (dict(w=P + 8), "EINVAL"), (dict(ko=P + 8), "EINVAL"),
    (dict(eps=-1.0), "EINVAL"), (dict(eps=float("nan")), "EINVAL"), (dict(tokens=-1), "EINVAL"),
    (dict(d=12), "EUNSUPPORTED"), (dict(d=264), "EUNSUPPORTED"), (dict(rot=8), "EUNSUPPORTED"),
    (dict(rot=144), "EUNSUPPORTED"), (dict(bt=24), "EUNSUPPORTED"), (dict(tokens=0), "OK"),
])
def test_write_refusals(nat, kw, status):
    a = dict(q=P, qs=12 * 128, ks=12 * 128, v=P, vs=12 * 128, w=None, eps=1e-6, table=P, mp=100, rot=128, pos=P,
             slots=P, tokens=5, d=128, qo=P, ko=None, bt=16)
    a.update(kw)
    if a["d"] > 128:
        a.update(qs=12 * a["d"], ks=12 * a["d"], vs=12 * a["d"])
    assert nat.lib.pkv_qk_norm_rope_append(a["q"], a["qs"], P, a["ks"], a["v"], a["vs"], a["w"], None, a["eps"],
                                           a["table"], a["mp"], a["rot"], 0, a["pos"], a["slots"], a["tokens"], 8, 2,
                                           a["d"], a["qo"], a["ko"], P, P, 10, a["bt"], None, None) == getattr(nat, "PKV_" + status)


def test_binding_refusals(nat):
    bf = dict(dtype=torch.bfloat16)
    q, c = torch.zeros(5, 8, 128, **bf), torch.zeros(4, 2, 16, 128, **bf)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        nat.attn_prefill(q, c, c, i(1, 4), i(1), i(2), 0.1)
    with pytest.raises(ValueError, match="bfloat16"):
        nat.attn_prefill(q.float(), c, c, i(1, 4), i(1), i(2), 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        nat.qk_norm_rope_append(q, q[:, :2], q[:, :2], None, None, torch.zeros(5, dtype=torch.int64), c, c)
    with pytest.raises(ValueError, match="contiguous"):
        nat.qk_norm_rope_append(q.transpose(0, 1)[:5], q[:5, :2], q[:5, :2], None, None,
                                torch.zeros(5, dtype=torch.int64), c, c)


def test_tree_masks(nat):
    assert nat.tree_masks([-1, 0, 0, 1, -1]) == [0b1, 0b11, 0b101, 0b1011, 0b10000]
    assert nat.tree_masks([]) == []
    chain = nat.tree_masks(list(range(-1, 63)))
    assert chain[63] == -1 and chain[62] == (1 << 63) - 1
    for bad in ([0], [-1, 1], [-2], [-1, 5]):
        with pytest.raises(ValueError):
            nat.tree_masks(bad)
    with pytest.raises(ValueError):
        nat.tree_masks([-1] * 65)


def test_rope_table(nat):
    t = nat.rope_table(70001, 64, base=1e6, device="cpu").numpy()
    p, i = np.array([0, 1, 70000])[:, None], np.arange(32)
    angle = p * 1e6 ** (-2.0 * i / 64)
    assert t.shape == (70001, 64) and t.dtype == np.float32
    assert np.abs(t[p[:, 0], :32] - np.cos(angle)).max() <= 2.0 ** -24
    assert np.abs(t[p[:, 0], 32:] - np.sin(angle)).max() <= 2.0 ** -24
    with pytest.raises(ValueError):
        nat.rope_table(10, 7)


def test_oracle_prompt_rows_are_decode_steps():
    """Row i of a prompt equals decode attention over the first p + 1 tokens."""
    b = Batch(1, [5, 0, 3], [21, 4, 3], 4, 2, 8)
    out = po.prompt_attention(b.q, b.k, b.v, b.tables, b.ctx, b.starts, b.scale)[0]
    for s, n in enumerate(b.new):
        for i in range(n):
            row = int(b.starts[s]) + i
            want = pa.paged_decode_attention(b.q[row][None], b.k, b.v, b.tables[s : s + 1],
                                             [b.held[s] - n + i + 1], b.scale)
            assert np.abs(out[row] - want[0]).max() <= 1e-14


def test_oracle_tree_of_a_chain_is_a_prompt():
    """A chain of drafts over a context: a prompt chunk whose tokens are cached."""
    b = Batch(2, [6], [20], 4, 2, 8)
    chain = np.array([(1 << (i + 1)) - 1 for i in range(6)], np.int64)
    tree = po.tree_attention(b.q, b.kd, b.vd, chain, b.k, b.v, b.tables, b.ctx, b.starts, b.scale)[0]
    c = Batch(2, [6], [26], 4, 2, 8)
    t = np.arange(26)
    for cache, old, new in ((c.k, b.k, b.kd), (c.v, b.v, b.vd)):
        cache[c.tables[0][t[:20] // 8], :, t[:20] % 8] = old[b.tables[0][t[:20] // 8], :, t[:20] % 8]
        cache[c.tables[0][t[20:] // 8], :, t[20:] % 8] = new
    want = po.prompt_attention(b.q, c.k, c.v, c.tables, c.ctx, c.starts, c.scale)[0]
    assert np.abs(tree - want).max() <= 1e-14


def test_oracle_rotation_and_norm():
    rng = np.random.default_rng(0)
    x = bits_of(rng.standard_normal((3, 2, 8)).astype(np.float32))
    half = 4
    table = np.concatenate([np.zeros((10, half)), np.ones((10, half))], axis=1).astype(np.float32)  # quarter turns
    y = po.norm_rope(x, None, 0.0, table, np.array([0, 5, 9]), False)
    f = floats(x).astype(np.float64)
    assert np.array_equal(y, np.concatenate([-f[..., half:], f[..., :half]], axis=-1))
    z = po.norm_rope(x, None, 0.0, table, np.array([0, 5, 9]), True)
    assert np.array_equal(z[..., 0::2], -f[..., 1::2]) and np.array_equal(z[..., 1::2], f[..., 0::2])
    one = bits_of(np.ones(8, np.float32))
    n = po.norm_rope(x, one, 0.0, None, None, False)
    assert np.abs((n * n).mean(axis=-1) - 1.0).max() <= 1e-12


def test_drafts_are_taken_once_and_only_in_their_place(nat):
    """Refusals that leave the block manager as it was; nothing is launched."""
    import torch
    from paged_kv_cache_49_gb300.engine import PagedKVEngine
    eng = PagedKVEngine(8, 2, 1, device="cpu")
    a, b = eng.bm.admit(14, 20), eng.bm.admit(3, 20)
    k = torch.zeros(4, 1, 128, dtype=torch.bfloat16)
    twice = eng.prepare_drafts([a, a], [[-1, 0], [-1, 0]])
    with pytest.raises(ValueError, match="takes one path"):
        eng.accept_drafts(twice, [[0], [0, 1]], k, k)
    db = eng.prepare_drafts([a, b], [[-1, 0], [-1, 0]])
    assert db.held == [14, 3] and db.positions.tolist() == [14, 15, 3, 4]
    eng.bm.prepare_append([b])
    with pytest.raises(ValueError, match="takes one path"):
        eng.accept_drafts(db, [[0], [0, 1]], k, k)
    assert [eng.bm.context_len(s) for s in (a, b)] == [14, 4]
