"""Beam search without a GPU: the oracle's selection against a plain search, the
manager's reorder against the oracle's, and what the calls refuse."""
import math
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import beam
from oracle import block_manager as obm


@pytest.fixture(scope="module")
def pkv():
    from tests.conftest import build_native
    build_native()
    import paged_kv_cache_49_gb300 as m
    return m


# ---- the oracle's selection ---------------------------------------------------


def test_selection_against_every_candidate():
    rng = np.random.default_rng(0)
    logits, scores = rng.standard_normal((6, 11)), -rng.random((2, 3))
    finished = np.array([[0, 1, 0], [0, 0, 0]], bool)
    got = beam.select(logits, scores, finished, 4, 5)
    for b in range(2):
        every = []
        for k in range(3):
            if finished[b, k]:
                every.append((-scores[b, k], k * 11 + 4))
                continue
            lse = math.log(sum(math.exp(x) for x in logits[b * 3 + k]))
            every += [(-(scores[b, k] + x - lse), k * 11 + v) for v, x in enumerate(logits[b * 3 + k])]
        every.sort()
        assert np.allclose(got[0][b], [-s for s, _ in every[:5]])
        assert (got[2][b] * 11 + got[1][b]).tolist() == [at for _, at in every[:5]]


def test_selection_of_ties_bars_and_missing_candidates():
    logits = np.zeros((2, 4))
    got = beam.select(logits, np.array([[-1.0, -1.0]]), np.zeros((1, 2), bool), -1, 6)
    assert got[1].tolist() == [[0, 1, 2, 3, 0, 1]] and got[2].tolist() == [[0, 0, 0, 0, 1, 1]]
    logits[0, 1:] = -np.inf
    logits[1] = np.nan
    got = beam.select(logits, np.array([[0.0, 0.0]]), np.zeros((1, 2), bool), -1, 3)
    assert got[1].tolist() == [[0, -1, -1]] and got[0][0, 0] == 0 and (got[0][0, 1:] == -np.inf).all()
    hist = np.arange(6, dtype=np.int32).reshape(1, 2, 3)
    got = beam.select(np.zeros((2, 4)), np.array([[-np.inf, -2.0]]), np.array([[False, True]]), 3, 2, hist,
                      np.array([[1, 2]], np.int32), np.full((1, 2, 3), 9, np.int32))
    assert got[1].tolist() == [[3, -1]] and got[3].tolist() == [[True, False]]
    assert got[4].tolist() == [[2, 0]] and got[5].tolist() == [[[3, 4, 9], [9, 9, 9]]]


def test_selection_of_large_logits():
    """Against sums of fractions: rows of masks alone, masks behind other logits, and
    logits so large that float64 does not hold what the beams' scores add."""
    rng = np.random.default_rng(3)
    for size in (1e9, 1e20, 1e30, 3e38):
        logits, scores = rng.standard_normal((4, 6)).astype(np.float32).astype(np.float64), -rng.random((2, 2))
        size = float(np.float32(size))
        logits[0, 2:], logits[1], logits[2, 1], logits[3, ::2] = -size, -size, size, size
        got = beam.select(logits, scores, np.zeros((2, 2), bool), -1, 12)
        for b in range(2):
            every = []
            for k in range(2):
                x = [Fraction(v) for v in logits[2 * b + k]]
                rest = math.log(sum(math.exp(float(v - max(x))) for v in x))
                every += [(-(v - max(x) + Fraction(scores[b, k] - rest)), k * 6 + i) for i, v in enumerate(x)]
            every.sort()
            assert (got[2][b] * 6 + got[1][b]).tolist() == [at for _, at in every]
            assert np.allclose(got[0][b], [-float(s) for s, _ in every])


# ---- reorder --------------------------------------------------------------------


def _same(o, n, ids):
    assert o.stats() == n.stats()
    for s in ids:
        assert o.table(s) == n.table(s) and o.context_len(s) == n.context_len(s)
    for b in range(o.num_blocks):
        assert o.ref[b] == n.refcount(b)


def _try(pkv, f):
    try:
        return f(), None
    except (obm.PoolExhausted, pkv.PoolExhausted):
        return None, "nomem"
    except (obm.ReservationExceeded, pkv.ReservationExceeded):
        return None, "nospc"
    except (obm.BlockManagerError, pkv.PkvError):
        return None, "inval"


@pytest.mark.parametrize("incremental", [False, True])
@pytest.mark.parametrize("seed", range(8))
def test_random_searches_match_the_oracle(pkv, seed, incremental):
    r = random.Random(seed)
    bt = r.choice([8, 16, 32])
    blocks = r.choice([24, 60, 200])
    o = obm.BlockManager(blocks, bt, incremental=incremental)
    n = pkv.BlockManager(blocks, bt, incremental=incremental)
    searches = []
    refused = 0
    for _ in range(120):
        what = r.random()
        if what < 0.12 or not searches:
            args = (r.randrange(1, 5 * bt), r.randrange(1, 4 * bt))
            a, b = _try(pkv, lambda: o.admit(*args)), _try(pkv, lambda: n.admit(*args))
            assert a == b
            if a[0] is None:
                continue
            k = r.randrange(0, 5)
            x, y = _try(pkv, lambda: o.fork(a[0], k)), _try(pkv, lambda: n.fork(a[0], k))
            assert x == y
            searches.append([a[0]] + (x[0] or []))
        elif what < 0.2:
            ids = searches.pop(r.randrange(len(searches)))
            for s in ids:
                o.free(s), n.free(s)
        elif what < 0.6:
            ids = r.choice(searches)
            a, b = _try(pkv, lambda: o.prepare_append(ids)), _try(pkv, lambda: n.prepare_append(ids))
            assert a[1] == b[1]
            if a[1] is None:
                assert [list(map(int, a[0][0])), [tuple(p) for p in a[0][1]]] == [b[0][0], b[0][1]]
        else:
            ids = r.choice(searches)
            parents = [r.randrange(len(ids)) for _ in ids]
            a, b = _try(pkv, lambda: o.reorder(ids, parents)), _try(pkv, lambda: n.reorder(ids, parents))
            assert a == b
            refused += a[1] is not None
        _same(o, n, [s for ids in searches for s in ids])
    for ids in searches:
        for s in ids:
            o.free(s), n.free(s)
    _same(o, n, [])
    assert n.stats()["free"] == blocks


@pytest.mark.parametrize("incremental", [False, True])
def test_reorder_shares_blocks_and_copies_on_write(pkv, incremental):
    bm = pkv.BlockManager(40, 16, incremental=incremental)
    a = bm.admit(20, 12)
    ids = [a] + bm.fork(a, 2)
    bm.prepare_append(ids)  # each its own partial block now
    tables = [bm.table(s) for s in ids]
    bm.reorder(ids, [1, 1, 1])
    assert [bm.table(s)[:2] for s in ids] == [tables[1][:2]] * 3 and bm.refcount(tables[1][1]) == 3
    assert bm.table(ids[1]) == tables[1]
    slots, pairs = bm.prepare_append(ids)
    assert len(set(s // 16 for s in slots)) == 3 and [p[0] for p in pairs] == [tables[1][1]] * 2
    bm.reorder(ids, [0, 1, 2])
    assert bm.stats()["cow_copies"] == 4
    for s in ids:
        bm.free(s)
    assert bm.stats()["free"] == 40


def test_a_permutation_moves_tables_only(pkv):
    bm = pkv.BlockManager(40, 16)
    ids = [bm.admit(5 + 16 * i, 4) for i in range(3)]
    tables, stats = [bm.table(s) for s in ids], bm.stats()
    bm.reorder(ids, [2, 0, 1])
    assert [bm.table(s) for s in ids] == [tables[2], tables[0], tables[1]] and bm.stats() == stats
    assert [bm.context_len(s) for s in ids] == [37, 5, 21]
    assert [bm.prompt[s] for s in ids] == [37, 5, 21]


def test_reorder_refuses(pkv):
    bm = pkv.BlockManager(8, 16)
    a, b = bm.admit(40, 8), bm.admit(8, 24)
    state = bm.stats(), bm.table(a), bm.table(b)
    for ids, parents in (([a, a], [0, 1]), ([a, 99], [0, 1]), ([a, b], [0, 2]), ([a, b], [-1, 0])):
        with pytest.raises(pkv.PkvError):
            bm.reorder(ids, parents)
    with pytest.raises(ValueError):
        bm.reorder([a, b], [0])
    c = bm.admit(1, 15)
    bm.preempt(c)
    with pytest.raises(pkv.PkvError):
        bm.reorder([a, c], [0, 0])
    assert (bm.table(a), bm.table(b)) == state[1:]
    bm.free(c)
    # a's rest and a spare, and b's release leaves too little for neither: 3 + 2 + 3 blocks
    full = pkv.BlockManager(7, 16)
    a, b = full.admit(20, 70), full.admit(1, 1)
    was = full.stats(), full.table(a), full.table(b)
    with pytest.raises(pkv.PoolExhausted):
        full.reorder([a, b], [0, 0])
    assert (full.stats(), full.table(a), full.table(b)) == was
    bm.reorder([], [])


# ---- refusals -------------------------------------------------------------------


def test_c_calls_refuse(pkv):
    from paged_kv_cache_49_gb300 import _native as nat
    L, P = nat.lib, 4096

    def call(x=P, stride=100, size=2, s=P, fin=None, eos=-1, g=2, k=4, n=8, v=100, h=None, ln=None, room=0, so=P, to=P, po=P,
             fo=P, lo=None, ho=None, ws=P, nb=1 << 20):
        return L.pkv_beam_select(x, stride, size, s, fin, eos, g, k, n, v, h, ln, room, so, to, po, fo, lo, ho, ws, nb, None,
                                 None)
    for bad in (dict(x=None), dict(s=None), dict(so=None), dict(to=None), dict(po=None), dict(fo=None), dict(ws=None), dict(g=0),
                dict(k=0), dict(n=0), dict(v=0), dict(stride=99), dict(eos=100), dict(eos=-2), dict(fin=P), dict(h=P),
                dict(h=P, ln=P, lo=P, ho=P), dict(h=P, ln=P, lo=P, room=4), dict(room=-1), dict(x=P + 1), dict(ws=P + 16),
                dict(nb=64)):
        assert call(**bad) == nat.PKV_EINVAL, bad
    for bad in (dict(k=33), dict(n=65), dict(size=1), dict(size=8)):
        assert call(**bad) == nat.PKV_EUNSUPPORTED, bad
    for bad in (dict(k=32, v=1 << 26, stride=1 << 26), dict(v=(1 << 30) + 1, stride=1 << 31, k=1), dict(g=1 << 21)):
        assert call(**bad) == nat.PKV_ERANGE, bad
    assert L.pkv_beam_workspace_size(2, 4, 8, 100) > 0
    for shape in ((0, 4, 8, 100), (2, 33, 8, 100), (2, 4, 65, 100), (2, 4, 8, 0)):
        assert L.pkv_beam_workspace_size(*shape) == 0


def _apart():
    """Arguments that the call takes, each at an address of its own."""
    names = ("x", "s", "fin", "h", "ln", "so", "to", "po", "fo", "lo", "ho", "ws")
    a = {name: (i + 1) << 24 for i, name in enumerate(names)}
    return dict(a, stride=100, size=2, eos=1, g=2, k=4, n=8, v=100, room=5, nb=1 << 20)


def _select(a):
    from paged_kv_cache_49_gb300 import _native as nat
    return nat.lib.pkv_beam_select(a["x"], a["stride"], a["size"], a["s"], a["fin"], a["eos"], a["g"], a["k"], a["n"], a["v"],
                                   a["h"], a["ln"], a["room"], a["so"], a["to"], a["po"], a["fo"], a["lo"], a["ho"], a["ws"],
                                   a["nb"], None, None)


@pytest.mark.parametrize("told", [True, False])
def test_each_argument_is_refused_by_its_own_check(pkv, told):
    """One argument at a time is wrong, the others are such as the call takes (as
    test_gpu_beam.py shows); each checked bound from its refused side."""
    from paged_kv_cache_49_gb300 import _native as nat
    ok = _apart()
    if not told:
        ok.update(h=None, ln=None, lo=None, ho=None, room=0)
    need = 256 * ((2 * 4 * 8 + 255) // 256) + 256 * ((2 * 4 * 8 * 8 + 255) // 256)  # one chunk a row
    bad = [dict(x=None), dict(s=None), dict(so=None), dict(to=None), dict(po=None), dict(fo=None), dict(ws=None), dict(g=0),
           dict(k=0), dict(n=0), dict(v=0), dict(g=-1), dict(stride=99), dict(stride=-100), dict(eos=100), dict(eos=-2), dict(eos=-1),
           dict(room=-1), dict(x=ok["x"] + 1), dict(x=ok["x"] + 2, size=4), dict(ws=ok["ws"] + 128), dict(nb=need - 1), dict(nb=0)]
    if told:
        bad += [dict(h=None), dict(ln=None), dict(lo=None), dict(ho=None), dict(room=0)]
    else:
        bad += [dict(h=1 << 26, room=5), dict(ln=1 << 26, room=5), dict(lo=1 << 26, room=5), dict(ho=1 << 26, room=5)]
    for change in bad:
        assert _select({**ok, **change}) == nat.PKV_EINVAL, change
    for change in (dict(k=33), dict(n=65), dict(size=1), dict(size=8)):
        assert _select({**ok, **change}) == nat.PKV_EUNSUPPORTED, change


def test_outputs_on_inputs_are_refused(pkv):
    """Whole, by their last byte and by their first."""
    from paged_kv_cache_49_gb300 import _native as nat
    g, k, n, v, room = 2, 4, 8, 100, 5
    inputs = {"x": (g * k - 1) * 128 * 2 + v * 2, "s": g * k * 4, "fin": g * k, "h": g * k * room * 4, "ln": g * k * 4}
    outputs = {"so": g * n * 4, "to": g * n * 4, "po": g * n * 4, "fo": g * n, "lo": g * n * 4, "ho": g * n * room * 4}
    at = {name: (i + 1) << 20 for i, name in enumerate([*inputs, *outputs])}
    for i, size in inputs.items():
        for o, length in outputs.items():
            for place in (at[i], at[i] + (size - 1) // 4 * 4, at[i] - length + 1):
                w = dict(at, **{o: place})
                got = nat.lib.pkv_beam_select(w["x"], 128, 2, w["s"], w["fin"], 1, g, k, n, v, w["h"], w["ln"], room, w["so"],
                                              w["to"], w["po"], w["fo"], w["lo"], w["ho"], 1 << 28, 1 << 20, None, None)
                assert got == nat.PKV_EINVAL, (i, o, place)


def test_python_calls_refuse(pkv):
    logits, scores = torch.zeros((4, 50)), torch.zeros((2, 2))
    with pytest.raises(ValueError, match="scores"):  # host tensors
        pkv.beam_select(logits, scores)
    for bad in (logits.half(), logits[0], logits.long()):
        with pytest.raises(ValueError, match="logits"):
            pkv.beam_select(bad, scores)
    with pytest.raises(pkv.PkvError):
        pkv.BeamWorkspace(1, 33, 4, 10, device="cpu")
