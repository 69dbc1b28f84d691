"""Beam selection on the GPU against the oracle: tokens, parents, flags and
histories exactly, scores to the rounding of fp32 and of the fp32 sums."""
import numpy as np
import pytest
import torch

from oracle import beam

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tests.conftest import build_native
    build_native()
    import paged_kv_cache_49_gb300 as m
    return m


def _near(got, want):
    """fp32 scores: half a step, 2^-24 of the value; the sum of exponentials, each
    off by exp2's 2^-22 and its argument's rounding (2^-24 of at most 30 for terms
    that count, times ln 2), summed in fp32 over 64 per thread and trees of 8
    levels (2^-24 each): under 2^-18 in all, and so the score by its logarithm. A
    score below -(2 - 2^-23) 2^127 = -3.4e38 by more than half a step of 2^104 has
    no nearer fp32 value than -inf: as 3e38 less than 3e38's negative is."""
    with np.errstate(over="ignore"):
        some = want.astype(np.float32) > -np.inf
    assert np.array_equal(some, got > -np.inf) and not np.isnan(got).any()
    diff = np.abs(np.where(some, got.astype(np.float64), 0) - np.where(some, want, 0))
    assert (diff <= np.where(some, np.abs(want) * 2.0 ** -24 + 2.0 ** -18, 0)).all(), diff.max()


def _check(pkv, logits, scores, finished=None, eos=-1, n=None, room=0, seed=0, given=True, **kw):
    """logits: a CUDA tensor [rows, vocab]; the rest numpy."""
    rng = np.random.default_rng(seed)
    groups, beams = scores.shape
    n = n or beams
    f = np.zeros(scores.shape, bool) if finished is None else finished
    hist = lens = None
    args = {}
    if room:
        hist = rng.integers(0, 1000, size=(groups, beams, room)).astype(np.int32)
        lens = rng.integers(0, room, size=(groups, beams)).astype(np.int32)
        args = dict(history=torch.from_numpy(hist).cuda(), lengths=torch.from_numpy(lens).cuda())
    if given:
        args["out"] = pkv.BeamBuffers(groups, n, room)
        args["workspace"] = pkv.BeamWorkspace(groups, beams, n, logits.shape[1])
        if room:
            args["out"].history.fill_(-9)
    else:
        args["candidates"] = n
    err = pkv.new_error_word()
    out = pkv.beam_select(logits, torch.from_numpy(scores.astype(np.float32)).cuda(),
                          None if finished is None else torch.from_numpy(finished).cuda(), eos, device_error=err, **args, **kw)
    torch.cuda.synchronize()
    assert pkv.read_device_error(err) == 0
    tail = None if not room else np.full((groups, n, room), -9 if given else 0, np.int32)
    want = beam.select(logits.double().cpu().numpy(), scores.astype(np.float32), f, eos, n, hist, lens, tail)
    for got, w in zip((out.tokens, out.parents, out.finished, out.lengths, out.history), want[1:]):
        assert np.array_equal(got.cpu().numpy(), w)
    _near(out.scores.cpu().numpy(), want[0])
    return out


def _logits(rng, rows, vocab, dtype=torch.bfloat16, size=2.0):
    return torch.from_numpy(size * rng.standard_normal((rows, vocab))).to(dtype).cuda()


def _scores(rng, groups, beams):
    return np.sort(-10 * rng.random((groups, beams)).astype(np.float32), axis=1)[:, ::-1].copy()


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 31, 64, 100, 255, 1000, 2047, 2048, 2049, 4099, 16384, 16385, 50001])
def test_vocabularies(pkv, vocab, dtype):
    rng = np.random.default_rng(vocab)
    _check(pkv, _logits(rng, 6, vocab, dtype), _scores(rng, 2, 3), n=6)


@pytest.mark.parametrize("groups,beams,n", [(1, 1, 1), (1, 1, 64), (3, 2, 5), (1, 32, 64), (70, 4, 8), (5, 16, 32), (400, 1, 2),
                                            (2, 32, 1), (7, 5, 9)])
def test_shapes(pkv, groups, beams, n):
    rng = np.random.default_rng(groups)
    finished = rng.random((groups, beams)) < 0.3
    _check(pkv, _logits(rng, groups * beams, 3001), _scores(rng, groups, beams), finished, 7, n, room=33, seed=n)
    _check(pkv, _logits(rng, groups * beams, 3001, torch.float32), _scores(rng, groups, beams), n=n, given=False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_chunks(pkv, dtype):
    """A vocabulary of many chunks a row, few rows; and many rows of large chunks."""
    rng = np.random.default_rng(1)
    _check(pkv, _logits(rng, 2, 1_000_003, dtype), _scores(rng, 1, 2), n=40)
    _check(pkv, _logits(rng, 320, 40_000, dtype), _scores(rng, 80, 4), n=8, room=5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_apart_and_off_boundaries(pkv, dtype):
    rng = np.random.default_rng(2)
    whole = _logits(rng, 9, 5000, dtype)
    for lo, hi in ((0, 4999), (1, 4000), (3, 5000), (2, 4997), (5, 13), (7, 16)):
        _check(pkv, whole[:8, lo:hi], _scores(rng, 4, 2), n=4)
    _check(pkv, whole[::2][:4, 6:], _scores(rng, 2, 2), n=4)


def test_the_first_step(pkv):
    """Beams that do not exist yet: one row counts, the others may hold NaN."""
    rng = np.random.default_rng(3)
    logits = _logits(rng, 8, 2000)
    logits[1:4] = float("nan")
    scores = np.zeros((2, 4), np.float32)
    scores[:, 1:] = -np.inf
    out = _check(pkv, logits, scores, np.zeros((2, 4), bool), 5, 4, room=6)
    assert (out.parents == 0).all()


def test_ties_go_to_the_lowest_index(pkv):
    """Equal logits by the thousand (more than a list holds), equal rows and scores
    off and on 16-byte boundaries."""
    for vocab in (20_000, 20_001):
        for dtype in DTYPES:
            logits = torch.zeros((4, vocab), dtype=dtype, device="cuda")
            out = _check(pkv, logits, np.array([[-1.0, -1.0], [-2.0, -1.0]], np.float32), n=9)
            assert out.tokens[0].tolist() == list(range(9)) and out.parents.tolist() == [[0] * 9, [1] * 9]
            logits[:, 777:15_000] = 1
            _check(pkv, logits, np.array([[-1.0, -1.0], [-2.0, -1.0]], np.float32), n=33)
            rng = np.random.default_rng(4)
            logits = _logits(rng, 1, vocab, dtype).repeat(4, 1).contiguous()
            _check(pkv, logits, np.array([[-1.0, -1.0], [-1.0, -1.0]], np.float32), n=12)
    # zeros of either sign are equal
    for dtype in DTYPES:
        logits = torch.zeros((2, 9000), dtype=dtype, device="cuda")
        logits[:, :4000] = -0.0
        logits[1, ::2] = -0.0
        _check(pkv, logits, np.array([[-1.0, -1.0]], np.float32), n=20)
        _check(pkv, logits - 3 * (torch.arange(9000, device="cuda") % 300 > 0).to(dtype), np.array([[0.0, -0.0]], np.float32), n=64)
    # logits of few values: thousands of ties with the last one taken
    coarse = torch.randint(0, 3, (6, 30_011), device="cuda").to(torch.bfloat16)
    _check(pkv, coarse, np.array([[-1.0, -1.5], [-2.0, -0.5], [0.0, 0.0]], np.float32), n=64)


def test_barred_tokens(pkv):
    rng = np.random.default_rng(5)
    logits = _logits(rng, 6, 10_000)
    allowed = torch.zeros(10_000, dtype=torch.bool)
    allowed[[17, 4000, 9999]] = True
    logits[:, ~allowed.cuda()] = float("-inf")
    _check(pkv, logits, _scores(rng, 3, 2), n=4)
    _check(pkv, logits, _scores(rng, 3, 2), n=16, room=3)  # fewer than n
    logits[:] = float("-inf")
    out = _check(pkv, logits, _scores(rng, 3, 2), n=3)
    assert (out.tokens == -1).all()


def test_nan_and_infinite_logits(pkv):
    rng = np.random.default_rng(6)
    logits = _logits(rng, 8, 5000, torch.float32)
    logits[0, 4321] = float("nan")
    logits[3, 0] = float("inf")
    logits[4] = float("nan")
    logits[6, :] = -3.0e38
    logits[6, 5] = 3.0e38
    scores = _scores(rng, 4, 2)
    scores[3, 1] = np.nan
    out = _check(pkv, logits, scores, n=5)
    assert (out.parents[0] == 1).all() and (out.parents[1] == 0).all()


MASKS = [-1.0e4, -65504.0, -1.0e9, -5.0e9, -1.0e10, -1.0e12, -1.0e18, -1.0e20, -1.0e30, -1.0e37, -3.3e38]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mask", MASKS)
def test_tokens_barred_by_a_large_finite_logit(pkv, mask, dtype):
    """Single tokens, the shares of whole warps, threads and chunks, all tokens but
    three, and whole rows."""
    rng = np.random.default_rng(13)
    vocab = 20_011
    for kept in (None, [17, 4000, 20_010]):
        logits = _logits(rng, 8, vocab, dtype)
        if kept is None:
            logits[:, rng.integers(0, vocab, 40)] = mask
            logits[1, :256] = mask
            logits[2, 4096:9001] = mask
            logits[3, 700:] = mask
        else:
            held = logits[:, kept].clone()
            logits[:] = mask
            logits[:, kept] = held
        logits[5] = mask
        logits[6:] = mask
        _check(pkv, logits, _scores(rng, 4, 2), n=8, room=3)
        _check(pkv, logits[:, 1:], _scores(rng, 2, 4), n=20)
    # many chunks a row
    logits = _logits(rng, 3, 400_000, dtype)
    logits[:, 1000:390_000] = mask
    logits[2] = mask
    _check(pkv, logits, _scores(rng, 1, 3), n=9)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [2.0e9, 1.0e20, 1.0e38, 3.0e38])
def test_rows_whose_largest_logit_is_large(pkv, size, dtype):
    rng = np.random.default_rng(14)
    logits = _logits(rng, 8, 9001, dtype)
    logits[0, 5000], logits[1, 8], logits[1, 7000] = size, size, size
    logits[2] += size
    logits[3] -= size
    logits[4], logits[4, ::3] = -size, -size / 2
    logits[5, 300:600] = -size
    logits[6], logits[6, 77] = size, size / 4
    _check(pkv, logits, _scores(rng, 4, 2), n=8)
    _check(pkv, logits, _scores(rng, 1, 8), n=30)


@pytest.mark.parametrize("at", [2.0 ** 24, -(2.0 ** 24), 2.0 ** 22, -(2.0 ** 22), 2.0 ** 23])
def test_logits_near_where_sums_are_formed_otherwise(pkv, at):
    """Neighbours of 2^24, of either sign, whose differences count: chunks and warps
    whose largest is below it beside others."""
    rng = np.random.default_rng(15)
    x = at + rng.integers(-9, 10, (6, 30_003))
    x[:, ::2] -= 40
    x[3:, 2048:] -= 8
    x[4, 25_000:] -= 30
    _check(pkv, torch.from_numpy(x).float().cuda(), _scores(rng, 3, 2), n=7)


@pytest.mark.parametrize("dtype", DTYPES)
def test_beams_with_scores_of_plus_infinity(pkv, dtype):
    """They come first, live and finished ones; of a live one the lowest tokens that are
    not barred, unless its logits are no numbers."""
    rng = np.random.default_rng(16)
    inf = np.inf
    scores = np.array([[-1.0, inf, -2.0], [inf, inf, -1.0], [inf, -3.0, inf], [-1.0, -2.0, inf], [inf, -inf, inf]], np.float32)
    finished = np.array([[0, 0, 0], [0, 1, 0], [0, 0, 0], [0, 1, 1], [1, 0, 1]], bool)
    for vocab in (5, 3000, 30_011):
        for n in (3, 20, 64):
            logits = _logits(rng, 15, vocab, dtype)
            logits[1, : vocab // 2] = -inf
            logits[3] = -inf
            logits[3, vocab - 1], logits[3, vocab // 2] = 1.0, -2.0
            logits[6, vocab // 3] = float("nan")
            logits[8] = -inf
            out = pkv.beam_select(logits, torch.from_numpy(scores).cuda(), torch.from_numpy(finished).cuda(), 2, candidates=n)
            want = beam.select(logits.double().cpu().numpy(), scores, finished, 2, n)
            for got, w in zip((out.tokens, out.parents, out.finished), want[1:]):
                assert np.array_equal(got.cpu().numpy(), w)
            got, large = out.scores.cpu().numpy(), want[0] == inf
            assert (got[large] == inf).all() and large.any(axis=1).tolist() == [True, True, False, True, True]
            _near(np.where(large, 0, got), np.where(large, 0, want[0]))


def test_all_beams_finished(pkv):
    rng = np.random.default_rng(7)
    logits = torch.full((4, 300), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = _check(pkv, logits, _scores(rng, 1, 4), np.ones((1, 4), bool), 2, 6, room=5)
    assert out.tokens.tolist() == [[2, 2, 2, 2, -1, -1]] and out.finished.tolist() == [[True] * 4 + [False] * 2]


def test_scores_far_apart_and_large(pkv):
    rng = np.random.default_rng(8)
    _check(pkv, _logits(rng, 4, 3000, torch.float32, 60.0), np.array([[-1000.0, -1001.0], [-3.0e4, -2.0]], np.float32), n=10)


def test_full_histories_are_reported(pkv):
    """A history without room takes no more; lengths outside it are clamped."""
    logits = torch.zeros((2, 10), device="cuda")
    logits[:, 3] = 5
    hist = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 2, 4)
    scores = torch.tensor([[-1.0, -9.0]], device="cuda")
    err = pkv.new_error_word()
    for length, want in ((4, [0, 1, 2, 3]), (3, [0, 1, 2, 3]), (9, [0, 1, 2, 3]), (-2, [3, 0, 0, 0])):
        lens = torch.tensor([[length, 0]], dtype=torch.int32, device="cuda")
        out = pkv.beam_select(logits, scores, history=hist, lengths=lens, candidates=1, device_error=err)
        assert out.history[0, 0].tolist() == want and out.lengths.tolist() == [[1 if length < 0 else 4]]
        assert pkv.read_device_error(err) == (0 if length == 3 else pkv.DEVERR_CONTEXT)


def test_steps_in_turn_on_streams_and_in_graphs(pkv):
    """Two buffers that take turns, as a search runs; captured and replayed."""
    rng = np.random.default_rng(9)
    groups, beams, vocab, room = 3, 4, 5003, 12
    logits = [_logits(rng, groups * beams, vocab) for _ in range(8)]

    def fresh():
        a, b = (pkv.BeamBuffers(groups, beams, room) for _ in range(2))
        a.scores[:, 1:] = float("-inf")
        return a, b

    ws = pkv.BeamWorkspace(groups, beams, beams, vocab)
    a, b = fresh()
    for x in logits:
        pkv.beam_select(x, a.scores, a.finished, 1, a.history, a.lengths, out=b, workspace=ws)
        a, b = b, a
    torch.cuda.synchronize()
    want = [t.clone() for t in (a.scores, a.tokens, a.finished, a.lengths, a.history)]
    # on the host, step by step
    s = np.zeros((groups, beams), np.float32)
    s[:, 1:] = -np.inf
    f, h, n = np.zeros((groups, beams), bool), np.zeros((groups, beams, room), np.int32), np.zeros((groups, beams), np.int32)
    for x in logits:
        best, _, _, f, n, h = beam.select(x.double().cpu().numpy(), s, f, 1, beams, h, n, np.zeros_like(h))
        s = best.astype(np.float32)
    assert np.array_equal(want[3].cpu().numpy(), n)
    for g in range(groups):
        for k in range(beams):
            assert want[4][g, k, :n[g, k]].tolist() == h[g, k, :n[g, k]].tolist()
    # the same from two graphs that share a workspace, on a side stream
    x = logits[0].clone()
    a, b = fresh()
    graphs = []
    side = torch.cuda.Stream()
    for src, dst in ((a, b), (b, a)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.beam_select(x, src.scores, src.finished, 1, src.history, src.lengths, out=dst, workspace=ws)
        graphs.append(g)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i, new in enumerate(logits):
            x.copy_(new)
            graphs[i % 2].replay()
    side.synchronize()
    assert all(torch.equal(g, w) for g, w in zip((a.scores, a.tokens, a.finished, a.lengths, a.history), want))
    for stream in (side, side.cuda_stream):
        out = pkv.beam_select(logits[3], torch.zeros((groups, beams), device="cuda"), stream=stream)
        side.synchronize()
        assert torch.equal(out.tokens, pkv.beam_select(logits[3], torch.zeros((groups, beams), device="cuda")).tokens)


def test_repeats_are_equal_to_the_bit(pkv):
    rng = np.random.default_rng(10)
    logits, scores = _logits(rng, 64, 30_001), torch.from_numpy(_scores(rng, 16, 4)).cuda()
    first = pkv.beam_select(logits, scores, candidates=8)
    for _ in range(10):
        again = pkv.beam_select(logits, scores, candidates=8)
        assert torch.equal(first.scores, again.scores) and torch.equal(first.tokens, again.tokens)


def test_two_calls_at_once(pkv):
    """On two streams, each with a workspace and buffers of its own, on one input."""
    rng = np.random.default_rng(12)
    logits = _logits(rng, 24, 30011, torch.bfloat16)
    scores = torch.from_numpy(-rng.random((6, 4), np.float32)).cuda()
    want = pkv.beam_select(logits, scores, candidates=8)
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [pkv.BeamWorkspace(6, 4, 8, 30011) for _ in range(2)]
    outs = [[pkv.BeamBuffers(6, 8) for _ in range(10)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(10):
        for st, w, o in zip(streams, spaces, outs):
            pkv.beam_select(logits, scores, out=o[i], workspace=w, stream=st)
    torch.cuda.synchronize()
    for x in (x for o in outs for x in o):
        assert torch.equal(x.scores, want.scores) and torch.equal(x.tokens, want.tokens) and torch.equal(x.parents, want.parents)


@pytest.mark.parametrize("told", [True, False])
def test_arguments_next_to_one_another_are_taken(pkv, told):
    """Inputs and outputs in one allocation, each output directly before or behind an
    input, with the least workspace: what the refusals' tests change one by one."""
    from paged_kv_cache_49_gb300 import _native as nat
    rng = np.random.default_rng(17)
    g, k, n, v, room = 2, 4, 8, 100, 5
    logits, scores = _logits(rng, g * k, v), _scores(rng, g, k)
    fin = rng.random((g, k)) < 0.3
    hist, lens = rng.integers(0, v, (g, k, room)).astype(np.int32), rng.integers(0, room, (g, k)).astype(np.int32)
    given = {"x": logits, "s": torch.from_numpy(scores), "fin": torch.from_numpy(fin), "h": torch.from_numpy(hist),
             "ln": torch.from_numpy(lens)}
    sizes = {"x": g * k * v * 2, "s": g * k * 4, "fin": g * k, "h": g * k * room * 4, "ln": g * k * 4, "so": g * n * 4, "to": g * n * 4,
             "po": g * n * 4, "fo": g * n, "lo": g * n * 4, "ho": g * n * room * 4}
    # sizes are multiples of 8 here; every output lies between two inputs or beside one
    order = ["so", "x", "to", "s", "po", "h", "fo", "fin", "lo", "ln", "ho"]
    space, at = torch.zeros(sum(sizes.values()), dtype=torch.uint8, device="cuda"), {}
    for name in order:
        at[name] = sum(sizes[o] for o in at)
    view = lambda name, dtype: space[at[name]:at[name] + sizes[name]].view(dtype)
    for name, t in given.items():
        view(name, t.dtype).copy_(t.reshape(-1))
    view("ho", torch.int32).fill_(-9)
    need = 256 * ((g * k * 8 + 255) // 256) + 256 * ((g * k * n * 8 + 255) // 256)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    p = {name: space.data_ptr() + at[name] if told or name not in ("h", "ln", "lo", "ho") else None for name in order}
    st = nat.lib.pkv_beam_select(p["x"], v, 2, p["s"], p["fin"], 1, g, k, n, v, p["h"], p["ln"], room if told else 0, p["so"], p["to"],
                                 p["po"], p["fo"], p["lo"], p["ho"], -(-ws.data_ptr() // 256) * 256, need, None,
                                 torch.cuda.current_stream().cuda_stream)
    assert st == nat.PKV_OK
    want = beam.select(logits.double().cpu().numpy(), scores, fin, 1, n, hist, lens, np.full((g, n, room), -9, np.int32))
    got = [view(name, dtype).cpu().numpy().reshape(g, n, -1) for name, dtype in (
        ("so", torch.float32), ("to", torch.int32), ("po", torch.int32), ("fo", torch.bool), ("lo", torch.int32), ("ho", torch.int32))]
    _near(got[0][..., 0], want[0])
    for a, b in list(zip(got[1:], want[1:]))[:5 if told else 3]:
        assert np.array_equal(a, b.reshape(a.shape))
    for name, t in given.items():  # as they were
        assert torch.equal(view(name, t.dtype).cpu(), t.reshape(-1).cpu())


def test_refusals_on_the_gpu(pkv):
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
    logits, scores, i32 = z(4, 50), z(2, 2), torch.int32
    hist, lens = z(2, 2, 5, dtype=i32), z(2, 2, dtype=i32)
    for a, kw in (((z(4, 50).half(), scores), {}), ((z(3, 50), scores), {}), ((z(50, 4).T, scores), {}), ((logits, scores.double()), {}),
                  ((logits, z(4)), {}), ((logits, scores, z(2, 2)), {}), ((logits, scores, z(2, 3, dtype=torch.bool)), {}),
                  ((logits, scores), dict(history=hist)), ((logits, scores), dict(history=hist, lengths=z(4, dtype=i32))),
                  ((logits, scores), dict(history=hist.long(), lengths=lens)), ((logits, scores), dict(out=pkv.BeamBuffers(1, 2))),
                  ((logits, scores), dict(history=hist, lengths=lens, out=pkv.BeamBuffers(2, 2))),
                  ((logits, scores), dict(history=hist, lengths=lens, out=pkv.BeamBuffers(2, 2, 6))),
                  ((logits, scores), dict(out=pkv.BeamBuffers(2, 2), candidates=3))):
        with pytest.raises(ValueError):
            pkv.beam_select(*a, **kw)
    both = pkv.BeamBuffers(2, 2, 5)
    with pytest.raises(ValueError):  # in place
        pkv.beam_select(logits, both.scores, both.finished, 1, both.history, both.lengths, out=both)
    for kw in (dict(eos=50), dict(finished=z(2, 2, dtype=torch.bool)), dict(candidates=65)):
        with pytest.raises(pkv.PkvError):
            pkv.beam_select(logits, scores, **kw)
    with pytest.raises(pkv.PkvError):  # a workspace of a smaller shape
        pkv.beam_select(z(400, 50), z(200, 2), workspace=pkv.BeamWorkspace(1, 1, 1, 5))
