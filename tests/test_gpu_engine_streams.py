"""Engine calls on a side stream whose inputs the caller lets go at once: their
memory is not given out anew before the stream is done with them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, HKV, D, T = 16, 4, 128, 200
SCALE = D ** -0.5


@pytest.fixture(scope="module")
def pkv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tests.conftest import build_native
    build_native()
    import paged_kv_cache_49_gb300 as m
    return m


def _inputs(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((n, h, D), generator=g, device="cuda").bfloat16() for h in (HQ, HKV, HKV)]


def _overwrite(shapes):
    """New tensors over what has been let go: zeros, which every index may be."""
    return [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(2)]


def _pass(pkv, side):
    """A prompt, a tree, its acceptance and plain appends; all results."""
    eng = pkv.PagedKVEngine(40, HQ, HKV, D)
    eng.k_cache.zero_(), eng.v_cache.zero_()
    ws = pkv.PrefillWorkspace()
    rope = pkv.RopeSpec(pkv.rope_table(400, D))
    a, b = eng.bm.admit(T, 30), eng.bm.admit(40, 30)
    results, kept = [], []

    def call(fn, *inputs):
        torch.cuda.synchronize()
        if side is not None:
            with torch.cuda.stream(side):
                torch.cuda._sleep(100_000_000)  # some 50 ms
        shapes = [(tuple(t.shape), t.dtype) for t in inputs]
        got = fn()
        return got, shapes

    def prompt():
        pb = eng.prepare_prefill([a], [T])
        q, k, v = _inputs(T, 1)
        got, shapes = call(lambda: eng.run_prefill(pb, q, k, v, SCALE, ws, rope, stream=side),
                           pb.positions, pb.tables, pb.ctx, pb.starts, pb.slots, q, k, v)
        return got, shapes

    def drafts():
        db = eng.prepare_drafts([a], [[-1, 0, 1, 0]])
        q, k, v = _inputs(4, 2)
        (out, keys), shapes = call(lambda: eng.run_drafts(db, q, k, v, SCALE, ws, rope, stream=side),
                                   db.positions, db.tables, db.ctx, db.starts, db.masks, db.slots, q, k, v)
        return (out, keys), shapes

    def accept():
        db = eng.prepare_drafts([a], [[-1, 0, 1, 0]])
        _, k, v = _inputs(4, 3)
        return call(lambda: eng.accept_drafts(db, [[0, 1, 2]], k, v, stream=side), k, v)

    def write():
        _, k, v = _inputs(40, 4)
        return call(lambda: eng.write_positions(b, 0, k, v, stream=side), k, v)

    def append():
        _, k, v = _inputs(2, 5)
        return call(lambda: eng.append_tokens([a, b], k, v, stream=side), k, v)

    for step in (prompt, drafts, accept, write, append):
        got, shapes = step()  # its inputs are gone now
        kept.append(_overwrite(shapes + [((n,), torch.int64) for n in (2, 4, 40)]))
        torch.cuda.synchronize()
        results += [x.clone() for x in (got if isinstance(got, tuple) else (got,)) if torch.is_tensor(x)]
        results += [eng.k_cache.clone(), eng.v_cache.clone()]
    assert ws.read_error() == 0 and pkv.read_device_error(eng.error) == 0
    return results


def test_inputs_let_go_while_a_side_stream_waits(pkv):
    want = _pass(pkv, None)
    got = _pass(pkv, torch.cuda.Stream())
    assert len(got) == len(want)
    for i, (g, w) in enumerate(zip(got, want)):
        assert torch.equal(g, w), i


@pytest.mark.parametrize("handle", ["side", "default"])
def test_streams_given_as_handles(pkv, handle):
    """cudaStream_t values, the default stream's zero among them."""
    side = torch.cuda.Stream() if handle == "side" else torch.cuda.default_stream()
    raw = side.cuda_stream
    assert raw == 0 or handle == "side"
    rope = pkv.RopeSpec(pkv.rope_table(400, D))
    results = []
    for stream in (None, raw):
        eng, ws = pkv.PagedKVEngine(40, HQ, HKV, D), pkv.PrefillWorkspace()
        eng.k_cache.zero_(), eng.v_cache.zero_()
        a, b = eng.bm.admit(T, 30), eng.bm.admit(1, 30)
        torch.cuda.synchronize()
        q, k, v = _inputs(T, 1)
        torch.cuda.synchronize()
        out = eng.run_prefill(eng.prepare_prefill([a], [T]), q, k, v, SCALE, ws, rope, stream=stream)
        eng.write_positions(b, 0, k[:1].contiguous(), v[:1].contiguous(), stream=stream)
        eng.append_tokens([a, b], k[:2].contiguous(), v[:2].contiguous(), stream=stream)
        torch.cuda.synchronize()
        results.append((out.clone(), eng.k_cache.clone(), eng.v_cache.clone()))
    assert all(torch.equal(x, y) for x, y in zip(*results))
