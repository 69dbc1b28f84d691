"""Refusals of the engine's prompt and draft calls (no GPU): each leaves the
block manager as it was, and nothing is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def engine():
    from tests.conftest import build_native
    build_native()
    from paged_kv_cache_49_gb300.engine import PagedKVEngine
    return lambda **kw: PagedKVEngine(40, 2, 1, device="cpu", **kw)


PARENTS = [-1, 0, 0, 1, -1]  # 0 and 4 follow the context; 1 and 2 follow 0, 3 follows 1


@pytest.mark.parametrize("path", [[2, 1], [1], [3, 1], [0, 3], [0, 1, 2], [0, 4], [4, 0], [1, 3], [0, 2, 3]])
def test_a_path_goes_from_parent_to_child(engine, path):
    """The keys of any other order are rotated for other positions."""
    eng = engine()
    a, b = eng.bm.admit(14, 20), eng.bm.admit(3, 20)
    db = eng.prepare_drafts([b, a], [[-1], PARENTS])
    assert db.parents == [[-1], PARENTS]
    k = torch.zeros(6, 1, 128, dtype=torch.bfloat16)
    before = eng.bm.stats()
    with pytest.raises(ValueError, match="parent"):
        eng.accept_drafts(db, [[0], path], k, k)
    assert [eng.bm.context_len(s) for s in (a, b)] == [14, 3] and eng.bm.stats() == before


@pytest.mark.parametrize("path", [[], [0], [4], [0, 1], [0, 2], [0, 1, 3]])
def test_paths_of_the_tree_pass_the_checks(engine, path, monkeypatch):
    import contextlib

    from paged_kv_cache_49_gb300 import _native as nat
    eng = engine()
    a = eng.bm.admit(14, 20)
    db = eng.prepare_drafts([a], [PARENTS])
    k = torch.zeros(5, 1, 128, dtype=torch.bfloat16)
    called = []
    monkeypatch.setattr(eng, "_on", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(nat, "append", lambda k, v, slots, *rest: called.append(slots.tolist()))
    slots = eng.accept_drafts(db, [path], k, k)
    assert called == [slots] and [i for i, s in enumerate(slots) if s >= 0] == sorted(path)
    assert eng.bm.context_len(a) == 14 + len(path)
    assert [slots[i] for i in path] == eng.bm.slots(a, 14, len(path))


def test_a_chunk_behind_tokens_that_nothing_wrote_says_where_it_starts(engine):
    """Without first a prompt's rows are its last ones: right for all of it, or for
    what follows tokens that are in the cache, not for its first chunk."""
    eng = engine()
    a, b = eng.bm.admit(100, 5), eng.bm.admit(40, 5)
    for counts in ([33, 40], [99, 40], [100, 39]):
        with pytest.raises(ValueError, match="first"):
            eng.prepare_prefill([a, b], counts)
    done = [0, 0]
    for counts in ([33, 0], [0, 40], [67, 0]):
        pb = eng.prepare_prefill([a, b], counts, done)
        assert pb.positions.tolist() == [f + i for f, c in zip(done, counts) for i in range(c)]
        done = [d + c for d, c in zip(done, counts)]
        assert pb.ctx.tolist() == done
    whole = eng.prepare_prefill([b, a], [40, 100])
    assert whole.positions.tolist() == [*range(40), *range(100)] and whole.ctx.tolist() == [40, 100]
    assert eng.prepare_prefill([a, b], [0, 40]).positions.tolist() == [*range(40)]


def test_the_rest_behind_cached_and_shared_tokens_needs_no_start(engine):
    eng = engine(prefix_cache=True)
    tokens = list(range(100))
    eng.bm.admit(100, 5, tokens=tokens)
    c = eng.bm.admit(110, 5, tokens=tokens + list(range(10)))
    with pytest.raises(ValueError, match="first"):
        eng.prepare_prefill([c], [13])
    assert eng.prepare_prefill([c], [14]).positions.tolist() == [*range(96, 110)]
    eng = engine()
    eng.bm.admit(70, 5, 0, 64)
    d = eng.bm.admit(80, 5, 0, 64)
    with pytest.raises(ValueError, match="first"):
        eng.prepare_prefill([d], [15])
    assert eng.prepare_prefill([d], [16]).positions.tolist() == [*range(64, 80)]
    eng = engine()
    e = eng.bm.admit(50, 5)
    f, = eng.bm.fork(e, 1)
    assert eng.prepare_prefill([f], [7]).positions.tolist() == [*range(43, 50)]


@pytest.mark.parametrize("counts,first", [([5, 1], [96, 0]), ([101, 1], [0, 0]), ([0, 1], [101, 0]), ([0, 1], [-1, 0]),
                                          ([3, 1], [-1, 0]), ([-1, 1], [5, 0]), ([1, 40], None), ([4, 3], [100, 0])])
def test_a_chunk_lies_within_its_sequence(engine, counts, first):
    """Reserved pages behind the context are the next steps'."""
    eng = engine()
    a, b = eng.bm.admit(100, 30), eng.bm.admit(3, 20)
    with pytest.raises(ValueError):
        eng.prepare_prefill([a, b], counts, first)
    with pytest.raises(ValueError):
        eng.prepare_prefill([a, b], [100, 3], [0])


def test_tokens_behind_a_prompt_that_has_come_need_no_start(engine):
    """A decode row, or the last chunk: what precedes it has been brought."""
    eng = engine()
    a, b = eng.bm.admit(100, 30), eng.bm.admit(3, 20)
    eng.prepare_prefill([a], [60], [0])
    assert eng.prepare_prefill([a, b], [40, 3]).positions.tolist() == [*range(60, 100), 0, 1, 2]
    child, = eng.bm.fork(a, 1)
    for _ in range(3):  # their appends are the decode steps'
        eng.bm.prepare_append([a, b, child])
    assert eng.prepare_prefill([a, b, child], [1, 1, 2]).positions.tolist() == [102, 5, 101, 102]
    # a chunk out of order does not count for what precedes it
    c = eng.bm.admit(50, 5)
    eng.prepare_prefill([c], [10], [40])
    with pytest.raises(ValueError, match="first"):
        eng.prepare_prefill([c], [20])
    # a preempted sequence comes back on fresh pages, all its tokens to be recomputed
    eng.bm.preempt(a)
    eng.bm.resume(a)
    for count in (1, 43):
        with pytest.raises(ValueError, match="first"):
            eng.prepare_prefill([a], [count])
    assert eng.prepare_prefill([a], [103]).positions.tolist() == [*range(103)]
    assert eng.prepare_prefill([a], [1]).positions.tolist() == [102]
    eng.bm.free(a)
    assert a not in eng.bm.prompt and a not in eng.bm.written


def test_written_positions_count(engine, monkeypatch):
    from paged_kv_cache_49_gb300 import _native as nat
    monkeypatch.setattr(nat, "append", lambda *a, **kw: None)
    eng = engine()
    a = eng.bm.admit(100, 30)
    k = torch.zeros(64, 1, 128, dtype=torch.bfloat16)
    eng.write_positions(a, 0, k, k)
    assert eng.prepare_prefill([a], [36]).positions.tolist() == [*range(64, 100)]


@pytest.mark.parametrize("stream,error", [("none", ValueError), (object(), TypeError)])
def test_a_refused_stream_leaves_the_device_as_it_was(engine, monkeypatch, stream, error):
    from paged_kv_cache_49_gb300 import _native as nat
    entered = []

    class Device:
        def __init__(self, index):
            pass

        def __enter__(self):
            entered.append(1)

        def __exit__(self, *exc):
            entered.pop()

    monkeypatch.setattr(torch.cuda, "device", Device)
    with pytest.raises(error):
        with nat._LaunchOn(1, stream):
            pass
    assert not entered


def test_inputs_on_the_host_are_refused_as_such(engine, monkeypatch):
    import contextlib
    eng = engine()
    monkeypatch.setattr(eng, "_on", lambda stream: contextlib.nullcontext())
    a = eng.bm.admit(10, 5)
    x = torch.zeros(10, 2, 128, dtype=torch.bfloat16)
    pb = eng.prepare_prefill([a], [10])
    with pytest.raises(ValueError, match="CUDA"):
        eng.run_prefill(pb, x, x[:, :1].contiguous(), x[:, :1].contiguous(), 0.1, None, stream=7)
