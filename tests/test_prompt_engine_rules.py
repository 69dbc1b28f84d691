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
