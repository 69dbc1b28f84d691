"""Prompt and tree attention at the edges of what the interface allows."""
import numpy as np
import pytest
import torch

from oracle import prompt_attention as po
from tests.prompt_batches import Batch
from tests.test_gpu_prompt_attention import _call, _check, _dev, _ref, _run, pkv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,held,hq,hkv,bt", [
    ([700], [256], 64, 8, 16),
    ([600], [448], 32, 8, 16),
    ([5, 900, 1], [400, 400, 396], 16, 2, 8),
    ([300, 2000, 40], [300, 0, 30], 8, 2, 32),
    ([3, 900, 1], [20011, 700, 300], 8, 2, 16),  # with a context that is cut
])
def test_chunks_longer_than_their_context(pkv, new, held, hq, hkv, bt):  # noqa: F811
    """The bit is set, rows before position 0 give zeros, all others are exact."""
    b = Batch(len(new) + new[0], new, held, hq, hkv, bt, first_row=1, rows_behind=2)
    d = _dev(pkv, b, False)
    ws = pkv.PrefillWorkspace()
    out = torch.full_like(d["q"], 7.0)
    _call(pkv, d, b.scale, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert ws.read_error() == pkv.DEVERR_CONTEXT
    lo, hi = int(b.starts[0]), int(b.starts[-1])
    assert (out[:lo] == 7.0).all() and (out[hi:] == 7.0).all()
    _check(out, _ref(b, False), slice(lo, hi))
    for s, (n, c) in enumerate(zip(new, held)):
        first = int(b.starts[s])
        assert (out[first : first + max(n - c, 0)] == 0).all()


def test_a_context_clamped_to_its_table(pkv):  # noqa: F811
    """More tokens than the table row holds: those that it holds are the context."""
    b = Batch(31, [700], [256], 16, 4, 16)
    d = _dev(pkv, b, False)
    ws = pkv.PrefillWorkspace()
    out = torch.full_like(d["q"], 7.0)
    d["ctx"][0] = 1 << 30
    _call(pkv, d, b.scale, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert ws.read_error() == pkv.DEVERR_CONTEXT
    _check(out, _ref(b, False))
    assert np.isfinite(out.float().cpu().numpy()).all()


def test_sequences_laid_over_the_same_rows(pkv):  # noqa: F811
    """query_starts that goes back: more items than the rows could have. The bit
    is set, and the sequence that has its rows to itself is exact."""
    held = [20011] * 10
    b = Batch(32, [320] + [0] * 8 + [40], held, 8, 1, 16)
    d = _dev(pkv, b, False)
    d["starts"].copy_(torch.tensor([0, 320] * 5 + [360], dtype=torch.int32))
    ws = pkv.PrefillWorkspace()
    out = torch.full_like(d["q"], 7.0)
    _call(pkv, d, b.scale, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert ws.read_error() == pkv.DEVERR_QUERY
    ref = po.prompt_attention(b.q[320:], b.k, b.v, b.tables[9:], b.ctx[9:], np.array([0, 40]), b.scale)
    _check(out[320:], ref)


@pytest.mark.parametrize("ctas", [1, 5, 100])
@pytest.mark.parametrize("tree", [False, True])
def test_a_workspace_of_fewer_ranges(pkv, tree, ctas):  # noqa: F811
    """Fewer CTAs do the work, and nothing behind the given bytes is touched."""
    b = Batch(33, [64, 33, 1], [9000, 2033, 700], 16, 2, 16)
    d = _dev(pkv, b, tree)
    ws = pkv.PrefillWorkspace()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # header and descriptions of split items, then as much for every CTA
    for full in range(40_000, 44_000, 16):
        if (ws.nbytes - full) % sms == 0 and (ws.nbytes - full) // sms % 256 == 0:
            break
    ws.nbytes = full + ctas * ((ws.nbytes - full) // sms)
    ws.tensor[ws.nbytes :].fill_(0x5A)
    out = torch.full_like(d["q"], 7.0)
    _call(pkv, d, b.scale, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert ws.read_error() == 0 and bool((ws.tensor[ws.nbytes :] == 0x5A).all())
    _check(out, _ref(b, tree))
    ws.nbytes = full
    with pytest.raises(pkv.PkvError):
        _call(pkv, d, b.scale, out=out, workspace=ws)


@pytest.mark.parametrize("hq,hkv,decode,chunks", [(16, 4, 24, [(180, 5000), (97, 97)]), (64, 8, 9, [(70, 8011)]),
                                                  (8, 1, 60, [(333, 3001), (1, 9000)])])
def test_a_step_of_chunks_and_decode_rows(pkv, hq, hkv, decode, chunks):  # noqa: F811
    """Long chunks and many single rows of grouped heads in one call."""
    lens = [(1, 500 + 37 * s % 1200) for s in range(decode)] + chunks
    lens = lens[1::2] + lens[::2]
    _run(pkv, Batch(hq + decode, [n for n, _ in lens], [c for _, c in lens], hq, hkv, 16, first_row=2, rows_behind=1), False)
