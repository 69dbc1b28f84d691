"""Prompt and tree attention at the edges of what the interface allows."""
import numpy as np
import pytest
import torch

from oracle import prompt_attention as po
from tests.prompt_batches import Batch
from tests.test_gpu_prompt_attention import _call, _check, _dev, _ref, pkv  # noqa: F401

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
