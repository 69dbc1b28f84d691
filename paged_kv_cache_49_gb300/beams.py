"""Beam search over an engine's sequences.

Every hypothesis is a sequence of the engine, and the hypotheses of a prompt
share its blocks, and those of their common beginnings, by reference (cs2680
Lecture 10, §10.4: forked sequences, copied on divergence). A step selects the
best continuations on the device (beam_select), brings the parents to the host,
where the block manager makes each sequence go on as its parent (reorder), and
leaves the copies of shared blocks to the next append.
"""
from __future__ import annotations

import torch

from . import _native as nat
from .engine import PagedKVEngine


class BeamSearch:
    """`beams` hypotheses of each of the running sequences `prompts`, whose tokens
    are all in the cache; they become the first hypotheses. At most max_length
    tokens are kept of each; eos ends one (-1: none does)."""

    def __init__(self, eng: PagedKVEngine, prompts, beams: int, vocab: int, max_length: int, eos: int = -1):
        prompts = list(prompts)
        if not prompts or beams < 1 or max_length < 1:
            raise ValueError("beam search needs a prompt, a beam and room for a token")
        self.eng, self.groups, self.beams, self.eos = eng, len(prompts), beams, int(eos)
        self.workspace = nat.BeamWorkspace(self.groups, beams, beams, vocab, device=eng.device)
        self.now, self._next = (nat.BeamBuffers(self.groups, beams, max_length, device=eng.device) for _ in range(2))
        # the hypotheses of a prompt are alike before the first step: one of them counts
        self.now.scores[:, 1:] = float("-inf")
        self.seq_ids: list[int] = []
        try:
            for s in prompts:
                self.seq_ids += [s] + eng.bm.fork(s, beams - 1)
        except nat.PkvError:
            for s in set(self.seq_ids) - set(prompts):
                eng.bm.free(s)
            raise
        self.live = [i for i in range(len(self.seq_ids)) if i % beams == 0]

    def step(self, logits) -> torch.Tensor:
        """One step: logits [groups * beams, vocab] of the hypotheses' next tokens, in
        the order of seq_ids (rows of hypotheses that are not in `live` are not
        read). Returns the tokens chosen, int32 [groups, beams]; seq_ids then go on
        as their parents, `live` lists those that take their token (neither finished
        nor missing), and `now` holds scores, parents, lengths and histories.
        Where the manager lacks pages (PoolExhausted) nothing has changed."""
        out = nat.beam_select(logits, self.now.scores, self.now.finished if self.eos >= 0 else None, self.eos, self.now.history,
                              self.now.lengths, out=self._next, workspace=self.workspace, device_error=self.eng.error)
        parents, ended = torch.stack([out.parents, out.finished.int()]).view(2, -1).cpu().tolist()
        rows = [i if p < 0 else i // self.beams * self.beams + p for i, p in enumerate(parents)]
        self.eng.reorder(self.seq_ids, rows)
        self.now, self._next = self._next, self.now
        self.live = [i for i, (p, e) in enumerate(zip(parents, ended)) if p >= 0 and not e]
        return out.tokens

    def histories(self) -> list[list[list[int]]]:
        """The tokens of every hypothesis, best first, by prompt."""
        lengths, rows = self.now.lengths.cpu().tolist(), self.now.history.cpu().tolist()
        return [[row[:n] for row, n in zip(g, ns)] for g, ns in zip(rows, lengths)]

    def free(self) -> None:
        """Ends the hypotheses' sequences."""
        for s in self.seq_ids:
            self.eng.bm.free(s)
        self.seq_ids, self.live = [], []
