"""Beam search's selection, restated in float64.

Candidate (k, v) of a group's beam k scores s_k + x_kv - log sum_v exp x_kv; a
finished beam has the one candidate (k, eos) with score s_k. The n best are
taken, equal scores by k * vocab + v; NaN and -inf are no candidates. Scores are
sums of two float64 numbers, so that logits of any size (a mask of -1e30, say)
leave what the others differ by. A taken
candidate's history is its parent's first `length` tokens and then the token,
unless the parent was finished (or has no room left).
"""
from __future__ import annotations

import numpy as np


def _two_sum(a, b):
    """a + b and what its rounding leaves (Knuth); nothing beside an infinity."""
    s = a + b
    t = s - a
    low = (a - (s - t)) + (b - t)
    return s, np.where(np.isfinite(s), low, 0.0)


def scores_of(logits, scores, finished, eos):
    """float64 [groups, beams * vocab], -inf where there is no candidate, and what
    their rounding leaves."""
    groups, beams = scores.shape
    x = np.asarray(logits, np.float64).reshape(groups, beams, -1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = x.max(axis=-1, keepdims=True)
        high, low = _two_sum(x, -top)
        total, more = _two_sum(high, scores[..., None] - np.log(np.exp(x - top).sum(axis=-1, keepdims=True)))
        total, low = _two_sum(total, low + more)
    for b, k in zip(*np.nonzero(finished)):
        total[b, k], low[b, k] = -np.inf, 0
        total[b, k, eos] = scores[b, k]
    total[~(scores > -np.inf)] = -np.inf
    none = ~(total > -np.inf)
    total, low = np.where(none, -np.inf, total), np.where(none, 0, low)
    return total.reshape(groups, -1), low.reshape(groups, -1)


def select(logits, scores, finished, eos, n, history=None, lengths=None, history_out=None):
    """(scores float64, tokens, parents, finished[, lengths, history]) [groups, n];
    history_out: what the rows' ends hold before."""
    scores = np.asarray(scores, np.float64)
    groups, beams = scores.shape
    total, low = scores_of(logits, scores, finished, eos)
    vocab = total.shape[1] // beams
    order = np.lexsort((-low, -total), axis=1)[:, :n]  # (stable)
    best = np.full((groups, n), -np.inf)
    tokens, parents = np.full((groups, n), -1, np.int32), np.full((groups, n), -1, np.int32)
    done = np.zeros((groups, n), bool)
    lens = np.zeros((groups, n), np.int32)
    hist = None if history is None else history_out.copy()
    for b in range(groups):
        for j, at in enumerate(order[b]):
            if not total[b, at] > -np.inf:
                break
            k, v = divmod(int(at), vocab)
            best[b, j], tokens[b, j], parents[b, j] = total[b, at], v, k
            done[b, j] = finished[b, k] or v == eos
            if history is not None:
                row = list(history[b, k, :lengths[b, k]]) + ([] if finished[b, k] else [v])
                row = row[:history.shape[2]]
                lens[b, j], hist[b, j, :len(row)] = len(row), row
    return (best, tokens, parents, done) + (() if history is None else (lens, hist))
