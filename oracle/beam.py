"""Beam search's selection, restated in float64.

Candidate (k, v) of a group's beam k scores s_k + x_kv - log sum_v exp x_kv; a
finished beam has the one candidate (k, eos) with score s_k. The n best are
taken, equal scores by k * vocab + v; NaN and -inf are no candidates. A taken
candidate's history is its parent's first `length` tokens and then the token,
unless the parent was finished (or has no room left).
"""
from __future__ import annotations

import numpy as np


def scores_of(logits, scores, finished, eos):
    """float64 [groups, beams * vocab], -inf where there is no candidate."""
    groups, beams = scores.shape
    x = np.asarray(logits, np.float64).reshape(groups, beams, -1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = x.max(axis=-1, keepdims=True)
        total = scores[..., None] + (x - (top + np.log(np.exp(x - top).sum(axis=-1, keepdims=True))))
    for b, k in zip(*np.nonzero(finished)):
        total[b, k] = -np.inf
        total[b, k, eos] = scores[b, k]
    total[~(scores > -np.inf)] = -np.inf
    return np.where(np.isnan(total), -np.inf, total).reshape(groups, -1)


def select(logits, scores, finished, eos, n, history=None, lengths=None, history_out=None):
    """(scores float64, tokens, parents, finished[, lengths, history]) [groups, n];
    history_out: what the rows' ends hold before."""
    scores = np.asarray(scores, np.float64)
    groups, beams = scores.shape
    total = scores_of(logits, scores, finished, eos)
    vocab = total.shape[1] // beams
    order = np.argsort(-total, axis=1, kind="stable")[:, :n]
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
