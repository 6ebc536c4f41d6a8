"""Beam search: selection over beams and vocabulary, and reordering of states.

TEST INFRASTRUCTURE ONLY: the rules of the package docstring apply (only
tests and ``smoke()`` import it).

Definitions this file fixes:

* ``score(w, v) = c_w + l_wv - ln sum_u exp l_wu``; the n best, by score
  descending, then beam, then token.  Scores here are fp64 (the sum through
  ``math.fsum``, correctly rounded, so that rows that are permutations of one
  another have equal sums and their candidates tie exactly).
* a finished beam offers ``(eos, c_w)`` alone; a beam at -inf and a token at
  -inf offer nothing, nor does a score that rounds to -inf in f32; places left
  over are (-inf, -1, -1).
* NaN or +inf among a live beam's logits, or a score that is NaN or +inf:
  the sequence is bad and every place is (-inf, -1, -1).
* reordering: slot w of sequence b takes what slot ``parents[b, w]`` held; a
  negative parent leaves its slot alone; with a length only the positions
  below it move.  A parent >= W or a length outside [0, T]: nothing of the
  sequence moves.
"""

from __future__ import annotations

import dataclasses
import math
from typing import Optional

import numpy as np

BAD_VALUE = 2
BAD_LAYOUT = 64


@dataclasses.dataclass
class BeamResult:
    scores: np.ndarray   # f64 [B, n]
    parents: np.ndarray  # i32 [B, n]
    tokens: np.ndarray   # i32 [B, n]
    status: np.ndarray   # u32 [B]
    gap: np.ndarray      # f64 [B]: smallest nonzero distance between neighbours of the order, the first left out included


def _log_softmax(row: np.ndarray) -> np.ndarray:
    """``l - ln sum exp l``, the maximum taken off first: added to the
    logarithm it would round that away where it is large (a row all at the
    lowest f32 is uniform: -ln V each, not 0)."""
    x = row - row.max()
    return x - math.log(math.fsum(np.exp(x)))


def beam_select(logits: np.ndarray, scores: np.ndarray, n: int, finished: Optional[np.ndarray] = None,
                eos: int = -1) -> BeamResult:
    """``logits [B, W, V]`` f64 (or f32) values, ``scores [B, W]``."""
    B, W, V = logits.shape
    out = BeamResult(np.full((B, n), -np.inf), np.full((B, n), -1, np.int32), np.full((B, n), -1, np.int32),
                     np.zeros(B, np.uint32), np.full(B, np.inf))
    for b in range(B):
        c = scores[b].astype(np.float64)
        ended = np.zeros(W, bool) if finished is None else np.asarray(finished[b], bool)
        live = ~ended & (c != -np.inf)
        x = logits[b].astype(np.float64)
        if np.isnan(c).any() or (c == np.inf).any() or np.isnan(x[live]).any() or (x[live] == np.inf).any():
            out.status[b] = BAD_VALUE
            continue
        s = np.full((W, V), -np.inf)
        for w in range(W):
            if ended[w]:
                s[w, eos] = c[w]
            elif live[w] and (x[w] > -np.inf).any():
                s[w] = c[w] + _log_softmax(x[w])
        s = s.reshape(-1)
        with np.errstate(over="ignore"):
            s[s.astype(np.float32) == -np.inf] = -np.inf
        order = np.argsort(-s, kind="stable")[:n + 1]
        order = order[s[order] > -np.inf]
        steps = -np.diff(s[order])
        if (steps > 0).any():
            out.gap[b] = steps[steps > 0].min()
        order = order[:n]
        k = len(order)
        out.scores[b, :k] = s[order]
        out.parents[b, :k] = order // V
        out.tokens[b, :k] = order % V
    return out


def beam_reorder(state: np.ndarray, parents: np.ndarray, lengths: Optional[np.ndarray] = None,
                 time_dim: Optional[int] = None):
    """(the state after, status [B]) for ``state [B, W, ...]``."""
    B, W = parents.shape
    new, status = state.copy(), np.zeros(B, np.uint32)
    for b in range(B):
        T = None if time_dim is None else state.shape[time_dim]
        if (parents[b] >= W).any() or (lengths is not None and not 0 <= lengths[b] <= (T if T is not None else 2**31)):
            status[b] = BAD_LAYOUT
            continue
        for w in range(W):
            p = int(parents[b, w])
            if p < 0:
                continue
            if time_dim is None:
                new[b, w] = state[b, p]
            else:
                keep = [slice(None)] * (time_dim - 2) + [slice(0, int(lengths[b]))]
                new[b, w][tuple(keep)] = state[b, p][tuple(keep)]
    return new, status
