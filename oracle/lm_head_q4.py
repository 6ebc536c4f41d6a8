"""The LM head on a projection in 4 bits with group scales.

TEST INFRASTRUCTURE ONLY: the rules of the package docstring apply (only
tests and ``smoke()`` import it).

``W[v, k] = scale[v, k // group] * (q[v, k] - zero[v, k // group])`` with q in
0..15 (byte j of a packed row: q[2j] in the low four bits, q[2j + 1] in the
high four) and zero 8 where none is given; ``logits = H W^T``.  Scales and
states are given as their values (f32 / f64 arrays); products are summed in
fp64.
"""

from __future__ import annotations

from typing import Optional

import numpy as np


def q4_weights(packed: np.ndarray, scales: np.ndarray, zeros: Optional[np.ndarray], group: int) -> np.ndarray:
    """``W [V, d]`` in fp64."""
    V, half = packed.shape
    q = np.empty((V, 2 * half))
    q[:, 0::2] = packed & 15
    q[:, 1::2] = packed >> 4
    for g in range(scales.shape[1]):
        part = slice(g * group, min((g + 1) * group, 2 * half))
        q[:, part] -= 8.0 if zeros is None else zeros[:, g:g + 1].astype(np.float64)
        q[:, part] *= scales[:, g:g + 1].astype(np.float64)
    return q


def q4_logits(states: np.ndarray, packed: np.ndarray, scales: np.ndarray, zeros: Optional[np.ndarray],
              group: int) -> np.ndarray:
    return states.astype(np.float64) @ q4_weights(packed, scales, zeros, group).T


def q4_abs_sums(states: np.ndarray, packed: np.ndarray, scales: np.ndarray, zeros: Optional[np.ndarray],
                group: int) -> np.ndarray:
    """sum_k |h_k W_k|: what rounding errors of a sum are relative to."""
    return np.abs(states.astype(np.float64)) @ np.abs(q4_weights(packed, scales, zeros, group)).T
