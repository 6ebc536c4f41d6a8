"""Trees of drafted tokens: greedy verification, and the attention over a paged
cache.

TEST INFRASTRUCTURE ONLY: the rules of the package docstring apply (only
tests and ``smoke()`` import it).

Definitions this file fixes:

* ``nodes(cu, B, n, total)``: (first row, nodes) per sequence, None where the
  offsets are bad;
* verification: node 0 first; a node's choice is its row's argmax (lowest
  index, NaN below -inf; an all-NaN row's is 0); the path goes to the lowest
  child whose token is the choice, and ends where there is none.  A NaN in a
  row of the path: BAD_VALUE; a child of a path node with a token outside
  [0, V): BAD_TOKEN, never followed;
* attention: in fp64, over the cached tokens and the node and its ancestors.
"""

from __future__ import annotations

import math

import numpy as np

BAD_TOKEN, BAD_VALUE, BAD_LAYOUT = 1, 2, 64


def nodes(cu, B: int, n: int, total: int):
    if cu is None:
        return [(b * n, n) for b in range(B)]
    return [(int(a), int(e - a)) if 0 <= a <= e <= total and e - a <= n else None
            for a, e in zip(np.asarray(cu, np.int64)[:-1], np.asarray(cu, np.int64)[1:])]


def parents_ok(parents) -> bool:
    return all(-1 <= p < i for i, p in enumerate(parents))


def _walk(tokens, parents, choice_of):
    """Path of one sequence; ``choice_of(i)`` gives (choice, status bits)."""
    path, status, at = [0], 0, 0
    while True:
        c, bits = choice_of(at)
        status |= bits
        to = [i for i in range(len(tokens)) if parents[i] == at and tokens[i] == c and c >= 0]
        if not to:
            return path, c, status
        at = to[0]
        path.append(at)


def _results(layout, n, one):
    acc, nxt, paths, st = [], [], [], []
    for b, at in enumerate(layout):
        if at is None:
            p, c, s = [], -1, BAD_LAYOUT
        elif at[1] == 0:
            p, c, s = [], -1, 0
        else:
            p, c, s = one(b, *at)
        acc.append(max(0, len(p) - 1))
        nxt.append(c)
        paths.append(p + [-1] * (n - len(p)))
        st.append(s)
    return (np.array(acc, np.int32), np.array(nxt, np.int32), np.array(paths, np.int32).reshape(len(layout), n),
            np.array(st, np.int32))


def _up(parents, first, N):
    return list(range(-1, N - 1)) if parents is None else [int(p) for p in parents[first:first + N]]


def verify_tree_greedy(target, tokens, parents, cu, B, n):
    """(n_accepted, next_token, path, status) for float64 rows ``target``."""
    V = target.shape[1]

    def one(b, first, N):
        up = _up(parents, first, N)
        if not parents_ok(up):
            return [], -1, BAD_LAYOUT
        tk = [int(t) for t in tokens[first:first + N]]

        def choice(i):
            row = target[first + i]
            bits = BAD_VALUE if np.isnan(row).any() else 0
            if any(up[j] == i and not 0 <= tk[j] < V for j in range(N)):
                bits |= BAD_TOKEN
            c = 0 if np.isnan(row).all() else int(np.flatnonzero(row == np.nanmax(row))[0])
            return c, bits

        return _walk(tk, up, choice)

    return _results(nodes(cu, B, n, len(tokens)), n, one)


def verify_tree(choices, tokens, parents, cu, B, n):
    def one(b, first, N):
        up = _up(parents, first, N)
        if not parents_ok(up):
            return [], -1, BAD_LAYOUT
        p, c, s = _walk([int(t) for t in tokens[first:first + N]], up, lambda i: (int(choices[first + i]), 0))
        return p, max(c, -1), s

    return _results(nodes(cu, B, n, len(tokens)), n, one)


def tree_attention(q, k, v, k_cache, v_cache, table, lengths, parents, cu, n, scale):
    """float64 arrays; returns (out, lse, sum_j p_j |v_j|, max_j scale sum_d |q_d k_jd|, status).
    Rows of bad sequences: 0, -inf; rows that no sequence has: NaN."""
    total, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    P, page = k_cache.shape[:2]
    B, width = table.shape
    out = np.full((total, Hq, D), np.nan)
    mag, lse, size = out.copy(), np.full((total, Hq), np.nan), np.full((total, Hq), np.nan)
    status = np.zeros(B, np.int32)
    for b, at in enumerate(nodes(cu, B, n, total)):
        if at is None:
            status[b] = BAD_LAYOUT
            continue
        first, N = at
        L = int(lengths[b])
        up = _up(parents, first, N)
        ids = table[b, :max(0, -(-L // page))]
        if not parents_ok(up) or not 0 <= L <= width * page or (ids < 0).any() or (ids >= P).any():
            status[b] = BAD_LAYOUT
            out[first:first + N], lse[first:first + N] = 0, -np.inf
            mag[first:first + N], size[first:first + N] = 0, 0
            continue
        kc = k_cache[ids].reshape(-1, Hkv, D)[:L]
        vc = v_cache[ids].reshape(-1, Hkv, D)[:L]
        for i in range(N):
            own = []
            j = i
            while j >= 0:
                own.append(first + j)
                j = up[j]
            for h in range(Hq):
                kk = np.concatenate((kc[:, h // G], k[own, h // G]))
                vv = np.concatenate((vc[:, h // G], v[own, h // G]))
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (kk @ q[first + i, h])
                    m = s.max()
                    e = np.exp(s - m)
                    z = e.sum()
                    out[first + i, h] = e @ vv / z
                    mag[first + i, h] = e @ np.abs(vv) / z
                    size[first + i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[first + i, h])).max()
                    lse[first + i, h] = m + math.log(z) if z > 0 else np.nan
    return out, lse, mag, size, status
