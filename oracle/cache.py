"""Pages of paged caches: appending, truncating, forking, one sequence after
another.

TEST INFRASTRUCTURE ONLY: the rules of the package docstring apply (only
tests and ``smoke()`` import it).

State: ``table`` [S, width], ``lengths`` [S], ``refs`` [P] integer arrays and
``pools``, a list of arrays [P, page, H, D]; the functions change them in
place and return the status.
"""

from __future__ import annotations

import numpy as np

from .tree import BAD_LAYOUT, nodes

NO_PAGES = 128


def _pages(tokens: int, page: int) -> int:
    return -(-tokens // page)


def append(table, lengths, refs, pools, rows, counts, path, cu, n):
    """``rows``: per pool [total, H, D]; ``counts``, ``path``, ``cu`` may be None."""
    S, width = table.shape
    page = pools[0].shape[1]
    total = rows[0].shape[0]
    status = np.zeros(S, np.int32)
    free = [p for p in range(len(refs)) if refs[p] == 0]
    copied = {}  # page: most of its tokens that a copy took
    for b, at in enumerate(nodes(cu, S, n, total)):
        if at is None:
            status[b] = BAD_LAYOUT
            continue
        first, N = at
        L = int(lengths[b])
        count = N if counts is None else int(counts[b])
        if not 0 <= count <= N or not 0 <= L <= width * page:
            status[b] = BAD_LAYOUT
            continue
        way = list(range(count)) if path is None else [int(x) for x in path[b][:count]]
        if any(not 0 <= x < N for x in way):
            status[b] = BAD_LAYOUT
            continue
        if count == 0:
            continue
        if L + count > width * page:
            status[b] = NO_PAGES
            continue
        copy = -1
        if L % page:
            last = int(table[b, L // page])
            if not 0 <= last < len(refs):
                status[b] = BAD_LAYOUT
                continue
            if refs[last] > 1 or copied.get(last, 0) > L % page:
                copy = last
        start = _pages(L, page) - (copy >= 0)
        need = _pages(L + count, page) - start
        if need > len(free):
            status[b] = NO_PAGES
            continue
        for j in range(need):
            p = free.pop(0)
            table[b, start + j] = p
            refs[p] = 1
        if copy >= 0:
            refs[copy] -= 1
            copied[copy] = max(copied.get(copy, 0), L % page)
            for pool in pools:
                pool[table[b, L // page], :L % page] = pool[copy, :L % page]
        for j, x in enumerate(way):
            for pool, new in zip(pools, rows):
                pool[table[b, (L + j) // page], (L + j) % page] = new[first + x]
        lengths[b] = L + count
    return status


def truncate(table, lengths, refs, page, to):
    S, width = table.shape
    status = np.zeros(S, np.int32)
    for b in range(S):
        L, t = int(lengths[b]), int(to[b])
        gone = table[b, _pages(max(t, 0), page):_pages(max(L, 0), page)]
        if not 0 <= t <= L <= width * page or (gone < 0).any() or (gone >= len(refs)).any():
            status[b] = BAD_LAYOUT
            continue
        for p in gone:
            refs[p] -= 1
        lengths[b] = t
    return status


def fork(table, lengths, refs, page, parents):
    """``parents`` [groups, W]."""
    groups, W = parents.shape
    width = table.shape[1]
    status = np.zeros(groups, np.int32)
    for g in range(groups):
        t, le = table[g * W:(g + 1) * W], lengths[g * W:(g + 1) * W]
        move = [(w, int(p)) for w, p in enumerate(parents[g]) if p >= 0 and p != w]
        ok = (parents[g] < W).all()
        for w in {x for m in move for x in m if x < W}:
            L = int(le[w])
            used = t[w, :_pages(max(0, min(L, width * page)), page)]
            ok = ok and 0 <= L <= width * page and (used >= 0).all() and (used < len(refs)).all()
        if not ok:
            status[g] = BAD_LAYOUT
            continue
        was, had = t.copy(), le.copy()
        for w, p in move:
            for x in was[w, :_pages(int(had[w]), page)]:
                refs[x] -= 1
            k = _pages(int(had[p]), page)
            t[w, :k] = was[p, :k]
            for x in was[p, :k]:
                refs[x] += 1
            le[w] = had[p]
    return status


def refs_of(table, lengths, page, P):
    """What refs has to be."""
    refs = np.zeros(P, np.int64)
    for row, L in zip(table, lengths):
        for p in row[:_pages(int(L), page)]:
            refs[p] += 1
    return refs
