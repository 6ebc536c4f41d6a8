"""The oracle of drafted trees and paged caches against brute force."""

import itertools

import numpy as np
import pytest

import oracle
from oracle import cache as oc


def random_tree(rng, n):
    return [-1] + [int(rng.integers(0, i)) for i in range(1, n)]


def test_a_chain_is_the_chain_verification():
    rng = np.random.default_rng(1)
    B, K, V = 40, 4, 3
    x = rng.normal(size=(B * (K + 1), V)).astype(np.float32)
    tokens = rng.integers(0, V, (B, K)).astype(np.int32)
    ref = oracle.verify_greedy(x, "f32", tokens.reshape(-1), B, K)
    nodes = np.concatenate((np.zeros((B, 1), np.int32), tokens), 1).reshape(-1)
    n, nxt, path, st = oracle.verify_tree_greedy(x.astype(np.float64), nodes, None, None, B, K + 1)
    assert np.array_equal(n, ref.n_accepted) and np.array_equal(nxt, ref.next_token) and not st.any()
    for b in range(B):
        assert list(path[b]) == list(range(n[b] + 1)) + [-1] * (K - n[b])


def test_path_is_the_plain_decoding_that_the_tree_holds():
    """Target rows of a table model: the path spells the model's own greedy
    continuation as far as the tree has it, the next token goes on with it."""
    rng = np.random.default_rng(2)
    V = 3
    best = {s: int(rng.integers(0, V)) for k in range(6) for s in itertools.product(range(V), repeat=k)}
    for _ in range(300):
        n = int(rng.integers(1, 9))
        up = random_tree(rng, n)
        tokens = rng.integers(0, V, n)
        said = [()]  # a node's tokens after node 0
        for i in range(1, n):
            said.append(said[up[i]] + (int(tokens[i]),))
        if max(map(len, said)) > 5 or len(set(said)) < n:  # (of two siblings alike only the first is followed)
            continue
        x = np.zeros((n, V))
        for i in range(n):
            x[i, best[said[i]]] = 1
        acc, nxt, path, _ = oracle.verify_tree_greedy(x, tokens, np.array(up), None, 1, n)
        s = ()
        while s + (best[s],) in said:
            s += (best[s],)
        assert acc[0] == len(s) and nxt[0] == best[s] and said[path[0][acc[0]]] == s


def test_attention_of_a_chain_is_causal_attention():
    rng = np.random.default_rng(3)
    L, N, H, D, page = 11, 5, 2, 8, 4
    k, v, q = (rng.normal(size=(L + N, H, D)) for _ in range(3))
    table = np.array([[2, 0, 3, 1]], np.int32)
    kc, vc = (np.zeros((4, page, H, D)) for _ in range(2))
    for t in range(L):
        kc[table[0, t // page], t % page], vc[table[0, t // page], t % page] = k[t], v[t]
    out, lse, _, _, st = oracle.tree_attention(q[L:], k[L:], v[L:], kc, vc, table, np.array([L]), None, None, N, 0.5)
    for i in range(N):
        for h in range(H):
            s = 0.5 * k[:L + i + 1, h] @ q[L + i, h]
            p = np.exp(s) / np.exp(s).sum()
            assert np.allclose(out[i, h], p @ v[:L + i + 1, h], rtol=1e-12, atol=1e-12)
            assert np.isclose(lse[i, h], np.log(np.exp(s).sum()), rtol=1e-12)
    assert st[0] == 0


@pytest.mark.parametrize("seed", range(6))
def test_pages_hold_what_separate_lists_hold(seed):
    """Random appends, forks and truncations: every sequence reads as a list of
    its own would, and the counts are those of the table."""
    rng = np.random.default_rng(seed)
    page, W, groups, width, P, D = 3, 4, 2, 9, 40, 2
    S = W * groups
    table, lengths, refs = np.zeros((S, width), np.int32), np.zeros(S, np.int32), np.zeros(P, np.int32)
    pool = np.zeros((P, page, 1, D))
    said = [[] for _ in range(S)]
    for step in range(60):
        kind = rng.integers(0, 3)
        if kind == 0:
            n = int(rng.integers(1, 6))
            new = rng.normal(size=(S * n, 1, D))
            counts = rng.integers(0, n + 1, S).astype(np.int32)
            path = np.stack([rng.permutation(n) for _ in range(S)]).astype(np.int32)
            st = oc.append(table, lengths, refs, [pool], [new], counts, path, None, n)
            for b in range(S):
                assert st[b] in (0, oc.NO_PAGES)
                if st[b] == 0:
                    said[b] += [new[b * n + x, 0] for x in path[b, :counts[b]]]
        elif kind == 1:
            parents = rng.integers(-1, W, (groups, W)).astype(np.int32)
            assert not oc.fork(table, lengths, refs, page, parents).any()
            said = [list(said[b // W * W + parents[b // W, b % W]]) if parents[b // W, b % W] >= 0 else said[b]
                    for b in range(S)]
        else:
            to = np.array([rng.integers(0, len(s) + 1) if rng.random() < 0.4 else len(s) for s in said], np.int32)
            assert not oc.truncate(table, lengths, refs, page, to).any()
            said = [s[:k] for s, k in zip(said, to)]
        assert np.array_equal(refs, oc.refs_of(table, lengths, page, P))
        for b in range(S):
            held = pool[table[b, :-(-len(said[b]) // page)], :, 0].reshape(-1, D)[:len(said[b])]
            assert lengths[b] == len(said[b]) and np.array_equal(held, np.array(said[b]).reshape(-1, D))
