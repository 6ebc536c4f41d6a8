"""Pins of the beam-search oracle: enumeration on tiny vocabularies, whole
searches against the probabilities of all sentences, hand-worked ties and
masks, reordering against plain copies; and of the 4-bit projection: hand
values and the quantiser's error."""

import itertools
import math

import numpy as np
import pytest

import oracle
from oracle import beam

torch = pytest.importorskip("torch")


def test_candidates_by_enumeration():
    rng = np.random.default_rng(1)
    for W, V, n in ((1, 1, 1), (2, 3, 4), (3, 5, 7), (4, 4, 16)):
        x = rng.normal(0, 2, (2, W, V))
        c = rng.normal(-5, 1, (2, W))
        r = oracle.beam_select(x, c, n)
        for b in range(2):
            all_ = [(-(c[b, w] + math.log(math.exp(x[b, w, v]) / sum(math.exp(y) for y in x[b, w]))), w, v)
                    for w in range(W) for v in range(V)]
            all_.sort()
            assert [(w, v) for _, w, v in all_[:n]] == list(zip(r.parents[b], r.tokens[b]))
            assert np.allclose(r.scores[b], [-s for s, _, _ in all_[:n]], rtol=0, atol=1e-12)


def test_wide_beam_search_is_exhaustive():
    """With as many beams as prefixes, three steps of selection find the most
    probable sentences of a table model (a table for each position, so that no
    two sentences tie), with their log-probabilities."""
    rng = np.random.default_rng(2)
    V = 4
    table = rng.normal(0, 1.5, (3, V, V))
    logp = table - np.log(np.exp(table).sum(2, keepdims=True))
    W = V * V
    toks = np.zeros((W, 4), np.int64)
    c = np.full((1, W), -np.inf)
    c[0, 0] = 0.0
    for t in range(3):
        r = oracle.beam_select(table[t, toks[:, t]][None], c, W)
        toks = toks[np.maximum(r.parents[0], 0)].copy()
        toks[:, t + 1] = np.maximum(r.tokens[0], 0)
        c = r.scores
    best = sorted((-sum(logp[t, a, b] for t, (a, b) in enumerate(zip((0, *s), s))), s)
                  for s in itertools.product(range(V), repeat=3))
    for (nl, s), got, sc in zip(best[:W], toks, c[0]):
        assert tuple(got[1:]) == s and abs(sc + nl) < 1e-12


def test_ties_masks_and_bad_values():
    z = np.zeros((1, 2, 3))
    r = oracle.beam_select(z, np.zeros((1, 2)), 4)
    assert r.parents.tolist() == [[0, 0, 0, 1]] and r.tokens.tolist() == [[0, 1, 2, 0]]
    # permuted rows tie exactly
    x = np.array([[[1.0, 0.25, -3.0], [-3.0, 1.0, 0.25]]])
    r = oracle.beam_select(x, np.zeros((1, 2)), 2)
    assert r.parents.tolist() == [[0, 1]] and r.tokens.tolist() == [[0, 1]] and r.scores[0, 0] == r.scores[0, 1]
    # a mask that leaves one token, one that leaves none, a dead beam with NaN logits, a finished beam
    x = np.full((1, 4, 3), -np.inf)
    x[0, 0, 2] = 7.0
    x[0, 2] = np.nan
    x[0, 3] = np.nan
    r = oracle.beam_select(x, np.array([[-1.0, -2.0, -np.inf, -3.0]]), 4, np.array([[0, 0, 0, 1]]), eos=1)
    assert r.status[0] == 0
    assert r.parents.tolist() == [[0, 3, -1, -1]] and r.tokens.tolist() == [[2, 1, -1, -1]]
    assert r.scores[0].tolist() == [-1.0, -3.0, -np.inf, -np.inf]
    for bad in (np.nan, np.inf):
        y = np.zeros((1, 2, 3))
        y[0, 1, 1] = bad
        assert oracle.beam_select(y, np.zeros((1, 2)), 2).status[0] == beam.BAD_VALUE
        assert oracle.beam_select(z, np.array([[0.0, bad]]), 2).status[0] == beam.BAD_VALUE


def test_reorder_by_hand():
    s = np.arange(2 * 3 * 4).reshape(2, 3, 4)
    new, st = oracle.beam_reorder(s, np.array([[2, 0, 0], [0, 3, 1]]))
    assert st.tolist() == [0, beam.BAD_LAYOUT]
    assert (new[0] == s[0][[2, 0, 0]]).all() and (new[1] == s[1]).all()
    new, st = oracle.beam_reorder(s, np.array([[-1, 0, 1], [1, 1, 1]]), np.array([2, 5]), 2)
    assert st.tolist() == [0, beam.BAD_LAYOUT]
    want = s.copy()
    want[0, 1, :2], want[0, 2, :2] = s[0, 0, :2], s[0, 1, :2]
    assert (new == want).all()


def test_q4_by_hand():
    packed = np.array([[0x98, 0xF0] + [0x88] * 14], np.uint8)  # q = 8, 9, 0, 15, then 8s
    w = oracle.q4_weights(packed, np.array([[0.5]]), None, 32)
    assert w[0, :4].tolist() == [0.0, 0.5, -4.0, 3.5] and (w[0, 4:] == 0).all()
    w = oracle.q4_weights(packed, np.array([[2.0]]), np.array([[9]], np.uint8), 32)
    assert w[0, :4].tolist() == [-2.0, 0.0, -18.0, 12.0]
    h = np.zeros((1, 32))
    h[0, 2] = 3.0
    assert oracle.q4_logits(h, packed, np.array([[0.5]]), None, 32)[0, 0] == -12.0


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,d", [(32, 32), (64, 160), (128, 224)])
def test_quantiser_error(zeros, group, d):
    """Every weight lies within half a step of its group (the scale's own
    rounding to bf16, 2^-8 of it, moves the ends of the range by at most 8 or
    15 times that)."""
    import speculative_decoding_verification_decode_gb300 as sv
    w = torch.randn(11, d, generator=torch.Generator().manual_seed(3))
    w[3] = 0.0
    p = sv.q4_quantize(w, group, zeros)
    s = p.scales.float().numpy()
    got = oracle.q4_weights(p.packed.numpy(), s, None if p.zeros is None else p.zeros.numpy(), group)
    step = np.repeat(s, group, 1)[:, :d]
    assert (np.abs(got - w.numpy()) <= step * (0.5 + 16 * 2.0 ** -8) + 1e-12).all()
    assert (got[3] == 0).all()
