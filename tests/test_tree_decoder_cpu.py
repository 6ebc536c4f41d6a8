"""TreeDecoder's own bookkeeping, with stand-ins for the calls that run on a GPU:
what it hands to the model, what stops a sequence, and what is committed."""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_decode_gb300 as sv  # noqa: E402
from speculative_decoding_verification_decode_gb300 import api, decoder  # noqa: E402

TREE = [-1, 0, 0, 1]
LAYERS = 3


class Stand:
    """The GPU's calls: attention whose status is set per layer, a verification
    that accepts node 1, and an append that counts."""

    def __init__(self, monkeypatch, B):
        self.bad = torch.zeros(LAYERS, B, dtype=torch.int32)
        self.calls, self.appended, self.B = 0, [], B
        monkeypatch.setattr(api, "tree_attention", self.attention)
        monkeypatch.setattr(api, "verify_tree_greedy", self.verify)
        monkeypatch.setattr(api, "cache_append", self.append)

    def attention(self, q, k, v, kc, vc, table, lengths, parents=None):
        self.calls += 1
        return api.TreeAttention(q.flatten(0, 1), None, self.bad[(self.calls - 1) % LAYERS].clone())

    def verify(self, logits, nodes, parents):
        B, n = nodes.shape
        w = lambda x: torch.tensor(x, dtype=torch.int32)
        path = torch.full((B, n), -1, dtype=torch.int32)
        path[:, 0], path[:, 1] = 0, 1
        return api.TreeResult(w([1] * B), w([9] * B), path, w([0] * B))

    def append(self, cache, keys, values, counts=None, path=None):
        self.appended.append(counts.clone())
        cache.lengths.add_(counts.to(torch.int32))
        return torch.zeros_like(cache.lengths)


def make(monkeypatch, lengths=(5, 7, 3), max_len=40, cached=None, seed=0, **kw):
    B = len(lengths)
    stand = Stand(monkeypatch, B)
    cache = sv.paged_cache(LAYERS, 16, 8, 1, 8, B, 5, device="cpu")
    seen = []

    def target(nodes, positions, attend):
        seen.append((nodes.clone(), positions.clone()))
        x = torch.zeros(*nodes.shape, 1, 8)
        for layer in range(LAYERS):
            attend(layer, x, x, x)
        return torch.zeros(*nodes.shape, 16)

    draft = lambda tokens, lengths: torch.ones(tokens.shape[0], len(TREE), dtype=torch.int32)
    tokens = torch.arange(B * max_len, dtype=torch.int32).view(B, max_len) % 11
    d = sv.TreeDecoder(draft, target, cache, tokens, torch.tensor(lengths, dtype=torch.int32), TREE, seed=seed, **kw)
    cache.lengths.copy_(torch.tensor([x - 1 for x in lengths] if cached is None else cached))
    return d, stand, seen


@pytest.mark.parametrize("layer", range(LAYERS))
@pytest.mark.parametrize("bits", [sv.SEQ_BAD_LAYOUT, sv.SEQ_TIMEOUT, sv.SEQ_BAD_LAYOUT | sv.SEQ_TIMEOUT])
def test_a_round_whose_attention_failed_commits_nothing(monkeypatch, layer, bits):
    d, stand, _ = make(monkeypatch)
    stand.bad[layer, 1] = bits
    tokens, lengths, held = d.tokens.clone(), d.lengths.clone(), d.cache.lengths.clone()
    d.round()
    assert d.status.tolist() == [0, bits, 0]
    assert stand.appended[-1].tolist() == [2, 0, 2]
    assert torch.equal(d.tokens[1], tokens[1]) and d.lengths[1] == lengths[1] and d.cache.lengths[1] == held[1]
    assert d.lengths.tolist() == [7, 7, 5]
    # and it stays as it is when the cause is gone
    stand.bad.zero_()
    d.round()
    assert d.status.tolist() == [0, bits, 0] and d.lengths.tolist() == [9, 7, 7]


def test_a_prefill_whose_attention_failed_appends_nothing(monkeypatch):
    d, stand, _ = make(monkeypatch, (5, 30, 3), cached=(0, 0, 0))
    stand.bad[1, 1] = sv.SEQ_TIMEOUT
    d.prefill(chunk=8)
    assert d.status.tolist() == [0, sv.SEQ_TIMEOUT, 0]
    assert d.cache.lengths.tolist() == [4, 0, 2]
    assert all(c[1] == 0 for c in stand.appended)


def test_a_prefill_stops_a_sequence_at_its_first_failure(monkeypatch):
    """What would come behind a chunk that is not there is not appended."""
    d, stand, _ = make(monkeypatch, (5, 30, 3), cached=(0, 0, 0))
    attention, chunks = stand.attention, []

    def once(*args, **kw):
        r = attention(*args, **kw)
        if stand.calls == 2:  # a layer of the first chunk
            r.status[1] = sv.SEQ_TIMEOUT
        return r

    monkeypatch.setattr(api, "tree_attention", once)
    d.prefill(chunk=8)
    assert d.status.tolist() == [0, sv.SEQ_TIMEOUT, 0]
    assert d.cache.lengths.tolist() == [4, 0, 2]


def test_a_sampled_round_whose_attention_failed_commits_nothing(monkeypatch):
    d, stand, _ = make(monkeypatch, temperature=torch.ones(3))
    monkeypatch.setattr(api, "accept_from_logits", lambda rows, *a, **kw: api.VerifyResult(None, torch.zeros(len(rows), dtype=torch.int32), None))
    monkeypatch.setattr(api, "verify_tree", lambda choices, nodes, parents: stand.verify(None, nodes, parents))
    stand.bad[0, 2] = sv.SEQ_BAD_LAYOUT
    d.round()
    assert d.status.tolist() == [0, 0, sv.SEQ_BAD_LAYOUT] and stand.appended[-1].tolist() == [2, 2, 0]
    assert d.lengths.tolist() == [7, 9, 3]


@pytest.mark.parametrize("lengths", [(5, 30, 3), (1, 40, 39), (37, 36, 38)])
def test_positions_are_within_the_sequences(monkeypatch, lengths):
    """Through a prefill whose chunk is longer than what a sequence may hold, and
    rounds of sequences that have stopped near their end."""
    d, stand, seen = make(monkeypatch, lengths, max_len=40, cached=(0, 0, 0))
    d.prefill()
    assert d.cache.lengths.tolist() == [x - 1 for x in lengths]
    for _ in range(25):
        d.round()
    assert (d.lengths > 40 - len(TREE)).all() and (d.lengths <= 40).all() and not d.status.any()
    assert all(0 <= int(p.min()) and int(p.max()) < 40 for _, p in seen)
    # nodes that count have their own place
    nodes, positions = seen[0]
    for b, n in enumerate(lengths):
        assert torch.equal(positions[b, :n - 1], torch.arange(n - 1, dtype=torch.int32))


def test_lengths_past_the_end_of_tokens(monkeypatch):
    """No place of such a sequence is looked at beyond the row; it stays as it is."""
    d, stand, seen = make(monkeypatch, (5, 41, 1000), max_len=40, cached=(4, 39, 39))
    before = d.tokens.clone()
    d.round()
    assert d.lengths.tolist() == [7, 41, 1000] and torch.equal(d.tokens[1:], before[1:])
    assert stand.appended[-1].tolist() == [2, 0, 0]


def test_a_prefill_of_lengths_past_the_end_of_tokens(monkeypatch):
    d, stand, _ = make(monkeypatch, (5, 41, 1000, 0), max_len=40, cached=(0, 0, 0, 0))
    d.prefill(chunk=16)
    assert d.cache.lengths.tolist() == [4, 39, 39, 0] and len(stand.appended) == 3


def test_an_empty_sequence_stays_empty(monkeypatch):
    """A slot without a token takes no part (padding of a batch)."""
    d, stand, _ = make(monkeypatch, (5, 0, 3), cached=(4, 0, 2))
    before = d.tokens.clone()
    d.round()
    assert stand.appended[-1].tolist() == [2, 0, 2] and d.lengths.tolist() == [7, 0, 5] and d.cache.lengths.tolist() == [6, 0, 4]
    assert torch.equal(d.tokens[1], before[1]) and not d.status.any()
