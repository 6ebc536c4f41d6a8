"""Rounds with drafted trees over a paged cache, as a program uses them: prompt
shared by forking, trees, commits with pages copied on write, graphs.

The model adds two attention layers (their q, k, v from the tokens' embeddings
and positions, rounded to bf16) to the embedding; its f64 twin takes the same
rounded q, k, v.  The kernel's attention may be off by e = 2 (2^-8) max|v|
(weights and result rounded to bf16, the oracle of the attention itself is
tested elsewhere) and a hundredth of that for all f32 sums; so a logit is off
by at most d = e sum |W| over a row of the two layers' product with the output
matrix, and a greedy token's own logit is within 2 d of the largest.
"""

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytestmark = pytest.mark.skip("needs a GPU")
else:
    pytestmark = pytest.mark.gpu

import __graft_entry__  # noqa: E402

DEV = torch.device("cuda", 0)
V, Hq, Hkv, D, E, LAYERS, SPAN = 97, 8, 2, 64, 64, 2, 512
TREE = [-1, 0, 0, 0, 1, 1, 2, 4, 4, 7]


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


class Model:
    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(DEV)
        self.emb, self.pos = r(V, E), r(SPAN, E)
        self.wq, self.wk, self.wv = r(LAYERS, E, Hq * D) / E ** 0.5, r(LAYERS, E, Hkv * D) / E ** 0.5, r(LAYERS, E, Hkv * D) / E ** 0.5
        self.out = r(LAYERS, Hq * D, V) / 8
        self.head = r(E, V) / 8

    def qkv(self, layer, nodes, positions):
        x = self.emb[nodes.long()] + self.pos[positions.long().clamp(0, SPAN - 1)]
        f = lambda w, h: (x @ w[layer]).to(torch.bfloat16).unflatten(-1, (h, D))
        return f(self.wq, Hq), f(self.wk, Hkv), f(self.wv, Hkv)

    def __call__(self, nodes, positions, attend):
        logits = self.emb[nodes.long()] @ self.head
        for layer in range(LAYERS):
            a = attend(layer, *self.qkv(layer, nodes, positions))
            logits = logits + a.float().flatten(-2) @ self.out[layer]
        return logits

    def exact(self, tokens):
        """f64 logits after every token of one sequence, and the bound d."""
        n = len(tokens)
        t = torch.tensor(tokens, device=DEV)[None]
        x = (self.emb[t.long()].double() @ self.head.double())[0]
        d = 0.0
        for layer in range(LAYERS):
            q, k, v = (y[0].double() for y in self.qkv(layer, t, torch.arange(n, device=DEV)[None]))
            s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(Hq // Hkv, 1)) / D ** 0.5
            s = s.masked_fill(~torch.ones(n, n, dtype=torch.bool, device=DEV).tril(), float("-inf"))
            a = torch.einsum("hij,jhd->ihd", s.softmax(2), v.repeat_interleave(Hq // Hkv, 1))
            x = x + a.flatten(1) @ self.out[layer].double()
            d += 1.01 * 2 * 2.0 ** -8 * float(v.abs().max()) * float(self.out[layer].abs().sum(0).max())
        return x, d


def guess(model):
    """A drafter that often knows: the model without attention, and noise."""
    table = (model.emb @ model.head).topk(8, dim=1).indices.int()

    def draft(tokens, lengths):
        last = tokens.gather(1, (lengths - 1).clamp(min=0).long()[:, None])
        n = torch.zeros(tokens.shape[0], len(TREE), dtype=torch.int32, device=DEV)
        n[:, :1] = last
        rank = [0] * len(TREE)
        for i, p in enumerate(TREE):
            if i:
                n[:, i] = table[n[:, p].long(), rank[p]]
                rank[p] += 1
        return n

    return draft


def knowing(model, said):
    """A drafter that knows the first of every node's children: the tokens ``said``."""
    base = guess(model)

    def draft(tokens, lengths):
        n = base(tokens, lengths)
        first = {}
        for i, p in enumerate(TREE):
            if i and p not in first:
                first[p] = i
        at, j = 0, 0
        while at in first:
            at = first[at]
            n[:, at] = said.gather(1, (lengths.long() + j).clamp(max=said.shape[1] - 1)[:, None])[:, 0]
            j += 1
        return n

    return draft


def decoder(model, B=5, prompts=(40, 1, 7, 130, 17), max_len=220, page=16, pages=90, draft=None, **kw):
    g = torch.Generator().manual_seed(1)
    tokens = torch.randint(0, V, (B, max_len), generator=g).int().to(DEV)
    lengths = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    cache = sv().paged_cache(LAYERS, pages, page, Hkv, D, B, -(-max_len // page), device=DEV)
    for t in (*cache.keys, *cache.values):
        t.fill_(float("nan"))  # nothing past a length may matter
    return sv().TreeDecoder(draft or guess(model), model, cache, tokens, lengths, TREE, **kw)


def check_greedy(model, d, prompts):
    accepted = 0
    for b, p in enumerate(prompts):
        n = int(d.lengths[b])
        tokens = d.tokens[b, :n].tolist()
        x, tol = model.exact(tokens[:-1])
        for i in range(p, n):
            assert x[i - 1, tokens[i]] >= x[i - 1].max() - 2 * tol, (b, i)
        accepted += n - p
    return accepted


@pytest.mark.parametrize("graph", [False, True])
def test_greedy_rounds_are_plain_greedy_decoding(graph):
    model, prompts = Model(), (40, 1, 7, 130, 17)
    d = decoder(model)
    d.prefill(chunk=48)
    assert d.cache.lengths.tolist() == [p - 1 for p in prompts]
    start = d.lengths.clone()
    d.run(9, graph)
    assert not d.status.any() and torch.equal(d.cache.lengths, d.lengths - 1)
    assert check_greedy(model, d, prompts) >= 9 * 5
    # a drafter that knows the answer is believed all the way down
    e = decoder(model, draft=knowing(model, d.tokens))
    e.prefill()
    r = e.round()
    deepest = int(e.depth.max())
    assert ((r.n_accepted == deepest) | (start + deepest >= d.lengths)).sum() >= 3
    check_greedy(model, e, prompts)


def test_a_shared_prompt():
    """One prompt, forked to all sequences: they share its pages, go their own
    ways by sampling, and the counts stay those of the tables."""
    from oracle import cache as oc
    model, B = Model(2), 6
    d = decoder(model, B, (37,) * B, temperature=torch.full((B,), 0.7), seed=5)
    d.tokens[:] = d.tokens[0].clone()
    full = d.lengths.clone()
    d.lengths[1:] = 1
    d.prefill()
    d.lengths.copy_(full)
    assert not sv().cache_fork(d.cache, torch.zeros(B, dtype=torch.int32, device=DEV)).any()
    assert d.cache.refs.max() == B and (d.cache.refs > 0).sum() == 3
    d.run(6)
    assert not d.status.any()
    t = d.cache
    want = oc.refs_of(t.table.cpu().numpy(), t.lengths.cpu().numpy(), 16, t.refs.numel())
    assert (t.refs.cpu().numpy() == want).all()
    said = {tuple(d.tokens[b, 37:int(d.lengths[b])].tolist()[:4]) for b in range(B)}
    assert len(said) > 1  # (six draws of four tokens at temperature 0.7 are not all alike)
    # temperature 0 by the sampling path is greedy
    e = decoder(model, B, (37,) * B, temperature=torch.zeros(B))
    e.prefill()
    e.run(4)
    check_greedy(model, e, (37,) * B)
    # the sequences' end: their pages are free again
    assert not sv().cache_truncate(e.cache, torch.zeros(B, dtype=torch.int32, device=DEV)).any()
    assert not e.cache.refs.any()


def test_sequences_that_cannot_go_on():
    model = Model(3)
    # room for whole trees up to max_len, then they stay
    d = decoder(model, 3, (5, 60, 66), max_len=70)
    d.prefill()
    d.run(66)  # (a round adds a token at least)
    assert (d.lengths > 70 - len(TREE)).all() and (d.lengths <= 70).all() and not d.status.any()
    kept = d.tokens.clone()
    d.run(2)
    assert torch.equal(kept, d.tokens)
    # pages run out: the status says so, the others go on
    d = decoder(model, 2, (40, 4), max_len=200, pages=6)
    d.prefill()
    d.run(60)
    assert (d.status == sv().SEQ_NO_PAGES).any()
    stopped = d.lengths.clone()
    d.run(2)
    assert torch.equal(stopped[d.status != 0], d.lengths[d.status != 0])
    check_greedy(model, d, (40, 4))


def test_what_lies_past_a_prompt_is_not_looked_at():
    model, prompts = Model(4), (40, 1, 7, 130, 17)
    d = decoder(model)
    e = decoder(model)
    for b, p in enumerate(prompts):
        e.tokens[b, p:] = -10 ** 6
    seen = []
    target = e.target_fn
    e.target_fn = lambda nodes, positions, attend: seen.append((int(nodes.min()), int(nodes.max()))) or target(nodes, positions, attend)
    for x in (d, e):
        x.prefill(chunk=50)
        x.run(5, graph=False)
    assert all(0 <= lo and hi < V for lo, hi in seen)
    assert torch.equal(d.lengths, e.lengths)
    for b in range(len(prompts)):
        assert torch.equal(d.tokens[b, :int(d.lengths[b])], e.tokens[b, :int(d.lengths[b])])


def test_refusals():
    model = Model()
    c = sv().paged_cache(1, 4, 8, Hkv, D, 2, 4, device=DEV)
    t, n = torch.zeros(2, 20, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    for parents in ([], [0], [-1, 1], [-1, -1], [-1, 0, 5]):
        with pytest.raises(ValueError, match="parents"):
            sv().TreeDecoder(guess(model), model, c, t, n, parents)
    with pytest.raises(ValueError, match="int32"):
        sv().TreeDecoder(guess(model), model, c, t.long(), n, TREE)
    with pytest.raises(ValueError, match="one sequence"):
        sv().TreeDecoder(guess(model), model, c, t[:1], n[:1], TREE)
    with pytest.raises(ValueError, match="every layer"):
        sv().TreeDecoder(guess(model), lambda nodes, positions, attend: torch.zeros(2, 10, V, device=DEV), c, t, n, TREE).round()
