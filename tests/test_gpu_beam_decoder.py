"""Beam search end to end on the GPU: hidden states -> 4-bit LM head -> beam
selection -> reordering of tokens and caches, as BeamDecoder runs it, eager
and replayed from a CUDA graph, against a search written out in fp64."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytestmark = pytest.mark.skip("needs a GPU")
else:
    pytestmark = pytest.mark.gpu

import __graft_entry__  # noqa: E402
import oracle  # noqa: E402

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


class TinyModel:
    """A recurrent model with a cache: the state of a beam is a running mix of
    its tokens' embeddings; the logits come from the state through a 4-bit
    head, so they depend on every earlier token of the beam."""

    def __init__(self, B, W, T, V, d, seed):
        g = torch.Generator().manual_seed(seed)
        self.emb = torch.randn(V, d, generator=g).to(DEV)
        self.head = sv().Q4Projection(*(None if t is None else t.to(DEV) for t in sv().q4_quantize(
            torch.randn(V, d, generator=g) * (3.0 / d ** 0.5), 64)[:3]), 64)
        self.state = torch.zeros(B, W, d, device=DEV)
        self.cache = torch.zeros(B, W, 2, T, 16, dtype=torch.bfloat16, device=DEV)
        self.rows = torch.arange(B, device=DEV)

    def __call__(self, tokens, lengths):
        at = (lengths.long() - 1).clamp(min=0)
        last = tokens[self.rows, :, at].long()  # [B, W]
        e = self.emb[last]
        self.state.mul_(0.7).add_(e)
        self.cache[self.rows, :, :, at] = e[:, :, :32].view(*e.shape[:2], 2, 16).to(torch.bfloat16)
        h = torch.tanh(self.state).to(torch.bfloat16)
        return sv().lm_head_logits(h, self.head).view(*tokens.shape[:2], -1)


def reference(model, tokens, lengths, steps, eos):
    """The same search with the oracle's selection and plain copies."""
    tokens, lengths = tokens.cpu().numpy().copy(), lengths.cpu().numpy().copy()
    B, W, _ = tokens.shape
    c = np.full((B, W), -np.inf, np.float32)
    c[:, 0] = 0
    fin = np.zeros((B, W), bool)
    gap = np.inf
    for _ in range(steps):
        logits = model(torch.from_numpy(tokens).to(DEV), torch.from_numpy(lengths).to(DEV)).cpu().numpy()
        r = oracle.beam_select(logits, c, W, fin if eos >= 0 else None, eos)
        gap = min(gap, r.gap.min())
        par = torch.from_numpy(np.where(r.parents < 0, np.arange(W), r.parents).astype(np.int64)).to(DEV)
        b = torch.arange(B, device=DEV)[:, None]
        model.state.copy_(model.state[b, par])
        model.cache.copy_(model.cache[b, par])
        tokens = np.take_along_axis(tokens, par.cpu().numpy()[:, :, None], 1)
        tokens[np.arange(B), :, lengths] = np.maximum(r.tokens, 0)
        fin = r.tokens == eos if eos >= 0 else fin
        c = r.scores.astype(np.float32)
        lengths = lengths + 1
    return tokens, c, gap


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("eos", [-1, 5])
@pytest.mark.parametrize("B,W,V", [(1, 4, 997), (3, 5, 2048)])
def test_search(B, W, V, eos, graph):
    T, steps, d = 24, 12, 128
    prompt = torch.randint(0, V, (B, 1, 4), generator=torch.Generator().manual_seed(B), dtype=torch.int32)
    tokens = torch.zeros(B, W, T, dtype=torch.int32)
    tokens[:, :, :4] = prompt
    tokens = tokens.to(DEV)
    lengths = torch.tensor([4, 2, 3][:B], dtype=torch.int32, device=DEV)
    ref = TinyModel(B, W, T, V, d, 1)
    want, scores, gap = reference(ref, tokens, lengths, steps, eos)
    assert gap > 1e-4  # the search is decided everywhere, also with f32 running scores
    m = TinyModel(B, W, T, V, d, 1)
    dec = sv().BeamDecoder(m, tokens, lengths, eos, [m.state, m.cache], [None, 3])
    got, ln, s = dec.run(steps, graph=graph)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), want)
    # every step rounds the running score once and adds the logarithm's error
    assert np.allclose(s.cpu().numpy(), scores, rtol=0, atol=steps * (2.0 ** -24 * np.abs(scores).max() + 2.0 ** -17))
    assert torch.equal(m.state, ref.state)
    for b in range(B):
        n = int(ln[b]) - 1
        assert torch.equal(m.cache[b, :, :, :n], ref.cache[b, :, :, :n])


@pytest.mark.parametrize("eos", [-1, 5])
def test_full_sequences_stay(eos):
    """A sequence that has filled its room stays as it is; the others go on as
    they would alone."""
    B, W, V, T, d, steps = 2, 4, 997, 10, 128, 6
    tokens = torch.zeros(B, W, T, dtype=torch.int32, device=DEV)
    tokens[:, :, :7] = torch.randint(0, V, (B, 1, 7), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    lengths = torch.tensor([4, 7], dtype=torch.int32, device=DEV)

    def table(tokens, lengths):  # logits by the last token and the position
        at = lengths.long() - 1
        last = tokens[torch.arange(B, device=DEV), :, at].long()
        return base[(last + 31 * at[:, None]) % 64]

    base = (3 * torch.randn(64, V, generator=torch.Generator().manual_seed(4))).to(DEV)
    short = sv().BeamDecoder(table, tokens.clone(), lengths.clone(), eos)
    short.run(3, graph=False)  # sequence 1 is full now
    kept = [t[1].clone() for t in (short.tokens, short.scores, short.finished)]
    wide = torch.zeros(B, W, 2 * T, dtype=torch.int32, device=DEV)
    wide[:, :, :T] = tokens
    ref = sv().BeamDecoder(table, wide, lengths.clone(), eos)
    ref.run(steps, graph=False)
    short.run(steps - 3, graph=False)
    for a, b in zip((short.tokens, short.scores, short.finished), kept):
        assert torch.equal(a[1], b)
    assert short.lengths.tolist() == [10, 10]
    assert torch.equal(short.tokens[0], ref.tokens[0, :, :T]) and torch.equal(short.scores[0], ref.scores[0])
