"""What BeamDecoder tells of sequences that it cannot carry on, eager and
replayed: a bad logit, a cache shorter than the sequence."""

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytestmark = pytest.mark.skip("needs a GPU")
else:
    pytestmark = pytest.mark.gpu

import __graft_entry__  # noqa: E402

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


class Table:
    """Logits by the last token and the position, the position's tokens kept
    in a cache of `room` positions; from length `bad` on, sequence 1's are NaN."""

    def __init__(self, B, W, V, room, bad=None):
        self.base = (3 * torch.randn(64, V, generator=torch.Generator().manual_seed(4))).to(DEV)
        self.cache = torch.zeros(B, W, room, dtype=torch.int32, device=DEV)
        self.rows, self.room, self.bad = torch.arange(B, device=DEV), room, bad

    def __call__(self, tokens, lengths):
        at = (lengths.long() - 1).clamp(min=0)
        last = tokens[self.rows, :, at]
        put = at.clamp(max=self.room - 1)
        self.cache[self.rows, :, put] = torch.where((at < self.room)[:, None], last, self.cache[self.rows, :, put])
        x = self.base[(last.long() + 31 * at[:, None]) % 64]
        if self.bad is not None:
            x = torch.where(((lengths >= self.bad) & (self.rows == 1))[:, None, None], float("nan"), x)
        return x


def start(B, W, V, T):
    tokens = torch.zeros(B, W, T, dtype=torch.int32, device=DEV)
    tokens[:, :, :4] = torch.randint(0, V, (B, 1, 4), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    return tokens, torch.full((B,), 4, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("eos", [-1, 5])
def test_a_bad_logit(eos, graph):
    """The sequence keeps what it had, and its status says so; the others go on."""
    B, W, V, T = 3, 4, 500, 16
    sound, broken = Table(B, W, V, T), Table(B, W, V, T, bad=8)
    tokens, lengths = start(B, W, V, T)
    a = sv().BeamDecoder(sound, tokens.clone(), lengths.clone(), eos, [sound.cache], [2])
    b = sv().BeamDecoder(broken, tokens.clone(), lengths.clone(), eos, [broken.cache], [2])
    a.run(4, graph=graph)
    kept = [x[1].clone() for x in (a.tokens, a.scores, a.finished, a.lengths)]
    a.run(4, graph=graph)
    b.run(8, graph=graph)
    torch.cuda.synchronize()
    assert a.status.tolist() == [0, 0, 0] and b.status.tolist() == [0, sv().SEQ_BAD_VALUE, 0]
    for i in (0, 2):
        for x, y in ((a.tokens, b.tokens), (a.scores, b.scores), (a.finished, b.finished), (a.lengths, b.lengths),
                     (sound.cache, broken.cache)):
            assert torch.equal(x[i], y[i])
    for x, y in zip((b.tokens, b.scores, b.finished, b.lengths), kept):
        assert torch.equal(x[1], y)
    assert b.lengths[1] == 8


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("room", [7, 11, 15, 16])
def test_a_short_cache(room, graph):
    """A cache with fewer positions than the sequences come to: they end where
    it does, and the status says so.  One position less than the tokens is
    enough, the last token's being never asked for."""
    B, W, V, T, steps = 2, 4, 500, 16, 14
    whole, short = Table(B, W, V, T), Table(B, W, V, room)
    tokens, lengths = start(B, W, V, T)
    lengths[1] = 2
    a = sv().BeamDecoder(whole, tokens.clone(), lengths.clone(), -1, [whole.cache], [2])
    b = sv().BeamDecoder(short, tokens.clone(), lengths.clone(), -1, [short.cache], [2])
    enough = room >= T - 1
    for i in range(B):  # the whole search, as far as the short one gets
        n = min(steps, (T if enough else room + 1) - int(lengths[i]))
        one = sv().BeamDecoder(whole, tokens.clone(), lengths.clone(), -1, [whole.cache], [2])
        whole.cache.zero_()
        one.run(n, graph=False)
        if i == 0:
            b.run(steps, graph=graph)
            torch.cuda.synchronize()
        assert torch.equal(one.tokens[i], b.tokens[i]) and torch.equal(one.scores[i], b.scores[i])
        assert one.lengths[i] == b.lengths[i]
        m = min(room, int(b.lengths[i]) - 1)
        assert torch.equal(whole.cache[i, :, :m], short.cache[i, :, :m])
    assert b.status.tolist() == [0 if enough else sv().SEQ_BAD_LAYOUT] * B
    a.run(steps, graph=graph)
    assert a.status.tolist() == [0] * B
