"""Beam selection and reordering at the ends of their ranges."""

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
F32_MAX = float(torch.finfo(torch.float32).max)


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("W,V", [(2, 20000), (3, 129281), (2, 5)])
@pytest.mark.parametrize("high", [1e30, 1e32, 3e38, F32_MAX])
def test_select_high_scores_on_the_lowest_logits(high, W, V, dtype):
    """A beam far above zero whose logits are all near the type's lowest
    value: the difference of its score and its logarithm leaves f32's range,
    its candidates' scores do not."""
    B, n = 2, 8
    x = torch.full((B, W, V), torch.finfo(dtype).min, dtype=dtype)
    x[:, 1:] = torch.randn(B, W - 1, V, generator=torch.Generator().manual_seed(V)).to(dtype)
    x[1, 0, V // 2] = 1.0  # one token far above the others: a second sequence without the overflow
    c = torch.full((B, W), -1.0)
    c[:, 0] = high
    r = sv().beam_select(x.to(DEV), c.to(DEV), n)
    o = oracle.beam_select(x.float().numpy(), c.numpy(), n)
    assert (r.status == 0).all()
    assert np.array_equal(r.parents.cpu().numpy(), o.parents) and np.array_equal(r.tokens.cpu().numpy(), o.tokens)
    # scores of 2^-24 relative, or of the logarithm's 2^-17 near zero
    assert np.all(np.abs(r.scores.cpu().numpy().astype(np.float64) - o.scores)[o.parents >= 0]
                  <= 2.0 ** -24 * np.abs(o.scores[o.parents >= 0]) + 2.0 ** -17)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [2.0 ** 20, 2.0 ** 30, 2.0 ** 40, -2.0 ** 40, 2.0 ** 100])
def test_select_order_with_logits_far_from_zero(at, dtype):
    """Rows of `count` equal maxima at a power of two, the other tokens twice
    as far down or more: log-probabilities -ln count, exactly, whatever the
    power.  Running scores take the beams to within an f32 step of one another;
    the order is that of c - ln count in 64 bits."""
    B, W, V, n = 16, 8, 700, 16
    rng = np.random.default_rng(5)
    low = -3.0 * abs(at)
    x = np.full((B, W, V), low)
    count = rng.integers(2, 60, (B, W))
    first = np.zeros((B, W, 16), np.int64)
    for b in range(B):
        for w in range(W):
            where = rng.permutation(V)[:count[b, w]]
            x[b, w, where] = at
            where.sort()
            first[b, w, :min(16, count[b, w])] = where[:16]
    c = (np.log(count) - 1.0).astype(np.float32)
    score = c.astype(np.float64) - np.log(count)
    for b in range(B):  # equal counts tie; the others are apart by more than 64-bit scores may be off
        assert np.diff(np.unique(score[b])).min(initial=1.0) >= 1e-10
    r = sv().beam_select(torch.from_numpy(x).to(dtype).to(DEV), torch.from_numpy(c).to(DEV), n)
    p, t = r.parents.cpu().numpy(), r.tokens.cpu().numpy()
    for b in range(B):
        want = sorted((-score[b, w], w, int(first[b, w, i])) for w in range(W) for i in range(min(16, count[b, w])))[:n]
        assert [(a, k) for a, k in zip(p[b].tolist(), t[b].tolist())] == [(w, v) for _, w, v in want]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("W,V", [(2, 3001), (4, 70000)])
def test_select_rows_all_at_the_lowest(W, V, dtype):
    """A row that a mask of the type's lowest value leaves nothing of is
    uniform: its candidates have log-probability -ln V."""
    n = 2 * W
    x = torch.randn(3, W, V, generator=torch.Generator().manual_seed(W)).to(dtype)
    x[0, 0] = x[1, 1] = x[2] = torch.finfo(dtype).min
    c = torch.full((3, W), -1.0)
    c[1, 1] = 20.0
    r = sv().beam_select(x.to(DEV), c.to(DEV), n)
    score = (c[:, :, None].double() + torch.log_softmax(x.double(), 2)).flatten(1)
    s, i = score.sort(dim=1, descending=True, stable=True)
    assert torch.equal(r.parents.cpu().long(), i[:, :n] // V) and torch.equal(r.tokens.cpu().long(), i[:, :n] % V)
    assert ((r.scores.cpu().double() - s[:, :n]).abs() <= 2.0 ** -24 * s[:, :n].abs() + 2.0 ** -17).all()
    assert (i[1, :n] // V == 1).all() and abs(float(s[1, 0]) - 20.0 + np.log(V)) < 1e-9


@pytest.mark.parametrize("low", [-1e9, -1e10, -1e20, -1e30, "lowest"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,W,V", [(3, 1, 513), (4, 3, 20000), (24, 2, 40000), (2, 8, 129281)])
def test_select_masked_stretches(B, W, V, dtype, low):
    """Stretches of a row at a mask's value, before, behind and around the
    tokens that are left: the masked ones add nothing to the row's sum,
    wherever a warp or a slice begins.  Beams far apart, so that no pair of
    them is near enough to have its logarithms taken again."""
    if low == "lowest" or dtype == torch.float16:
        low = torch.finfo(dtype).min
    n = 6
    g = torch.Generator().manual_seed(V)
    x = torch.randn(B, W, V, generator=g)
    left = [slice(V - V // 5, V), slice(0, V // 7), slice(V // 2, V // 2 + 9), slice(V - 7, V)]
    for b in range(B):
        for w in range(W):
            keep = x[b, w, left[(b + w) % 4]].clone()
            x[b, w] = low
            x[b, w, left[(b + w) % 4]] = keep
    x = x.to(dtype)
    c = -20.0 * torch.arange(W)[None, :] - torch.rand(B, W, generator=g)
    r = sv().beam_select(x.to(DEV), c.to(DEV), n)
    o = oracle.beam_select(x.double().numpy(), c.numpy(), n)
    assert (r.status == 0).all()
    assert np.array_equal(r.parents.cpu().numpy(), o.parents) and np.array_equal(r.tokens.cpu().numpy(), o.tokens)
    d = np.abs(r.scores.cpu().numpy().astype(np.float64) - o.scores)
    assert (d <= 2.0 ** -24 * np.abs(o.scores) + 2.0 ** -17).all(), d.max()


@pytest.mark.parametrize("ended", [False, True])
def test_select_minus_zero(ended):
    """A score of -0 ties with one of 0: the lower beam first."""
    W, V = 4, 3
    x = torch.full((2, W, V), -float("inf"))
    x[:, :, 1] = torch.tensor([-0.0, 0.0, 0.0, -0.0])
    c = torch.tensor([[-0.0, 0.0, -0.0, 0.0], [0.0, -0.0, 0.0, -0.0]])
    fin = torch.tensor([[True, False, True, False], [True, True, True, True]]) if ended else None
    for n in (1, 2, 4):
        r = sv().beam_select(x.to(DEV), c.to(DEV), n, None if fin is None else fin.to(DEV), 1 if ended else -1)
        assert r.parents.tolist() == [list(range(n))] * 2 and (r.tokens == 1).all() and (r.scores == 0).all()


def test_reorder_many_sequences():
    """More sequences than 46340: their square is no size of anything."""
    B, W = 50000, 3
    g = torch.Generator().manual_seed(1)
    t = torch.randint(0, 1 << 30, (B, W), generator=g, dtype=torch.int32)
    u = torch.randint(0, 1 << 30, (B, W, 9), generator=g, dtype=torch.int32)
    parents = torch.randint(-1, W, (B, W), generator=g, dtype=torch.int32)
    take = torch.where(parents < 0, torch.arange(W), parents).long()
    lengths = torch.randint(0, 10, (B,), generator=g, dtype=torch.int32)
    dt, du = t.to(DEV), u.to(DEV)
    st = sv().beam_reorder([dt, du], parents.to(DEV), lengths.to(DEV), [None, 2])
    assert (st == 0).all()
    rows = torch.arange(B)[:, None]
    assert torch.equal(dt.cpu(), t[rows, take])
    live = torch.arange(9)[None, None] < lengths[:, None, None]
    assert torch.equal(du.cpu(), torch.where(live, u[rows, take], u))


@pytest.mark.parametrize("B,elements", [(64, 16384), (64, 16383), (300, 4096), (49, 16384)])
def test_reorder_one_segment_per_beam(B, elements):
    """A state of one segment per beam for many sequences."""
    W = 4
    g = torch.Generator().manual_seed(B)
    t = torch.randn(B, W, elements, generator=g)
    parents = torch.randint(0, W, (B, W), generator=g, dtype=torch.int32)
    d = t.to(DEV)
    assert (sv().beam_reorder(d, parents.to(DEV)) == 0).all()
    assert torch.equal(d.cpu(), t[torch.arange(B)[:, None], parents.long()])


def test_reorder_refuses_its_own_arguments_as_states():
    """Parents or lengths that would move while they are read."""
    p = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    ln = torch.zeros(2, dtype=torch.int32, device=DEV)
    q = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    t = torch.zeros(2, 3, 8, device=DEV)
    for states, kw in (([t, p], {}), (p, {}), (ln[:, None], dict(parents=q, lengths=ln))):
        with pytest.raises(ValueError, match="while it is read"):
            sv().beam_reorder(states, **{"parents": p, **kw})
    assert (sv().beam_reorder([t, p], p.long()) == 0).all()  # (a copy of them is read)
