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
