"""Beam selection and reordering at the ends of their ranges."""

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
