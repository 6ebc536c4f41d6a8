"""The LM head on a 4-bit projection where the states of a row differ by far.

A state that meets a code equal to its zero adds nothing to a logit, however
large it is: products are formed with the integers q - zero, so they count
relative to sum |h W| alone.  The bound is the one of the ordinary cases: a
group's sum of exact products takes at most 128 truncations of 2^-23 of the
running sum of magnitudes, its scaling and the sum over the groups 2 more
roundings per group, and 2^-16 of sum |h W| holds them with the group sums'
truncations all falling the same way (128 2^-23 = 2^-16).
"""

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytestmark = pytest.mark.skip("needs a GPU")
else:
    pytestmark = pytest.mark.gpu

import __graft_entry__  # noqa: E402

DEV = torch.device("cuda", 0)
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


def near_zero_codes(seed, V, d, group, zeros, scale="bf16"):
    """A projection whose codes are their zero or one beside it, and those zeros per weight."""
    g = torch.Generator().manual_seed(seed)
    G = -(-d // group)
    z = torch.randint(1, 15, (V, G), generator=g, dtype=torch.uint8) if zeros else torch.full((V, G), 8, dtype=torch.uint8)
    of = z.repeat_interleave(group, 1)[:, :d]
    q = of + torch.randint(0, 3, (V, d), generator=g, dtype=torch.uint8) - 1
    scales = ((torch.rand(V, G, generator=g) + 0.3) / d ** 0.5).to(DT[scale])
    return q, of, scales, z if zeros else None


def projection(q, scales, z, group):
    return sv().Q4Projection((q[:, 0::2] | (q[:, 1::2] << 4)).to(DEV), scales.to(DEV), None if z is None else z.to(DEV),
                             group)


def check(h, p):
    d = h.shape[1]
    b = p.packed
    q = torch.stack((b & 15, b >> 4), 2).flatten(1).double()
    z = 8.0 if p.zeros is None else p.zeros.double().repeat_interleave(p.group, 1)[:, :d]
    w = (q - z) * p.scales.double().repeat_interleave(p.group, 1)[:, :d]
    x = h.to(DEV).double()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv().lm_head_logits(h.to(DEV), p, err=err)
    assert err.item() == 0
    off, mag = (got.double() - x @ w.T).abs(), x.abs() @ w.abs().T
    assert (off <= REL * mag).all(), (off / mag).max().item()
    return got


@pytest.mark.parametrize("rows", [1, 8, 16, 17, 40])
@pytest.mark.parametrize("dtype,large", [("bf16", 1e3), ("bf16", 1e4), ("bf16", 1e5), ("bf16", 1e30), ("f16", 1e3), ("f16", 6e4)])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False), (128, True)])
def test_large_states_on_codes_equal_to_their_zero(group, zeros, dtype, large, rows):
    """One state per group far above the others, at every place of eight
    neighbouring columns, on codes equal to their zero."""
    V, d = 300, 1056
    q, of, scales, z = near_zero_codes(rows, V, d, group, zeros)
    h = torch.randn(rows, d, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    for i, at in enumerate(range(3, d, 31)):  # (31: every place modulo 32)
        q[:, at] = of[:, at]
        h[:, at] = large if i % 2 else -large
    check(h, projection(q, scales, z, group))


@pytest.mark.parametrize("rows", [7, 16, 17])
@pytest.mark.parametrize("group", [32, 128])
def test_states_of_many_magnitudes(group, rows):
    """Magnitudes from 2^-60 to 2^60 in one row; a vocabulary row sees one band
    of them, the other codes being equal to their zero."""
    V, d = 240, 512
    g = torch.Generator().manual_seed(2)
    band = torch.randint(0, 12, (d,), generator=g)
    h = (torch.randn(rows, d, generator=g) * torch.exp2(10.0 * band - 60)).to(torch.bfloat16)
    q = torch.randint(0, 16, (V, d), generator=g, dtype=torch.uint8)
    q[(torch.arange(V) % 12)[:, None] != band[None]] = 8
    scales = ((torch.rand(V, -(-d // group), generator=g) + 0.3)).to(torch.bfloat16)
    check(h, projection(q, scales, None, group))


@pytest.mark.parametrize("rows", [5, 16, 17])
@pytest.mark.parametrize("dtype,scale", [("bf16", 2.0 ** 110), ("bf16", 2.0 ** -100), ("f16", 2.0 ** 12), ("f16", 2.0 ** -9)])
def test_rows_near_the_ends_of_the_range(dtype, scale, rows):
    """Large and small rows beside one of ordinary size."""
    V, d, group = 300, 544, 64
    q, of, scales, z = near_zero_codes(3, V, d, group, True, "f32")
    h = torch.randn(rows, d, generator=torch.Generator().manual_seed(4)).clamp(-4, 4)
    h[1:] *= scale
    check(h.to(DT[dtype]), projection(q, scales, z, group))
