"""Weights that a projection in 4 bits cannot hold are refused, and those at the
end of the scales' range are held (host only)."""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_decode_gb300 as sv  # noqa: E402


def values(p, d):
    q = torch.stack((p.packed & 15, p.packed >> 4), 2).flatten(1).double()
    z = 8.0 if p.zeros is None else p.zeros.double().repeat_interleave(p.group, 1)[:, :d]
    return (q - z) * p.scales.double().repeat_interleave(p.group, 1)[:, :d]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_weights_that_are_not_finite(bad, zeros):
    w = torch.randn(4, 96, generator=torch.Generator().manual_seed(1))
    w[2, 70] = bad
    with pytest.raises(ValueError, match="finite"):
        sv.q4_quantize(w, 32, zeros)


@pytest.mark.parametrize("zeros", [False, True])
def test_scales_past_their_type(zeros):
    w = torch.randn(4, 96, generator=torch.Generator().manual_seed(1))
    w[1, 5] = 2e6
    with pytest.raises(ValueError, match="too large"):
        sv.q4_quantize(w, 32, zeros, torch.float16)
    w[1, 5] = 4e5  # a scale of 57143 or 26667
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        p = sv.q4_quantize(w, 32, zeros, dt)
        step = p.scales.double().repeat_interleave(32, 1)
        # half a step, and at the group's end 15 times what rounding the scale takes off a step
        off = (values(p, 96) - w.double()).abs()
        assert (off <= step * (0.5 + 15 * torch.finfo(dt).eps / 2) * (1 + 1e-6)).all()
