"""The decoders' counter-based uniforms on the CPU: any seed is taken, what small
seeds and early rounds gave stays, and (seed, round) pairs have draws of their own."""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_decode_gb300 as sv  # noqa: E402

B, N, K = 3, 5, 4


def tree(seed):
    c = sv.paged_cache(1, 8, 8, 1, 8, B, 2, device="cpu")
    return sv.TreeDecoder(None, None, c, torch.zeros(B, 16, dtype=torch.int32), torch.ones(B, dtype=torch.int32), [-1, 0, 1, 2, 3], seed=seed)


def chain(seed):
    return sv.SpeculativeDecoder(None, None, torch.zeros(B, 16, dtype=torch.int32), torch.ones(B, dtype=torch.int32), K, 100, seed=seed)


def draws(make, seed, round_):
    d = make(seed)
    d.counter.fill_(round_)
    if make is tree:
        return d._uniforms().reshape(-1)
    return torch.cat([d._uniforms(i).reshape(-1) for i in range(2)])


def words(x):
    """The mix as it stands for seeds below 2^16 and rounds below 2^16, in whole numbers."""
    M = (1 << 64) - 1
    out = []
    for v in x:
        for mul, sh in ((0x5851F42D4C957F2D, 33), (0x2545F4914F6CDD1D, 29), (0x14057B7EF767814F, 31)):
            v = ((v ^ (v >> sh)) * mul) & M
        out.append((v >> 40) & 0xFFFFFF)
    return out


@pytest.mark.parametrize("seed", [0, 1, 5, 40000, 65535])
@pytest.mark.parametrize("round_", [0, 1, 77, 16383])
def test_small_seeds_and_early_rounds_keep_their_draws(seed, round_):
    want = words([i + (round_ << 32) + (seed << 48) for i in range(B * N)])
    assert (draws(tree, seed, round_) * (1 << 24)).long().tolist() == want
    want = words([i + ((4 * round_ + s) << 32) + (seed << 48) for s in range(2) for i in range(B * (K + 1))])
    assert (draws(chain, seed, round_) * (1 << 24)).long().tolist() == want


@pytest.mark.parametrize("make", [tree, chain])
def test_seeds_and_rounds_differ(make):
    seen = {}
    for seed in (0, 1, 2, 5, 65535, 65536, 65537, 65541, 1 << 20, 1 << 30, (1 << 31) - 1):
        for round_ in (0, 1, 16383, 16384, 32768, 65535, 65536, 131072, 1 << 20, 1 << 33, 1 << 45):
            u = draws(make, seed, round_)
            assert ((u >= 0) & (u < 1)).all()
            key = tuple(u.tolist())
            assert key not in seen, (seed, round_, seen[key])
            seen[key] = (seed, round_)


@pytest.mark.parametrize("make", [tree, chain])
def test_draws_of_neighbouring_seeds_do_not_share_a_place(make):
    """No draw of one (seed, round) stands anywhere in another's: by chance two
    sets of 30 words of 24 bits meet once in 2^24 / 900."""
    sets = [set(draws(make, s, r).tolist()) for s, r in ((0, 0), (1, 0), (0, 65536), (0, 16384), (65536, 0), (65537, 0), (1, 131072))]
    for i, a in enumerate(sets):
        for b in sets[:i]:
            assert not a & b
