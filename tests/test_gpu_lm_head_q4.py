"""The LM head on a 4-bit projection, on the GPU, against fp64 products.

Tolerance: products of a state with an integer are exact in f32 (8 or 11
significant bits times 4); a group's sum is accumulated in f32, at most one
truncation (2^-23 of the running sum of magnitudes) per accumulation step of
at least 16 products or one rounding per product, so at most 128 steps; then
one product and one addition per group.  With d / 32 <= 512 groups every
logit is within (128 + 2 * 512) 2^-23 < 2^-12 of sum |h W| at worst; these
tests ask for 2^-16 of it, which bounds the sum of at most 128 truncations
even if all of them fall the same way, and leaves no room for a weight rounded
to bf16 or f16 (2^-9, 2^-12).
"""

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
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


def make(seed, rows, V, d, group, dtype="bf16", scale="bf16", zeros=False):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(rows, d, generator=g).to(DT[dtype])
    G = -(-d // group)
    packed = torch.randint(0, 256, (V, d // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand(V, G, generator=g) - 0.3) / d ** 0.5).to(DT[scale])
    z = torch.randint(0, 16, (V, G), generator=g, dtype=torch.uint8) if zeros else None
    return h, sv().Q4Projection(packed, scales, z, group)


def on_dev(p):
    return sv().Q4Projection(*(None if t is None else t.to(DEV) for t in p[:3]), p.group)


def reference(h, p):
    """(logits, sum |h W|) in fp64, on the GPU (the oracle's definition)."""
    z = 8.0 if p.zeros is None else p.zeros.to(DEV).double().repeat_interleave(p.group, 1)[:, :h.shape[1]]
    b = p.packed.to(DEV)
    q = torch.stack((b & 15, b >> 4), 2).flatten(1).double()
    w = (q - z) * p.scales.to(DEV).double().repeat_interleave(p.group, 1)[:, :h.shape[1]]
    x = h.to(DEV).double()
    return x @ w.T, x.abs() @ w.abs().T


def check(h, p, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = sv().lm_head_logits(h.to(DEV), on_dev(p), err=err, **kw)[:, :p.packed.shape[0]]
    want, mag = reference(h, p)
    assert err.item() == 0
    off = (got.double() - want).abs()
    assert (off <= REL * mag).all(), ((off / mag.clamp(min=1e-300)).max().item())
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,V,d,group", [
    (1, 1, 32, 32), (1, 5, 64, 64), (3, 300, 96, 32), (7, 1000, 160, 128), (8, 257, 256, 64), (9, 255, 512, 128),
    (16, 2048, 1024, 32), (17, 1025, 2080, 128), (33, 700, 288, 64), (64, 512, 544, 32), (65, 300, 128, 128),
    (130, 900, 1056, 128), (11, 32000, 4096, 128), (1, 50257, 2080, 64), (5, 3000, 16384, 128),
    (16, 700, 8192, 32), (14, 5000, 10016, 64), (16, 40000, 8192, 128), (12, 39000, 1024, 32), (2, 160000, 64, 32),
])
def test_logits_shapes(dtype, rows, V, d, group):
    h, p = make(rows + V + d, rows, V, d, group, dtype, "f16" if dtype == "f16" else "bf16", zeros=rows % 2 == 0)
    check(h, p)


@pytest.mark.parametrize("scale", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_logits_scales_and_zeros(scale, zeros, group):
    h, p = make(group, 6, 777, 1184, group, "bf16", scale, zeros)
    check(h, p)


def test_logits_against_the_oracle_exactly_in_integers():
    """States in small integers and power-of-two scales: every sum is exact in
    f32, so the logits equal the oracle's bit for bit."""
    g = torch.Generator().manual_seed(3)
    for d, group, dt in ((256, 32, torch.bfloat16), (1088, 64, torch.float16), (2048, 128, torch.bfloat16)):
        h = torch.randint(-8, 9, (5, d), generator=g).to(dt)
        G = -(-d // group)
        p = sv().Q4Projection(torch.randint(0, 256, (401, d // 2), generator=g, dtype=torch.uint8),
                              torch.ldexp(torch.ones(401, G), torch.randint(-3, 2, (401, G), generator=g)).to(dt),
                              torch.randint(0, 16, (401, G), generator=g, dtype=torch.uint8), group)
        got = sv().lm_head_logits(h.to(DEV), on_dev(p)).cpu().numpy()
        want = oracle.q4_logits(h.float().numpy(), p.packed.numpy(), p.scales.float().numpy(), p.zeros.numpy(), group)
        assert np.array_equal(got, want.astype(np.float32)) and np.array_equal(want, want.astype(np.float32))


def test_every_code_and_position():
    """One-hot states pick single weights: every code of 0..15 at every place
    of a 64-weight stretch, exactly."""
    d, V = 64, 16
    q = (torch.arange(V)[:, None] + torch.arange(d)[None, :]) % 16
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8)
    for zeros in (None, torch.full((V, 2), 3, dtype=torch.uint8)):
        p = sv().Q4Projection(packed, torch.ones(V, 2), zeros, 32)
        for dt in (torch.bfloat16, torch.float16):
            got = sv().lm_head_logits(torch.eye(d, dtype=dt, device=DEV), on_dev(p)).cpu()
            assert torch.equal(got.T, (q - (8 if zeros is None else 3)).float())


def test_logits_out_and_around():
    """`out` with a longer stride: what lies behind the vocabulary stays; the
    states may be a 3-D view; host inputs come back to the host."""
    h, p = make(5, 10, 999, 256, 64)
    out = torch.full((12, 1100), 7.0, device=DEV)
    check(h, p, out=out[:10])
    assert (out[:, 999:] == 7).all() and (out[10:] == 7).all()
    a = sv().lm_head_logits(h.to(DEV).view(2, 5, 256), on_dev(p))
    assert torch.equal(a, out[:10, :999])
    b = sv().lm_head_logits(h, p)
    assert b.device.type == "cpu" and torch.equal(b, a.cpu())


def test_values_pass_through():
    """NaN and infinities in a state's row reach that row's logits only; a NaN
    scale its vocabulary row only."""
    h, p = make(6, 4, 300, 256, 64)
    h[1, 17] = float("nan")
    h[2, 200] = float("inf")
    p.scales[5, 2] = float("nan")
    got = sv().lm_head_logits(h.to(DEV), on_dev(p)).cpu()
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[2]).any()
    assert torch.isnan(got[:, 5]).all()
    keep = torch.ones(300, dtype=torch.bool)
    keep[5] = False
    assert torch.isfinite(got[[0, 3]][:, keep]).all()


def test_far_offsets():
    """A projection beyond 2^32 nibbles and logits beyond 2^31 elements."""
    V, d = 300000, 16384
    g = torch.Generator().manual_seed(7)
    packed = torch.zeros(V, d // 2, dtype=torch.uint8, device=DEV)
    packed[-200:] = torch.randint(0, 256, (200, d // 2), generator=g, dtype=torch.uint8).to(DEV)
    scales = torch.full((V, d // 128), 2.0 ** -6, dtype=torch.bfloat16, device=DEV)
    h = torch.randn(2, d, generator=g).to(torch.bfloat16)
    got = sv().lm_head_logits(h.to(DEV), sv().Q4Projection(packed, scales, None, 128))
    tail = sv().Q4Projection(packed[-200:].cpu(), scales[-200:].cpu(), None, 128)
    want, mag = reference(h, tail)
    assert ((got[:, -200:].double() - want).abs() <= REL * mag).all()
    ld = (1 << 30) + 4
    out = torch.empty(3 * ld, dtype=torch.float32, device=DEV).as_strided((3, 200), (ld, 1))
    h3 = torch.randn(3, d, generator=g).to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv().lm_head_logits(h3.to(DEV), on_dev(tail), out=out, err=err)
    want, mag = reference(h3, tail)
    assert ((out.double() - want).abs() <= REL * mag).all()


def test_refusals():
    h, p = make(8, 2, 40, 64, 32)
    h, p = h.to(DEV), on_dev(p)
    for bad in (p._replace(group=48), p._replace(scales=p.scales[:, :1]), p._replace(scales=p.scales.double()),
                p._replace(zeros=torch.zeros(40, 1, dtype=torch.uint8, device=DEV)),
                p._replace(packed=p.packed.to(torch.int32))):
        with pytest.raises(ValueError):
            sv().lm_head_logits(h, bad)
    with pytest.raises(ValueError):
        sv().lm_head_logits(h.float(), p)
    with pytest.raises(ValueError):
        sv().lm_head_logits(h[:, :32], p)
    with pytest.raises(ValueError):
        sv().lm_head_logits(h, p, out=torch.empty(2, 39, device=DEV))
    with pytest.raises(ValueError):
        sv().lm_head_verify_static(h, h, p, torch.ones(1), torch.zeros(1), torch.zeros(2))


def test_output_refusals():
    """Rows of `out` that share memory, and words elsewhere, are refused."""
    h, p = make(8, 3, 40, 64, 32)
    h, p = h.to(DEV), on_dev(p)
    with pytest.raises(ValueError, match="out"):
        sv().lm_head_logits(h, p, out=torch.empty(1, 40, device=DEV).expand(3, 40))
    with pytest.raises(ValueError, match="out"):
        sv().lm_head_logits(h, p, out=torch.empty(200, device=DEV).as_strided((3, 40), (32, 1)))
    with pytest.raises(ValueError, match="err"):
        sv().lm_head_logits(h, p, err=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="err"):
        sv().lm_head_logits(h, p, err=torch.zeros(1, dtype=torch.uint8, device=DEV))
    one = sv().lm_head_logits(h[:1], p, out=torch.empty(1, 40, device=DEV).expand(1, 40))
    assert torch.equal(one, sv().lm_head_logits(h[:1], p))


def test_streams_and_graphs():
    cases = [make(30 + i, 6, 8000, 1024, 64, zeros=bool(i)) for i in range(2)]
    cases = [(h.to(DEV), on_dev(p)) for h, p in cases]
    want = [sv().lm_head_logits(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            for _ in range(3):
                r = sv().lm_head_logits(*c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s, capture_error_mode="relaxed"):
            outs.append(sv().lm_head_logits(*c))
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_verify_from_states():
    """lm_head_verify on a 4-bit projection: the logits it read are the 4-bit
    product's, and its results the verification of those logits."""
    from workloads.lm_head import make_lm_head
    wl = make_lm_head(seed=5, B=7, K=3, V=5001, d=512)
    wl.temperature[::3] = 0.0
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(DEV).view(torch.bfloat16)
    w = bf(wl.w)
    T, tok, u = (torch.from_numpy(a).to(DEV) for a in (wl.temperature, wl.tokens, wl.uniforms))
    for zeros, dt in ((False, torch.bfloat16), (True, torch.float16)):
        p = sv().q4_quantize(w, 64, zeros)
        ht, hd = bf(wl.h_target).to(dt), bf(wl.h_draft).to(dt)
        r = sv().lm_head_verify(ht, hd, p, T, tok, u)
        for h, got in ((ht, r.target_logits), (hd, r.draft_logits)):
            want, mag = reference(h, p)
            assert ((got.double() - want).abs() <= REL * mag).all()
        v = sv().accept_from_logits(r.target_logits.contiguous(), r.draft_logits.contiguous(), T, tok, u)
        for a, b in zip(r[:3], v):
            assert torch.equal(a, b)
    # ragged: K_b in 0..3
    cu = torch.tensor([0, 3, 3, 4, 6, 9, 11, 12], dtype=torch.int32, device=DEV)
    r = sv().lm_head_verify(ht[:19], hd[:12], p, T, tok[:12], u[:19], cu_k=cu, k=3)
    v = sv().accept_from_logits(r.target_logits.contiguous(), r.draft_logits.contiguous(), T, tok[:12], u[:19],
                                cu_k=cu, k=3)
    for a, b in zip(r[:3], v):
        assert torch.equal(a, b)


def test_empty_and_single():
    """No rows, one row given as a vector, no drafts, no sequences."""
    h, p = make(50, 3, 300, 128, 64)
    h, q = h.to(DEV), on_dev(p)
    assert sv().lm_head_logits(h[:0], q).shape == (0, 300)
    all_rows = sv().lm_head_logits(h, q)
    assert torch.equal(sv().lm_head_logits(h[1], q), sv().lm_head_logits(h[1:2], q))
    T = torch.zeros(3, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    r = sv().lm_head_verify(h, h[:0], q, T, none, torch.rand(3, device=DEV))
    assert torch.equal(r.next_token.long(), all_rows.argmax(1)) and (r.n_accepted == 0).all()
    r = sv().lm_head_verify(h[:0], h[:0], q, T[:0], none, T[:0])
    assert r.n_accepted.shape == (0,)


@pytest.mark.parametrize("rows", [3, 30])
def test_a_workspace_is_enough(rows):
    """A verification in the caller's workspace, twice: the same results, and
    nothing written behind it."""
    V, d, B = 1003, 256, rows
    h, p = make(51, 2 * B, V, d, 128)
    h, q = h.to(DEV), on_dev(p)
    tok = torch.randint(0, V, (B,), generator=torch.Generator().manual_seed(2), dtype=torch.int32).to(DEV)
    u = torch.rand(2 * B, generator=torch.Generator().manual_seed(3)).to(DEV)
    T = torch.full((B,), 0.7, device=DEV)
    need = sv().lm_head_workspace(B, B, V).numel()
    buf = torch.full((need + 4096,), 171, dtype=torch.uint8, device=DEV)
    a = sv().lm_head_verify(h, h[:B], q, T, tok, u)
    for _ in range(2):
        b = sv().lm_head_verify(h, h[:B], q, T, tok, u, workspace=buf[:need])
        assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    assert (buf[need:] == 171).all()
