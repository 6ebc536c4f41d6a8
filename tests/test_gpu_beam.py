"""Beam selection and state reordering on the GPU against the oracle.

Scores: the kernel's f32 output may be off the exact score by the output's own
rounding (2^-24 relative) and by the error of its logarithm of the row's sum.
That sum is taken in f32: per term 3 roundings of an exponent of mean size
H - H_min <= 18 bits (12.5 half steps of 2^-24 each), the exponential (2^-21),
and at most 40 additions on the way of a term, so at most
(3 * 18 * ln 2 + 8 + 40) 2^-24 < 2^-17 relative, which is the logarithm's error.
Order: the kernel orders by the scores in 64 bits; the oracle's smallest gap
between neighbours says where that order is decided (gaps of 1e-10 and more).
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
LSE_TOL = 2.0 ** -17
GAP = 1e-10
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


def make(seed, B, W, V, dtype, pad=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(B, W, V, generator=g)
    buf = torch.full((B * W, V + pad), 1e4 if dtype != "f16" else 6e4, dtype=DT[dtype])  # past the row: never read
    buf[:, :V] = x.view(B * W, V).to(DT[dtype])
    c = -10.0 - torch.cumsum(torch.rand(B, W, generator=g), 1)
    return buf.to(DEV)[:, :V].unflatten(0, (B, W)), c.to(DEV)


def check(x, c, n, finished=None, eos=-1, need_gap=True, **kw):
    r = sv().beam_select(x, c, n, finished, eos, **kw)
    fin = None if finished is None else finished.cpu().numpy()
    o = oracle.beam_select(x.float().cpu().numpy(), c.cpu().numpy(), n, fin, eos)
    s, p, t, st = (v.cpu().numpy() for v in r)
    assert np.array_equal(st, o.status.astype(np.int32))
    decided = o.gap >= GAP
    if need_gap:
        assert decided.all()
    assert np.array_equal(p[decided], o.parents[decided])
    assert np.array_equal(t[decided], o.tokens[decided])
    none = o.parents < 0
    assert (s[none] == -np.inf).all()
    d = np.abs(s[~none].astype(np.float64) - o.scores[~none])
    assert (d <= 2.0 ** -24 * np.abs(o.scores[~none]) + LSE_TOL).all(), d.max()
    return r, o


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,W,V,n,pad", [
    (1, 1, 1, 1, 0), (2, 1, 1, 3, 0), (2, 2, 5, 4, 3), (3, 4, 257, 8, 0), (1, 64, 300, 128, 7), (5, 3, 1000, 6, 1),
    (2, 2, 4096, 16, 0), (2, 5, 4097, 10, 0), (1, 4, 32000, 8, 0), (2, 16, 8191, 32, 8), (40, 2, 2049, 4, 5),
    (2, 5, 129281, 10, 0), (1, 3, 262144, 128, 0),
])
def test_select_shapes(dtype, B, W, V, n, pad):
    x, c = make(B * 1000 + V, B, W, V, dtype, pad)
    check(x, c, n, need_gap=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_any_alignment(dtype):
    """Rows that start at every element offset of a 16-byte line."""
    buf = 3 * torch.randn(3 * 5001 + 64, generator=torch.Generator().manual_seed(5)).to(DT[dtype])
    buf = buf.to(DEV)
    c = torch.tensor([[-1.0, -1.5, -1.25]], device=DEV)
    for off in range(9):
        x = buf[off:off + 3 * 5001].view(1, 3, 5001)
        check(x, c, 6, need_gap=False)


def test_select_ties():
    """Equal scores go to the lower beam, then the lower token: uniform rows,
    rows in coarse steps, equal rows, permuted rows (equal sums, so exact
    ties between beams), ties across the whole of a large row."""
    z = torch.zeros(2, 4, 1000, device=DEV)
    r, _ = check(z, torch.zeros(2, 4, device=DEV), 8)
    assert r.tokens.tolist() == [list(range(8))] * 2
    check(z, torch.tensor([[-1.0, -1.0, 0.0, 0.0]] * 2, device=DEV), 100)
    g = torch.Generator().manual_seed(6)
    for V in (300, 40000):
        q = torch.randint(-4, 5, (3, 4, V), generator=g).float().div(4)
        for dt in (torch.float32, torch.bfloat16):
            x = q.to(dt).to(DEV)
            check(x, torch.zeros(3, 4, device=DEV) - 2.0, 17, need_gap=False)
            same = x[:, :1].expand(3, 4, V).contiguous()
            check(same, torch.zeros(3, 4, device=DEV) - 2.0, 17)
            perm = torch.stack([same[:, w][:, torch.randperm(V, generator=g).to(DEV)] for w in range(4)], 1)
            check(perm, torch.zeros(3, 4, device=DEV) - 2.0, 17)
    big = torch.zeros(1, 8, 128256, dtype=torch.bfloat16, device=DEV)
    big[0, 3, 77777] = 0.25
    r, _ = check(big, torch.zeros(1, 8, device=DEV), 16, need_gap=False)


@pytest.mark.parametrize("delta", [3e-6, 1e-6, 2e-7, 3e-8])
def test_select_near_ties(delta):
    """Beams whose best scores differ by less than f32 sums can tell: the
    order is that of the scores in 64 bits."""
    g = torch.Generator().manual_seed(7)
    B, W, V = 16, 4, 5000
    x = (2 * torch.randn(B, W, V, generator=g)).double()
    x -= torch.logsumexp(x, 2, keepdim=True)
    x[:, :, 0] = -1.0
    for _ in range(3):  # the best token at log-probability -1 exactly, up to f32 rounding of the logits
        rest = torch.logsumexp(x[:, :, 1:], 2, keepdim=True)
        x[:, :, 1:] += float(np.log1p(-np.exp(-1.0))) - rest
    x = x.float().to(DEV)
    c = (torch.rand(B, W, generator=g) * delta).to(DEV)
    check(x, c, 4, need_gap=False)
    o = oracle.beam_select(x.cpu().numpy(), c.cpu().numpy(), 4)
    assert (o.gap < 4 * delta).mean() > 0.5  # the case is what it says
    check(x, c, 8, need_gap=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_select_masks(dtype):
    """Masked tokens (-inf and the type's lowest value), rows that a mask
    leaves with one token or none, dead beams, ended beams, fewer candidates
    than asked for."""
    x, c = make(8, 6, 4, 3001, dtype)
    x[0, :, 100:] = -float("inf")
    x[1, 1:] = -float("inf")
    x[1, 0, 1:] = -float("inf")
    x[2] = -float("inf")
    x[3, :, ::2] = torch.finfo(DT[dtype]).min
    x[4, 2] = torch.finfo(DT[dtype]).min
    x[5, :, 1:] = -float("inf")
    check(x, c, 8)
    c[0, 1] = c[3, 0] = c[4, 0] = -float("inf")
    x[0, 1] = float("nan")  # a dead beam's row is not read
    fin = torch.zeros(6, 4, dtype=torch.bool, device=DEV)
    fin[3, 2] = fin[5, 0] = fin[5, 3] = True
    x[5, 0] = float("nan")  # nor an ended one's
    r, o = check(x, c, 8, fin, 7)
    assert (o.tokens[5] == 7).sum() == 2 and (r.parents[2] == -1).all()
    c[1] = -float("inf")
    fin[4] = True
    check(x, c, 128, fin, 3000, need_gap=False)


def test_select_bad_values():
    x, c = make(9, 6, 3, 5003, "bf16")
    x[0, 1, 5002] = float("nan")
    x[1, 0, 0] = float("inf")
    c[2, 1], c[3, 2] = float("nan"), float("inf")
    x[4, 2] = float("nan")
    r, o = check(x, c, 6)
    assert (o.status != 0).tolist() == [True] * 5 + [False]
    assert (r.tokens[:5] == -1).all() and (r.parents[:5] == -1).all()


def test_select_extreme_logits():
    x, c = make(10, 3, 2, 4000, "f32")
    x[0] *= 1e-30
    x[1] *= 1e30
    x[2, 0, 17], x[2, 1, 18] = 3e38, -3e38
    check(x, c, 5, need_gap=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("low", [-1e9, -1e30, float(torch.finfo(torch.float32).min)])
def test_select_beams_at_the_lowest(dtype, low):
    """Beams held off by a huge negative score (a search's first step): they
    change nothing while the others have candidates enough, and follow them
    where they have not.  With tokens at the type's lowest value as well, a
    score can lie below f32's range: that is no candidate."""
    x, c = make(14, 4, 4, 20000, dtype)
    c[:, 1:] = low
    c[1, 2] = c[0, 0]
    x[2, 0, 5:] = -float("inf")
    x[3] = torch.finfo(DT[dtype]).min
    x[3, :, 77] = 1.0
    check(x, c, 8, need_gap=False)
    check(x, c, 128, need_gap=False)


def test_select_empty_and_single():
    """No sequences; one beam whose rows lie apart; scores and flags of other types."""
    r = sv().beam_select(torch.zeros(0, 3, 50, device=DEV), torch.zeros(0, 3, device=DEV), 5)
    assert r.scores.shape == (0, 5) and r.status.shape == (0,)
    x, c = make(16, 4, 5, 900, "bf16")
    check(x[:, 2:3], c[:, 2:3], 3)  # [4, 1, 900], rows five apart
    fin = torch.zeros(4, 5, dtype=torch.int64, device=DEV)
    fin[1, 2] = 3
    a = sv().beam_select(x, c.double(), 6, fin, 4)
    b = sv().beam_select(x, c, 6, fin != 0, 4)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("B,W,V", [(1, 4, 32000), (19, 2, 4000), (20, 2, 4000), (3, 16, 48000), (3, 16, 52000)])
def test_select_one_kernel_and_two(B, W, V):
    """Both sides of the rule that takes small calls in one kernel, the
    workspace asked for being enough and nothing written behind it."""
    x, c = make(17, B, W, V, "bf16")
    n = 2 * W
    need = sv().beam_select_workspace(B, W, V, n).numel()
    buf = torch.full((need + 4096,), 171, dtype=torch.uint8, device=DEV)
    check(x, c, n, need_gap=False, workspace=buf[:need])
    assert (buf[need:] == 171).all()


@pytest.mark.parametrize("dtype,W,V,n", [
    ("bf16", 8, 2402, 16), ("f16", 64, 32000, 128), ("bf16", 64, 128256, 128), ("f32", 64, 128256, 128),
    ("f32", 64, 200001, 128), ("f32", 64, 300000, 128), ("f32", 16, 8000, 32), ("bf16", 4, 300, 8),
])
def test_select_one_live_beam(dtype, W, V, n):
    """A search's first step: one beam alive, so fewer groups of logits than
    candidates asked for; beside it, in another sequence, ended beams and a
    masked row."""
    x, c = make(18, 2, W, V, dtype)
    c[0, 1:] = -float("inf")
    c[1, 3:] = -float("inf")
    fin = torch.zeros(2, W, dtype=torch.bool, device=DEV)
    fin[1, 1] = True
    x[1, 2] = -float("inf")
    check(x, c, n, fin, 2, need_gap=False)


def test_select_refusals():
    x, c = make(15, 2, 3, 500, "bf16")
    with pytest.raises(ValueError, match="workspace"):
        sv().beam_select(x, c, 4, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    for kw in (dict(n=1 << 32), dict(n=4, eos=(1 << 32) + 5)):
        with pytest.raises(ValueError, match="below"):
            sv().beam_select(x, c, **kw)
    for n in (0, -1, 129, 1 << 30):
        with pytest.raises(sv().SVError):
            sv().beam_select(x, c, n)


def test_select_far_offsets():
    """Rows beyond 2^31 elements from the first."""
    V, stride = 1500, (1 << 28) + 8
    buf = torch.empty(9 * stride, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((3, 3, V), (3 * stride, stride, 1))
    x.copy_(3 * torch.randn(3, 3, V, generator=torch.Generator().manual_seed(11)))
    check(x, torch.full((3, 3), -2.0, device=DEV) - torch.arange(3, device=DEV), 6)


def test_select_many_sequences():
    x, c = make(12, 3000, 2, 300, "f16")
    check(x, c, 4, need_gap=False)


def test_select_host_inputs_and_workspace():
    x, c = make(13, 3, 4, 2000, "f32")
    a = sv().beam_select(x, c, 8)
    h = sv().beam_select(x.cpu(), c.cpu(), 8)
    ws = sv().beam_select_workspace(3, 4, 2000, 8)
    ws.fill_(255)  # no initial contents needed
    b = sv().beam_select(x, c, 8, workspace=ws)
    b2 = sv().beam_select(x, c, 8, workspace=ws)
    for u, v, w, z in zip(a, h, b, b2):
        assert v.device.type == "cpu" and torch.equal(u.cpu(), v) and torch.equal(u, w) and torch.equal(u, z)
    with pytest.raises(sv().SVError):
        sv().beam_select(x, c, 129)
    with pytest.raises(ValueError):
        sv().beam_select(x, c[:2], 8)
    with pytest.raises(ValueError):
        sv().beam_select(x.double(), c, 8)


def test_select_streams_and_graphs():
    """Calls on two streams at once, and two captured graphs replayed
    together: each has its own workspace."""
    xs = [make(20 + i, 8, 4, 50000, "bf16") for i in range(2)]
    want = [sv().beam_select(x, c, 8) for x, c in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(sv().beam_select(*xs[i], 8))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(want[i], r))
    graphs, outs = [], []
    for i, s in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(sv().beam_select(*xs[i], 8))
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, r in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, r))


# ------------------------------------------------------------------ reordering

def states_for(seed, B, W, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    if dtype.is_floating_point:
        return torch.randn(B, W, *shape, generator=g).to(dtype)
    return torch.randint(0, 127, (B, W, *shape), generator=g, dtype=torch.int32).to(dtype)


def bits(t):
    return t.contiguous().cpu().view(torch.uint8).numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8, torch.int64])
@pytest.mark.parametrize("B,W,shape,td", [
    (1, 1, (5,), None), (2, 2, (1,), None), (3, 4, (8, 100, 16), 3), (2, 5, (3, 77, 5), 3), (2, 16, (40, 6, 8), 2),
    (1, 64, (2, 33, 24), 3), (2, 33, (129,), 2), (4, 17, (3, 1000), None), (1, 9, (70000,), None), (2, 3, (0, 5), 2),
])
def test_reorder_shapes(dtype, B, W, shape, td):
    t = states_for(B * W, B, W, shape, dtype)
    g = torch.Generator().manual_seed(W)
    parents = torch.randint(-1, W, (B, W), generator=g, dtype=torch.int32)
    parents[0] = torch.arange(W).roll(1)  # a cycle through every slot
    T = None if td is None else t.shape[td]
    lengths = None if td is None else torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    want, st = oracle.beam_reorder(t.view(torch.int16).numpy() if dtype == torch.bfloat16 else t.numpy(),
                                   parents.numpy(), None if lengths is None else lengths.numpy(), td)
    d = t.to(DEV)
    got = sv().beam_reorder(d, parents.to(DEV), None if lengths is None else lengths.to(DEV), td)
    assert got.tolist() == st.tolist()
    assert np.array_equal(bits(d).reshape(-1), np.ascontiguousarray(want).view(np.uint8).reshape(-1))


def test_reorder_views_and_several_states():
    """Parts of longer buffers, keys and values of one fused buffer, tokens,
    recurrent states, different lengths of time: one call; what lies around
    the views and past the lengths stays."""
    B, W = 3, 6
    g = torch.Generator().manual_seed(1)
    fused = torch.randn(B, W, 2, 4, 50, 8, generator=g).to(torch.bfloat16).to(DEV)
    toks = torch.randint(0, 999, (B, W, 61), generator=g, dtype=torch.int32).to(DEV)
    rec = torch.randn(B, W, 7, 9, generator=g).to(DEV)
    odd = torch.randint(0, 255, (B + 1, W, 3, 31, 7), generator=g, dtype=torch.uint8).to(DEV)
    parents = torch.randint(0, W, (B, W), generator=g, dtype=torch.int32)
    lengths = torch.tensor([0, 17, 29], dtype=torch.int32)
    olds = [x.clone() for x in (fused, toks, rec, odd)]
    views = [fused[:, :, 0, :, :40], fused[:, :, 1, :, :40], toks[:, :, 1:], rec[:, :, :, 2:5], odd[1:, :, 1:, :30]]
    dims = [3, 3, 2, None, 3]
    wants = [oracle.beam_reorder(v.cpu().view(torch.int16).numpy() if v.dtype == torch.bfloat16 else v.cpu().numpy(),
                                 parents.numpy(), lengths.numpy(), td)[0] for v, td in zip(views, dims)]
    st = sv().beam_reorder(views, parents.to(DEV), lengths.to(DEV), dims)
    assert (st == 0).all()
    for v, w in zip(views, wants):
        assert np.array_equal(bits(v).reshape(-1), np.ascontiguousarray(w).view(np.uint8).reshape(-1))
    new_f, new_t, new_r, new_o = fused, toks, rec, odd
    assert torch.equal(new_f[:, :, :, :, 40:], olds[0][:, :, :, :, 40:])
    assert torch.equal(new_t[:, :, 0], olds[1][:, :, 0])
    assert torch.equal(new_r[:, :, :, :2], olds[2][:, :, :, :2]) and torch.equal(new_r[:, :, :, 5:], olds[2][:, :, :, 5:])
    assert torch.equal(new_o[0], olds[3][0]) and torch.equal(new_o[:, :, 0], olds[3][:, :, 0])
    assert torch.equal(new_o[:, :, :, 30], olds[3][:, :, :, 30])


def test_reorder_many_states_one_call():
    """More states than one launch describes."""
    B, W = 2, 3
    ts = [states_for(i, B, W, (4, 10 + i, 8), torch.float32).to(DEV) for i in range(101)]
    parents = torch.tensor([[1, 2, 0], [2, 2, -1]], dtype=torch.int32)
    lengths = torch.tensor([10, 3], dtype=torch.int32)
    wants = [oracle.beam_reorder(t.cpu().numpy(), parents.numpy(), lengths.numpy(), 3)[0] for t in ts]
    st = sv().beam_reorder(ts, parents.to(DEV), lengths.to(DEV), 3)
    assert (st == 0).all()
    for t, w in zip(ts, wants):
        assert np.array_equal(t.cpu().numpy(), w)


def test_reorder_bad_sequences_stay():
    """A parent or a length out of range: that sequence is left as it was in
    every state, the others move."""
    B, W = 5, 4
    a, b = states_for(1, B, W, (2, 20, 8), torch.float32), states_for(2, B, W, (12,), torch.float32)
    parents = torch.tensor([[1, 0, 3, 2]] * B, dtype=torch.int32)
    parents[1, 3] = W
    parents[4, 0] = -7
    lengths = torch.tensor([20, 20, 21, -1, 5], dtype=torch.int32)
    da, db = a.to(DEV), b.to(DEV)
    st = sv().beam_reorder([da, db], parents.to(DEV), lengths.to(DEV), [3, None])
    assert st.tolist() == [0, 64, 64, 64, 0]
    wa, _ = oracle.beam_reorder(a.numpy(), parents.numpy(), lengths.numpy(), 3)
    for i in (1, 2, 3):
        assert torch.equal(da[i].cpu(), a[i]) and torch.equal(db[i].cpu(), b[i])
    assert np.array_equal(da.cpu().numpy(), wa)
    assert torch.equal(db[0].cpu(), b[0][[1, 0, 3, 2]])


def test_reorder_far_offsets():
    """A state larger than 4 GB: the last sequence and the last positions."""
    t = torch.zeros(2, 3, 1, 1 << 20, 768, dtype=torch.uint8, device=DEV)  # 4.8 GB
    for w in range(3):
        t[1, w, 0, -1000:] = w + 1
        t[1, w, 0, :1000] = 10 + w
    parents = torch.tensor([[0, 1, 2], [2, 0, 0]], dtype=torch.int32, device=DEV)
    lengths = torch.full((2,), 1 << 20, dtype=torch.int32, device=DEV)
    assert (sv().beam_reorder(t, parents, lengths, 3) == 0).all()
    for w, p in enumerate((2, 0, 0)):
        assert (t[1, w, 0, -1000:] == p + 1).all() and (t[1, w, 0, :1000] == 10 + p).all()
    assert (t[0] == 0).all()


def test_reorder_refusals():
    t = torch.zeros(2, 3, 4, 5, device=DEV)
    p = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    ln = torch.zeros(2, dtype=torch.int32, device=DEV)
    bad = [dict(states=[t, t]), dict(states=t[:, :2]), dict(states=t, time_dim=2), dict(states=t, time_dim=1, lengths=ln),
           dict(states=t.transpose(2, 3), time_dim=3, lengths=ln), dict(states=t[:, :1].expand(2, 3, 4, 5)),
           dict(states=t, lengths=ln[:1], time_dim=3), dict(states=[t], time_dim=[3, 3], lengths=ln),
           dict(states=t.clone().requires_grad_()), dict(states=[t.cpu()]), dict(states=[t, t.cpu()])]
    for kw in bad:
        with pytest.raises(ValueError):
            sv().beam_reorder(parents=p, **kw)


def test_reorder_replayed():
    t = states_for(3, 2, 4, (2, 30, 8), torch.bfloat16).to(DEV)
    p = torch.tensor([[1, 2, 3, 0]] * 2, dtype=torch.int32, device=DEV)
    ln = torch.tensor([30, 11], dtype=torch.int32, device=DEV)
    old = t.clone()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        sv().beam_reorder(t, p, ln, 3)
    for _ in range(4):  # a cycle of four: four replays bring everything back
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(t, old)
    g.replay()
    p.copy_(torch.tensor([[0, 1, 2, 3]] * 2))
    torch.cuda.synchronize()
    assert torch.equal(t[0], old[0][[1, 2, 3, 0]])
