"""Tree attention on the GPU against the oracle in 64 bits.

Tolerances, for an element o = sum_j p_j v_j with A = sum_j p_j |v_j|, e half a
step of the type relative to a value (bf16 2^-8, f16 2^-11) and u = 2^-24:

* the result is rounded to the type: e |o| (f16: at least half its smallest
  step, 2^-25);
* a weight exp(s_j - m) is rounded to the type before it multiplies v_j: e A; one
  below the type's smallest normal number (f16: 2^-14) is off by up to 2^-25
  instead, which is at most n 2^-25 max|v| in all, since z is at least 1 (the m
  that the weights are taken against is no larger than the largest score);
* a score's f32 dot product over D terms is off by at most (D + 2) 2 u S, S the largest
  scale sum_d |q_d k_jd| (f32 adds, with one more bit for tensor-core adds that truncate), its
  product with scale log2(e) and the maximum's subtraction by 4 u (S + S), and
  the exponential by 2^-22: d = ((D + 2) 2 + 8) u S + 2^-22 relative in
  each weight, so 2 d A in the quotient;
* sums over n keys in f32: 2 n u A for the products and n u for z, bounded as
  4 n u A.

lse = m + ln z is off by d + n u + 2^-22 (|lse| + 1).

A row with a score whose terms pass f32's range has no defined result (the
products are summed in f32); such rows are not compared, those beside them are.
"""

import math
from types import SimpleNamespace

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
BF, HF = torch.bfloat16, torch.float16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


def f64(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, seed, N, lengths, Hq, Hkv, D, page, dtype, tree=True, spare=3, junk=float("nan"), q_scale=1.5, width=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.n, self.lengths = max(max(N), 1), np.array(lengths, np.int32)
        self.cu = np.concatenate(([0], np.cumsum(N))).astype(np.int32)
        total = int(self.cu[-1])
        r = lambda *s: torch.randn(*s, generator=g).to(dtype)
        self.q, self.k, self.v = (q_scale * r(total, Hq, D)).to(dtype), r(total, Hkv, D), r(total, Hkv, D)
        self.parents = np.array([-1 if i == 0 else (int(rng.integers(max(-1, i - 9), i)) if tree else i - 1) for n in N for i in range(n)],
                                np.int32)
        pages = [-(-int(x) // page) for x in lengths]
        P = sum(pages) + spare
        at = rng.permutation(P)
        width = max(pages + [1]) if width is None else width
        self.table = rng.integers(-5, P + 5, (len(N), width)).astype(np.int32)  # past the length: anything
        # what no sequence holds is junk
        self.kc, self.vc = (torch.full((P, page, Hkv, D), junk).to(dtype) for _ in range(2))
        o = 0
        for b, L in enumerate(lengths):
            self.table[b, :pages[b]] = at[o:o + pages[b]]
            for j in range(pages[b]):
                k = min(page, L - j * page)
                self.kc[at[o + j], :k], self.vc[at[o + j], :k] = r(k, Hkv, D), r(k, Hkv, D)
            o += pages[b]
        self.scale, self.dtype, self.D, self.page = 1 / math.sqrt(D), dtype, D, page

    def dev(self):
        d = lambda a: torch.as_tensor(a).to(DEV)
        return dict(q=d(self.q), k=d(self.k), v=d(self.v), k_cache=d(self.kc), v_cache=d(self.vc), table=d(self.table),
                    lengths=d(self.lengths), parents=d(self.parents), cu_nodes=d(self.cu), n=self.n)

    def oracle(self, **kw):
        a = dict(parents=self.parents, cu=self.cu, scale=self.scale, table=self.table, lengths=self.lengths)
        a.update(kw)
        return oracle.tree_attention(f64(self.q), f64(self.k), f64(self.v), f64(self.kc), f64(self.vc), a["table"],
                                     a["lengths"], a["parents"], a["cu"], self.n, a["scale"])

    def check(self, r, ref=None, keys=None):
        out, lse, mag, size, status = self.oracle() if ref is None else ref
        assert np.array_equal(r.status.cpu().numpy(), status)
        got, got_lse = f64(r.out)[:len(out)], f64(r.lse)[:len(out)]
        n = (int(np.clip(self.lengths, 0, None).max()) if keys is None else keys) + self.n
        e, tiny = (2.0 ** -8, 0.0) if self.dtype == BF else (2.0 ** -11, 2.0 ** -25)
        d = ((self.D + 2) * 2 + 8) * U * size + 2.0 ** -22
        vmax = max((float(x.abs().nan_to_num(0, 0, 0).max()) for x in (self.v, self.vc) if x.numel()), default=0.0)
        tol = e * np.abs(out) + tiny + (e + 2 * d[..., None] + 4 * n * U) * mag + (n * tiny * vmax if tiny else 0)
        known = ~np.isnan(lse) & ~(size > 2.0 ** 126 * self.scale)  # rows of a sequence
        fine = known[..., None] & np.isfinite(out)
        with np.errstate(invalid="ignore"):
            err = np.abs(got - out)
        assert (err[fine] <= tol[fine]).all(), (err - tol)[fine].max()
        lt = d + n * U + 2.0 ** -22 * (np.abs(lse) + 1)
        real = known & np.isfinite(lse)
        assert (np.abs(got_lse - lse)[real] <= lt[real]).all(), np.abs(got_lse - lse)[real].max()
        empty = known & np.isneginf(lse)
        assert np.isneginf(got_lse[empty]).all() and (got[empty] == 0).all()
        return err[fine].max() if fine.any() else 0.0


def run(c, **kw):
    return sv().tree_attention(**{**c.dev(), **kw})


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 128), (4, 1, 64), (8, 2, 128), (7, 1, 80), (6, 2, 8), (10, 2, 96), (3, 3, 72),
                                      (64, 1, 128), (128, 1, 64), (127, 1, 32)])
def test_heads_and_widths(dtype, Hq, Hkv, D):
    c = Case(D + Hq, [5, 1, 0, 19, 2], [300, 0, 77, 129, 1], Hq, Hkv, D, 16, dtype)
    c.check(run(c))


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 56, 64, 128, 200, 256, 384])
def test_pages(page):
    """Every end of a page, a tile and a sequence."""
    c = Case(page, [3] * 12, [0, 1, 7, 8, 9, 127, 128, 129, 255, 256, 385, 1000], 4, 2, 64, page, BF)
    c.check(run(c))


@pytest.mark.parametrize("N", [1, 2, 17, 31, 32, 33, 64, 100, 127, 128, 129, 200, 255, 256])
@pytest.mark.parametrize("tree", [False, True])
def test_nodes(N, tree):
    c = Case(N, [N, 1, N, max(1, N - 1)], [200, 130, 0, 5], 8, 2, 128, 16, BF, tree)
    c.check(run(c))
    if not tree:
        a, b = run(c), run(c, parents=None)
        assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


@pytest.mark.parametrize("L", [2000, 5003, 20011])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_long_contexts(L, dtype):
    """Keys split over many CTAs, beside short sequences and idle ones."""
    c = Case(L, [6, 1, 0, 3], [L, 3, 100, 1], 8, 2, 128, 64, dtype, tree=False)
    c.check(run(c))


def test_many_sequences():
    """More items than CTAs, ends of items all over the tiles."""
    rng = np.random.default_rng(1)
    B = 150
    c = Case(1, rng.integers(0, 9, B), rng.integers(0, 700, B), 4, 2, 64, 16, BF)
    c.check(run(c))
    c = Case(2, rng.integers(20, 60, 40), rng.integers(0, 300, 40), 16, 2, 128, 32, HF)
    c.check(run(c))


@pytest.mark.parametrize("B", [385, 1100])
def test_more_sequences_than_threads(B):
    """Several sequences to a thread of the plan; long ones among short ones and
    idle ones."""
    rng = np.random.default_rng(B)
    lengths = rng.integers(0, 40, B)
    lengths[rng.integers(0, B, 5)] = 3000
    c = Case(B, rng.integers(0, 4, B), lengths, 4, 2, 64, 32, BF)
    c.check(run(c))
    c = Case(B + 1, rng.integers(0, 70, B) * (rng.random(B) < 0.1), lengths, 8, 1, 64, 32, BF)
    c.check(run(c))


def test_one_sequence_among_idle_ones():
    for at in (0, 31, 32, 200, 399):
        N, lengths = np.zeros(400, int), np.full(400, 50)
        N[at], lengths[at] = 37, 2000
        c = Case(at, N, lengths, 8, 2, 128, 16, BF)
        c.check(run(c))


def test_equal_trees_in_four_dimensions():
    c = Case(3, [6] * 5, [70, 5, 128, 0, 300], 8, 4, 64, 16, BF)
    a = c.dev()
    r = run(c)
    s = sv().tree_attention(a["q"].view(5, 6, 8, 64), a["k"].view(5, 6, 4, 64), a["v"].view(5, 6, 4, 64), a["k_cache"],
                            a["v_cache"], a["table"], a["lengths"].long(), a["parents"].view(5, 6).long())
    assert torch.equal(r.out, s.out) and torch.equal(r.lse, s.lse)
    c.check(s)


def test_strides():
    """q, k and v inside a fused projection, heads-first caches, table rows
    apart, out with a stride; rows past the last sequence stay."""
    c = Case(4, [6, 2, 7], [70, 5, 333], 8, 2, 64, 16, BF)
    a = c.dev()
    total = a["q"].shape[0]
    fused = torch.randn(total, 12, 72, device=DEV).to(BF)
    for name, lo, hi in (("q", 0, 8), ("k", 8, 10), ("v", 10, 12)):
        fused[:, lo:hi, :64] = a[name]
        a[name] = fused[:, lo:hi, :64]
    for name in ("k_cache", "v_cache"):
        a[name] = a[name].transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.full((3, a["table"].shape[1] + 5), -7, dtype=torch.int32, device=DEV)
    wide[:, :a["table"].shape[1]] = a["table"]
    a["table"] = wide[:, :a["table"].shape[1]]
    buf = torch.full((total + 4, 10, 64), 7.0, dtype=BF, device=DEV)
    r = sv().tree_attention(**a, out=buf[:, 1:9])
    c.check(r)
    assert (buf[total:] == 7).all() and (buf[:, 0] == 7).all() and (buf[:, 9] == 7).all()
    assert r.out.data_ptr() == buf[:, 1:9].data_ptr()
    # rows that start at odd addresses are laid out first
    for name in ("q", "k", "v"):
        x = torch.empty(a[name].numel() + 1, dtype=BF, device=DEV)[1:].view(a[name].shape)
        a[name] = x.copy_(a[name])
    c.check(sv().tree_attention(**a))


def test_rows_past_the_last_sequence():
    c = Case(5, [3, 4], [40, 9], 4, 2, 64, 8, BF)
    a = c.dev()
    pad = lambda t: torch.cat((t, torch.full_like(t[:1], float("nan")).expand(5, *t.shape[1:])))
    a["q"], a["k"], a["v"] = pad(a["q"]), pad(a["k"]), pad(a["v"])
    a["parents"] = torch.cat((a["parents"], torch.full((5,), 99, dtype=torch.int32, device=DEV)))
    out = torch.full_like(a["q"], 3.0)
    r = sv().tree_attention(**a, out=out)
    c.check(r)
    assert (out[7:] == 3).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), 3e38])
@pytest.mark.parametrize("D,Hq", [(128, 8), (80, 6)])
def test_what_a_node_does_not_see(bad, D, Hq):
    """A node's key and value that are no numbers reach it and its descendants
    and nobody else, in its own head."""
    c = Case(6, [40, 9], [150, 3], Hq, 2, D, 16, BF)
    x = torch.tensor(bad).to(BF)
    c.v[5, 0, :3] = x
    c.v[17, 1] = x
    c.k[30, 0] = x if bad == bad else float("nan")
    c.v[44, 1, D - 1] = x
    ref = c.oracle()
    r = run(c)
    c.check(r, ref)
    got = f64(r.out)[:len(ref[0])]
    odd = ~np.isfinite(ref[0]) & (bad != 3e38)
    assert (~np.isfinite(got[odd])).all()
    if bad == bad and abs(bad) > 1e38:
        inf = np.isinf(ref[0])
        assert (got[inf] == ref[0][inf]).all()
    # nodes that see none of them
    assert np.isfinite(got).any()


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), 3e38, 0.0])
def test_unused_places_of_the_cache(junk):
    c = Case(7, [4, 1, 1, 130], [1, 17, 120, 250], 4, 1, 128, 64, BF, junk=junk)
    c.check(run(c))


def test_large_scores():
    """Scores in the hundreds: a few keys take it all; the maximum moves late."""
    for q_scale in (20.0, 60.0):
        c = Case(8, [6, 3], [900, 2000], 4, 2, 64, 16, BF, q_scale=q_scale)
        for b, L in enumerate(c.lengths):  # the largest keys last
            for t in range(L):
                c.kc[c.table[b, t // 16], t % 16] *= (t + 1) / L
        c.check(run(c))


def test_scores_that_pass_the_range():
    """Keys so far along a query that every f32 exponential but one is 0, and equal
    ones."""
    c = Case(9, [2, 2], [300, 40], 2, 1, 64, 8, BF)
    c.q.fill_(1.0)
    c.kc.nan_to_num_(0.0).clamp_(-1, 1)
    c.kc[c.table[0, 3], 5] = 200.0
    c.k.fill_(-100.0)
    c.check(run(c))
    c.q.fill_(0.0)  # all alike
    c.check(run(c))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scale(scale):
    c = Case(10, [5, 4], [100, 300], 4, 2, 64, 16, HF)
    c.check(run(c, scale=scale), c.oracle(scale=scale))


def test_bad_layouts():
    c = Case(11, [4] * 6, [40, 50, 60, 70, 80, 90], 4, 2, 64, 16, BF, width=6)
    a = c.dev()
    lengths, table, parents = c.lengths.copy(), c.table.copy(), c.parents.copy()
    lengths[0], lengths[1] = -1, 97
    table[2, 1], table[3, 4] = -1, c.kc.shape[0]
    parents[18] = 2
    kw = dict(lengths=lengths, table=table, parents=parents)
    ref = c.oracle(**kw)
    assert list(ref[4]) == [64, 64, 64, 64, 64, 0]
    c.check(sv().tree_attention(**{**a, **{k: torch.as_tensor(v).to(DEV) for k, v in kw.items()}}), ref)
    for cu in ([0, 4, 3, 8, 12, 16, 20], [0, 4, 9, 13, 17, 21, 25], [-1, 3, 7, 11, 15, 19, 23], [0, 0, 0, 0, 0, 0, 0]):
        cu = np.array(cu, np.int32)
        out = torch.full_like(a["q"], 5.0)
        r = sv().tree_attention(**{**a, "cu_nodes": torch.as_tensor(cu).to(DEV), "parents": None}, out=out)
        ref = c.oracle(cu=cu, parents=None)
        c.check(r, ref)
        assert (out[torch.as_tensor(np.isnan(ref[1][:, 0])).to(DEV)] == 5).all()


def test_empty_calls():
    c = Case(12, [0, 0, 0], [10, 0, 30], 4, 2, 64, 16, BF)
    r = run(c)
    assert r.out.shape == (0, 4, 64) and not r.status.any()
    a = c.dev()
    a["cu_nodes"], a["table"], a["lengths"] = a["cu_nodes"][:1], a["table"][:0], a["lengths"][:0]
    assert sv().tree_attention(**a).status.shape == (0,)
    c = Case(13, [2, 1], [0, 0], 4, 2, 64, 16, BF)  # no cache at all
    a = c.dev()
    c.table = c.table[:, :0]
    c.check(sv().tree_attention(**{**a, "table": a["table"][:, :0]}))


def test_the_same_call_gives_the_same_bits():
    rng = np.random.default_rng(4)
    c = Case(14, rng.integers(0, 20, 30), rng.integers(0, 3000, 30), 8, 2, 128, 16, BF)
    a, b = run(c), run(c)
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_offsets_past_32_bits():
    """Pools of more than 2^32 bytes (and 2^31 elements); pages near their ends."""
    c = Case(15, [6, 2], [500, 77], 8, 8, 128, 16, BF, tree=False)
    a = c.dev()
    P, big = c.kc.shape[0], 150000
    for name in ("k_cache", "v_cache"):
        x = torch.empty(big, *c.kc.shape[1:], dtype=BF, device=DEV)
        x[big - P:] = a[name]
        a[name] = x
    a["table"] = a["table"].clamp(0, P - 1) + (big - P)
    c.check(sv().tree_attention(**a))


def test_streams_and_graphs():
    """Two captured calls replayed together on two streams, and eager ones among
    them."""
    cs = [Case(16 + i, [5, 9, 1], [700, 90, 2500], 8, 2, 128, 16, BF) for i in range(2)]
    args = [c.dev() for c in cs]
    want = [sv().tree_attention(**a).out.clone() for a in args]
    for c, w, a in zip(cs, want, args):
        c.check(sv().tree_attention(**a))
    graphs, outs = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            outs.append(sv().tree_attention(**a))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, g in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        eager = sv().tree_attention(**args[0]).out
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for o, w in zip(outs, want):
            assert torch.equal(o.out, w)
        assert torch.equal(eager, want[0])


def test_a_graph_follows_its_inputs():
    """Lengths, nodes and pages change between replays: from one long sequence to
    many short ones and back."""
    rng = np.random.default_rng(5)
    B = 12
    shapes = [(rng.integers(0, 20, B), rng.integers(0, 3000, B)) for _ in range(4)]
    shapes[1][0][:] = 0
    shapes[1][0][7] = 20
    total, width, P = 20 * B, 200, 12 * 200
    g = torch.Generator().manual_seed(3)
    a = dict(q=torch.randn(total, 8, 64, generator=g), k=torch.randn(total, 2, 64, generator=g), v=torch.randn(total, 2, 64, generator=g),
             k_cache=torch.randn(P, 16, 2, 64, generator=g), v_cache=torch.randn(P, 16, 2, 64, generator=g))
    a = {k: v.to(HF).to(DEV) for k, v in a.items()}
    i32 = lambda x: torch.as_tensor(np.asarray(x, np.int32)).to(DEV)
    a.update(table=i32(rng.permutation(P).reshape(B, width)), lengths=i32(np.zeros(B)), cu_nodes=i32(np.zeros(B + 1)), n=20,
             parents=i32(np.zeros(total)))

    def fill(N, lengths):
        a["lengths"].copy_(i32(lengths))
        a["cu_nodes"].copy_(i32(np.concatenate(([0], np.cumsum(N)))))
        up = [int(rng.integers(-1, i)) for n in N for i in range(n)]
        a["parents"].copy_(i32(up + [0] * (total - len(up))))

    fill(*shapes[0])
    out = torch.zeros_like(a["q"])
    sv().tree_attention(**a, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        r = sv().tree_attention(**a, out=out)
    for N, lengths in shapes + shapes[:1]:
        fill(N, lengths)
        graph.replay()
        again = sv().tree_attention(**a)
        rows = int(sum(N))
        assert torch.equal(r.out[:rows], again.out[:rows]) and not r.status.any()
        ref = oracle.tree_attention(*(f64(a[k]) for k in ("q", "k", "v", "k_cache", "v_cache")), a["table"].cpu().numpy(), lengths,
                                    a["parents"].cpu().numpy(), a["cu_nodes"].cpu().numpy(), 20, 0.125)
        Case.check(SimpleNamespace(lengths=np.array(lengths), n=20, dtype=HF, D=64, scale=0.125, v=a["v"].cpu(), vc=a["v_cache"].cpu()),
                   SimpleNamespace(out=r.out, lse=r.lse, status=r.status), ref)


def test_refusals():
    m = sv()
    c = Case(17, [2, 2], [10, 20], 4, 2, 64, 16, BF)
    a = c.dev()
    call = lambda **kw: m.tree_attention(**{**a, **kw})
    for kw, what in ((dict(q=a["q"].float()), "bfloat16"), (dict(k=a["k"].half()), "type"), (dict(v_cache=a["v_cache"].cpu()), "device"),
                     (dict(q=a["q"][:3]), "total"), (dict(k_cache=a["k_cache"][:, :, :1]), "caches"),
                     (dict(table=a["table"].long()), "table"), (dict(lengths=a["lengths"][:1]), "lengths"),
                     (dict(n=None), "n "), (dict(cu_nodes=a["cu_nodes"][:2]), "cu_nodes"), (dict(parents=a["parents"][:3]), "parents"),
                     (dict(out=torch.empty(3, 4, 64, dtype=BF, device=DEV)), "out"),
                     (dict(out=a["q"]), "input"),
                     (dict(q=a["q"].clone().requires_grad_()), "backward")):
        with pytest.raises(ValueError, match=what):
            call(**kw)
    for kw, what in ((dict(q=a["q"][:, :3], out=None), "multiple"), (dict(n=300), "256")):
        with pytest.raises(m.SVError, match=what):
            call(**kw)
    x = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)
    with pytest.raises(m.SVError, match="dim"):
        m.tree_attention(x(1, 1, 136), x(1, 1, 136), x(1, 1, 136), x(2, 8, 1, 136), x(2, 8, 1, 136),
                         torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, device=DEV, dtype=torch.int32))
    with pytest.raises(m.SVError, match="page_size"):
        m.tree_attention(x(1, 1, 64), x(1, 1, 64), x(1, 1, 64), x(2, 4, 1, 64), x(2, 4, 1, 64),
                         torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, device=DEV, dtype=torch.int32))
