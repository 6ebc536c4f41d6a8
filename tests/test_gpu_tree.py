"""Verification of drafted trees on the GPU, equal to the oracle."""

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


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


def dev(a):
    return None if a is None else torch.as_tensor(np.asarray(a), device=DEV)


def make(seed, N, V, dtype, pad=0, follow=0.8, chain=False, offset=0):
    """Trees of N[b] nodes whose rows choose a child's token with probability
    ``follow``; returns (target view, tokens, parents, cu)."""
    rng = np.random.default_rng(seed)
    total = int(sum(N))
    cu = np.concatenate(([0], np.cumsum(N))).astype(np.int32)
    parents, tokens, choice = [], rng.integers(0, V, total), []
    for b, n in enumerate(N):
        up = [i - 1 if chain else int(rng.integers(0, max(i, 1))) for i in range(n)] if n else []
        if n:
            up[0] = -1
        for i in range(n):
            kids = [j for j in range(n) if up[j] == i]
            choice.append(tokens[cu[b] + rng.choice(kids)] if kids and rng.random() < follow else rng.integers(0, V))
        parents += up
    g = torch.Generator().manual_seed(seed)
    flat = torch.full((offset + total * (V + pad),), 6e4, dtype=DT[dtype])  # between the rows: never read
    x = flat[offset:].view(total, V + pad)[:, :V] if total else flat[:0].view(0, V)
    x.copy_(torch.randn(total, V, generator=g))
    if total:
        x.scatter_(1, torch.as_tensor(np.array(choice))[:, None].long(), 9.0)
    y = flat.to(DEV)
    y = y[offset:].view(total, V + pad)[:, :V] if total else y[:0].view(0, V)
    return y, tokens.astype(np.int32), np.array(parents, np.int32), cu


def same(r, ref):
    for got, want in zip(r, ref):
        assert np.array_equal(got.cpu().numpy(), want), (got.cpu().numpy()[:20], want[:20])


def check(x, tokens, parents, cu, n):
    B = len(cu) - 1
    r = sv().verify_tree_greedy(x, dev(tokens), dev(parents), dev(cu), n)
    ref = oracle.verify_tree_greedy(x.double().cpu().numpy(), tokens, parents, cu, B, n)
    same(r, ref)
    return ref


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,pad,offset", [(1, 0, 0), (2, 1, 0), (7, 0, 1), (127, 0, 0), (1000, 24, 0), (4099, 5, 3),
                                          (32000, 0, 0), (129281, 3, 1)])
def test_ragged_trees(dtype, V, pad, offset):
    N = [5, 0, 1, 13, 31, 2] if V > 20000 else [5, 0, 1, 40, 256, 2, 0, 64, 65, 17]
    ref = check(*make(V, N, V, dtype, pad, offset=offset), n=max(N))
    assert ref[0].max() > 1 or V < 3


@pytest.mark.parametrize("B,n,V", [(1, 1, 5000), (1, 16, 32000), (3, 256, 501), (200, 7, 1003), (64, 33, 4000)])
def test_equal_trees_and_layouts(B, n, V):
    x, tokens, parents, cu = make(B, [n] * B, V, "bf16")
    ref = oracle.verify_tree_greedy(x.double().cpu().numpy(), tokens, parents, None, B, n)
    t, p = dev(tokens), dev(parents)
    same(sv().verify_tree_greedy(x.view(B, n, V), t.view(B, n), p.view(B, n)), ref)
    same(sv().verify_tree_greedy(x, t, p, n=n), ref)
    same(sv().verify_tree_greedy(x, t.long(), p.long(), n=n), ref)
    same([v.to(DEV) for v in sv().verify_tree_greedy(x.cpu(), t.cpu(), p.cpu(), n=n)], ref)


def test_a_chain_needs_no_parents():
    x, tokens, parents, cu = make(3, [6] * 9, 777, "f16", chain=True)
    ref = oracle.verify_tree_greedy(x.double().cpu().numpy(), tokens, None, None, 9, 6)
    assert ref[0].max() > 2
    same(sv().verify_tree_greedy(x, dev(tokens), n=6), ref)
    r = sv().verify_greedy(x, dev(tokens.reshape(9, 6)[:, 1:].copy()))
    assert np.array_equal(r.n_accepted.cpu().numpy(), ref[0]) and np.array_equal(r.next_token.cpu().numpy(), ref[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_ties_zeros_and_values_that_are_no_numbers(dtype):
    V, n = 3001, 9
    x, tokens, parents, cu = make(5, [n] * 12, V, dtype, follow=1.0)
    ref = oracle.verify_tree_greedy(x.double().cpu().numpy(), tokens, parents, cu, 12, n)
    ways = ref[2]
    first = lambda b, j=0: cu[b] + ways[b][j]
    x[first(0)] = 1.0  # a row of ties
    x[first(1)] = 0.0
    x[first(1), ::2] = -0.0  # -0 and 0 tie
    x[first(2)] = float("-inf")
    x[first(3)] = float("nan")
    x[first(4), 5] = float("nan")
    x[first(5), V - 1] = float("inf")
    x[first(6), 17] = float("inf")
    x[first(6), 16] = float("nan")
    x[first(7)] = torch.finfo(DT[dtype]).min
    x[first(8), :] = float("-inf")
    x[first(8), 2999] = torch.finfo(DT[dtype]).min
    x[first(8), 3000] = float("nan")
    off = [i for i in range(n) if i not in ways[9]]
    if off:
        x[cu[9] + off[0]] = float("nan")  # off the path: not looked at
    ref = check(x, tokens, parents, cu, n)
    assert list(ref[3][:10]) == [0, 0, 0, 2, 2, 0, 2, 0, 2, 0]


def test_tokens_out_of_range_and_siblings_alike():
    V, n = 500, 6
    parents = np.array([-1, 0, 0, 0, 2, 2] * 4 + [-1, -1, 0, 0, 2, -1], np.int32)
    tokens = np.array([0, 7, 9, 9, 4, 4, 0, -1, V, 9, 1, 2, 10**6, 9, 8, 9, -5, 4, 3, 9, 9, 9, V + 7, -9, 0, 9, 9, 8, 4, 4],
                      np.int32)
    x = torch.zeros(30, V, device=DEV)
    x[:, 9] = 1
    x[2::6, 4] = 2
    ref = check(x, tokens, parents, np.arange(0, 31, 6, dtype=np.int32), n)
    assert list(ref[2][0][:3]) == [0, 2, 4] and list(ref[3]) == [0, 1, 0, 0, 0]


def test_bad_offsets_and_parents():
    V, n = 300, 4
    x, tokens, parents, _ = make(8, [4] * 6, V, "bf16")
    for cu in ([0, 4, 3, 8, 12, 24, 20], [0, 4, 9, 13, 17, 21, 25], [-1, 3, 7, 11, 15, 19, 23], [0] * 7, [24] * 7):
        check(x, tokens, parents, np.array(cu, np.int32), n)
    p = parents.copy()
    p[5], p[9], p[14], p[19] = 1, 3, -2, 100
    ref = check(x, tokens, p, np.arange(0, 25, 4, dtype=np.int32), n)
    assert list(ref[3]) == [0, 64, 64, 64, 64, 0]


def test_empty_calls():
    z = torch.zeros(0, 100, device=DEV)
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    r = sv().verify_tree_greedy(z, e, e, torch.zeros(1, dtype=torch.int32, device=DEV), 5)
    assert r.path.shape == (0, 5)
    r = sv().verify_tree_greedy(z, e, e, torch.zeros(4, dtype=torch.int32, device=DEV), 5)
    assert r.next_token.tolist() == [-1] * 3 and r.path.tolist() == [[-1] * 5] * 3
    r = sv().verify_tree(e, e, e, torch.zeros(4, dtype=torch.int32, device=DEV), 0)
    assert r.next_token.tolist() == [-1] * 3 and r.path.shape == (3, 0)


@pytest.mark.parametrize("chain", [False, True])
def test_choices(chain):
    rng = np.random.default_rng(4)
    N = [5, 0, 1, 40, 256, 2, 0, 64]
    x, tokens, parents, cu = make(11, N, 50, "f32", chain=chain)
    choices = x.argmax(1).int().cpu().numpy()
    choices[rng.random(len(choices)) < 0.05] = -1
    r = sv().verify_tree(dev(choices), dev(tokens), None if chain else dev(parents), dev(cu), 256)
    same(r, oracle.verify_tree(choices, tokens, None if chain else parents, cu, len(N), 256))


def test_sampled_choices_follow_the_target():
    """Choices drawn by the verification's own inverse CDF on the nodes' rows:
    the first emitted token has the target's law whatever the tree holds."""
    V, B = 6, 40000
    rng = np.random.default_rng(5)
    p = torch.tensor([0.3, 0.05, 0.25, 0.2, 0.15, 0.05])
    x = p.log().to(DEV).expand(B * 3, V).contiguous()
    tokens = torch.tensor([[0, 2, 4]] * B, dtype=torch.int32, device=DEV)
    parents = torch.tensor([[-1, 0, 0]] * B, dtype=torch.int32, device=DEV)
    u = torch.as_tensor(rng.random(B * 3, np.float32), device=DEV)
    draw = sv().accept_from_logits(x, x[:0], torch.ones(B * 3, device=DEV), tokens[:0].reshape(-1), u)
    r = sv().verify_tree(draw.next_token, tokens, parents)
    kid = r.path.gather(1, r.n_accepted.long()[:, None])[:, 0]
    first = torch.where(r.n_accepted > 0, tokens.gather(1, kid.long()[:, None])[:, 0], r.next_token)
    seen = torch.bincount(first.cpu().long(), minlength=V).double() / B
    assert (seen - p).abs().max() < 5 * (0.25 / B) ** 0.5  # five standard deviations


def test_another_stream_and_a_captured_call():
    x, tokens, parents, cu = make(6, [17] * 20, 5003, "bf16")
    t, p = dev(tokens), dev(parents)
    ref = oracle.verify_tree_greedy(x.double().cpu().numpy(), tokens, parents, None, 20, 17)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = sv().verify_tree_greedy(x, t, p, n=17)
    s.synchronize()
    same(r, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        r = sv().verify_tree_greedy(x, t, p, n=17)
    x2, tokens2, parents2, _ = make(7, [17] * 20, 5003, "bf16")
    x.copy_(x2), t.copy_(dev(tokens2)), p.copy_(dev(parents2))
    g.replay()
    g.replay()
    same(r, oracle.verify_tree_greedy(x2.double().cpu().numpy(), tokens2, parents2, None, 20, 17))


def test_refusals():
    f = lambda *s: torch.zeros(*s, device=DEV)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    m = sv()
    for call, what in ((lambda: m.verify_tree_greedy(f(4, 9), i(5), i(5), n=5), "one row"),
                       (lambda: m.verify_tree_greedy(f(4, 9), i(4), i(3), n=4), "parents"),
                       (lambda: m.verify_tree_greedy(f(4, 9), i(4), i(4)), "n "),
                       (lambda: m.verify_tree_greedy(f(4, 9), i(4), i(4), i(3)), "n "),
                       (lambda: m.verify_tree_greedy(f(4, 9), i(4), i(4), n=3), "n rows"),
                       (lambda: m.verify_tree_greedy(f(4, 9).double(), i(4), i(4), n=4), "float"),
                       (lambda: m.verify_tree_greedy(f(4, 9), f(4), i(4), n=4), "whole"),
                       (lambda: m.verify_tree(i(3), i(4), i(4), n=4), "choices")):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(m.SVError, match="256"):
        m.verify_tree_greedy(f(257, 9), i(257), i(257), n=257)
