"""Paged caches on the GPU, equal to the oracle byte for byte: pools, page
tables, lengths and counts."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytestmark = pytest.mark.skip("needs a GPU")
else:
    pytestmark = pytest.mark.gpu

import __graft_entry__  # noqa: E402
from oracle import cache as oc  # noqa: E402

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def sv():
    import speculative_decoding_verification_decode_gb300 as m
    return m


class Pair:
    """A cache on the GPU and the oracle's copy of it."""

    def __init__(self, seed, layers, P, page, H, D, S, width, dtype=torch.float32, heads_first=False, lengths=None, share=0.0):
        self.rng = rng = np.random.default_rng(seed)
        self.page, self.n_seq, self.layers, self.D, self.H, self.dtype = page, S if isinstance(S, int) else S[0] * S[1], layers, D, H, dtype
        c = sv().paged_cache(layers, P, page, H, D, S, width, dtype, DEV)
        if heads_first:  # pools stored [P, H, page, D]
            c = c._replace(keys=[torch.empty(P, H, page, D, dtype=dtype, device=DEV).transpose(1, 2) for _ in range(layers)],
                           values=[torch.empty(P, H, page, D, dtype=dtype, device=DEV).transpose(1, 2) for _ in range(layers)])
        for t in (*c.keys, *c.values):
            t.copy_(torch.as_tensor(rng.integers(-60, 60, t.shape)))
        self.c = c
        self.table = rng.integers(0, P, (self.n_seq, width)).astype(np.int32)  # entries past the length mean nothing
        self.lengths, self.refs = np.zeros(self.n_seq, np.int32), np.zeros(P, np.int32)
        self.pools = [t.float().cpu().numpy() for t in (*c.keys, *c.values)]
        if lengths is not None:
            at = list(rng.permutation(P))
            for b, L in enumerate(lengths):
                k = -(-L // page)
                if b and rng.random() < share:
                    self.table[b], self.lengths[b] = self.table[b - 1], self.lengths[b - 1]
                    k = -(-self.lengths[b] // page)
                else:
                    self.table[b, :k], self.lengths[b] = [at.pop() for _ in range(k)], L
                for p in self.table[b, :k]:
                    self.refs[p] += 1
        self.push()

    def push(self):
        self.c.table.copy_(torch.as_tensor(self.table).view(self.c.table.shape))
        self.c.lengths.copy_(torch.as_tensor(self.lengths).view(self.c.lengths.shape))
        self.c.refs.copy_(torch.as_tensor(self.refs))

    def rows(self, total):
        new = [self.rng.integers(-60, 60, (total, self.H, self.D)).astype(np.float32) for _ in self.pools]
        t = [torch.as_tensor(x).to(self.dtype).to(DEV) for x in new]
        return new, t[:self.layers], t[self.layers:]

    def append(self, n, counts=None, path=None, cu=None, total=None, wrap=lambda x: x):
        new, keys, values = self.rows(self.n_seq * n if cu is None else total)
        d = lambda a: None if a is None else torch.as_tensor(np.asarray(a, np.int32), device=DEV)
        st = sv().cache_append(self.c, wrap(keys), wrap(values), d(counts), d(path), d(cu), n)
        ref = oc.append(self.table, self.lengths, self.refs, self.pools, new, counts, path, cu, n)
        return self.same(st, ref)

    def fork(self, parents):
        st = sv().cache_fork(self.c, torch.as_tensor(parents.astype(np.int32), device=DEV))
        return self.same(st, oc.fork(self.table, self.lengths, self.refs, self.page, parents))

    def truncate(self, to):
        st = sv().cache_truncate(self.c, torch.as_tensor(np.asarray(to, np.int32), device=DEV))
        return self.same(st, oc.truncate(self.table, self.lengths, self.refs, self.page, to))

    def same(self, st, ref):
        assert np.array_equal(st.cpu().numpy().reshape(-1), ref), (st.cpu().numpy().reshape(-1)[:20], ref[:20])
        assert np.array_equal(self.c.lengths.cpu().numpy().reshape(-1), self.lengths)
        assert np.array_equal(self.c.refs.cpu().numpy(), self.refs)
        assert np.array_equal(self.c.table.cpu().numpy().reshape(self.table.shape), self.table)
        for t, p in zip((*self.c.keys, *self.c.values), self.pools):
            assert np.array_equal(t.float().cpu().numpy(), p)
        return ref


@pytest.mark.parametrize("dtype,D,heads_first", [(torch.float32, 8, False), (torch.bfloat16, 64, False), (torch.float16, 20, True),
                                                 (torch.uint8, 7, False), (torch.bfloat16, 3, True), (torch.int8, 16, False)])
@pytest.mark.parametrize("page", [1, 4, 7, 16])
def test_random_use(dtype, D, heads_first, page):
    """Appends, forks and truncations in turn, through a pool that is at times
    too small."""
    x = Pair(page, 2, 30, page, 2, D, (3, 4), 9, torch.int8 if dtype == torch.uint8 else dtype, heads_first)
    rng, refused = x.rng, 0
    for step in range(40):
        kind = rng.integers(0, 4)
        if kind <= 1:
            n = int(rng.integers(1, 2 * page + 3))
            counts = rng.integers(0, n + 1, 12)
            path = np.stack([rng.permutation(n) for _ in range(12)])
            refused += int((x.append(n, counts, path if step % 2 else None) > 0).sum())
        elif kind == 2:
            x.fork(rng.integers(-1, 4, (3, 4)))
        else:
            x.truncate(np.array([rng.integers(0, L + 1) if rng.random() < 0.5 else L for L in x.lengths]))
        assert np.array_equal(x.refs, oc.refs_of(x.table, x.lengths, page, 30))
    assert refused


@pytest.mark.parametrize("S", [1, 31, 257, 1500, 2100])
def test_many_sequences(S):
    """More sequences than the deciding CTA has threads; shared last pages all
    over."""
    rng = np.random.default_rng(S)
    x = Pair(S, 1, 4 * S + 10, 8, 1, 4, S, 4, torch.bfloat16, lengths=rng.integers(0, 20, S), share=0.5)
    x.append(5, rng.integers(0, 6, S))
    x.append(3)
    x.truncate(np.maximum(0, x.lengths - rng.integers(0, 9, S)))
    x.append(2, rng.integers(0, 3, S))


def test_one_page_shared_by_all():
    """The first of the sequences that append copy, the last keeps the page;
    where one does not append, all copy."""
    for idle in (None, 3):
        x = Pair(9, 1, 40, 8, 2, 8, 12, 3, lengths=[13] * 12, share=1.0)
        shared = x.table[0, 1]
        counts = np.ones(12, int)
        if idle is not None:
            counts[idle] = 0
        x.append(1, counts)
        assert x.refs[shared] == 1
        assert (x.table[:, 1] == shared).sum() == 1 and (x.table[-1, 1] == shared) == (idle is None)


def test_too_few_pages():
    """Sequences in order take what there is; one that needs more than is left is
    refused and a later, smaller one served; a refused one keeps sharing."""
    x = Pair(2, 2, 14, 4, 1, 8, 5, 8, lengths=[6, 6, 3, 1, 0], share=0.0)
    x.table[1], x.refs[:] = x.table[0], 0
    x.lengths[1] = 6
    x.refs[:] = oc.refs_of(x.table, x.lengths, 4, 14)
    used = [p for p in range(14) if x.refs[p]]
    for p in range(14):  # only three pages are free
        if p not in used and sum(x.refs == 0) > 3:
            x.refs[p] = 1
    x.push()
    st = x.append(20, np.array([20, 1, 1, 9, 4]))
    assert list(st) == [oc.NO_PAGES, 0, 0, 0, oc.NO_PAGES]
    st = x.append(4, np.array([0, 0, 0, 0, 4]))
    st = x.append(33, np.array([0, 33, 0, 0, 0]))  # the table row is full first
    assert st[1] == oc.NO_PAGES


def test_a_prompt():
    """Thousands of tokens of one sequence, ragged with short ones."""
    x = Pair(5, 3, 700, 16, 2, 16, 3, 400, torch.float16, lengths=[0, 5, 333])
    x.append(5003, None, None, np.array([0, 5003, 5003, 5020]), total=5020)
    x.append(5003, np.array([1, 0, 17]), None, np.array([0, 3, 3, 20]), total=20)


def test_rows_of_any_layout():
    """Rows inside larger ones (a fused projection's), four dimensions, and
    arrays that differ in their strides."""
    x = Pair(6, 2, 40, 8, 2, 8, 4, 5, torch.bfloat16, lengths=[3, 9, 0, 16])

    def inside(ts):
        out = []
        for t in ts:
            big = torch.zeros(t.shape[0], 6, 8, dtype=t.dtype, device=DEV)
            big[:, 2:4] = t
            out.append(big[:, 2:4])
        return out

    def mixed(ts):
        out = inside(ts)
        out[-1] = ts[-1].transpose(1, 2).contiguous().transpose(1, 2)
        return out

    for wrap in (inside, mixed, lambda ts: [t.view(4, 3, 2, 8) for t in ts], lambda ts: mixed(ts)[::1]):
        x.append(3, np.array([1, 3, 0, 2]), np.array([[2, 0, 1]] * 4), wrap=wrap)
        x.truncate(x.lengths - np.array([1, 3, 0, 2]))
    x.append(3, np.array([1, 0, 0, 2]), None, np.array([0, 1, 1, 1, 4]), total=4)


def test_many_layers():
    x = Pair(7, 70, 20, 8, 1, 8, 2, 5, lengths=[3, 9], share=0.0)
    x.append(9, np.array([9, 2]))


def test_bad_input_changes_nothing():
    x = Pair(8, 1, 30, 4, 1, 4, 8, 4, lengths=[5, 6, 7, 0, 3, 16, 2, 9])
    x.lengths[3], x.lengths[4] = -1, 17
    x.table[0, 1], x.table[6, 0] = -1, 30
    x.push()
    st = x.append(3, np.array([1, 4, -1, 1, 1, 1, 1, 3]))
    assert list(st) == [64, 64, 64, 64, 64, 128, 64, 0]
    path = np.array([[0, 1, 2]] * 8)
    path[1, 1], path[2, 0], path[5, 2], path[7, 2] = 3, -1, 9, 77
    x.append(3, np.array([0, 2, 2, 0, 0, 0, 0, 2]), path)
    for cu in ([0, 3, 2, 5, 5, 5, 5, 5, 5], [-2, 1, 2, 2, 2, 2, 2, 2, 2], [0, 4, 4, 4, 4, 4, 4, 4, 9]):
        x.append(3, None, None, np.array(cu), total=8)
    x.truncate(np.array([5, -1, 9, 0, 0, 4, 2, 0]))
    x.truncate(np.array([0, 0, 0, 0, 0, 0, 0, 0]))
    y = Pair(8, 1, 30, 4, 1, 4, (4, 2), 4, lengths=[5, 6, 7, 0, 3, 16, 2, 9])
    y.lengths[1], y.table[4, 0] = 17, 30
    y.push()
    st = y.fork(np.array([[1, -1], [2, 0], [-1, 0], [-5, 0]]))
    assert list(st) == [64, 64, 64, 0]


@pytest.mark.parametrize("groups,W,width", [(1, 1, 5), (3, 64, 700), (40, 3, 33), (1, 1000, 40), (2, 1024, 9), (1, 7, 9000)])
def test_forks(groups, W, width):
    rng = np.random.default_rng(W)
    page = 4
    most = width * page
    P = min(60000, groups * W * width + 1)
    lengths = rng.integers(0, max(1, min(most, P // (groups * W) * page)) + 1, groups * W)
    x = Pair(W, 1, P, page, 1, 1, (groups, W), width, torch.int8, lengths=lengths, share=0.3)
    for _ in range(3):
        x.fork(rng.integers(-1, W, (groups, W)))
    x.fork(np.zeros((groups, W), int))
    assert np.array_equal(x.refs, oc.refs_of(x.table, x.lengths, page, P))


def test_one_group_of_all_and_permutations():
    x = Pair(3, 1, 50, 4, 1, 4, 6, 5, lengths=[5, 0, 20, 7, 4, 13])
    st = sv().cache_fork(x.c, torch.tensor([1, 2, 3, 4, 5, 0], dtype=torch.int64, device=DEV))
    x.same(st, oc.fork(x.table, x.lengths, x.refs, 4, np.array([[1, 2, 3, 4, 5, 0]])))


def test_captured_calls_and_another_stream():
    """A round (append, truncate, fork) in a graph, replayed, equal to the same
    rounds one after another."""
    x = Pair(4, 2, 60, 4, 2, 8, (2, 3), 8, torch.bfloat16, lengths=[5, 9, 3, 0, 8, 2])
    new, keys, values = x.rows(6 * 3)
    counts = torch.tensor([1, 3, 2, 0, 3, 1], dtype=torch.int32, device=DEV)
    parents = torch.tensor([[1, 1, 2], [0, 2, 0]], dtype=torch.int32, device=DEV)
    back = torch.tensor([[4, 6, 5], [0, 2, 0]], dtype=torch.int32, device=DEV)
    kept = [t.clone() for t in (*x.c.keys, *x.c.values, x.c.table, x.c.lengths, x.c.refs)]

    def round_():
        sv().cache_fork(x.c, parents)
        return sv().cache_append(x.c, keys, values, counts, n=3), sv().cache_truncate(x.c, torch.minimum(back, x.c.lengths))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        round_()
    s.synchronize()
    for t, k in zip((*x.c.keys, *x.c.values, x.c.table, x.c.lengths, x.c.refs), kept):
        t.copy_(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        out = round_()
    for _ in range(4):
        g.replay()
        oc.fork(x.table, x.lengths, x.refs, 4, parents.cpu().numpy())
        ref = oc.append(x.table, x.lengths, x.refs, x.pools, new, counts.cpu().numpy(), None, None, 3)
        x_to = np.minimum(back.cpu().numpy().reshape(-1), x.lengths)
        st = oc.truncate(x.table, x.lengths, x.refs, 4, x_to)
        assert np.array_equal(out[0].cpu().numpy().reshape(-1), ref)
        x.same(out[1], st)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes; pages near its end."""
    P, page, H, D = 150000, 16, 8, 128
    c = sv().paged_cache(1, P, page, H, D, 2, 4, torch.bfloat16, DEV)
    c.refs.fill_(1)
    c.refs[P - 3:] = 0
    new = torch.randn(2, 20, H, D, device=DEV, dtype=torch.bfloat16)
    st = sv().cache_append(c, new, new + 1, torch.tensor([20, 3], device=DEV))
    assert not st.any() and c.table[0, :2].tolist() == [P - 3, P - 2] and int(c.table[1, 0]) == P - 1
    assert torch.equal(c.keys[0][P - 3], new[0, :16]) and torch.equal(c.values[0][P - 2, :4], new[0, 16:] + 1)
    assert torch.equal(c.keys[0][P - 1, :3], new[1, :3])


def test_refusals():
    m = sv()
    c = m.paged_cache(2, 5, 8, 1, 8, 3, 4, device=DEV)
    r = torch.zeros(3, 1, 8, dtype=torch.bfloat16, device=DEV)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    for call, what in ((lambda: m.cache_append(c, [r], [r, r]), "layers"),
                       (lambda: m.cache_append(c, [r, r], [r, r.float()]), "pools' type"),
                       (lambda: m.cache_append(c, [r, r[:2]], [r, r]), "new rows"),
                       (lambda: m.cache_append(c, [r, r], [r, r], counts=i(2)), "counts"),
                       (lambda: m.cache_append(c, [r, r], [r, r], path=i(3, 2)), "n rows"),
                       (lambda: m.cache_append(c, [r, r], [r, r], counts=torch.zeros(3, device=DEV)), "whole"),
                       (lambda: m.cache_append(c._replace(values=[c.keys[0], c.values[1]]), [r, r], [r, r]), "twice"),
                       (lambda: m.cache_append(c._replace(refs=i(6)), [r, r], [r, r]), "refs"),
                       (lambda: m.cache_append(c._replace(lengths=i(4)), [r, r], [r, r]), "lengths"),
                       (lambda: m.cache_append(c._replace(table=c.table.long()), [r, r], [r, r]), "int32"),
                       (lambda: m.cache_append(c._replace(keys=[c.keys[0], c.keys[1][:, :, :, ::2]]), [r, r], [r, r]), "alike"),
                       (lambda: m.cache_truncate(c, i(2)), "lengths"),
                       (lambda: m.cache_fork(c, i(2, 2)), "parents"),
                       (lambda: m.cache_fork(c, c.lengths), "parents")):
        with pytest.raises(ValueError, match=what):
            call()
