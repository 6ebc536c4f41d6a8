"""Rounds and prefills whose attention has no result: the sequence stops, its
status says why, and its tokens, length and pages stay as they are."""

import functools

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytestmark = pytest.mark.skip("needs a GPU")
else:
    pytestmark = pytest.mark.gpu

import __graft_entry__  # noqa: E402
from test_gpu_tree_decoder import Model, check_greedy, decoder, sv  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def state(d, b):
    return [t.clone() for t in (d.tokens[b], d.lengths[b], d.cache.lengths[b], d.cache.table[b], d.cache.refs)]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("sampled", [False, True])
def test_a_page_that_does_not_exist(graph, sampled):
    model, prompts = Model(6), (40, 1, 7, 130, 17)
    d = decoder(model, temperature=torch.full((5,), 0.5) if sampled else None)
    d.prefill(chunk=48)
    page = int(d.cache.table[3, 2])
    d.cache.table[3, 2] = -1  # in the middle of sequence 3
    before = state(d, 3)
    held = int((d.cache.table[3, :9] >= 0).sum())
    d.run(5, graph)
    assert d.status.tolist() == [0, 0, 0, sv().SEQ_BAD_LAYOUT, 0]
    after = state(d, 3)
    assert all(torch.equal(x, y) for x, y in zip(before[:4], after[:4])) and d.cache.refs[page] == 1 and held == 8
    assert all(int(d.lengths[b]) >= prompts[b] + 5 for b in (0, 1, 2, 4))
    d.cache.table[3, 2] = page
    if not sampled:
        check_greedy(model, d, prompts)


def test_a_prefill_over_a_page_that_does_not_exist():
    model = Model(7)
    d = decoder(model)
    d.prefill(chunk=48)
    assert d.cache.lengths[3] == 129
    d.tokens[3, 130:200] = 5
    d.lengths[3] = 200  # a longer prompt
    d.cache.table[3, 1] = d.cache.refs.numel()
    before = state(d, 3)
    d.prefill(chunk=48)
    assert d.status.tolist() == [0, 0, 0, sv().SEQ_BAD_LAYOUT, 0]
    assert all(torch.equal(x, y) for x, y in zip(before, state(d, 3)))


def test_a_wait_that_gave_up(monkeypatch):
    from speculative_decoding_verification_decode_gb300 import api
    d = decoder(Model(8))
    d.prefill()
    before = [state(d, b) for b in range(5)]
    with monkeypatch.context() as m:
        m.setattr(api, "tree_attention", functools.partial(api.tree_attention, flags=sv().FLAG_EXPIRE_EXCHANGE))
        d.round()
    assert (d.status == sv().SEQ_TIMEOUT).all()
    d.round()
    for b in range(5):
        assert all(torch.equal(x, y) for x, y in zip(before[b], state(d, b)))
    # in a prefill
    d = decoder(Model(8))
    with monkeypatch.context() as m:
        m.setattr(api, "tree_attention", functools.partial(api.tree_attention, flags=sv().FLAG_EXPIRE_EXCHANGE))
        d.prefill(chunk=50)
    assert (d.status == sv().SEQ_TIMEOUT).all() and not d.cache.lengths.any() and not d.cache.refs.any()


@pytest.mark.parametrize("sampled", [False, True])
def test_positions_are_below_max_len(sampled):
    model, prompts, max_len = Model(9), (5, 60, 66), 70
    d = decoder(model, 3, prompts, max_len=max_len, temperature=torch.full((3,), 0.5) if sampled else None)
    seen, target = [], d.target_fn
    d.target_fn = lambda nodes, positions, attend: seen.append((int(positions.min()), int(positions.max()))) or target(nodes, positions, attend)
    d.prefill()
    assert d.cache.lengths.tolist() == [p - 1 for p in prompts]
    d.run(66, graph=False)
    assert (d.lengths > max_len - d.n).all() and not d.status.any()
    assert all(0 <= lo and hi < max_len for lo, hi in seen)
    if not sampled:
        check_greedy(model, d, prompts)
