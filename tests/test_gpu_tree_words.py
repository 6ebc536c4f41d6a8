"""Tokens, parents, offsets and lengths in 64 bits that do not fit 32: never
followed, and their sequence's layout is bad."""

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


def i64(*x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def test_verification():
    V, rows = 50, torch.zeros(3, 50, device=DEV)
    rows[0, 5] = rows[1, 7] = rows[2, 9] = 1.0
    r = sv().verify_tree_greedy(rows, i64(0, 5, 7), n=3, cu_nodes=i64(0, 3))
    assert r.n_accepted.tolist() == [2] and r.next_token.tolist() == [9] and r.status.tolist() == [0]
    r = sv().verify_tree_greedy(rows, i64(0, 2**32 + 5, 7), n=3, cu_nodes=i64(0, 3))
    assert r.n_accepted.tolist() == [0] and r.next_token.tolist() == [5] and r.status.tolist() == [sv().SEQ_BAD_TOKEN]
    r = sv().verify_tree_greedy(rows, i64(0, 5, 7), i64(-1, 2**32, 1), n=3, cu_nodes=i64(0, 3))
    assert r.next_token.tolist() == [-1] and r.status.tolist() == [sv().SEQ_BAD_LAYOUT]
    r = sv().verify_tree_greedy(rows, i64(0, 5, 7), n=3, cu_nodes=i64(0, 2**32 + 3))
    assert r.next_token.tolist() == [-1] and r.status.tolist() == [sv().SEQ_BAD_LAYOUT]
    r = sv().verify_tree(i64(2**32 + 5, 7, 9), i64(0, 5, 7), n=3, cu_nodes=i64(0, 3))
    assert r.n_accepted.tolist() == [0]


def test_attention_and_pages():
    x = lambda *s: torch.randn(*s, device=DEV).to(torch.bfloat16)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    r = sv().tree_attention(x(2, 2, 64), x(2, 1, 64), x(2, 1, 64), x(8, 8, 1, 64), x(8, 8, 1, 64), table, i64(2**32 + 3, 3), n=1)
    assert r.status.tolist() == [sv().SEQ_BAD_LAYOUT, 0] and not r.out[0].any() and r.out[1].any()
    c = sv().paged_cache(1, 8, 8, 1, 64, 2, 4, device=DEV)
    rows = x(6, 1, 64)
    status = sv().cache_append(c, rows, rows, counts=i64(2**32 + 2, 2), n=3)
    assert status.tolist() == [sv().SEQ_BAD_LAYOUT, 0] and c.lengths.tolist() == [0, 2]
    assert sv().cache_truncate(c, i64(0, -2**32 + 1)).tolist() == [0, sv().SEQ_BAD_LAYOUT] and c.lengths.tolist() == [0, 2]
    assert sv().cache_fork(c, i64(2**32 + 1, 1)).tolist() == [sv().SEQ_BAD_LAYOUT] and c.lengths.tolist() == [0, 2]
