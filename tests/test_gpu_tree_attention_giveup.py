"""The tree attention's bounded waits.  With the testing flag
FLAG_EXPIRE_EXCHANGE every wait for outputs gives up at once, so that a CTA
leaves the items behind its first one undone: the call returns, every sequence
says SEQ_TIMEOUT, nothing but the sequences' own rows is written, whatever
records the workspace held before, and the next ordinary call is as ever."""

import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytestmark = pytest.mark.skip("needs a GPU")
else:
    pytestmark = pytest.mark.gpu

import __graft_entry__  # noqa: E402
from test_gpu_tree_attention import BF, HF, Case, sv  # noqa: E402

DEV = torch.device("cuda", 0)
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def shapes():
    ctas = min(152, torch.cuda.get_device_properties(0).multi_processor_count)
    half = ctas // 2
    return [
        # as many items as CTAs, long and short by turns: pieces of several items
        ([1] * (2 * half), [5000, 100] * half, 1, 1, 64, BF),
        ([3, 0, 2] * 8, [3000, 10, 90] * 8, 8, 4, 128, HF),
        # more items than CTAs
        ([2] * 90, [700, 30, 0] * 30, 8, 4, 64, BF),
        # one item in many pieces
        ([60], [8191], 8, 1, 128, BF),
        ([200, 1], [300, 5], 16, 2, 128, HF),
    ]


@pytest.mark.parametrize("which", range(5))
def test_expired_waits(which, monkeypatch):
    N, lengths, Hq, Hkv, D, dtype = shapes()[which]
    c = Case(which, N, lengths, Hq, Hkv, D, 64, dtype)
    a = c.dev()
    total = a["q"].shape[0]
    want = sv().tree_attention(**a)
    c.check(want)
    # the workspace full of records of an item far away: (parts, slot, CTA, sequence, head, pair, nodes, err)
    record = np.array([1, 0, 0, 0, 1 << 14, 1 << 10, 256, 0], np.int32)
    empty, poisoned = torch.empty, []

    def poison(*args, **kw):
        t = empty(*args, **kw)
        if kw.get("dtype") is torch.uint8:
            n = t.numel() // 32
            t[:32 * n].view(torch.int32).view(n, 8).copy_(torch.from_numpy(record).to(DEV).expand(n, 8))
            poisoned.append(t.numel())
        return t

    buf = empty((total + 2 * GUARD, Hq, D), dtype=dtype, device=DEV).fill_(7.0)
    monkeypatch.setattr(torch, "empty", poison)
    t = time.perf_counter()
    r = sv().tree_attention(**a, out=buf[GUARD:GUARD + total], flags=sv().FLAG_EXPIRE_EXCHANGE)
    torch.cuda.synchronize()
    assert time.perf_counter() - t < 10.0  # no wait ran to its full limit
    monkeypatch.undo()
    assert poisoned
    assert ((r.status & sv().SEQ_TIMEOUT) != 0).all()
    assert (buf[:GUARD] == 7).all() and (buf[GUARD + total:] == 7).all()
    again = sv().tree_attention(**a)
    assert torch.equal(again.out, want.out) and torch.equal(again.lse, want.lse) and not again.status.any()


def test_records_of_another_call_do_not_matter(monkeypatch):
    """The same poisoned workspace under an ordinary call."""
    empty = torch.empty
    for which in range(5):
        N, lengths, Hq, Hkv, D, dtype = shapes()[which]
        c = Case(which, N, lengths, Hq, Hkv, D, 64, dtype)
        a = c.dev()
        want = sv().tree_attention(**a)
        monkeypatch.setattr(torch, "empty", lambda *s, **kw: empty(*s, **kw).fill_(1) if kw.get("dtype") is torch.uint8 else empty(*s, **kw))
        got = sv().tree_attention(**a)
        monkeypatch.undo()
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse) and not got.status.any()


def test_unknown_flags_are_refused():
    c = Case(9, [1], [5], 2, 1, 64, 8, BF)
    with pytest.raises(sv().SVError, match="flag"):
        sv().tree_attention(**c.dev(), flags=1)
