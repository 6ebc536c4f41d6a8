"""Host-side checks of the drafted-tree and paged-cache calls (no GPU: nothing
is launched on any of these paths)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import __graft_entry__  # noqa: E402
import speculative_decoding_verification_decode_gb300 as sv  # noqa: E402
from speculative_decoding_verification_decode_gb300 import _lib  # noqa: E402

P = 1 << 12


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


def greedy(lib, **kw):
    a = dict(x=P, dt=1, stride=1000, tok=P, par=P, cu=None, B=2, n=4, total=8, V=1000, acc=P, nxt=P, path=P, st=P, stream=None)
    a.update(kw)
    return lib.sv_verify_tree_greedy(*a.values())


@pytest.mark.parametrize("kw,frag", [
    (dict(B=-1), b"batch"),
    (dict(n=-1), b"n ("),
    (dict(total=-1), b"total"),
    (dict(total=7), b"total must equal"),
    (dict(V=0), b"vocab"),
    (dict(stride=999), b"row_stride"),
    (dict(dt=3), b"dtype"),
    (dict(x=None), b"target"),
    (dict(x=P + 1), b"aligned"),
    (dict(tok=None), b"tokens"),
    (dict(acc=None), b"output"),
    (dict(nxt=None), b"output"),
    (dict(path=None), b"output"),
    (dict(st=None), b"output"),
])
def test_greedy_argument_errors(lib, kw, frag):
    assert greedy(lib, **kw) == _lib.SV_ERR_ARG
    assert frag in lib.sv_last_error()


def test_greedy_limits_and_empty_calls(lib):
    assert greedy(lib, n=257, total=514) == _lib.SV_ERR_UNSUPPORTED
    assert b"256" in lib.sv_last_error()
    assert greedy(lib, B=0, total=0, x=None, tok=None, acc=None, nxt=None, path=None, st=None) == _lib.SV_OK


def test_choices_argument_errors(lib):
    a = dict(c=P, tok=P, par=P, cu=None, B=2, n=4, total=8, acc=P, nxt=P, path=P, st=P, stream=None)
    call = lambda **kw: lib.sv_verify_tree(*{**a, **kw}.values())
    for kw, frag in ((dict(c=None), b"choices"), (dict(total=9), b"total"), (dict(st=None), b"output"), (dict(B=-3), b"batch")):
        assert call(**kw) == _lib.SV_ERR_ARG
        assert frag in lib.sv_last_error()
    assert call(n=300, total=600) == _lib.SV_ERR_UNSUPPORTED
    assert call(B=0, total=0) == _lib.SV_OK


FIELDS = dict(dtype=1, q_heads=8, kv_heads=2, dim=64, q=P, k=P, v=P, q_row=512, q_head=64, k_row=128, k_head=64,
              v_row=128, v_head=64, k_cache=P, v_cache=P, kc_page=2048, kc_token=128, kc_head=64, vc_page=2048,
              vc_token=128, vc_head=64, pages=10, page_size=16, table=P, table_stride=5, max_pages=5, lengths=P,
              parents=P, cu_nodes=0, batch=2, n=4, total=8, out=P, out_row=512, out_head=64, lse=P, status=P)


def attention(lib, scale=0.125, ws=P, wb=1 << 34, **kw):
    assert not set(kw) - set(FIELDS)
    words = list({**FIELDS, **kw}.values())
    return lib.sv_tree_attention((ctypes.c_int64 * len(words))(*words), scale, ws, wb, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(dtype=0), b"dtype"),
    (dict(dtype=7), b"dtype"),
    (dict(q_heads=7), b"multiple"),
    (dict(kv_heads=0), b"kv_heads"),
    (dict(batch=-1), b"batch"),
    (dict(total=9), b"total must equal"),
    (dict(pages=0), b"pages"),
    (dict(max_pages=-1), b"pages"),
    (dict(table_stride=4), b"table_stride"),
    (dict(table=0), b"table"),
    (dict(lengths=0), b"lengths"),
    (dict(status=0), b"status"),
    (dict(q=0), b"q, k, v"),
    (dict(out=0), b"out"),
    (dict(k_cache=0), b"cache"),
    (dict(q=P + 8), b"aligned"),
    (dict(v_cache=P + 2), b"aligned"),
    (dict(q_row=516), b"multiples of 8"),
    (dict(vc_token=-128), b"negative"),
    (dict(out_row=56), b"overlap"),
    (dict(out_head=0), b"overlap"),
    (dict(scale=3e38), b"scale"),
    (dict(scale=float("nan")), b"scale"),
    (dict(scale=float("inf")), b"scale"),
])
def test_attention_argument_errors(lib, kw, frag):
    assert attention(lib, **kw) == _lib.SV_ERR_ARG
    assert frag in lib.sv_last_error()


@pytest.mark.parametrize("kw,frag", [
    (dict(dim=136), b"dim"),
    (dict(dim=60), b"dim"),
    (dict(page_size=12), b"page_size"),
    (dict(page_size=4), b"page_size"),
    (dict(n=257, total=514), b"256"),
    (dict(q_heads=258), b"128"),
    (dict(max_pages=1 << 24, table_stride=1 << 24), b"tokens"),
])
def test_attention_limits(lib, kw, frag):
    assert attention(lib, **kw) == _lib.SV_ERR_UNSUPPORTED
    assert frag in lib.sv_last_error()


def test_attention_empty_batch(lib):
    assert attention(lib, batch=0, total=0, q=0, k=0, v=0, out=0, lengths=0, status=0, table=0) == _lib.SV_OK


def pages(**kw):
    a = dict(table=P, stride=6, max_pages=6, lengths=P, refs=P, pages=20, page=16, S=4)
    a.update(kw)
    return (ctypes.c_int64 * 8)(*a.values())


def append(lib, cache=None, where=None, n_pools=2, counts=None, path=None, cu=None, n=3, total=12, st=P, ws=P, wb=1 << 30,
           pools=(P, P), rows=(P, P)):
    w = (ctypes.c_int64 * 7)(*(where or (4096, 256, 128, 512, 128, 2, 128)))
    return lib.sv_cache_append(cache or pages(), w, (ctypes.c_int64 * 2)(*pools), (ctypes.c_int64 * 2)(*rows), n_pools,
                               counts, path, cu, n, total, st, ws, wb, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(cache=pages(S=-1)), b"sequences"),
    (dict(cache=pages(pages=0)), b"pages"),
    (dict(cache=pages(page=0)), b"page_size"),
    (dict(cache=pages(max_pages=-1)), b"max_pages"),
    (dict(cache=pages(stride=5)), b"table_stride"),
    (dict(cache=pages(lengths=0)), b"NULL"),
    (dict(cache=pages(refs=0)), b"NULL"),
    (dict(n_pools=0), b"pool"),
    (dict(n=-1), b"n ("),
    (dict(total=11), b"total must equal"),
    (dict(st=None), b"status"),
    (dict(pools=(P, 0)), b"NULL"),
    (dict(rows=(0, P)), b"NULL"),
    (dict(where=(4096, 256, 128, 512, 128, -1, 128)), b"heads"),
    (dict(where=(4096, -256, 128, 512, 128, 2, 128)), b"negative"),
    (dict(ws=None), b"workspace"),
    (dict(wb=16), b"workspace"),
    (dict(ws=P + 8), b"16-byte"),
])
def test_append_argument_errors(lib, kw, frag):
    assert append(lib, **kw) == _lib.SV_ERR_ARG
    assert frag in lib.sv_last_error()


def test_fork_and_truncate_argument_errors(lib):
    assert lib.sv_cache_fork(pages(), P, 0, P, None) == _lib.SV_ERR_ARG and b"width" in lib.sv_last_error()
    assert lib.sv_cache_fork(pages(), P, 1025, P, None) == _lib.SV_ERR_ARG and b"width" in lib.sv_last_error()
    assert lib.sv_cache_fork(pages(), P, 3, P, None) == _lib.SV_ERR_ARG and b"multiple" in lib.sv_last_error()
    assert lib.sv_cache_fork(pages(), None, 2, P, None) == _lib.SV_ERR_ARG and b"NULL" in lib.sv_last_error()
    assert lib.sv_cache_truncate(pages(), None, P, None) == _lib.SV_ERR_ARG and b"NULL" in lib.sv_last_error()
    assert lib.sv_cache_truncate(None, P, P, None) == _lib.SV_ERR_ARG and b"cache" in lib.sv_last_error()
    assert lib.sv_cache_truncate(pages(S=0, table=0, lengths=0), None, None, None) == _lib.SV_OK
    assert lib.sv_cache_fork(pages(S=0), None, 2, None, None) == _lib.SV_OK


def test_workspace_sizes(lib):
    assert lib.sv_cache_append_workspace_size(-1, 1, 1, 1) == 0
    assert lib.sv_cache_append_workspace_size(0, 5, 100, 16) < 64
    big = lib.sv_cache_append_workspace_size(1 << 20, 1 << 20, 1 << 20, 16)  # no more pages than there are
    assert (1 << 25) <= big <= (1 << 25) + (1 << 22) + 64


def test_binding_refuses_before_any_device_work():
    f = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        sv.tree_attention(f(2, 2, 8), f(2, 1, 8), f(2, 1, 8), f(3, 8, 1, 8), f(3, 8, 1, 8), f(1, 3), f(1))
    c = sv.paged_cache(2, 5, 8, 1, 8, 3, 4, device="cpu")
    for call in (lambda: sv.cache_append(c, f(3, 1, 8), f(3, 1, 8)), lambda: sv.cache_truncate(c, f(3)),
                 lambda: sv.cache_fork(c, f(3))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
