"""Arrays of the tree attention whose strides are 0: the C call refuses them
where a dimension has more than one entry (a tensor map cannot say it), the
binding copies such queries, keys and values (no GPU: nothing is launched)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import __graft_entry__  # noqa: E402
from speculative_decoding_verification_decode_gb300 import _lib, api  # noqa: E402

P = 1 << 12
FIELDS = dict(dtype=1, q_heads=8, kv_heads=2, dim=64, q=P, k=P, v=P, q_row=512, q_head=64, k_row=128, k_head=64,
              v_row=128, v_head=64, k_cache=P, v_cache=P, kc_page=2048, kc_token=128, kc_head=64, vc_page=2048,
              vc_token=128, vc_head=64, pages=10, page_size=16, table=P, table_stride=5, max_pages=5, lengths=P,
              parents=P, cu_nodes=0, batch=2, n=4, total=8, out=1 << 20, out_row=512, out_head=64, lse=1 << 21, status=1 << 22)


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


def attention(lib, **kw):
    assert not set(kw) - set(FIELDS)
    words = list({**FIELDS, **kw}.values())
    return lib.sv_tree_attention((ctypes.c_int64 * len(words))(*words), 0.125, 1 << 24, 1 << 34, None)


@pytest.mark.parametrize("name", ["q_row", "q_head", "k_row", "k_head", "v_row", "v_head", "kc_page", "kc_token", "kc_head",
                                  "vc_page", "vc_token", "vc_head"])
def test_a_stride_of_0_is_refused(lib, name):
    assert attention(lib, **{name: 0}) == _lib.SV_ERR_ARG
    assert b"stride of 0" in lib.sv_last_error() and name.encode() in lib.sv_last_error()


def test_views_that_the_binding_copies():
    x = torch.arange(6 * 4 * 16, dtype=torch.bfloat16).view(6, 4, 16)
    views = [x[:, :1].expand(-1, 4, -1), x[:1].expand(6, -1, -1), x[:1, :1].expand(6, 4, -1)]
    for v in views:
        y = api._aligned(v)
        assert y.is_contiguous() and torch.equal(y, v)
    # a dimension of one entry may have any stride
    for v in (x[:, :1].expand(-1, 1, -1), x[:1].as_strided((1, 4, 16), (0, 16, 1)), x[:, 1:2].as_strided((6, 1, 16), (64, 0, 1))):
        assert api._aligned(v) is v
