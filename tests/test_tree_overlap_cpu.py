"""An out of the tree attention that shares memory with another array of the call
is refused, wherever it begins (no GPU: nothing is launched)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import __graft_entry__  # noqa: E402
from speculative_decoding_verification_decode_gb300 import _lib  # noqa: E402

M = 1 << 20  # bytes between the arrays
FIELDS = dict(dtype=1, q_heads=8, kv_heads=2, dim=64, q=M, k=2 * M, v=3 * M, q_row=512, q_head=64, k_row=128, k_head=64,
              v_row=128, v_head=64, k_cache=4 * M, v_cache=5 * M, kc_page=2048, kc_token=128, kc_head=64, vc_page=2048,
              vc_token=128, vc_head=64, pages=10, page_size=16, table=6 * M, table_stride=5, max_pages=5, lengths=7 * M,
              parents=8 * M, cu_nodes=0, batch=2, n=4, total=8, out=9 * M, out_row=512, out_head=64, lse=10 * M, status=11 * M)
OUT = 8 * 512 * 2  # bytes of out


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _lib.load()


def refused(lib, **kw):
    """Whether the host checks refuse the call (here a call that passes them ends at the missing GPU)."""
    assert not set(kw) - set(FIELDS)
    words = list({**FIELDS, **kw}.values())
    rc = lib.sv_tree_attention((ctypes.c_int64 * len(words))(*words), 0.125, 12 * M, 1 << 34, None)
    if rc == _lib.SV_ERR_ARG:
        assert b"out" in lib.sv_last_error(), lib.sv_last_error()
    return rc == _lib.SV_ERR_ARG


# bytes of each array from its first to its last element
SIZES = dict(q=OUT, k=8 * 128 * 2, v=8 * 128 * 2, k_cache=10 * 2048 * 2, v_cache=10 * 2048 * 2, table=10 * 4, lengths=2 * 4,
             parents=8 * 4, lse=8 * 8 * 4, status=2 * 4)


@pytest.mark.parametrize("name", sorted(SIZES))
def test_an_out_that_reaches_into_another_array(lib, name):
    at, size = FIELDS[name], SIZES[name]
    end = (size + 15) // 16 * 16
    for o in (at, at + 16 * ((size - 1) // 16), at - OUT + 16, at + 16 * (size // 32)):
        assert refused(lib, out=o), (name, o - at)
    for o in (at + end, at - OUT):  # side by side
        assert not refused(lib, out=o), (name, o - at)


def test_ragged_layouts(lib):
    kw = dict(cu_nodes=20 * M, batch=2, total=8)
    assert not refused(lib, **kw)
    assert refused(lib, **kw, out=20 * M) and refused(lib, **{**kw, "cu_nodes": FIELDS["out"] + OUT - 16})
    assert not refused(lib, **{**kw, "cu_nodes": FIELDS["out"] + OUT})


def test_an_out_beside_its_inputs_in_one_projection(lib):
    """q, k, v and out as column ranges of one [total, heads, dim] tensor: rows lie
    between one another's, elements do not meet."""
    row = 20 * 64
    kw = dict(q=M, k=M + 8 * 128, v=M + 10 * 128, q_row=row, k_row=row, v_row=row, out_row=row)
    assert not refused(lib, **kw, out=M + 12 * 128)
    assert refused(lib, **kw, out=M + 11 * 128)
    assert refused(lib, **kw, out=M + 4 * 128)
    # beginning in the row before
    kw = dict(q=M + 8 * 128, k=M + 16 * 128, v=M + 18 * 128, q_row=row, k_row=row, v_row=row, out_row=row)
    assert not refused(lib, **kw, out=M)
    assert refused(lib, **kw, out=M + 16) and refused(lib, **kw, out=M + 16 * 128)
    # the same rows, but not as far apart
    assert refused(lib, **{**kw, "out_row": row + 64}, out=M)


@pytest.mark.parametrize("kw", [dict(out_row=64, out_head=64), dict(out_row=64, out_head=128), dict(out_row=256, out_head=64),
                                dict(out_row=448, out_head=64)])
def test_an_out_whose_rows_overlap(lib, kw):
    assert refused(lib, **kw)


@pytest.mark.parametrize("kw", [dict(out_row=64, out_head=512), dict(out_row=512, out_head=64), dict(out_row=64, out_head=520),
                                dict(out_row=1024, out_head=72), dict(out_row=0, out_head=64, total=1, n=1, batch=1),
                                dict(out_row=64, out_head=0, q_heads=1, kv_heads=1, q_head=0, k_head=0, kc_head=0, vc_head=0)])
def test_an_out_of_any_order(lib, kw):
    assert not refused(lib, **kw)


def test_no_rows_no_overlap(lib):
    assert not refused(lib, batch=2, n=0, total=0, out=M)
