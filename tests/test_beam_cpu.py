"""Host-side checks of the beam-search and 4-bit LM-head calls (no GPU: nothing
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


def select(lib, **kw):
    a = dict(x=P, dt=1, stride=1000, c=P, fin=None, eos=-1, B=2, W=4, V=1000, n=8, s=P, p=P, t=P, st=P, ws=P,
             wb=1 << 30, stream=None)
    a.update(kw)
    return lib.sv_beam_select(*a.values())


@pytest.mark.parametrize("kw,frag", [
    (dict(B=-1), b"batch"),
    (dict(W=0), b"beams"),
    (dict(W=65), b"beams"),
    (dict(V=0), b"vocab"),
    (dict(n=0), b"n ("),
    (dict(n=129), b"n ("),
    (dict(stride=999), b"row_stride"),
    (dict(dt=3), b"dtype"),
    (dict(fin=P), b"eos"),
    (dict(fin=P, eos=1000), b"eos"),
    (dict(B=1 << 29, W=8), b"batch"),
    (dict(x=None), b"NULL"),
    (dict(c=None), b"NULL"),
    (dict(st=None), b"NULL"),
    (dict(x=P + 1), b"aligned"),
    (dict(ws=None), b"workspace"),
    (dict(wb=8), b"workspace"),
    (dict(ws=P + 8), b"workspace"),
])
def test_select_argument_errors(lib, kw, frag):
    assert select(lib, **kw) == _lib.SV_ERR_ARG
    assert frag in lib.sv_last_error()


def test_select_sizes(lib):
    assert select(lib, V=1 << 29, stride=1 << 29) == _lib.SV_ERR_UNSUPPORTED  # flat index beyond 31 bits
    assert select(lib, B=0, x=None, c=None, s=None, p=None, t=None, st=None, ws=None, wb=0) == _lib.SV_OK
    assert lib.sv_beam_select_workspace_size(2, 4, 1000, 8) > 0
    for bad in ((-1, 4, 1000, 8), (2, 0, 1000, 8), (2, 65, 1000, 8), (2, 4, 0, 8), (2, 4, 1000, 129)):
        assert lib.sv_beam_select_workspace_size(*bad) == 0


def state(**kw):
    a = dict(data=P, seq_stride=4 * 4096, beam_stride=4096, seg_stride=1024, token_bytes=64, segs=4, tokens=16,
             timed=1, reserved=0)
    a.update(kw)
    return _lib.BeamState(*a.values())


@pytest.mark.parametrize("kw,frag", [
    (dict(segs=-1), b"size"),
    (dict(tokens=-1), b"size"),
    (dict(token_bytes=-1), b"size"),
    (dict(seq_stride=-16), b"stride"),
    (dict(beam_stride=512), b"stride"),
    (dict(seg_stride=512), b"stride"),
    (dict(data=None), b"data"),
    (dict(token_bytes=1 << 45), b"too large"),
])
def test_reorder_state_errors(lib, kw, frag):
    s = (_lib.BeamState * 1)(state(**kw))
    assert lib.sv_beam_reorder(s, 1, P, P, 2, 4, P, None) == _lib.SV_ERR_ARG
    assert frag in lib.sv_last_error()


def test_reorder_argument_errors(lib):
    s = (_lib.BeamState * 1)(state())
    call = lambda **kw: lib.sv_beam_reorder(*{**dict(s=s, n=1, p=P, ln=P, B=2, W=4, st=P, stream=None), **kw}.values())
    assert call(B=-1) == _lib.SV_ERR_ARG
    assert call(W=65) == _lib.SV_ERR_ARG and b"beams" in lib.sv_last_error()
    assert call(n=0) == _lib.SV_ERR_ARG and b"state" in lib.sv_last_error()
    assert call(ln=None) == _lib.SV_ERR_ARG and b"lengths" in lib.sv_last_error()
    assert call(p=None) == _lib.SV_ERR_ARG
    assert call(st=None) == _lib.SV_ERR_ARG
    assert call(B=0, p=None, st=None) == _lib.SV_OK
    huge = (_lib.BeamState * 1)(state(token_bytes=1 << 30, tokens=1 << 15, segs=1, timed=0, beam_stride=1 << 46))
    assert lib.sv_beam_reorder(huge, 1, P, P, 1 << 12, 4, P, None) == _lib.SV_ERR_UNSUPPORTED


def q4(lib, proj=True, group=128, sdt=1, packed=P, scales=P, **kw):
    pr = _lib.Q4Proj(packed, scales, None, sdt, group)
    a = dict(h=P, dt=1, proj=ctypes.byref(pr) if proj else None, rows=3, V=100, d=256, out=P, ld=100, err=None,
             stream=None)
    a.update(kw)
    return lib.sv_lm_head_q4_logits(*a.values())


@pytest.mark.parametrize("kw,frag", [
    (dict(rows=-1), b"rows"),
    (dict(V=0), b"rows"),
    (dict(proj=False), b"proj"),
    (dict(dt=0), b"states"),
    (dict(sdt=4), b"scale"),
    (dict(group=16), b"group"),
    (dict(group=256), b"group"),
    (dict(d=40), b"multiple of 32"),
    (dict(ld=99), b"ld"),
    (dict(h=None), b"NULL"),
    (dict(packed=None), b"NULL"),
    (dict(scales=None), b"NULL"),
    (dict(h=P + 8), b"aligned"),
    (dict(packed=P + 8), b"aligned"),
    (dict(scales=P + 1), b"aligned"),
    (dict(out=P + 2), b"aligned"),
])
def test_q4_argument_errors(lib, kw, frag):
    assert q4(lib, **kw) == _lib.SV_ERR_ARG
    assert frag in lib.sv_last_error()


def test_q4_verify_argument_errors(lib):
    pr = ctypes.byref(_lib.Q4Proj(P, P, None, 1, 128))
    need = lib.sv_lm_head_workspace_size(2, 6, 100)
    args = dict(ht=P, hd=P, dt=1, proj=pr, d=256, T=P, tok=P, u=P, cu=None, B=2, K=3, sk=6, V=100, n=P, nx=P, st=P,
                ws=P, wb=need, flags=0, stream=None)
    call = lambda **kw: lib.sv_lm_head_q4_verify(*{**args, **kw}.values())
    assert q4(lib, rows=0, h=None, out=None) == _lib.SV_OK
    assert call(B=0, sk=0) == _lib.SV_OK
    assert call(wb=need - 4) == _lib.SV_ERR_ARG and b"workspace_bytes" in lib.sv_last_error()
    assert call(flags=16) == _lib.SV_ERR_ARG
    assert call(sk=5) == _lib.SV_ERR_ARG
    assert call(hd=None) == _lib.SV_ERR_ARG
    assert call(ws=P + 8) == _lib.SV_ERR_ARG
    assert call(T=None) == _lib.SV_ERR_ARG


def test_binding_refusals():
    """Shapes and types the binding refuses before any device work."""
    with pytest.raises(ValueError, match="scores"):
        sv.beam_select(torch.zeros(2, 3, 8), torch.zeros(6))
    with pytest.raises(ValueError, match="CUDA"):
        sv.beam_reorder(torch.zeros(2, 3, 8), torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="state"):
        sv.beam_reorder([], torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="group"):
        sv.q4_quantize(torch.zeros(4, 64), group=48)
    with pytest.raises(ValueError, match="multiple of 32"):
        sv.q4_quantize(torch.zeros(4, 40))
    with pytest.raises(ValueError, match="max_len"):
        sv.BeamDecoder(None, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_state_descriptions():
    """Strides of the layouts a cache may have, and those that cannot move in place."""
    from speculative_decoding_verification_decode_gb300.api import _beam_layout

    def _beam_state(t, td):
        words = (t.data_ptr(), *_beam_layout(t, td))
        return ctypes.cast((ctypes.c_int64 * 7)(*words), ctypes.POINTER(_lib.BeamState))[0]

    assert ctypes.sizeof(_lib.BeamState) == 56
    t = torch.zeros(2, 3, 4, 10, 16, dtype=torch.bfloat16)  # heads before time
    d = _beam_state(t, 3)
    assert (d.segs, d.tokens, d.token_bytes, d.seg_stride, d.beam_stride, d.timed) == (4, 10, 32, 320, 1280, 1)
    d = _beam_state(t, 2)  # time first: [B, W, T, H, D]
    assert (d.segs, d.tokens, d.token_bytes) == (1, 4, 320)
    d = _beam_state(t[:, :, :, :7], 3)  # part of a longer buffer
    assert (d.segs, d.tokens, d.token_bytes, d.seg_stride) == (4, 7, 32, 320)
    d = _beam_state(t, None)
    assert (d.segs, d.tokens, d.token_bytes, d.timed) == (1, 1, 1280, 0)
    d = _beam_state(t[:, :, :, :, :5], None)  # rows with gaps
    assert (d.segs, d.token_bytes, d.seg_stride) == (40, 10, 32)
    d = _beam_state(torch.zeros(2, 3, dtype=torch.int32), None)  # one value per beam
    assert (d.segs, d.tokens, d.token_bytes) == (1, 1, 4)
    with pytest.raises(ValueError, match="broadcast"):
        _beam_state(t[:, :1].expand(2, 3, 4, 10, 16), None)
    for bad, td in ((t.transpose(3, 4), 4), (t[..., ::2], None), (t[:, :, ::1, :, ::2], 3), (t[:, :, :, :7], 2)):
        with pytest.raises(ValueError):
            _beam_state(bad, td)
