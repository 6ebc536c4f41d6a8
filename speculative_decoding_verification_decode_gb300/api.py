"""PyTorch binding of libsv: argument marshalling only.

Every step of verification runs in the CUDA kernel behind the C ABI; these
functions only check shapes, pick the current CUDA stream and pass device
pointers.  When the inputs live in host memory the call copies them to the
GPU (from pinned memory when they are pinned), runs the kernel and copies the
results back, which is how an end-to-end caller with host buffers uses it.
"""

from __future__ import annotations

import ctypes
import functools
import struct
from operator import attrgetter
from typing import NamedTuple, Optional, Sequence, Union

import torch

from . import _lib

_DTYPES = {torch.float32: _lib.SV_F32, torch.bfloat16: _lib.SV_BF16, torch.float16: _lib.SV_F16}


class VerifyResult(NamedTuple):
    n_accepted: torch.Tensor  # int32 [B]
    next_token: torch.Tensor  # int32 [B]; -1 when the sequence's inputs are invalid
    status: torch.Tensor  # int32 [B]; OR of SV_SEQ_* bits


class SVError(RuntimeError):
    pass


def _check(rc: int):
    if rc != _lib.SV_OK:
        lib = _lib.load()
        raise SVError(f"{lib.sv_status_string(rc).decode()}: {lib.sv_last_error().decode()}")


def _rows(x: torch.Tensor) -> torch.Tensor:
    """[rows, V] view of a 2-D or 3-D ([B, rows_per_seq, V]) input with unit
    stride along V."""
    if x.dim() == 3:
        x = x.reshape(-1, x.shape[-1])
    if x.dim() != 2:
        raise ValueError("rows must be 2-D [rows, V] or 3-D [B, rows, V]")
    if x.stride(1) != 1:
        x = x.contiguous()
    return x


def _layout(n_target_rows: int, tokens: torch.Tensor, cu_k, k):
    sum_k = int(tokens.numel())
    if cu_k is None:
        B = n_target_rows - sum_k
        if B < 0 or (B and sum_k % B):
            raise ValueError("target rows must be B*(K+1) for B*K draft tokens")
        K = sum_k // B if B else 0
        return B, K, sum_k
    B = int(cu_k.numel()) - 1
    if k is None:
        raise ValueError("k (the largest K_b) is required with cu_k")
    if n_target_rows < sum_k + B:
        raise ValueError("target must hold sum(K_b) + B rows")
    return B, int(k), sum_k


class _Marshal:
    """Moves host inputs to the device (and results back) for one call."""

    def __init__(self, ref: torch.Tensor):
        self.host = ref.device.type != "cuda"
        self.device = torch.device("cuda", torch.cuda.current_device()) if self.host else ref.device

    def dev(self, t: Optional[torch.Tensor], dtype=None) -> Optional[torch.Tensor]:
        if t is None:
            return None
        if dtype is not None and t.dtype != dtype:
            t = t.to(dtype)
        if t.device != self.device:
            t = t.to(self.device, non_blocking=True)
        return t.contiguous() if t.dim() == 1 else t

    def outputs(self, B: int):
        mk = lambda: torch.empty(B, dtype=torch.int32, device=self.device)
        return mk(), mk(), mk()

    def finish(self, res: VerifyResult) -> VerifyResult:
        if not self.host:
            return res
        return VerifyResult(*(x.to("cpu") for x in res))

    def stream(self):
        return ctypes_ptr(torch.cuda.current_stream(self.device).cuda_stream)


def ctypes_ptr(v):
    return None if v is None else int(v)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(dev: torch.device, fn, *args):
    """``fn(*args, stream)`` on ``dev``'s current stream, the device made
    current only where it is not (host time counts in the calls of a few
    microseconds that this serves)."""
    i = dev.index
    if i == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            rc = fn(*args, _raw_stream(i))
    if rc != _lib.SV_OK:
        _check(rc)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def verify_greedy(target: torch.Tensor, draft_tokens: torch.Tensor,
                  cu_k: Optional[torch.Tensor] = None, k: Optional[int] = None,
                  flags: int = 0) -> VerifyResult:
    """Greedy verification (spec-verify card, "Method"): ``target`` holds the
    K_b + 1 rows of every sequence (probabilities or logits, f32/bf16/f16)."""
    m = _Marshal(target)
    tg = _rows(m.dev(target))
    tok = m.dev(draft_tokens.reshape(-1), torch.int32)
    cu = m.dev(cu_k, torch.int32)
    B, K, sum_k = _layout(tg.shape[0], tok, cu, k)
    n, nxt, st = m.outputs(B)
    lib = _lib.load()
    with torch.cuda.device(m.device):
        _check(lib.sv_verify_greedy(_p(tg), _DTYPES[tg.dtype], tg.stride(0), _p(tok), _p(cu), B, K,
                                    sum_k, tg.shape[1], _p(n), _p(nxt), _p(st), flags, m.stream()))
    return m.finish(VerifyResult(n, nxt, st))


def accept(target_probs: torch.Tensor, draft_probs: torch.Tensor, draft_tokens: torch.Tensor,
           uniforms: torch.Tensor, cu_k: Optional[torch.Tensor] = None, k: Optional[int] = None,
           flags: int = 0) -> VerifyResult:
    """Speculative sampling on f32 probability rows with explicit uniforms
    (``K_b + 1`` per sequence; the last one draws the correction or bonus)."""
    m = _Marshal(target_probs)
    tg = _rows(m.dev(target_probs, torch.float32))
    dr = _rows(m.dev(draft_probs, torch.float32))
    if dr.stride(0) != tg.stride(0):
        dr = dr.contiguous()
        tg = tg.contiguous()
    tok = m.dev(draft_tokens.reshape(-1), torch.int32)
    u = m.dev(uniforms.reshape(-1), torch.float32)
    cu = m.dev(cu_k, torch.int32)
    B, K, sum_k = _layout(tg.shape[0], tok, cu, k)
    n, nxt, st = m.outputs(B)
    lib = _lib.load()
    with torch.cuda.device(m.device):
        _check(lib.sv_accept(_p(tg), _p(dr), tg.stride(0), _p(tok), _p(u), _p(cu), B, K, sum_k,
                             tg.shape[1], _p(n), _p(nxt), _p(st), flags, m.stream()))
    return m.finish(VerifyResult(n, nxt, st))


def accept_from_logits(target_logits: torch.Tensor, draft_logits: torch.Tensor,
                       temperature: torch.Tensor, draft_tokens: torch.Tensor,
                       uniforms: torch.Tensor, cu_k: Optional[torch.Tensor] = None,
                       k: Optional[int] = None, warped_out: Optional[tuple] = None,
                       flags: int = 0, top_k: Optional[torch.Tensor] = None,
                       top_p: Optional[torch.Tensor] = None,
                       floors: Optional[tuple] = None) -> VerifyResult:
    """Mixed greedy / sampled verification from logits with a fused
    per-sequence temperature softmax (``temperature[b] == 0`` is greedy).

    ``warped_out``: optional pair of f32 device tensors ``[target_rows, V]``
    and ``[draft_rows, V]`` that receive the warped weights of every row the
    kernel reached (a testing aid).

    ``top_k`` (int32 ``[B]``) / ``top_p`` (f32 ``[B]``): the sampler filters of
    include/sv_filter.h, applied alike to target and draft rows, in one call of
    ``sv_accept_from_logits_filtered`` (the fused top-k plan where it applies,
    the floors and the floored verification for the rest; with ``warped_out``
    the two calls instead).  ``floors``: a pair of f32 device tensors
    ``[target_rows]``, ``[draft_rows]`` of precomputed floors (used instead of
    top_k / top_p; either may be None)."""
    m = _Marshal(target_logits)
    tg = _rows(m.dev(target_logits))
    dr = _rows(m.dev(draft_logits, tg.dtype))
    if dr.stride(0) != tg.stride(0):
        dr = dr.contiguous()
        tg = tg.contiguous()
    tok = m.dev(draft_tokens.reshape(-1), torch.int32)
    u = m.dev(uniforms.reshape(-1), torch.float32)
    T = m.dev(temperature.reshape(-1), torch.float32)
    cu = m.dev(cu_k, torch.int32)
    B, K, sum_k = _layout(tg.shape[0], tok, cu, k)
    wt, wd = (None, None) if warped_out is None else warped_out
    n, nxt, st = m.outputs(B)
    lib = _lib.load()
    if floors is None and (top_k is not None or top_p is not None):
        tk, tp = m.dev(top_k, torch.int32), m.dev(top_p, torch.float32)
        if warped_out is None:
            with torch.cuda.device(m.device):
                _check(lib.sv_accept_from_logits_filtered(_p(tg), _p(dr), _DTYPES[tg.dtype], tg.stride(0), _p(T),
                                                          _p(tk), _p(tp), _p(tok), _p(u), _p(cu), B, K, sum_k,
                                                          tg.shape[1], _p(n), _p(nxt), _p(st), flags, m.stream()))
            return m.finish(VerifyResult(n, nxt, st))
        floors = _floors(lib, m, tg, dr, T, tk, tp, cu, B, K, sum_k)
    with torch.cuda.device(m.device):
        if floors is None:
            _check(lib.sv_accept_from_logits(_p(tg), _p(dr), _DTYPES[tg.dtype], tg.stride(0), _p(T),
                                             _p(tok), _p(u), _p(cu), B, K, sum_k, tg.shape[1], _p(n),
                                             _p(nxt), _p(st), _p(wt), _p(wd), flags, m.stream()))
        else:
            ft, fd = (m.dev(f, torch.float32) for f in floors)
            _check(lib.sv_accept_from_logits_floored(_p(tg), _p(dr), _DTYPES[tg.dtype], tg.stride(0),
                                                     _p(T), _p(tok), _p(u), _p(cu), B, K, sum_k,
                                                     tg.shape[1], _p(ft), _p(fd), _p(n), _p(nxt),
                                                     _p(st), _p(wt), _p(wd), flags, m.stream()))
    return m.finish(VerifyResult(n, nxt, st))


def _floors(lib, m, tg, dr, T, tk, tp, cu, B, K, sum_k, out=None):
    if out is not None:
        ft, fd = out
    else:
        ft = torch.full((sum_k + B,), float("-inf"), dtype=torch.float32, device=m.device)
        fd = torch.full((sum_k,), float("-inf"), dtype=torch.float32, device=m.device)
    with torch.cuda.device(m.device):
        _check(lib.sv_sampler_floors(_p(tg), _p(dr), _DTYPES[tg.dtype], tg.stride(0), _p(T), _p(tk),
                                     _p(tp), _p(cu), B, K, sum_k, tg.shape[1], _p(ft), _p(fd),
                                     m.stream()))
    return ft, fd


def sampler_floors(target_logits: torch.Tensor, draft_logits: torch.Tensor,
                   temperature: torch.Tensor, top_k: Optional[torch.Tensor] = None,
                   top_p: Optional[torch.Tensor] = None, cu_k: Optional[torch.Tensor] = None,
                   k: Optional[int] = None, sum_k: Optional[int] = None, out: Optional[tuple] = None):
    """Per-row floors of the top-k / top-p filters (include/sv_filter.h):
    ``(floor_target [target_rows], floor_draft [draft_rows])`` f32; the rows a
    filter keeps are those with logit >= floor (-inf keeps all, NaN marks an
    invalid top-p).  Without ``cu_k`` the layout is B*(K+1) target rows and
    B*K draft rows with ``k`` = K.  ``out``: optional preallocated f32 device
    tensors for the two results (device inputs only; rows the kernel does not
    reach keep their values)."""
    n_t = target_logits.reshape(-1, target_logits.shape[-1]).shape[0]
    n_d = draft_logits.reshape(-1, draft_logits.shape[-1]).shape[0]
    if cu_k is None:
        B = int(temperature.numel())
        K = (n_t - B) // B if B else 0
        sk = B * K
        if n_t != B * (K + 1) or n_d != sk:
            raise ValueError(f"without cu_k the rows must be B*(K+1) target and B*K draft rows for "
                             f"B = {B} temperatures (got {n_t} and {n_d})")
    else:
        B = int(cu_k.numel()) - 1
        if k is None or sum_k is None:
            raise ValueError("k and sum_k are required with cu_k")
        K, sk = int(k), int(sum_k)
        if n_t < sk + B or n_d < sk:
            raise ValueError(f"cu_k needs {sk + B} target and {sk} draft rows (got {n_t} and {n_d})")
    m = _Marshal(target_logits)
    tg = _rows(m.dev(target_logits))
    dr = _rows(m.dev(draft_logits, tg.dtype))
    if dr.stride(0) != tg.stride(0):
        dr = dr.contiguous()
        tg = tg.contiguous()
    T = m.dev(temperature.reshape(-1), torch.float32)
    cu = m.dev(cu_k, torch.int32)
    ft, fd = _floors(_lib.load(), m, tg, dr, T, m.dev(top_k, torch.int32), m.dev(top_p, torch.float32),
                     cu, B, K, sk, None if m.host else out)
    if m.host:
        return ft.cpu(), fd.cpu()
    return ft, fd


# ---------------------------------------------------------------- draft-length gate

class GateResult(NamedTuple):
    n_submit: torch.Tensor  # int32 [B]: drafts each sequence submits
    cu_k: torch.Tensor  # int32 [B+1]: their exclusive prefix sum (the verify calls' cu_k)


def gate_draft_lengths(confidence: torch.Tensor, edges: torch.Tensor, hits: torch.Tensor,
                       total: torch.Tensor, k_drafted: Optional[torch.Tensor] = None,
                       logit_margin: Optional[torch.Tensor] = None, margin: float = 1.15,
                       draft_ms: float = 196.0, verify_base_ms: float = 300.0,
                       verify_slope_ms: float = 109.0, plain_ms: float = 303.0,
                       margin_threshold: float = 0.0, min_draft: int = 0) -> GateResult:
    """Draft-length gate (include/sv_gate.h; PocketLLM dspark.md): ``confidence``
    is ``[B, K]`` f32; ``edges`` ``[n_buckets - 1]`` f32; ``hits`` / ``total``
    ``[n_buckets]`` f64 calibration counts.  Defaults are the page's."""
    if confidence.dim() != 2:
        raise ValueError("confidence must be [B, K]")
    dev = confidence.device
    if dev.type != "cuda":
        raise ValueError("gate inputs must be CUDA tensors")
    conf = confidence.to(torch.float32).contiguous()
    B, K = conf.shape
    e = edges.to(device=dev, dtype=torch.float32).contiguous()
    h = hits.to(device=dev, dtype=torch.float64).contiguous()
    t = total.to(device=dev, dtype=torch.float64).contiguous()
    kd = None if k_drafted is None else k_drafted.to(device=dev, dtype=torch.int32).contiguous()
    lm = None if logit_margin is None else logit_margin.to(device=dev, dtype=torch.float32).contiguous()
    n = torch.empty(B, dtype=torch.int32, device=dev)
    cu = torch.empty(B + 1, dtype=torch.int32, device=dev)
    prm = _lib.GateParams(margin, draft_ms, verify_base_ms, verify_slope_ms, plain_ms,
                          margin_threshold, min_draft)
    lib = _lib.load()
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        _check(lib.sv_gate_draft_lengths(_p(conf), _p(kd), _p(lm), _p(e), _p(h), _p(t), h.numel(), B, K,
                                         ctypes.byref(prm), _p(n), _p(cu), stream))
    return GateResult(n, cu)


def gate_update(confidence: torch.Tensor, n_submitted: torch.Tensor, n_accepted: torch.Tensor,
                edges: torch.Tensor, hits: torch.Tensor, total: torch.Tensor, decay: float = 0.9) -> None:
    """One round of calibration, in place on ``hits`` / ``total`` (f64 CUDA
    tensors, contiguous): positions before the accepted length are hits, the
    first rejected position is a miss, later ones are not recorded."""
    if confidence.dim() != 2:
        raise ValueError("confidence must be [B, K]")
    dev = confidence.device
    for x in (hits, total):
        if x.device != dev or x.dtype != torch.float64 or not x.is_contiguous():
            raise ValueError("hits / total must be contiguous f64 tensors on the confidence's device")
    conf = confidence.to(torch.float32).contiguous()
    B, K = conf.shape
    e = edges.to(device=dev, dtype=torch.float32).contiguous()
    ns = n_submitted.to(device=dev, dtype=torch.int32).contiguous()
    na = n_accepted.to(device=dev, dtype=torch.int32).contiguous()
    lib = _lib.load()
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        _check(lib.sv_gate_update(_p(conf), _p(ns), _p(na), _p(e), _p(hits), _p(total), hits.numel(), B, K,
                                  float(decay), stream))



# ---------------------------------------------------------------- LM head in front of verification

def _bf16_rows(x: torch.Tensor, m: "_Marshal") -> torch.Tensor:
    if not isinstance(x, torch.Tensor):
        raise ValueError("states and projection must be bfloat16 tensors (this call takes no 4-bit projection)")
    x = m.dev(x)
    if x.dtype != torch.bfloat16:
        raise ValueError("states and projection must be bfloat16")
    return x.reshape(-1, x.shape[-1]).contiguous()


class Q4Projection(NamedTuple):
    """A vocabulary projection in 4 bits (include/sv_lm_head_q4.h):
    ``W[v, k] = scales[v, k // group] * (q[v, k] - zeros[v, k // group])``.
    ``lm_head_logits`` and ``lm_head_verify`` take it in place of the bf16
    matrix; ``q4_quantize`` makes one from such a matrix."""
    packed: torch.Tensor  # uint8 [V, d / 2]: q[2j] in the low four bits of byte j, q[2j + 1] in the high four
    scales: torch.Tensor  # f32 / bf16 / f16 [V, ceil(d / group)]
    zeros: Optional[torch.Tensor] = None  # uint8 [V, ceil(d / group)] in 0..15; None: 8 everywhere
    group: int = 128  # weights per scale: 32, 64 or 128


def q4_quantize(weight: torch.Tensor, group: int = 128, zeros: bool = False,
                scale_dtype: torch.dtype = torch.bfloat16) -> Q4Projection:
    """A ``[V, d]`` matrix in 4 bits, each weight rounded to the nearest step
    of its group.  Without ``zeros`` the steps are -8..7 times the scale, the
    largest magnitude at 7; with them 0..15 from the group's smallest to its
    largest value (0 always among them).  A weight that is not finite, or a
    group whose scale is past ``scale_dtype``'s largest number, is refused.
    Done once, where the weights are laid out; any device."""
    if weight.dim() != 2 or group not in (32, 64, 128):
        raise ValueError("weight must be [V, d], group 32, 64 or 128")
    if weight.shape[1] % 32:
        raise ValueError("d must be a multiple of 32")
    if scale_dtype not in _DTYPES:
        raise ValueError("scale_dtype must be float32, bfloat16 or float16")
    V, d = weight.shape
    G = -(-d // group)
    w = torch.nn.functional.pad(weight.float(), (0, G * group - d)).view(V, G, group)
    if zeros:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scale = ((hi - lo) / 15).to(scale_dtype)
        step = torch.where(scale > 0, scale.float(), 1.0)
        z = (-lo / step).round().clamp(0, 15)
    else:
        scale = (w.abs().amax(2) / 7).to(scale_dtype)
        step = torch.where(scale > 0, scale.float(), 1.0)
        z = torch.full_like(step, 8.0)
    if not bool(torch.isfinite(scale).all()):  # (an infinite scale would make every weight of its group NaN)
        raise ValueError(f"a group of weights is not finite, or too large for scales in {scale_dtype}")
    q = ((w / step[..., None]).round() + z[..., None]).clamp(0, 15).to(torch.uint8).view(V, G * group)[:, :d]
    packed = q[:, 0::2] | (q[:, 1::2] << 4)
    return Q4Projection(packed.contiguous(), scale, z.to(torch.uint8) if zeros else None, group)


def _q4_arg(p: Q4Projection, dev: torch.device):
    """(V, d, sv_q4_proj, tensors it points into) of a checked projection."""
    packed, scales, zeros, group = p
    if packed.dim() != 2 or packed.dtype != torch.uint8:
        raise ValueError("packed must be uint8 [V, d / 2]")
    V, d = packed.shape
    d *= 2
    if V >= 2**31 or d >= 2**31:
        raise ValueError("a projection's sizes must be below 2^31")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    shape = (V, -(-d // group))
    code = _DTYPES.get(scales.dtype)
    if code is None or scales.shape != shape:
        raise ValueError(f"scales must be f32, bf16 or f16 {list(shape)}")
    if zeros is not None:
        if zeros.dtype != torch.uint8 or zeros.shape != shape:
            raise ValueError(f"zeros must be uint8 {list(shape)}")
        zeros = _like(zeros, dev, torch.uint8)
    packed, scales = _like(packed, dev, torch.uint8), _like(scales, dev, scales.dtype)
    arg = _lib.Q4Proj(packed.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(), code, group)
    return V, d, arg, (packed, scales, zeros)


def _q4_states(x: torch.Tensor, d: int) -> torch.Tensor:
    if x.dtype != torch.bfloat16 and x.dtype != torch.float16:
        raise ValueError("states must be bfloat16 or float16")
    if x.shape[-1] != d:
        raise ValueError("states and projection must have the same last dimension")
    return (x if x.dim() == 2 else x.reshape(-1, d)).contiguous()


def lm_head_logits(states: torch.Tensor, proj: Union[torch.Tensor, Q4Projection], out: Optional[torch.Tensor] = None,
                   err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``states [rows, d] . proj[V, d]^T`` in fp32 on the tensor cores
    (include/sv_lm_head.h).  ``proj``: bf16 ``[V, d]``, or a ``Q4Projection``
    (include/sv_lm_head_q4.h; the states may then be f16 too).  ``out``:
    optional f32 ``[rows, >= V]`` device tensor with unit stride along V;
    ``err``: optional int32 ``[1]`` device word that receives bit 0 if a
    device wait gave up."""
    if isinstance(proj, Q4Projection):
        if not states.is_cuda:
            return lm_head_logits(_Marshal(states).dev(states), proj, out, err).cpu()
        dev = states.device
        V, d, arg, keep = _q4_arg(proj, dev)
        h = _q4_states(states, d)
        rows = h.shape[0]
        if out is None:
            out = torch.empty((rows, (V + 3) // 4 * 4), dtype=torch.float32, device=dev)
            if V % 4:  # rows start on 16-byte boundaries
                out = out[:, :V]
        elif (out.device != dev or out.dtype != torch.float32 or out.dim() != 2 or out.shape[0] < rows
              or out.shape[1] < V or (out.stride(1) != 1 and V > 1) or (out.stride(0) < V and rows > 1)):
            raise ValueError("out must be f32 [rows, >= V] on the states' device with unit stride along V, "
                             "its rows apart from one another")
        if err is not None and (err.device != dev or err.dtype != torch.int32 or err.numel() < 1):
            raise ValueError("err must be an int32 word on the states' device")
        _launch(dev, _lib.load().sv_lm_head_q4_logits, h.data_ptr(), _DTYPES[h.dtype], arg, rows, V, d,
                out.data_ptr(), max(out.stride(0), V), None if err is None else err.data_ptr())
        return out
    m = _Marshal(states)
    h = _bf16_rows(states, m)
    w = _bf16_rows(proj, m)
    if h.shape[1] != w.shape[1]:
        raise ValueError("states and projection must have the same last dimension")
    rows, V = h.shape[0], w.shape[0]
    if out is None:
        out = torch.empty(rows, (V + 3) // 4 * 4, dtype=torch.float32, device=m.device)[:, :V]
    lib = _lib.load()
    with torch.cuda.device(m.device):
        _check(lib.sv_lm_head_logits(_p(h), _p(w), rows, V, h.shape[1], _p(out), out.stride(0), _p(err),
                                     m.stream()))
    return out.cpu() if m.host else out


class LMHeadResult(NamedTuple):
    n_accepted: torch.Tensor
    next_token: torch.Tensor
    status: torch.Tensor
    target_logits: Optional[torch.Tensor]  # f32 [target rows, V] the verification read (views of the workspace)
    draft_logits: Optional[torch.Tensor]


def lm_head_workspace(batch: int, sum_k: int, vocab: int, device=None) -> torch.Tensor:
    """A workspace for sv_lm_head_verify of this size (uninitialised bytes)."""
    n = int(_lib.load().sv_lm_head_workspace_size(batch, sum_k, vocab))
    return torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda", torch.cuda.current_device()))


def lm_head_verify(target_states: torch.Tensor, draft_states: torch.Tensor,
                   proj: Union[torch.Tensor, Q4Projection],
                   temperature: torch.Tensor, draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                   cu_k: Optional[torch.Tensor] = None, k: Optional[int] = None, flags: int = 0,
                   workspace: Optional[torch.Tensor] = None) -> LMHeadResult:
    """Verification from hidden states (include/sv_lm_head.h): the target and
    draft positions' logits through the one projection ``proj`` (bf16
    ``[V, d]``, or a ``Q4Projection``, include/sv_lm_head_q4.h, whose states may
    be f16 too), then the mixed greedy / sampled verification of accept_from_logits.
    Returns the verification results and, for device inputs, the fp32 logits
    it read (views of the workspace, valid until it is reused)."""
    m = _Marshal(target_states)
    q4 = isinstance(proj, Q4Projection)
    if q4:
        V, d, arg, keep = _q4_arg(proj, m.device)
        ht, hd = _q4_states(m.dev(target_states), d), m.dev(draft_states)
        hd = _q4_states(hd, d) if hd.numel() else hd
        if hd.dtype != ht.dtype:
            raise ValueError("target and draft states must have the same dtype")
    else:
        ht, hd, w = _bf16_rows(target_states, m), _bf16_rows(draft_states, m), _bf16_rows(proj, m)
        V, d = w.shape
        if ht.shape[1] != d or (hd.numel() and hd.shape[1] != d):
            raise ValueError("states and projection must have the same last dimension")
    tok = m.dev(draft_tokens.reshape(-1), torch.int32)
    u = m.dev(uniforms.reshape(-1), torch.float32)
    T = m.dev(temperature.reshape(-1), torch.float32)
    cu = m.dev(cu_k, torch.int32)
    B, K, sum_k = _layout(ht.shape[0], tok, cu, k)
    lib = _lib.load()
    need = int(lib.sv_lm_head_workspace_size(B, sum_k, V))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = lm_head_workspace(B, sum_k, V, m.device)
    n, nxt, st = m.outputs(B)
    with torch.cuda.device(m.device):
        tail = (d, _p(T), _p(tok), _p(u), _p(cu), B, K, sum_k, V, _p(n), _p(nxt), _p(st), _p(workspace),
                workspace.numel() * workspace.element_size(), flags, m.stream())
        if q4:
            _check(lib.sv_lm_head_q4_verify(_p(ht), _p(hd), _DTYPES[ht.dtype], arg, *tail))
        else:
            _check(lib.sv_lm_head_verify(_p(ht), _p(hd), _p(w), *tail))
    res = m.finish(VerifyResult(n, nxt, st))
    lt = ld = None
    if not m.host:
        ldv = (V + 3) // 4 * 4
        f = workspace[256:256 + (2 * sum_k + B) * ldv * 4].view(torch.float32).view(-1, ldv)
        lt, ld = f[:sum_k + B, :V], f[sum_k + B:, :V]
    return LMHeadResult(res.n_accepted, res.next_token, res.status, lt, ld)


def lm_head_verify_static(target_states: torch.Tensor, draft_states: torch.Tensor, proj: torch.Tensor,
                          temperature: torch.Tensor, draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                          cu_k: Optional[torch.Tensor] = None, k: Optional[int] = None,
                          flags: int = 0) -> VerifyResult:
    """lm_head_verify on the library's own fixed device scratch
    (sv_lm_head_verify_static, include/sv_lm_head.h): no workspace is
    allocated or passed.  Calls larger than the scratch raise SVError; calls
    that overlap on the GPU race on the scratch (issue them on one stream)."""
    m = _Marshal(target_states)
    ht = _bf16_rows(target_states, m)
    hd = _bf16_rows(draft_states, m)
    w = _bf16_rows(proj, m)
    tok = m.dev(draft_tokens.reshape(-1), torch.int32)
    u = m.dev(uniforms.reshape(-1), torch.float32)
    T = m.dev(temperature.reshape(-1), torch.float32)
    cu = m.dev(cu_k, torch.int32)
    B, K, sum_k = _layout(ht.shape[0], tok, cu, k)
    V, d = w.shape
    n, nxt, st = m.outputs(B)
    lib = _lib.load()
    with torch.cuda.device(m.device):
        _check(lib.sv_lm_head_verify_static(_p(ht), _p(hd), _p(w), d, _p(T), _p(tok), _p(u), _p(cu), B, K, sum_k,
                                            V, _p(n), _p(nxt), _p(st), flags, m.stream()))
    return m.finish(VerifyResult(n, nxt, st))


# ---------------------------------------------------------------- penalties (in place)

def apply_penalties(target_logits: torch.Tensor, draft_logits: torch.Tensor, draft_tokens: torch.Tensor,
                    repetition: torch.Tensor, frequency: torch.Tensor, presence: torch.Tensor,
                    hist_offsets: Optional[torch.Tensor] = None, hist_tokens: Optional[torch.Tensor] = None,
                    cu_k: Optional[torch.Tensor] = None, k: Optional[int] = None) -> torch.Tensor:
    """Repetition / frequency / presence penalties on the raw logits rows, in
    place (include/sv_penalties.h): row i of a sequence sees its history plus
    the drafts before position i.  The rows must be CUDA tensors with unit
    stride along V.  Returns the per-sequence status (int32 [B])."""
    for x in (target_logits, draft_logits):
        if x.device.type != "cuda" or x.stride(-1) != 1:
            raise ValueError("the rows must be CUDA tensors with unit stride along V (modified in place)")
    dev = target_logits.device
    tg = target_logits.reshape(-1, target_logits.shape[-1])
    dr = draft_logits.reshape(-1, draft_logits.shape[-1])
    if tg.data_ptr() != target_logits.data_ptr() or dr.data_ptr() != draft_logits.data_ptr():
        raise ValueError("the rows must be addressable as [rows, V] in place")
    if dr.numel() and dr.stride(0) != tg.stride(0):
        raise ValueError("target and draft rows must have the same row stride")
    m = _Marshal(target_logits)
    tok = m.dev(draft_tokens.reshape(-1), torch.int32)
    cu = m.dev(cu_k, torch.int32)
    B, K, sum_k = _layout(tg.shape[0], tok, cu, k)
    f = lambda x: m.dev(x.reshape(-1), torch.float32)
    r, fr, pr = f(repetition), f(frequency), f(presence)
    ho = m.dev(hist_offsets, torch.int32)
    ht = m.dev(hist_tokens, torch.int32)
    st = torch.empty(B, dtype=torch.int32, device=dev)
    lib = _lib.load()
    with torch.cuda.device(dev):
        _check(lib.sv_apply_penalties(_p(tg), _p(dr), _DTYPES[tg.dtype], tg.stride(0), _p(ho), _p(ht),
                                      0 if ht is None else ht.numel(), _p(tok), _p(cu), B, K, sum_k, tg.shape[1],
                                      _p(r), _p(fr), _p(pr), _p(st), m.stream()))
    return st


# ---------------------------------------------------------------- beam search

class BeamCandidates(NamedTuple):
    scores: torch.Tensor  # f32 [B, n]: accumulated log-probabilities, best first; -inf where there is none
    parents: torch.Tensor  # int32 [B, n]: the beam each candidate extends; -1 where there is none
    tokens: torch.Tensor  # int32 [B, n]; -1 where there is none
    status: torch.Tensor  # int32 [B]; SEQ_BAD_VALUE or 0


@functools.lru_cache(maxsize=256)
def _select_bytes(batch: int, beams: int, vocab: int, n: int) -> int:
    return int(_lib.load().sv_beam_select_workspace_size(batch, beams, vocab, n))


def _like(t: torch.Tensor, dev: torch.device, dtype: torch.dtype) -> torch.Tensor:
    """``t`` contiguous on ``dev`` in ``dtype`` (itself where it is)."""
    if t.dtype != dtype or t.device != dev:
        t = t.to(device=dev, dtype=dtype)
    return t.contiguous()


def beam_select_workspace(batch: int, beams: int, vocab: int, n: int, device=None) -> torch.Tensor:
    """A workspace for sv_beam_select of this size (uninitialised bytes)."""
    return torch.empty(_select_bytes(batch, beams, vocab, n), dtype=torch.uint8,
                       device=device or torch.device("cuda", torch.cuda.current_device()))


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n: Optional[int] = None,
                finished: Optional[torch.Tensor] = None, eos: int = -1,
                workspace: Optional[torch.Tensor] = None) -> BeamCandidates:
    """The ``n`` best continuations (default: as many as beams) of every
    sequence's beams (include/sv_beam.h): ``logits [B, W, V]`` (or the
    ``[B * W, V]`` rows) in f32 / bf16 / f16, ``scores [B, W]`` the beams'
    accumulated log-probabilities (-inf: a dead beam); a candidate's score is
    its beam's plus the token's log-softmax; equal ones go by the lower beam,
    then the lower token.  ``finished [B, W]``: beams that have ended offer
    only ``(eos, their score)``.  ``workspace``: optional bytes of
    ``beam_select_workspace``; calls that overlap on the GPU must not share
    one."""
    if scores.dim() != 2:
        raise ValueError("scores must be [B, W]")
    if not logits.is_cuda:
        m = _Marshal(logits)
        r = beam_select(m.dev(logits), m.dev(scores), n, m.dev(finished), eos, workspace)
        return BeamCandidates(*(x.cpu() for x in r))
    B, W = scores.shape
    dev, dtype = logits.device, _DTYPES.get(logits.dtype)
    if dtype is None:
        raise ValueError("logits must be float32, bfloat16 or float16")
    if logits.dim() == 3 and logits.shape[0] == B and logits.shape[1] == W:
        V = logits.shape[2]
        s0, stride, s2 = logits.stride()
        if (s2 != 1 and V > 1) or (s0 != W * stride and B > 1):
            logits = logits.contiguous()
            stride = V
    else:
        logits = _rows(logits)
        if logits.shape[0] != B * W:
            raise ValueError(f"logits must hold one row for each of the {B} x {W} scores (got {logits.shape[0]})")
        V, stride = logits.shape[1], logits.stride(0)
    if stride < V:  # one row, or rows that share memory
        if B * W > 1 and W * B != 0:
            logits = logits.contiguous()
        stride = V
    if finished is not None:
        if finished.shape != scores.shape:
            raise ValueError("finished must have the shape of scores")
        if finished.dtype != torch.bool:
            finished = finished != 0
        finished = _like(finished, dev, torch.bool)
    scores = _like(scores, dev, torch.float32)
    n = W if n is None else int(n)
    if max(V, W, abs(n), abs(eos)) >= 2**31:
        raise ValueError("sizes, n and eos must be below 2^31")
    lib = _lib.load()
    need = _select_bytes(B, W, V, n)
    have = 0
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous on the logits' device")
        have = workspace.numel() * workspace.element_size()
    if have < need:
        workspace, have = torch.empty(need, dtype=torch.uint8, device=dev), need
    shape = (B, n if 0 < n <= 128 else 0)  # (any other n is refused below)
    out = torch.empty(shape, dtype=torch.float32, device=dev)
    par = torch.empty(shape, dtype=torch.int32, device=dev)
    tok = torch.empty(shape, dtype=torch.int32, device=dev)
    st = torch.empty(B, dtype=torch.int32, device=dev)
    _launch(dev, lib.sv_beam_select, logits.data_ptr(), dtype, stride, scores.data_ptr(),
            None if finished is None else finished.data_ptr(), int(eos), B, W, V, n, out.data_ptr(), par.data_ptr(),
            tok.data_ptr(), st.data_ptr(), None if workspace is None else workspace.data_ptr(), have)
    return BeamCandidates(out, par, tok, st)


def _flat_stride(shape, strides, lo: int, hi: int, what: str):
    """Extent and stride (elements) of dimensions lo..hi-1 taken as one."""
    size, stride = 1, None
    for d in range(hi - 1, lo - 1, -1):
        if shape[d] == 1:
            continue
        if stride is None:
            size, stride = shape[d], strides[d]
        elif strides[d] == size * stride:
            size *= shape[d]
        else:
            raise ValueError(f"{what} are not addressable in place with one stride")
    return size, 0 if stride is None else stride


def _beam_layout(t: torch.Tensor, time_dim: Optional[int]) -> tuple:
    """The words of sv_beam_state after its pointer: four strides and sizes in
    bytes, then (segs, tokens) and (timed, 0) as pairs of 32 bits."""
    shape, strides, e = tuple(t.shape), t.stride(), t.element_size()
    dims = len(shape)
    for n, s in zip(shape, strides):
        if s == 0 and n > 1:
            raise ValueError("a state is a broadcast view (modified in place)")
    if time_dim is None:
        span, k = 1, dims  # the run of memory at the end of the shape, then segments of it
        while k > 2 and (shape[k - 1] == 1 or strides[k - 1] == span):
            span *= shape[k - 1]
            k -= 1
        if k == dims and k > 2:
            raise ValueError("a state's last dimension must have unit stride (moved in place)")
        segs, seg = _flat_stride(shape, strides, 2, k, "a state's dimensions after [B, W]")
        if segs >= 2**31:
            raise ValueError("a state has too many segments")
        return (strides[0] * e, strides[1] * e, seg * e, span * e, segs | 1 << 32, 0)
    segs, seg = _flat_stride(shape, strides, 2, time_dim, "a state's dimensions between the beams and the time")
    if max(segs, shape[time_dim]) >= 2**31:
        raise ValueError("a state has too many segments or tokens")
    span, stride = _flat_stride(shape, strides, time_dim + 1, dims, "a state's dimensions after the time")
    if (span > 1 and stride != 1) or (shape[time_dim] > 1 and strides[time_dim] != span):
        raise ValueError("a state's tokens must be contiguous: unit stride after the time, one after another along it")
    return (strides[0] * e, strides[1] * e, seg * e, span * e, segs | shape[time_dim] << 32, 1)


def beam_reorder(states: Union[torch.Tensor, Sequence[torch.Tensor]], parents: torch.Tensor,
                 lengths: Optional[torch.Tensor] = None,
                 time_dim: Union[None, int, Sequence[Optional[int]]] = None) -> torch.Tensor:
    """Moves beam states to their new slots, in place (include/sv_beam.h):
    slot ``w`` of sequence ``b`` receives what slot ``parents[b, w]`` held
    before the call; a negative parent leaves its slot as it is.  ``states``:
    one CUDA tensor ``[B, W, ...]`` or several, of any types; none may share
    memory with another, nor with ``parents`` or ``lengths``.  ``lengths [B]`` with ``time_dim`` (one dimension for
    all states, or one per state, None for a state without time): only the
    first ``lengths[b]`` positions along it are in use and move.  Returns the
    per-sequence status (int32 ``[B]``)."""
    if isinstance(states, torch.Tensor):
        states = [states]
    dims = time_dim if isinstance(time_dim, (list, tuple)) else [time_dim] * len(states)
    if not states or len(dims) != len(states):
        raise ValueError("at least one state is needed, and one time_dim for all or for each")
    if parents.dim() != 2:
        raise ValueError("parents must be [B, W]")
    B, W = parents.shape
    dev = states[0].device
    if dev.type != "cuda":
        raise ValueError("the states must be CUDA tensors (modified in place)")
    grad = torch.is_grad_enabled()
    words, seen, layout, last = [], set(), None, None
    for t, td in zip(states, dims):
        key = (t.shape, t.stride(), t.dtype, td)
        if key != last or t.device != dev:  # a layer's states are alike: one layout serves them all
            if t.device != dev or t.dim() < 2 or t.shape[0] != B or t.shape[1] != W:
                raise ValueError(f"a state must be a CUDA tensor [{B}, {W}, ...] on {dev} (got {list(t.shape)} on {t.device})")
            d = td
            if d is not None:
                d = d + t.dim() if d < 0 else d
                if not 2 <= d < t.dim():
                    raise ValueError("time_dim must be a dimension after the beams")
                if lengths is None:
                    raise ValueError("time_dim needs lengths")
            layout, last = _beam_layout(t, d), key
        if grad and t.requires_grad:
            raise ValueError("a state requires a gradient: it is modified in place")
        p = t.data_ptr()
        words.append(p)
        words.extend(layout)
        if p:
            if p in seen:
                raise ValueError("a state is listed twice")
            seen.add(p)
    parents = _like(parents, dev, torch.int32)
    if lengths is not None:
        if lengths.numel() != B:
            raise ValueError("lengths must be [B]")
        lengths = _like(lengths, dev, torch.int32)
    if parents.data_ptr() in seen or lengths is not None and lengths.data_ptr() in seen:
        raise ValueError("parents or lengths is a state too: it would move while it is read")
    st = torch.empty(B, dtype=torch.int32, device=dev)
    _launch(dev, _lib.load().sv_beam_reorder, (ctypes.c_int64 * len(words))(*words), len(states), parents.data_ptr(),
            None if lengths is None else lengths.data_ptr(), B, W, st.data_ptr())
    return st


# ---------------------------------------------------------------- trees of drafted tokens

class TreeResult(NamedTuple):
    n_accepted: torch.Tensor  # int32 [B]: nodes accepted after node 0
    next_token: torch.Tensor  # int32 [B]: the target's token after the last of them; -1 where there is none
    path: torch.Tensor  # int32 [B, n]: node 0, then the accepted nodes, then -1
    status: torch.Tensor  # int32 [B]; OR of SEQ_* bits


class TreeAttention(NamedTuple):
    out: torch.Tensor  # [total, Hq, D], the queries' type
    lse: torch.Tensor  # f32 [total, Hq]: natural logarithm of each row's sum of exponentials
    status: torch.Tensor  # int32 [B]; SEQ_BAD_LAYOUT or 0


def _words(t: Optional[torch.Tensor], dev: torch.device, what: str) -> Optional[torch.Tensor]:
    """``t`` as contiguous int32 on ``dev``; numbers that do not fit become the
    type's ends, which are out of every range too."""
    if t is None:
        return None
    if t.dtype is not torch.int32:
        if t.is_floating_point() or t.is_complex() or t.dtype == torch.bool:
            raise ValueError(f"{what} must be whole numbers")
        if t.dtype.itemsize >= 4:
            wide = t.to(torch.int64)
            if t.dtype is torch.uint64:
                wide = torch.where(wide < 0, 2**31 - 1, wide)  # (2^63 and above)
            t = wide.clamp(-2**31, 2**31 - 1)
        t = t.to(torch.int32)
    if t.device != dev:
        t = t.to(dev)
    return t.contiguous()


def _tree_layout(total: int, B: Optional[int], cu_nodes: Optional[torch.Tensor], n: Optional[int], what: str):
    """(B, n) of ``total`` rows of nodes."""
    if cu_nodes is not None:
        if n is None:
            raise ValueError("n (the most nodes of a sequence) is required with cu_nodes")
        if cu_nodes.numel() < 1 or B is not None and cu_nodes.numel() != B + 1:
            raise ValueError("cu_nodes must be [B + 1]")
        return cu_nodes.numel() - 1, int(n)
    if n is None:
        if not B:
            raise ValueError("n (the nodes of a sequence) is required")
        n = total // B
    n = int(n)
    if B is None:
        B = total // n if n > 0 else 0
    if n < 0 or B * n != total:
        raise ValueError(f"without cu_nodes, {what} must hold n rows for every sequence")
    return B, n


def _verify_tree(rows, choices, tokens, parents, cu_nodes, n) -> TreeResult:
    ref = rows if choices is None else choices
    if not ref.is_cuda:
        m = _Marshal(ref)
        r = _verify_tree(m.dev(rows), m.dev(choices), m.dev(tokens), m.dev(parents), m.dev(cu_nodes), n)
        return TreeResult(*(x.cpu() for x in r))
    dev = ref.device
    B = None
    if tokens.dim() == 2:
        B = tokens.shape[0]
    if n is None and tokens.dim() == 2:
        n = tokens.shape[1]
    total = tokens.numel()
    B, n = _tree_layout(total, B, cu_nodes, n, "tokens")
    if max(total, n) >= 2**31:
        raise ValueError("sizes must be below 2^31")
    tokens, cu = _words(tokens, dev, "tokens"), _words(cu_nodes, dev, "cu_nodes")
    if parents is not None:
        if parents.numel() != total:
            raise ValueError("parents must have one entry for each token")
        parents = _words(parents, dev, "parents")
    out = torch.empty((3, B), dtype=torch.int32, device=dev)
    path = torch.empty((B, max(n, 0)), dtype=torch.int32, device=dev)
    p = out.data_ptr()
    where = (p, p + 4 * B, path.data_ptr(), p + 8 * B)  # n_accepted, next_token, path, status
    lib = _lib.load()
    if choices is None:
        dtype = _DTYPES.get(rows.dtype)
        if dtype is None:
            raise ValueError("target must be float32, bfloat16 or float16")
        if rows.dim() != 3 and rows.dim() != 2:
            raise ValueError("target must be [total, V] or [B, n, V]")
        rows = _rows(rows)
        V, stride = rows.shape[1], rows.stride(0)
        if rows.shape[0] != total:
            raise ValueError(f"target must hold one row for each of the {total} tokens (got {rows.shape[0]})")
        if V >= 2**31:
            raise ValueError("sizes must be below 2^31")
        if stride < V and total > 1:
            rows, stride = rows.contiguous(), V
        _launch(dev, lib.sv_verify_tree_greedy, rows.data_ptr(), dtype, stride, tokens.data_ptr(), _p(parents), _p(cu),
                B, n, total, V, *where)
    else:
        if choices.numel() != total:
            raise ValueError("choices must have one entry for each token")
        choices = _words(choices, dev, "choices")
        _launch(dev, lib.sv_verify_tree, choices.data_ptr(), tokens.data_ptr(), _p(parents), _p(cu), B, n, total, *where)
    return TreeResult(out[0], out[1], path, out[2])


def verify_tree_greedy(target: torch.Tensor, tokens: torch.Tensor, parents: Optional[torch.Tensor] = None,
                       cu_nodes: Optional[torch.Tensor] = None, n: Optional[int] = None) -> TreeResult:
    """Greedy verification of a drafted tree (include/sv_tree.h): from node 0 of
    every sequence, whose children's tokens follow the target's argmax the
    furthest.  ``target [total, V]`` (or ``[B, n, V]``): the rows after each
    node, probabilities or logits, f32 / bf16 / f16.  ``tokens`` and
    ``parents``, ``[total]`` or ``[B, n]``: a node's token (node 0's is not
    looked at) and the earlier node it continues, -1 for none; without
    ``parents`` every node continues the one before.  ``cu_nodes [B + 1]`` with
    ``n`` (the most nodes of a sequence): ragged trees.  At most 256 nodes each."""
    return _verify_tree(target, None, tokens, parents, cu_nodes, n)


def verify_tree(choices: torch.Tensor, tokens: torch.Tensor, parents: Optional[torch.Tensor] = None,
                cu_nodes: Optional[torch.Tensor] = None, n: Optional[int] = None) -> TreeResult:
    """verify_tree_greedy for choices that have been drawn: ``choices`` (int32,
    one per node) is the target's token after it.  For sampling they come from
    ``accept_from_logits`` on the nodes' rows without drafts (its
    ``next_token``); what is emitted then follows the target's distribution
    whatever the tree holds."""
    return _verify_tree(None, choices, tokens, parents, cu_nodes, n)


_ATTENTION = struct.Struct("37q")  # sv_tree_attn (include/sv_tree.h)


@functools.lru_cache(maxsize=64)
def _attention_bytes(dim: int) -> int:
    return int(_lib.load().sv_tree_attention_workspace_size(dim))


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """``t [., H, D]`` itself where its last dimension has unit stride and the
    others, and its address, are multiples of 16 bytes, none broadcast; else a
    copy."""
    s = t.stride()
    if ((s[2] != 1 and t.shape[2] > 1) or s[0] % 8 or s[1] % 8 or t.data_ptr() % 16
            or s[0] == 0 and t.shape[0] > 1 or s[1] == 0 and t.shape[1] > 1):
        t = torch.empty(t.shape, dtype=t.dtype, device=t.device).copy_(t)
    return t


def tree_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   table: torch.Tensor, lengths: torch.Tensor, parents: Optional[torch.Tensor] = None,
                   cu_nodes: Optional[torch.Tensor] = None, n: Optional[int] = None, scale: Optional[float] = None,
                   out: Optional[torch.Tensor] = None, flags: int = 0) -> TreeAttention:
    """Attention of drafted nodes over their sequence's cached tokens and their
    own ancestors (include/sv_tree.h).  ``q [total, Hq, D]``, ``k``, ``v
    [total, Hkv, D]`` (or ``[B, n, H, D]``): the nodes' own; ``k_cache``,
    ``v_cache [pages, page_size, Hkv, D]`` with ``table [B, max_pages]`` and
    ``lengths [B]``: token t of sequence b is in page ``table[b, t //
    page_size]``.  All in bf16 or all in f16; ``q``, ``k``, ``v`` views of any
    strides (copied where the kernel cannot take them), the caches no broadcast
    views.  ``parents``, ``cu_nodes``, ``n``
    as ``verify_tree_greedy`` takes them (without ``parents`` a chain, so one
    token per sequence is plain decoding); at most 256 nodes per sequence.
    ``scale``: default ``D ** -0.5``.  ``out``: optional tensor for the result,
    sharing no memory with an input; rows past the last sequence are left as they
    are.  ``flags``:
    FLAG_EXPIRE_EXCHANGE is a testing aid."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("q must be a CUDA tensor (the caches stay where they are)")
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad
                                    or k_cache.requires_grad or v_cache.requires_grad):
        raise ValueError("tree_attention has no backward pass: call it under torch.no_grad()")
    dtype = _DTYPES.get(q.dtype)
    if dtype is None or dtype == _lib.SV_F32:
        raise ValueError("q must be bfloat16 or float16")
    kind = q.dtype
    if not (k.dtype == v.dtype == k_cache.dtype == v_cache.dtype == kind
            and k.device == v.device == k_cache.device == v_cache.device == dev):
        raise ValueError("k, v, k_cache and v_cache must have the type and device of q")
    if q.dim() == 4 and k.dim() == 4 and v.dim() == 4 and cu_nodes is None:
        if n is None:
            n = q.shape[1]
        q, k, v = q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1)
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("q must be [total, Hq, D], k and v [total, Hkv, D]")
    total, Hq, D = q.shape
    Hkv = k.shape[1]
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or k_cache.shape[2] != Hkv or k_cache.shape[3] != D:
        raise ValueError(f"the caches must be [pages, page_size, {Hkv}, {D}]")
    if table.dim() != 2 or table.dtype != torch.int32 or table.device != dev or table.stride(1) != 1 and table.shape[1] > 1:
        raise ValueError("table must be int32 [B, max_pages] on q's device with unit stride along a row")
    B = table.shape[0]
    if lengths.numel() != B:
        raise ValueError("lengths must be [B]")
    _, n = _tree_layout(total, B, cu_nodes, n, "q")
    if max(total, abs(n), Hq) >= 2**31:
        raise ValueError("sizes must be below 2^31")
    lengths, cu = _words(lengths, dev, "lengths"), _words(cu_nodes, dev, "cu_nodes")
    if parents is not None:
        if parents.numel() != total:
            raise ValueError("parents must have one entry for each row of q")
        parents = _words(parents, dev, "parents")
    q, k, v = _aligned(q), _aligned(k), _aligned(v)
    kc, vc = k_cache.stride(), v_cache.stride()
    kp, vp = k_cache.data_ptr(), v_cache.data_ptr()
    if (kc[3] != 1 or vc[3] != 1) and D > 1 or (kc[0] | kc[1] | kc[2] | vc[0] | vc[1] | vc[2]) % 8 or (kp | vp) % 16:
        raise ValueError("the caches must have unit stride along the head dimension, their addresses and other strides multiples of 16 bytes")
    if 0 in kc or 0 in vc:
        for s in (kc, vc):
            if any(x == 0 and size > 1 for x, size in zip(s, k_cache.shape)):
                raise ValueError("the caches must be no broadcast views (one key head serves several query heads as it is)")
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty((total, Hq, D), dtype=kind, device=dev)
    elif (out.shape[0] < total or out.shape[1:] != q.shape[1:] or out.dtype != q.dtype or out.device != dev or out.stride(2) != 1
          or out.stride(0) % 8 or out.stride(1) % 8 or out.data_ptr() % 16):
        raise ValueError("out must be like q with at least its rows, its address and strides multiples of 16 bytes")
    elif total and out.data_ptr() in (q.data_ptr(), k.data_ptr(), v.data_ptr(), kp, vp):
        raise ValueError("out is an input too: it would change while it is read")
    lse = torch.empty((total, Hq), dtype=torch.float32, device=dev)
    status = torch.empty(B, dtype=torch.int32, device=dev)
    need = _attention_bytes(D)
    workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
    words = _ATTENTION.pack(dtype, Hq, Hkv, D, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
             kp, vp, kc[0], kc[1], kc[2], vc[0], vc[1], vc[2], k_cache.shape[0],
             k_cache.shape[1], table.data_ptr(), table.stride(0), table.shape[1], lengths.data_ptr(), _p(parents) or 0,
             _p(cu) or 0, B, n, total, out.data_ptr(), os[0], os[1], lse.data_ptr(), status.data_ptr())
    _launch(dev, _lib.load().sv_tree_attention_flagged, words,
            D ** -0.5 if scale is None else float(scale), flags, workspace.data_ptr(), need)
    return TreeAttention(out, lse, status)


# ---------------------------------------------------------------- paged caches

class PagedCache(NamedTuple):
    """A model's key / value caches in pages (include/sv_cache.h).  One page
    table serves the pools of all layers; ``paged_cache`` makes an empty one."""
    keys: Sequence[torch.Tensor]  # per layer [pages, page_size, Hkv, D]
    values: Sequence[torch.Tensor]
    table: torch.Tensor  # int32 [..., max_pages], a row per sequence; entries past its length mean nothing
    lengths: torch.Tensor  # int32 [...]: tokens of each sequence
    refs: torch.Tensor  # int32 [pages]: table entries in use that name each page; 0: free


def paged_cache(layers: int, pages: int, page_size: int, heads: int, dim: int, sequences: Union[int, Sequence[int]],
                max_pages: int, dtype: torch.dtype = torch.bfloat16, device=None) -> PagedCache:
    """An empty cache of ``layers`` layers; ``sequences``: their number, or
    ``(groups, width)`` for the groups that ``cache_fork`` takes (beams).  The
    pools are not initialised: nothing past a sequence's length is ever used."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    shape = (sequences,) if isinstance(sequences, int) else tuple(sequences)
    pool = lambda: [torch.empty(pages, page_size, heads, dim, dtype=dtype, device=dev) for _ in range(layers)]
    word = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    return PagedCache(pool(), pool(), word(*shape, max_pages), word(*shape), word(pages))


_PAGES = struct.Struct("8q")  # sv_cache_pages (include/sv_cache.h)
_ROWS = struct.Struct("7q")  # sv_cache_rows
_kind = attrgetter("dtype")
_shape = attrgetter("shape")


def _pages_arg(c: PagedCache) -> tuple:
    """(words of sv_cache_pages, sequences, device) of a checked cache."""
    table, lengths, refs, pool = c.table, c.lengths, c.refs, c.keys[0] if len(c.keys) else None
    at, i32 = table.get_device(), torch.int32
    if at < 0:
        raise ValueError("the cache must be CUDA tensors (modified in place)")
    if (table.dtype is not i32 or lengths.dtype is not i32 or refs.dtype is not i32 or lengths.get_device() != at
            or refs.get_device() != at):
        raise ValueError("table, lengths and refs must be int32 on one device")
    shape, sequences, pages = table.shape, lengths.numel(), refs.numel()
    width = shape[-1]
    if lengths.shape != shape[:-1] or not lengths.is_contiguous() or refs.dim() != 1 or not refs.is_contiguous():
        raise ValueError("lengths must be contiguous with one entry per table row, refs contiguous [pages]")
    stride = width
    if not table.is_contiguous():
        if table.dim() != 2 or table.stride(1) != 1 or table.stride(0) < width:
            raise ValueError("table must be contiguous, or [sequences, max_pages] with rows apart from one another")
        stride = table.stride(0)
    if pool is None or len(c.values) != len(c.keys):
        raise ValueError("the cache needs at least one layer, keys and values of each")
    if pool.dim() != 4 or pool.shape[0] != pages or pool.shape[1] < 1:
        raise ValueError("the pools must be [pages, page_size, Hkv, D], one page for each entry of refs")
    page = pool.shape[1]
    if max(sequences, pages, page, width) >= 2**31:
        raise ValueError("sizes must be below 2^31")
    words = _PAGES.pack(table.data_ptr(), stride, width, lengths.data_ptr(), refs.data_ptr(), pages, page, sequences)
    return words, sequences, table.device


@functools.lru_cache(maxsize=256)
def _append_bytes(sequences: int, n: int, pages: int, page: int) -> int:
    return int(_lib.load().sv_cache_append_workspace_size(sequences, n, pages, page))


def cache_append(cache: PagedCache, keys: Union[torch.Tensor, Sequence[torch.Tensor]],
                 values: Union[torch.Tensor, Sequence[torch.Tensor]], counts: Optional[torch.Tensor] = None,
                 path: Optional[torch.Tensor] = None, cu_nodes: Optional[torch.Tensor] = None,
                 n: Optional[int] = None) -> torch.Tensor:
    """Appends tokens to every sequence of a paged cache, in place
    (include/sv_cache.h): ``keys[layer]``, ``values[layer]`` hold the rows
    ``[total, Hkv, D]`` (or ``[sequences, n, Hkv, D]``) of the new tokens, as
    ``tree_attention`` took them; the first ``counts`` of ``path`` (``path
    [sequences, n]`` and ``n_accepted + 1`` of a verification) go behind the
    sequence; without ``path`` its first ``counts`` rows, without ``counts`` all.
    New pages are the lowest free ones, in sequence order; a shared last page is
    copied first.  No new row may lie in a pool.  ``lengths`` grow by ``counts``.  Returns the per-sequence
    status: SEQ_NO_PAGES where pages or table entries do not suffice,
    SEQ_BAD_LAYOUT; such a sequence is left as it is."""
    if isinstance(keys, torch.Tensor):
        keys = [keys]
    if isinstance(values, torch.Tensor):
        values = [values]
    pages, S, dev = _pages_arg(cache)
    layers = len(cache.keys)
    if len(keys) != layers or len(values) != layers:
        raise ValueError(f"keys and values must hold rows for each of the {layers} layers")
    pool = cache.keys[0]
    P, page, H, D = pool.shape
    strides, dtype = pool.stride(), pool.dtype
    if strides[3] != 1 and D > 1 or any(s == 0 and n > 1 for n, s in zip(pool.shape, strides)):
        raise ValueError("the pools must have unit stride along the head dimension, and be no broadcast views")
    first = keys[0]
    if first.dim() == 4 and cu_nodes is None:
        if n is None:
            n = first.shape[1]
        total = first.shape[0] * first.shape[1]
    else:
        total = first.shape[0]
    if n is None and path is not None:
        n = path.shape[-1]
    _, n = _tree_layout(total, S, cu_nodes, n, "keys")
    # (the same few questions to every tensor of every layer: asked in C, the answers gathered in sets)
    held, new = (*cache.keys, *cache.values), [*keys, *values]
    kinds = {dtype}
    compact = torch.Tensor.is_contiguous  # (a cheaper question than the strides)
    if (set(map(_shape, held)) != {pool.shape}
            or not (pool.numel() and all(map(compact, held))) and set(map(torch.Tensor.stride, held)) != {strides}
            or set(map(_kind, held)) != kinds or set(map(torch.Tensor.get_device, held)) != {dev.index}):
        raise ValueError("the pools must be alike: shape, strides, type, device")
    if first.dim() == 4 and cu_nodes is None:
        new = [x.flatten(0, 1) for x in new]
    if (set(map(_shape, new)) != {(total, H, D)} or set(map(_kind, new)) != kinds
            or set(map(torch.Tensor.get_device, new)) != {dev.index}):
        raise ValueError(f"new rows must be [{total}, {H}, {D}] of the pools' type, on their device")
    if torch.is_grad_enabled() and (pool.requires_grad or held[-1].requires_grad or new[0].requires_grad or new[-1].requires_grad):
        raise ValueError("the cache is modified in place: no gradients")  # (layers are alike)
    if not (total and all(map(compact, new))) and (len(set(map(torch.Tensor.stride, new))) > 1
                                                   or new[0].stride(2) != 1 and D > 1):
        new = [x.contiguous() for x in new]  # (one layout serves all)
        new = [x if x.stride() == new[0].stride() else torch.empty_like(new[0]).copy_(x) for x in new]
    layout = new[0].stride()
    pools, rows = list(map(torch.Tensor.data_ptr, held)), list(map(torch.Tensor.data_ptr, new))
    seen = set(pools)
    if len(seen) != len(pools):
        raise ValueError("a pool is listed twice")
    if not seen.isdisjoint(rows) and total:
        raise ValueError("new rows are a pool too: they would change while they are read")
    counts, path, cu = _words(counts, dev, "counts"), _words(path, dev, "path"), _words(cu_nodes, dev, "cu_nodes")
    if counts is not None and counts.numel() != S:
        raise ValueError("counts must have one entry per sequence")
    if path is not None and path.numel() != S * n:
        raise ValueError(f"path must be [{S}, {n}]")
    if max(total, n) >= 2**31:
        raise ValueError("sizes must be below 2^31")
    e = pool.element_size()
    status = torch.empty_like(cache.lengths)
    need = _append_bytes(S, n, P, page)
    workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    where = _ROWS.pack(strides[0] * e, strides[1] * e, strides[2] * e, layout[0] * e, layout[1] * e, H, D * e)
    addresses = struct.Struct(f"{len(pools)}q")
    _launch(dev, _lib.load().sv_cache_append, pages, where, addresses.pack(*pools), addresses.pack(*rows), len(pools),
            _p(counts), _p(path), _p(cu), n, total, status.data_ptr(), workspace.data_ptr(), need)
    return status


def cache_truncate(cache: PagedCache, lengths: torch.Tensor) -> torch.Tensor:
    """Takes every sequence of a paged cache back to ``lengths`` tokens, in
    place (include/sv_cache.h): the pages past them are given up; 0 frees the
    sequence.  Returns the per-sequence status: SEQ_BAD_LAYOUT for a length
    below 0 or above the sequence's (it is left as it is)."""
    pages, S, dev = _pages_arg(cache)
    if lengths.numel() != S:
        raise ValueError("lengths must have one entry per sequence")
    to = _words(lengths, dev, "lengths")
    status = torch.empty_like(cache.lengths)
    _launch(dev, _lib.load().sv_cache_truncate, pages, to.data_ptr(), status.data_ptr())
    return status


def cache_fork(cache: PagedCache, parents: torch.Tensor) -> torch.Tensor:
    """Lets sequences share others' pages, in place (include/sv_cache.h): slot
    ``w`` of group ``g`` takes what slot ``parents[g, w]`` of the group held
    before the call (its pages, shared, and its length) and gives up its own; a
    negative parent, or ``w``, leaves it as it is.  ``parents [groups, width]``,
    or ``[sequences]`` for one group of all; at most 1024 slots per group.
    Nothing is copied until a shared last page is appended to.  Returns the
    status per group (int32 ``[groups]``)."""
    pages, S, dev = _pages_arg(cache)
    if parents.dim() not in (1, 2) or parents.numel() != S:
        raise ValueError("parents must be [groups, width] or [sequences], one entry per sequence")
    width = parents.shape[-1]
    par = _words(parents, dev, "parents")
    if par.data_ptr() == cache.lengths.data_ptr() and S:
        raise ValueError("parents is the cache's lengths: it would change while it is read")
    status = torch.empty(S // width if width else 0, dtype=torch.int32, device=dev)
    if S:
        _launch(dev, _lib.load().sv_cache_fork, pages, par.data_ptr(), width, status.data_ptr())
    return status
