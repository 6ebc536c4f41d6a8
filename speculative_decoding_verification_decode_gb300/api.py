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
