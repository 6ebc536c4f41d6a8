// Host side of the LM head on a projection in 4 bits
// (include/sv_lm_head_q4.h); the kernel is in sv_lm_head_q4.cuh.
#include "../../include/sv_lm_head.h"
#include "sv_lm_head_q4.cuh"

namespace svq {

sv_status start_bf16(const Args& g, int n, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st);
sv_status start_few_bf16(const Args& g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st);
sv_status start_few_f16(const Args& g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st);
sv_status start_f16(const Args& g, int n, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st);

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Host checks of a projection against the call's sizes.
sv_status check(const sv_q4_proj* p, sv_dtype dtype, int vocab, int dim) {
  if (!p) return svh::fail(SV_ERR_ARG, "proj is NULL");
  if (dtype != SV_BF16 && dtype != SV_F16)
    return svh::fail(SV_ERR_ARG, "states must be SV_BF16 or SV_F16 (dtype %d)", static_cast<int>(dtype));
  if (p->scale_dtype != SV_F32 && p->scale_dtype != SV_BF16 && p->scale_dtype != SV_F16)
    return svh::fail(SV_ERR_ARG, "unknown scale dtype %d", static_cast<int>(p->scale_dtype));
  if (p->group != 32 && p->group != 64 && p->group != 128)
    return svh::fail(SV_ERR_ARG, "group (%d) must be 32, 64 or 128", p->group);
  if (dim % 32) return svh::fail(SV_ERR_ARG, "dim (%d) must be a multiple of 32", dim);
  if (vocab > (1 << 24)) return svh::fail(SV_ERR_UNSUPPORTED, "vocab %d too large", vocab);
  return SV_OK;
}

sv_status check_pointers(const sv_q4_proj* p) {
  if (!p->packed || !p->scales) return svh::fail(SV_ERR_ARG, "a projection pointer is NULL");
  if (!aligned16(p->packed)) return svh::fail(SV_ERR_ARG, "packed must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(p->scales) % (p->scale_dtype == SV_F32 ? 4 : 2))
    return svh::fail(SV_ERR_ARG, "scales must be aligned to their elements");
  return SV_OK;
}

// rows0 rows of s0 into out0 and rows1 rows of s1 into out1, in one launch:
// the two sets follow one another as rows of one product, the second from a
// multiple of 8.
sv_status launch(const void* s0, int rows0, const void* s1, int rows1, sv_dtype dtype, const sv_q4_proj* proj,
                 int vocab, int dim, float* out0, float* out1, long long ld, unsigned* err, cudaStream_t stream) {
  if (!encoder()) return svh::fail(SV_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  Args g;
  g.scales = proj->scales;
  g.zeros = proj->zeros;
  g.scale_dtype = proj->scale_dtype;
  g.G = (dim + proj->group - 1) / proj->group;
  g.out0 = out0;
  g.out1 = out1;
  g.err = err;
  g.ld = ld;
  g.rows0 = rows0;
  g.rows1 = rows1;
  g.V = vocab;
  g.d = dim;
  // up to 16 rows whose states fit in shared memory: the kernel for few rows
  // (128256 x 4096, groups of 128: 1 row 60 us against the other's 134, 11 rows
  // 79 against 134, 16 rows 97 against 136; groups of 32: 82, 100, 139 against
  // 157, 157, 159)
  if (static_cast<long long>(rows0) + rows1 <= 16) {
    const sv_status few = dtype == SV_BF16 ? start_few_bf16(g, proj, s0, s1, stream) : start_few_f16(g, proj, s0, s1, stream);
    if (few != SV_ERR_UNSUPPORTED) return few;
  }
  const long long split = rows1 ? (static_cast<long long>(rows0) + 7) / 8 * 8 : 0x40000000LL;
  const long long all = rows1 ? split + rows1 : rows0;
  if (all > 0x3FFFFFFFLL) return svh::fail(SV_ERR_UNSUPPORTED, "too many rows");
  g.split = static_cast<int>(split);
  g.blocks = static_cast<int>((all + 63) / 64);
  const int n = static_cast<int>(((all + g.blocks - 1) / g.blocks + 15) / 16 * 16);
  g.blocks = static_cast<int>((all + n - 1) / n);
  return dtype == SV_BF16 ? start_bf16(g, n, proj, s0, s1, stream) : start_f16(g, n, proj, s0, s1, stream);
}

}  // namespace svq

extern "C" {

sv_status sv_lm_head_q4_logits(const void* states, sv_dtype dtype, const sv_q4_proj* proj, int32_t rows,
                               int32_t vocab, int32_t dim, float* logits, int64_t ld, uint32_t* err, void* stream) {
  svh::clear_error();
  if (rows < 0 || vocab < 1 || dim < 1) return svh::fail(SV_ERR_ARG, "rows, vocab, dim out of range");
  sv_status s = svq::check(proj, dtype, vocab, dim);
  if (s != SV_OK) return s;
  if (ld < vocab) return svh::fail(SV_ERR_ARG, "ld (%lld) must be >= vocab", (long long)ld);
  if (rows == 0) return SV_OK;
  if (!states || !logits) return svh::fail(SV_ERR_ARG, "states or logits is NULL");
  s = svq::check_pointers(proj);
  if (s != SV_OK) return s;
  if (!svq::aligned16(states)) return svh::fail(SV_ERR_ARG, "states must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(logits) % 4) return svh::fail(SV_ERR_ARG, "logits must be 4-byte aligned");
  return svq::launch(states, rows, nullptr, 0, dtype, proj, vocab, dim, logits, nullptr, ld, err,
                     static_cast<cudaStream_t>(stream));
}

sv_status sv_lm_head_q4_verify(const void* target_states, const void* draft_states, sv_dtype dtype,
                               const sv_q4_proj* proj, int32_t dim, const float* temperature,
                               const int32_t* draft_tokens, const float* uniforms, const int32_t* cu_k,
                               int32_t batch, int32_t k, int32_t sum_k, int32_t vocab, int32_t* n_accepted,
                               int32_t* next_token, uint32_t* status, void* workspace, size_t workspace_bytes,
                               uint32_t flags, void* stream) {
  svh::clear_error();
  if (batch < 0 || sum_k < 0 || vocab < 1 || dim < 1) return svh::fail(SV_ERR_ARG, "size out of range");
  sv_status s = svq::check(proj, dtype, vocab, dim);
  if (s != SV_OK) return s;
  if (batch == 0) return SV_OK;
  if (static_cast<long long>(sum_k) + batch > 0x7FFFFFFFLL) return svh::fail(SV_ERR_ARG, "too many rows");
  if (!target_states || (sum_k > 0 && !draft_states)) return svh::fail(SV_ERR_ARG, "a states pointer is NULL");
  s = svq::check_pointers(proj);
  if (s != SV_OK) return s;
  if (!svq::aligned16(target_states) || (sum_k > 0 && !svq::aligned16(draft_states)))
    return svh::fail(SV_ERR_ARG, "states must be 16-byte aligned");
  const size_t need = sv_lm_head_workspace_size(batch, sum_k, vocab);
  if (!workspace || workspace_bytes < need)
    return svh::fail(SV_ERR_ARG, "workspace_bytes (%zu) < the %zu bytes sv_lm_head_workspace_size() asks for",
                     workspace_bytes, need);
  if (!svq::aligned16(workspace)) return svh::fail(SV_ERR_ARG, "workspace must be 16-byte aligned");
  const long long ldv = (static_cast<long long>(vocab) + 3) / 4 * 4;
  const int t_rows = sum_k + batch;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  uint32_t* err = reinterpret_cast<uint32_t*>(ws);
  float* lt = reinterpret_cast<float*>(ws + 256);
  float* ld = lt + static_cast<size_t>(t_rows) * ldv;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // the verification's host checks first, so that nothing is enqueued when
  // they fail (a zero batch of the same arguments enqueues nothing)
  s = svh::accept_logits(lt, ld, SV_F32, ldv, temperature, draft_tokens, uniforms, cu_k, 0, k, 0, vocab, nullptr,
                         nullptr, n_accepted, next_token, status, nullptr, nullptr, nullptr, flags, stream);
  if (s != SV_OK) return s;
  if (!cu_k && static_cast<long long>(batch) * k != sum_k)
    return svh::fail(SV_ERR_ARG, "without cu_k, sum_k must equal batch * k");
  if (!temperature || !uniforms || (sum_k > 0 && !draft_tokens) || !n_accepted || !next_token || !status)
    return svh::fail(SV_ERR_ARG, "a verification pointer is NULL");
  const cudaError_t e = cudaMemsetAsync(err, 0, sizeof(uint32_t), st);
  if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
  s = svq::launch(target_states, t_rows, draft_states, sum_k, dtype, proj, vocab, dim, lt, ld, ldv, err, st);
  if (s != SV_OK) return s;
  return svh::accept_logits(lt, ld, SV_F32, ldv, temperature, draft_tokens, uniforms, cu_k, batch, k, sum_k, vocab,
                            nullptr, nullptr, n_accepted, next_token, status, nullptr, nullptr, err, flags, stream);
}

}  // extern "C"
