// The LM head with a projection in 4 bits (include/sv_lm_head_q4.h).
//
// First form: one warp per vocabulary row; a lane takes 32 consecutive
// weights at a time (16 bytes, inside one group), sums their products with
// the states in f32, scales the sum by its group's scale, and the lanes' sums
// are added at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/sv_lm_head.h"
#include "../../include/sv_lm_head_q4.h"
#include "sv_host.h"

namespace svq {

constexpr int kThreads = 256, kRows = 8;

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

struct Args {
  const uint4* packed;
  const void* scales;
  const unsigned char* zeros;
  const void* h[2];
  float* out[2];
  int rows[2];
  int V, d, group, G;
  long long ld;
};

template <typename H, typename S>
__global__ void __launch_bounds__(kThreads) simple_kernel(Args g) {
  const int v = blockIdx.x * (kThreads / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (v >= g.V) return;
  int r0 = blockIdx.y * kRows, part = 0;
  const int first = (g.rows[0] + kRows - 1) / kRows * kRows;
  if (r0 >= first) {
    r0 -= first;
    part = 1;
  }
  const H* h = static_cast<const H*>(g.h[part]);
  const int rows = g.rows[part];
  float acc[kRows] = {};
  for (int c = lane; c < g.d / 32; c += 32) {
    const uint4 q4 = g.packed[static_cast<long long>(v) * (g.d / 32) + c];
    const unsigned q[4] = {q4.x, q4.y, q4.z, q4.w};
    const long long gi = static_cast<long long>(v) * g.G + c * 32 / g.group;
    const float s = to_f32(static_cast<const S*>(g.scales)[gi]);
    const int z = g.zeros ? g.zeros[gi] & 15 : 8;
    for (int r = 0; r < kRows && r0 + r < rows; ++r) {
      float p = 0.f;
      for (int j = 0; j < 32; ++j)
        p += static_cast<float>(static_cast<int>(q[j / 8] >> (4 * (j % 8)) & 15u) - z) *
             to_f32(h[static_cast<long long>(r0 + r) * g.d + c * 32 + j]);
      acc[r] += s * p;
    }
  }
  for (int r = 0; r < kRows; ++r) {
    for (int o = 16; o > 0; o /= 2) acc[r] += __shfl_xor_sync(0xFFFFFFFFu, acc[r], o);
    if (lane == 0 && r0 + r < rows) g.out[part][static_cast<long long>(r0 + r) * g.ld + v] = acc[r];
  }
}

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

// rows0 rows of s0 into out0 and rows1 rows of s1 into out1.
sv_status launch(const void* s0, int rows0, const void* s1, int rows1, sv_dtype dtype, const sv_q4_proj* proj,
                 int vocab, int dim, float* out0, float* out1, long long ld, unsigned* err, cudaStream_t stream) {
  (void)err;
  Args g;
  g.packed = static_cast<const uint4*>(proj->packed);
  g.scales = proj->scales;
  g.zeros = proj->zeros;
  g.h[0] = s0;
  g.h[1] = s1;
  g.out[0] = out0;
  g.out[1] = out1;
  g.rows[0] = rows0;
  g.rows[1] = rows1;
  g.V = vocab;
  g.d = dim;
  g.group = proj->group;
  g.G = (dim + proj->group - 1) / proj->group;
  g.ld = ld;
  const dim3 grid((vocab + kThreads / 32 - 1) / (kThreads / 32), (rows0 + kRows - 1) / kRows + (rows1 + kRows - 1) / kRows);
  if (grid.y > 65535) return svh::fail(SV_ERR_UNSUPPORTED, "too many rows");
  auto go = [&](void (*kern)(Args)) -> sv_status {
    kern<<<grid, kThreads, 0, stream>>>(g);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return SV_OK;
  };
  if (dtype == SV_BF16) {
    if (proj->scale_dtype == SV_F32) return go(simple_kernel<__nv_bfloat16, float>);
    if (proj->scale_dtype == SV_BF16) return go(simple_kernel<__nv_bfloat16, __nv_bfloat16>);
    return go(simple_kernel<__nv_bfloat16, __half>);
  }
  if (proj->scale_dtype == SV_F32) return go(simple_kernel<__half, float>);
  if (proj->scale_dtype == SV_BF16) return go(simple_kernel<__half, __nv_bfloat16>);
  return go(simple_kernel<__half, __half>);
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
