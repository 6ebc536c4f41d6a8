// Attention of a tree of drafted tokens over a paged cache
// (include/sv_tree.h).
//
// A warp takes a node and a query head and walks the keys that the node sees,
// with the running maximum and sum of a softmax.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sv_tree.h"
#include "sv_host.h"
#include "sv_ptx.cuh"

namespace sva {

constexpr int kWarps = 4;

__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T rounded(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 rounded(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half rounded(float x) {
  return __float2half_rn(x);
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) simple_kernel(const __grid_constant__ sv_tree_attn A, float scale) {
  const int lane = threadIdx.x & 31;
  const long long id = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int h = static_cast<int>(id % A.q_heads), i = static_cast<int>(id / A.q_heads % A.n);
  const int b = static_cast<int>(id / A.q_heads / A.n);
  if (b >= A.batch) return;
  long long first = b * A.n, N = A.total ? A.n : 0;
  if (A.cu_nodes) {
    first = A.cu_nodes[b];
    const long long end = A.cu_nodes[b + 1];
    N = end - first;
    if (first < 0 || end < first || end > A.total || N > A.n) {
      if (lane == 0 && i == 0 && h == 0) A.status[b] = SV_SEQ_BAD_LAYOUT;
      return;
    }
  }
  const int len = A.lengths[b], page = static_cast<int>(A.page_size);
  bool ok = len >= 0 && len <= A.max_pages * A.page_size;
  if (ok)
    for (int j = lane; j < (len + page - 1) / page; j += 32) {
      const int p = A.table[b * A.table_stride + j];
      ok = ok && p >= 0 && p < A.pages;
    }
  if (A.parents)
    for (int j = lane; j < N; j += 32) ok = ok && A.parents[first + j] >= -1 && A.parents[first + j] < j;
  ok = __all_sync(0xFFFFFFFFu, ok);
  if (lane == 0 && i == 0 && h == 0) A.status[b] = ok ? 0u : SV_SEQ_BAD_LAYOUT;
  if (i >= N) return;
  const int D = static_cast<int>(A.dim), kh = h / static_cast<int>(A.q_heads / A.kv_heads);
  T* out = static_cast<T*>(A.out) + (first + i) * A.out_row + h * A.out_head;
  float* lse = A.lse ? A.lse + (first + i) * A.q_heads + h : nullptr;
  if (!ok) {
    for (int d = lane; d < D; d += 32) out[d] = rounded<T>(0.0f);
    if (lse && lane == 0) *lse = -INFINITY;
    return;
  }
  float q[4] = {}, o[4] = {}, m = -INFINITY, z = 0;
  for (int d = 0; d < 4; ++d)
    if (lane + 32 * d < D) q[d] = value(static_cast<const T*>(A.q)[(first + i) * A.q_row + h * A.q_head + lane + 32 * d]);
  auto step = [&](const T* k, const T* v) {
    float s = 0;
    for (int d = 0; d < 4; ++d)
      if (lane + 32 * d < D) s += q[d] * value(k[lane + 32 * d]);
    for (int x = 16; x; x /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    s *= scale;
    const float was = m;
    m = fmaxf(m, s);
    const float keep = was == m ? 1.0f : expf(was - m), p = expf(s - m);
    z = z * keep + p;
    for (int d = 0; d < 4; ++d)
      if (lane + 32 * d < D) o[d] = o[d] * keep + p * value(v[lane + 32 * d]);
  };
  for (int t = 0; t < len; ++t) {
    const long long p = A.table[b * A.table_stride + t / page], at = t % page;
    step(static_cast<const T*>(A.k_cache) + p * A.kc_page + at * A.kc_token + kh * A.kc_head,
         static_cast<const T*>(A.v_cache) + p * A.vc_page + at * A.vc_token + kh * A.vc_head);
  }
  for (int j = i; j >= 0; j = A.parents ? A.parents[first + j] : j - 1)
    step(static_cast<const T*>(A.k) + (first + j) * A.k_row + kh * A.k_head,
         static_cast<const T*>(A.v) + (first + j) * A.v_row + kh * A.v_head);
  for (int d = 0; d < 4; ++d)
    if (lane + 32 * d < D) out[lane + 32 * d] = rounded<T>(o[d] / z);
  if (lse && lane == 0) *lse = m + logf(z);
}

}  // namespace sva

extern "C" {

size_t sv_tree_attention_workspace_size(int32_t dim) {
  (void)dim;
  return 0;
}

sv_status sv_tree_attention(const sv_tree_attn* args, float scale, void* workspace, size_t workspace_bytes,
                            void* stream) {
  svh::clear_error();
  if (!args) return svh::fail(SV_ERR_ARG, "args is NULL");
  const sv_tree_attn& a = *args;
  constexpr long long kMax = 0x7FFFFFFFLL;
  if (a.dtype != SV_BF16 && a.dtype != SV_F16) return svh::fail(SV_ERR_ARG, "dtype (%lld) must be SV_BF16 or SV_F16", (long long)a.dtype);
  if (a.kv_heads < 1 || a.q_heads < 1 || a.q_heads > kMax || a.q_heads % a.kv_heads)
    return svh::fail(SV_ERR_ARG, "q_heads (%lld) must be a multiple of kv_heads (%lld)", (long long)a.q_heads, (long long)a.kv_heads);
  if (a.q_heads / a.kv_heads > 128)
    return svh::fail(SV_ERR_UNSUPPORTED, "more than 128 query heads per key head");
  if (a.dim < 8 || a.dim > 128 || a.dim % 8) return svh::fail(SV_ERR_UNSUPPORTED, "dim (%lld) must be a multiple of 8 up to 128", (long long)a.dim);
  if (a.page_size < 8 || a.page_size > kMax || a.page_size % 8)
    return svh::fail(SV_ERR_UNSUPPORTED, "page_size (%lld) must be a multiple of 8", (long long)a.page_size);
  if (a.batch < 0 || a.n < 0 || a.total < 0 || a.batch > kMax || a.total > kMax)
    return svh::fail(SV_ERR_ARG, "batch, n and total must be in [0, 2^31)");
  if (a.n > SV_TREE_MAX_NODES) return svh::fail(SV_ERR_UNSUPPORTED, "n (%lld) is more than %d nodes", (long long)a.n, SV_TREE_MAX_NODES);
  if (!a.cu_nodes && a.batch * a.n != a.total) return svh::fail(SV_ERR_ARG, "without cu_nodes, total must equal batch * n");
  if (a.pages < 1 || a.pages > kMax || a.max_pages < 0 || a.max_pages > kMax)
    return svh::fail(SV_ERR_ARG, "pages or max_pages out of range");
  if (a.table_stride < a.max_pages && a.batch > 1) return svh::fail(SV_ERR_ARG, "table_stride (%lld) is less than max_pages", (long long)a.table_stride);
  if (!(scale == scale) || scale - scale != 0) return svh::fail(SV_ERR_ARG, "scale must be finite");
  if (a.batch == 0) return SV_OK;
  if (!a.status || !a.lengths || (!a.table && a.max_pages > 0)) return svh::fail(SV_ERR_ARG, "status, lengths or table is NULL");
  if (a.total > 0 && (!a.q || !a.k || !a.v || !a.out)) return svh::fail(SV_ERR_ARG, "q, k, v or out is NULL");
  if (!a.k_cache || !a.v_cache) return svh::fail(SV_ERR_ARG, "a cache is NULL");
  const int64_t strides[] = {a.q_row, a.q_head, a.k_row, a.k_head, a.v_row, a.v_head, a.kc_page, a.kc_token,
                             a.kc_head, a.vc_page, a.vc_token, a.vc_head, a.out_row, a.out_head};
  for (const int64_t x : strides)
    if (x < 0 || x % 8) return svh::fail(SV_ERR_ARG, "strides must be multiples of 8 elements, not negative");
  for (const void* p : {a.q, a.k, a.v, a.k_cache, a.v_cache, static_cast<const void*>(a.out)})
    if (reinterpret_cast<uintptr_t>(p) & 15) return svh::fail(SV_ERR_ARG, "q, k, v, the caches and out must be 16-byte aligned");
  const long long warps = a.batch * (a.n > 0 ? a.n : 1) * a.q_heads;
  sv_tree_attn b = a;
  if (b.n == 0) {  // (one warp per sequence and head writes the status)
    b.n = 1;
    b.total = 0;
  }
  const long long grid = (warps + sva::kWarps - 1) / sva::kWarps;
  if (grid > kMax) return svh::fail(SV_ERR_UNSUPPORTED, "the call is too large");
  if (a.dtype == SV_BF16)
    sva::simple_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), 32 * sva::kWarps, 0, static_cast<cudaStream_t>(stream)>>>(b, scale);
  else
    sva::simple_kernel<__half><<<static_cast<unsigned>(grid), 32 * sva::kWarps, 0, static_cast<cudaStream_t>(stream)>>>(b, scale);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SV_OK : svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
