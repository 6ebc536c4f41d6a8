// Beam search's selection over beams and vocabulary (include/sv_beam.h).
//
// First form: one CTA per row takes the row's maximum and sum of exponentials
// in 64 bits; then one CTA per sequence takes the n candidates one after
// another, each the best that comes after the one before it in the order
// (score descending, beam W + token ascending).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/sv_beam.h"
#include "sv_host.h"

namespace svs {

constexpr int kThreads = 512;

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

struct Params {
  const void* logits;
  long long stride;
  const float* scores;
  const unsigned char* finished;
  int eos, B, W, V, n;
  double* lse;  // [B W]: -inf: no candidates; NaN: bad value
  float* out_s;
  int* out_p;
  int* out_t;
  unsigned* st;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) row_kernel(Params P) {
  const long long r = blockIdx.x;
  __shared__ double red[kThreads];
  const float c = P.scores[r];
  if ((P.finished && P.finished[r]) || c == -INFINITY) return;
  const T* row = static_cast<const T*>(P.logits) + r * P.stride;
  float m = -INFINITY;
  bool bad = false;
  for (int v = threadIdx.x; v < P.V; v += kThreads) {
    const float x = to_f32(row[v]);
    bad |= isnan(x) || x == INFINITY;
    m = fmaxf(m, x);
  }
  red[threadIdx.x] = bad ? static_cast<double>(NAN) : static_cast<double>(m);
  __syncthreads();
  for (int h = kThreads / 2; h > 0; h /= 2) {
    if (threadIdx.x < h) {
      const double a = red[threadIdx.x], b = red[threadIdx.x + h];
      red[threadIdx.x] = isnan(a) ? a : isnan(b) ? b : fmax(a, b);
    }
    __syncthreads();
  }
  const double mx = red[0];
  __syncthreads();
  if (isnan(mx) || mx == -INFINITY) {
    if (threadIdx.x == 0) P.lse[r] = mx;
    return;
  }
  // the sum in units of 2^-60, exact whatever the order: rows that are
  // permutations of one another get equal sums, so their candidates tie
  unsigned long long hi = 0, lo = 0;
  for (int v = threadIdx.x; v < P.V; v += kThreads) {
    const auto q = static_cast<unsigned long long>(exp(static_cast<double>(to_f32(row[v])) - mx) * 1152921504606846976.0);
    hi += q >> 32;
    lo += q & 0xFFFFFFFFu;
  }
  __shared__ unsigned long long ih[kThreads], il[kThreads];
  ih[threadIdx.x] = hi;
  il[threadIdx.x] = lo;
  __syncthreads();
  for (int h = kThreads / 2; h > 0; h /= 2) {
    if (threadIdx.x < h) {
      ih[threadIdx.x] += ih[threadIdx.x + h];
      il[threadIdx.x] += il[threadIdx.x + h];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double total = static_cast<double>(ih[0] + (il[0] >> 32)) + static_cast<double>(il[0] & 0xFFFFFFFFu) * 0x1p-32;
    P.lse[r] = mx + log(total * 0x1p-28);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) pick_kernel(Params P) {
  const int b = blockIdx.x;
  __shared__ double rs[kThreads];
  __shared__ int ri[kThreads];
  bool bad = false;
  for (int w = 0; w < P.W; ++w) {
    const float c = P.scores[b * P.W + w];
    bad |= isnan(c) || c == INFINITY;
    if (!(P.finished && P.finished[b * P.W + w]) && c != -INFINITY) bad |= isnan(P.lse[b * P.W + w]);
  }
  double last = INFINITY;
  int last_i = -1;
  for (int k = 0; k < P.n; ++k) {
    double best = -INFINITY;
    int bi = 0x7FFFFFFF;
    auto offer = [&](double s, int i) {
      if (s > -INFINITY && (s < last || (s == last && i > last_i)) && (s > best || (s == best && i < bi))) {
        best = s;
        bi = i;
      }
    };
    for (int w = 0; !bad && w < P.W; ++w) {
      const long long r = static_cast<long long>(b) * P.W + w;
      const float c = P.scores[r];
      if (c == -INFINITY) continue;
      if (P.finished && P.finished[r]) {
        offer(c, w * P.V + P.eos);
        continue;
      }
      const double lse = P.lse[r];
      if (lse == -INFINITY) continue;
      const T* row = static_cast<const T*>(P.logits) + r * P.stride;
      for (int v = threadIdx.x; v < P.V; v += kThreads)
        offer(static_cast<double>(c) + (static_cast<double>(to_f32(row[v])) - lse), w * P.V + v);
    }
    rs[threadIdx.x] = best;
    ri[threadIdx.x] = bi;
    __syncthreads();
    for (int h = kThreads / 2; h > 0; h /= 2) {
      if (threadIdx.x < h) {
        const double s = rs[threadIdx.x + h];
        const int i = ri[threadIdx.x + h];
        if (s > rs[threadIdx.x] || (s == rs[threadIdx.x] && i < ri[threadIdx.x])) {
          rs[threadIdx.x] = s;
          ri[threadIdx.x] = i;
        }
      }
      __syncthreads();
    }
    last = rs[0];
    last_i = ri[0];
    if (threadIdx.x == 0) {
      const bool none = last == -INFINITY;
      P.out_s[b * P.n + k] = static_cast<float>(last);
      P.out_p[b * P.n + k] = none ? -1 : last_i / P.V;
      P.out_t[b * P.n + k] = none ? -1 : last_i % P.V;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) P.st[b] = bad ? SV_SEQ_BAD_VALUE : 0u;
}

}  // namespace svs

extern "C" {

size_t sv_beam_select_workspace_size(int32_t batch, int32_t beams, int32_t vocab, int32_t n) {
  if (batch < 0 || beams < 1 || beams > SV_BEAM_MAX_BEAMS || vocab < 1 || n < 1 || n > SV_BEAM_MAX_CANDIDATES) return 0;
  return (static_cast<size_t>(batch) * beams * sizeof(double) + 15) / 16 * 16;
}

sv_status sv_beam_select(const void* logits, sv_dtype dtype, int64_t row_stride, const float* scores,
                         const uint8_t* finished, int32_t eos, int32_t batch, int32_t beams, int32_t vocab, int32_t n,
                         float* out_scores, int32_t* out_parents, int32_t* out_tokens, uint32_t* status,
                         void* workspace, size_t workspace_bytes, void* stream) {
  svh::clear_error();
  if (batch < 0) return svh::fail(SV_ERR_ARG, "batch (%d) must be >= 0", batch);
  if (beams < 1 || beams > SV_BEAM_MAX_BEAMS)
    return svh::fail(SV_ERR_ARG, "beams (%d) must be in [1, %d]", beams, SV_BEAM_MAX_BEAMS);
  if (vocab < 1) return svh::fail(SV_ERR_ARG, "vocab (%d) must be >= 1", vocab);
  if (static_cast<long long>(beams) * vocab > 0x7FFFFFFFLL)
    return svh::fail(SV_ERR_UNSUPPORTED, "beams * vocab must be below 2^31");
  if (n < 1 || n > SV_BEAM_MAX_CANDIDATES)
    return svh::fail(SV_ERR_ARG, "n (%d) must be in [1, %d]", n, SV_BEAM_MAX_CANDIDATES);
  if (row_stride < vocab) return svh::fail(SV_ERR_ARG, "row_stride < vocab");
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16)
    return svh::fail(SV_ERR_ARG, "unknown dtype %d", static_cast<int>(dtype));
  if (finished && (eos < 0 || eos >= vocab))
    return svh::fail(SV_ERR_ARG, "eos (%d) must be in [0, vocab) when finished is given", eos);
  if (static_cast<long long>(batch) * (beams > n ? beams : n) > 0x7FFFFFFFLL)
    return svh::fail(SV_ERR_ARG, "batch (%d) too large", batch);
  if (batch == 0) return SV_OK;
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens || !status)
    return svh::fail(SV_ERR_ARG, "a logits, scores or output pointer is NULL");
  const size_t elem = dtype == SV_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % elem) return svh::fail(SV_ERR_ARG, "logits must be aligned to their elements");
  const size_t need = sv_beam_select_workspace_size(batch, beams, vocab, n);
  if (!workspace || workspace_bytes < need)
    return svh::fail(SV_ERR_ARG, "workspace_bytes (%zu) < the %zu bytes sv_beam_select_workspace_size() asks for",
                     workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) % 16) return svh::fail(SV_ERR_ARG, "workspace must be 16-byte aligned");
  svs::Params p{logits, row_stride, scores, finished, eos, batch, beams, vocab, n, static_cast<double*>(workspace),
                out_scores, out_parents, out_tokens, status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](void (*rows)(svs::Params), void (*pick)(svs::Params)) -> sv_status {
    rows<<<static_cast<unsigned>(batch * beams), svs::kThreads, 0, st>>>(p);
    pick<<<static_cast<unsigned>(batch), svs::kThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return SV_OK;
  };
  switch (dtype) {
    case SV_F32: return go(svs::row_kernel<float>, svs::pick_kernel<float>);
    case SV_BF16: return go(svs::row_kernel<__nv_bfloat16>, svs::pick_kernel<__nv_bfloat16>);
    default: return go(svs::row_kernel<__half>, svs::pick_kernel<__half>);
  }
}

}  // extern "C"
