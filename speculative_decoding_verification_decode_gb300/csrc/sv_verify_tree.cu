// Greedy verification of a drafted tree (include/sv_tree.h).
//
// The path visits few of a tree's rows, one after another: a thread-block
// cluster takes a sequence, shares the row of the current node among its CTAs,
// exchanges their best (value, index) pairs through distributed shared memory,
// and all of them look up the child to go to.  A step is a trip to memory, a
// reduction by shuffles and one barrier of the cluster, some 2.5 us; what is read
// is the path's rows and nothing else, so a call takes as long as its longest path.
//
// Measured (calls in a graph; from Python 24 to 30 us, the host's share 24): 64 trees of 32 nodes, V = 128256 bf16 (38 MB of 525 read): 24.6 us.
// Threads a CTA: 128 26.6, 512 33.7 (fewer clusters at a time); clusters of four
// 28.8; four loads of 16 bytes in flight instead of eight 25.7; elements one at a time
// 48.  One tree of 16, V = 32000 f32: 11.1 us (clusters of four 12.8).
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sv_tree.h"
#include "sv_host.h"
#include "sv_ptx.cuh"

namespace svt {

constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxCluster = 8;

struct Tree {
  const int* tokens;
  const int* parents;
  const int* cu;
  int n, total;
  int* n_accepted;
  int* next_token;
  int* path;
  unsigned* status;
};

struct Rows {
  const void* data;
  long long stride;
  int V;
};

// First row and number of nodes of sequence b; false: its offsets are bad.
__device__ __forceinline__ bool nodes_of(const Tree& T, int b, int& first, int& N) {
  first = b * T.n;
  N = T.n;
  if (!T.cu) return true;
  first = T.cu[b];
  const int end = T.cu[b + 1];
  N = end - first;
  return first >= 0 && end >= first && end <= T.total && N <= T.n;
}

// Ordered so that a larger key is a larger value, or an equal one at a lower
// index; 0 is below every key.  (x + 0 makes -0 a 0.)
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<uint64_t>(o) << 32 | ~static_cast<uint32_t>(index);
}
__device__ __forceinline__ int index_of(uint64_t key) { return key ? static_cast<int>(~static_cast<uint32_t>(key)) : 0; }

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(__half x) { return __half2float(x); }

// Largest of a 16-byte vector's elements; NaN if there is one among them.
template <typename E>
__device__ __forceinline__ float top_of(uint4 v);
template <>
__device__ __forceinline__ float top_of<float>(uint4 v) {
  return svk::fmax_nan(svk::fmax_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                       svk::fmax_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
}
template <>
__device__ __forceinline__ float top_of<__nv_bfloat16>(uint4 v) {
  const uint32_t m = svk::bf16x2_max_nan(svk::bf16x2_max_nan(v.x, v.y), svk::bf16x2_max_nan(v.z, v.w));
  return svk::fmax_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float top_of<__half>(uint4 v) {
  const uint32_t m = svk::f16x2_max_nan(svk::f16x2_max_nan(v.x, v.y), svk::f16x2_max_nan(v.z, v.w));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
  return svk::fmax_nan(f.x, f.y);
}

// Best of elements lo..hi of a row for this thread; `nan` tells of any NaN.  A
// 16-byte vector counts through its largest element; only the vector that
// holds the thread's best is looked at again.
template <typename E>
__device__ __forceinline__ uint64_t best_of(const E* row, int lo, int hi, bool& nan) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(E));
  uint64_t best = 0;
  auto one = [&](int i) {
    const float x = value(row[i]);
    nan = nan || x != x;
    const uint64_t k = x != x ? 0 : key_of(x, i);
    best = best > k ? best : k;
  };
  const int t = static_cast<int>(threadIdx.x);
  // elements before the first 16-byte boundary, and behind the last
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row + lo) & 15) / sizeof(E));
  int first = lo + (off ? kVec - off : 0);
  first = first < hi ? first : hi;
  const int vectors = (hi - first) / kVec, rest = first + vectors * kVec;
  if (t < first - lo) one(lo + t);
  if (t < hi - rest) one(rest + t);
  const uint4* p = reinterpret_cast<const uint4*>(row + first);
  float top = -INFINITY;
  int at = -1;
  constexpr int kFly = 8;  // loads in flight
  for (int i = t; i < vectors; i += kFly * kThreads) {
    uint4 v[kFly];
#pragma unroll
    for (int j = 0; j < kFly; ++j)
      if (i + j * kThreads < vectors) v[j] = __ldg(p + i + j * kThreads);
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      if (i + j * kThreads >= vectors) break;
      float x = top_of<E>(v[j]);
      if (x != x) {  // one element at a time
        for (int e = 0; e < kVec; ++e) one(first + (i + j * kThreads) * kVec + e);
        continue;
      }
      if (at < 0 || x > top) top = x, at = i + j * kThreads;
    }
  }
  if (at >= 0) {
    int e = 0;
    while (e < kVec - 1 && value(row[first + at * kVec + e]) != top) ++e;
    const uint64_t k = key_of(top, first + at * kVec + e);
    best = best > k ? best : k;
  }
  return best;
}

struct __align__(16) Shared {
  uint4 slot[2][kMaxCluster * kWarps];  // [step parity][warp of the cluster]: its best, whether it saw a NaN
  int token[SV_TREE_MAX_NODES], parent[SV_TREE_MAX_NODES];
  int next;
};

// Loads the tree; false: a parent is out of range.
__device__ __forceinline__ bool load_tree(const Tree& T, int first, int N, Shared& sm) {
  bool ok = true;
  for (int i = static_cast<int>(threadIdx.x); i < N; i += static_cast<int>(blockDim.x)) {
    const int p = T.parents ? T.parents[first + i] : i - 1;
    ok = ok && p >= -1 && p < i;
    sm.parent[i] = p;
    sm.token[i] = T.tokens[first + i];
  }
  return __syncthreads_and(ok);
}

__global__ void __launch_bounds__(256) walk_kernel(const __grid_constant__ Tree T, const int* choices) {
  __shared__ Shared sm;
  __shared__ int s_choice[SV_TREE_MAX_NODES];
  const int b = static_cast<int>(blockIdx.x), t = static_cast<int>(threadIdx.x);
  int first, N;
  const bool good = nodes_of(T, b, first, N);
  if (!good) N = 0;
  for (int i = t; i < N; i += 256) s_choice[i] = choices[first + i];
  const bool ok = load_tree(T, first, N, sm) && good;
  int* path = T.path + static_cast<long long>(b) * T.n;
  int at = 0, steps = 0, next = -1;
  if (ok && N > 0)
    for (;;) {
      if (t == 0) path[steps] = at;
      ++steps;
      const int c = s_choice[at];
      if (t == 0) sm.next = N;
      __syncthreads();
      if (c >= 0 && t > at && t < N && sm.parent[t] == at && sm.token[t] == c) atomicMin(&sm.next, t);
      __syncthreads();
      const int to = sm.next;
      __syncthreads();
      next = c >= 0 ? c : -1;
      if (to >= N) break;
      at = to;
    }
  for (int i = steps + t; i < T.n; i += 256) path[i] = -1;
  if (t == 0) {
    T.n_accepted[b] = steps ? steps - 1 : 0;
    T.next_token[b] = next;
    T.status[b] = ok ? 0u : SV_SEQ_BAD_LAYOUT;
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads, 4) greedy_kernel(const __grid_constant__ Tree T, const __grid_constant__ Rows R) {
  __shared__ Shared sm;
  const int rank = static_cast<int>(svk::cluster_rank()), size = static_cast<int>(svk::cluster_size());
  const int b = static_cast<int>(blockIdx.x) / size, t = static_cast<int>(threadIdx.x), lane = t & 31;
  int first, N;
  const bool good = nodes_of(T, b, first, N);
  if (!good) N = 0;
  const bool ok = load_tree(T, first, N, sm) && good;
  svk::cluster_sync_all();  // every CTA runs before another writes to it
  int* path = T.path + static_cast<long long>(b) * T.n;
  int at = 0, steps = 0, next = -1;
  unsigned status = ok ? 0u : SV_SEQ_BAD_LAYOUT;
  if (ok && N > 0) {
    const int lo = static_cast<int>(static_cast<long long>(R.V) * rank / size);
    const int hi = static_cast<int>(static_cast<long long>(R.V) * (rank + 1) / size);
    for (;;) {
      const int par = steps & 1;
      if (rank == 0 && t == 0) path[steps] = at;
      ++steps;
      bool nan = false;
      uint64_t best = best_of(static_cast<const E*>(R.data) + (static_cast<long long>(first) + at) * R.stride, lo, hi, nan);
      nan = __any_sync(0xFFFFFFFFu, nan);
#pragma unroll
      for (int d = 16; d; d /= 2) {
        const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, best, d);
        best = best > o ? best : o;
      }
      // every warp tells every CTA of the cluster, and every warp there works
      // out the same: one barrier of the cluster a step, none of the CTA
      if (lane < size)
        svk::dsmem_st_v4(svk::dsmem_addr(&sm.slot[par][rank * kWarps + t / 32], lane),
                         make_uint4(static_cast<uint32_t>(best), static_cast<uint32_t>(best >> 32), nan, 0));
      svk::cluster_sync_all();
      uint64_t top = 0;
      nan = false;
      for (int i = lane; i < size * kWarps; i += 32) {
        const uint4 v = sm.slot[par][i];
        const uint64_t k = static_cast<uint64_t>(v.y) << 32 | v.x;
        top = top > k ? top : k;
        nan = nan || v.z;
      }
#pragma unroll
      for (int d = 16; d; d /= 2) {
        const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, top, d);
        top = top > o ? top : o;
      }
      if (__any_sync(0xFFFFFFFFu, nan)) status |= SV_SEQ_BAD_VALUE;
      next = index_of(top);
      bool bad = false;
      int to = N;
      for (int i = at + 1 + lane; i < N; i += 32)
        if (sm.parent[i] == at) {
          bad = bad || sm.token[i] < 0 || sm.token[i] >= R.V;
          if (sm.token[i] == next) to = to < i ? to : i;
        }
      if (__any_sync(0xFFFFFFFFu, bad)) status |= SV_SEQ_BAD_TOKEN;
      to = __reduce_min_sync(0xFFFFFFFFu, to);
      if (to >= N) break;
      at = to;
    }
  }
  if (rank) return;
  for (int i = steps + t; i < T.n; i += kThreads) path[i] = -1;
  if (t == 0) {
    T.n_accepted[b] = steps ? steps - 1 : 0;
    T.next_token[b] = next;
    T.status[b] = status;
  }
}

// Checks that both calls share.
sv_status check(const Tree& T, int batch) {
  if (batch < 0) return svh::fail(SV_ERR_ARG, "batch (%d) must be >= 0", batch);
  if (T.n < 0 || T.total < 0) return svh::fail(SV_ERR_ARG, "n (%d) and total (%d) must be >= 0", T.n, T.total);
  if (T.n > SV_TREE_MAX_NODES)
    return svh::fail(SV_ERR_UNSUPPORTED, "n (%d) is more than %d nodes", T.n, SV_TREE_MAX_NODES);
  if (!T.cu && static_cast<long long>(batch) * T.n != T.total)
    return svh::fail(SV_ERR_ARG, "without cu_nodes, total must equal batch * n");
  if (batch == 0) return SV_OK;
  if (T.total > 0 && !T.tokens) return svh::fail(SV_ERR_ARG, "tokens is NULL");
  if (!T.n_accepted || !T.next_token || (T.n > 0 && !T.path) || !T.status)
    return svh::fail(SV_ERR_ARG, "an output pointer is NULL");
  return SV_OK;
}

template <typename E>
sv_status launch(const Tree& T, const Rows& R, int batch, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMaxCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(batch) * kMaxCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, greedy_kernel<E>, T, R);
  return e == cudaSuccess ? SV_OK : svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
}

}  // namespace svt

extern "C" {

sv_status sv_verify_tree_greedy(const void* target, sv_dtype dtype, int64_t row_stride, const int32_t* tokens,
                                const int32_t* parents, const int32_t* cu_nodes, int32_t batch, int32_t n,
                                int32_t total, int32_t vocab, int32_t* n_accepted, int32_t* next_token,
                                int32_t* path, uint32_t* status, void* stream) {
  svh::clear_error();
  const svt::Tree T = {tokens, parents, cu_nodes, n, total, n_accepted, next_token, path, status};
  const sv_status s = svt::check(T, batch);
  if (s != SV_OK) return s;
  if (vocab < 1) return svh::fail(SV_ERR_ARG, "vocab (%d) must be >= 1", vocab);
  if (row_stride < vocab && total > 1) return svh::fail(SV_ERR_ARG, "row_stride (%lld) is less than vocab", (long long)row_stride);
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return svh::fail(SV_ERR_ARG, "dtype (%d) is unknown", (int)dtype);
  if (batch == 0) return SV_OK;
  if (batch > 0x7FFFFFFF / 16) return svh::fail(SV_ERR_UNSUPPORTED, "batch %d too large", batch);
  if (total > 0 && !target) return svh::fail(SV_ERR_ARG, "target is NULL");
  const size_t e = dtype == SV_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(target) % e) return svh::fail(SV_ERR_ARG, "target is not aligned to its type");
  const svt::Rows R = {target, row_stride, vocab};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SV_F32) return svt::launch<float>(T, R, batch, st);
  if (dtype == SV_BF16) return svt::launch<__nv_bfloat16>(T, R, batch, st);
  return svt::launch<__half>(T, R, batch, st);
}

sv_status sv_verify_tree(const int32_t* choices, const int32_t* tokens, const int32_t* parents,
                         const int32_t* cu_nodes, int32_t batch, int32_t n, int32_t total, int32_t* n_accepted,
                         int32_t* next_token, int32_t* path, uint32_t* status, void* stream) {
  svh::clear_error();
  const svt::Tree T = {tokens, parents, cu_nodes, n, total, n_accepted, next_token, path, status};
  const sv_status s = svt::check(T, batch);
  if (s != SV_OK || batch == 0) return s;
  if (total > 0 && !choices) return svh::fail(SV_ERR_ARG, "choices is NULL");
  svt::walk_kernel<<<static_cast<unsigned>(batch), 256, 0, static_cast<cudaStream_t>(stream)>>>(T, choices);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SV_OK : svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
