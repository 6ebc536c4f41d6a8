// Reordering of beam states in place (include/sv_beam.h).
//
// A slot's new contents are another slot's old ones, and one parent may go to
// several slots while its own slot is overwritten.  A thread therefore owns a
// column: the same bytes of every beam of one sequence.  It loads the column
// of every moving slot's parent into registers, then stores; nobody else
// touches those bytes, so the permutation with repetitions needs no second
// buffer, no order among the slots and no barrier.  A slot that keeps its
// parent costs nothing.
//
// That wants 16-byte accesses: the bytes in flight carry a copy (151 MB whose
// beams lie 4 bytes off one another took 69 us with one 4-byte register per
// access, 49 with four times as many).  Where addresses or extents forbid them,
// a CTA owns a range of columns instead: it brings the range of every parent to
// shared memory in the aligned 16-byte blocks that hold it, waits, and writes
// every moving slot in its own aligned blocks, put together from 32-bit words.
#include <cuda_runtime.h>

#include "../../include/sv_beam.h"
#include "sv_host.h"

namespace svb {

constexpr int kThreads = 256;
// The staged path's CTAs per SM and shared memory of each: many small ones, whose
// reading and writing overlap (151 MB whose beams lie 4 bytes off one another:
// two of 96 KB 38 us, four of 48 KB 35, eight of 24 KB 33.8).
constexpr int kStagedCtas = 8, kStageBytes = 24 * 1024;
constexpr int kStates = 48;    // per launch: their descriptions are kernel parameters
// Bytes of one segment that a CTA takes (of every beam).  Staged: 8 KB (64 x 4
// beams of 64 KB 10 us, with 64 KB 33; 16 x 4 of 512 KB in 16 states 129 and
// 135, with 4 KB 153).  Aligned: some 128 KB of all beams together, a few rounds
// of a CTA's registers (4 beams, 16 states of 512 KB: 32 KB 106 us, 64 KB 109,
// 8 KB 157; 16 beams, 4 states of 2 MB: 8 KB 98, 32 KB 110), but less where that
// would leave SMs without a CTA (64 x 4 beams of 32 KB: 8 KB 4.3, 32 KB 5.9).
constexpr int kMinChunk = 8192, kMaxChunk = 65536, kChunkOfAll = 131072, kSms = 152;

struct State {
  char* data;
  long long seq, beam, seg;  // strides, bytes
  long long token_bytes;
  int segs, tokens, timed;
  int unit;    // bytes that divide every address, stride and extent; 16 at most
  int chunks;  // CTAs per segment
  unsigned first;  // first CTA of this state
};

struct Params {
  State s[kStates];
  const int* parents;
  const int* lengths;
  unsigned* status;  // NULL: another launch writes it
  int n, B, W, min_tokens, status_ctas, chunk_bytes;
};

// Columns lo + tid, lo + tid + kThreads, ... < hi of one segment, M moves at
// most, N columns at a time per thread: N x M accesses in flight.  (`volatile`:
// offsets kept in registers over the loop would push the data out of them; 16
// moves took 276 us where they take 132.)
template <typename U, int M, int N>
__device__ __forceinline__ void move_columns(char* base, const volatile long long* src, const volatile long long* dst, int m,
                                             long long lo, long long hi) {
  for (long long c = lo + threadIdx.x; c < hi; c += N * kThreads) {
    U v[N][M];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < M; ++j)
        if (j < m && c + i * kThreads < hi)
          v[i][j] = *reinterpret_cast<const U*>(base + src[j] + (c + i * kThreads) * sizeof(U));
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < M; ++j)
        if (j < m && c + i * kThreads < hi)
          *reinterpret_cast<U*>(base + dst[j] + (c + i * kThreads) * sizeof(U)) = v[i][j];
  }
}

// Bytes lo..hi of one segment in 16-byte accesses: 64 registers of data per
// thread whatever the number of moves; more moves take narrower accesses.
__device__ __forceinline__ void move_aligned(char* base, const volatile long long* src, const volatile long long* dst, int m,
                                             long long lo, long long hi) {
  if (m <= 2)
    move_columns<uint4, 2, 8>(base, src, dst, m, lo / 16, hi / 16);
  else if (m <= 4)
    move_columns<uint4, 4, 4>(base, src, dst, m, lo / 16, hi / 16);
  else if (m <= 8)
    move_columns<uint4, 8, 2>(base, src, dst, m, lo / 16, hi / 16);
  else if (m <= 16)
    move_columns<uint4, 16, 1>(base, src, dst, m, lo / 16, hi / 16);
  else if (m <= 32)
    move_columns<uint2, 32, 1>(base, src, dst, m, lo / 8, hi / 8);
  else
    move_columns<unsigned, 64, 1>(base, src, dst, m, lo / 4, hi / 4);
}

// Bytes lo..hi of one segment at any alignment, through shared memory.  The
// blocks at a range's ends may hold neighbours' bytes; those are not used.
__device__ __forceinline__ void move_staged(char* base, const long long* src, const long long* dst, int m, long long lo,
                                         long long hi, int unit) {
  extern __shared__ __align__(16) unsigned char stage[];
  const int room = kStageBytes / m / 16 * 16;  // per move, the blocks at both ends included
  for (long long at = lo; at < hi; at += room - 32) {
    const int bytes = static_cast<int>(hi - at < room - 32 ? hi - at : room - 32);
    for (int j = 0; j < m; ++j) {
      const uintptr_t from = reinterpret_cast<uintptr_t>(base) + src[j] + at;
      const uintptr_t first = from & ~static_cast<uintptr_t>(15);
      const int blocks = static_cast<int>((from + bytes - first + 15) / 16);
      const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(stage + j * room));
      for (int k = threadIdx.x; k < blocks; k += kThreads)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * k), "l"(first + 16 * k) : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    for (int j = 0; j < m; ++j) {
      const uintptr_t from = reinterpret_cast<uintptr_t>(base) + src[j] + at;
      const uintptr_t to = reinterpret_cast<uintptr_t>(base) + dst[j] + at, end = to + bytes;
      const uintptr_t first = to & ~static_cast<uintptr_t>(15);
      const unsigned char* held = stage + j * room + (from & 15);  // the byte for `to`
      const int blocks = static_cast<int>((end - first + 15) / 16);
      for (int k = threadIdx.x; k < blocks; k += kThreads) {
        const uintptr_t p = first + 16 * static_cast<uintptr_t>(k);
        if (p >= to && p + 16 <= end) {
          const unsigned char* q = held + (p - to);
          const unsigned o = static_cast<unsigned>(reinterpret_cast<uintptr_t>(q) & 3);
          const unsigned* w = reinterpret_cast<const unsigned*>(q - o);
          uint4 v;
          if (o == 0) {
            v = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
            v.x = __funnelshift_r(w[0], w[1], 8 * o);
            v.y = __funnelshift_r(w[1], w[2], 8 * o);
            v.z = __funnelshift_r(w[2], w[3], 8 * o);
            v.w = __funnelshift_r(w[3], w[4], 8 * o);
          }
          *reinterpret_cast<uint4*>(p) = v;
        } else {
          for (uintptr_t x = p > to ? p : to; x < p + 16 && x < end; x += unit) {
            const unsigned char* q = held + (x - to);
            if (unit == 8)
              *reinterpret_cast<uint2*>(x) = *reinterpret_cast<const uint2*>(q);
            else if (unit == 4)
              *reinterpret_cast<unsigned*>(x) = *reinterpret_cast<const unsigned*>(q);
            else if (unit == 2)
              *reinterpret_cast<unsigned short*>(x) = *reinterpret_cast<const unsigned short*>(q);
            else
              *reinterpret_cast<unsigned char*>(x) = *q;
          }
        }
      }
    }
    __syncthreads();  // read before the next range arrives
  }
}

__device__ __forceinline__ bool sequence_ok(const Params& P, int b) {
  for (int w = 0; w < P.W; ++w)
    if (P.parents[b * P.W + w] >= P.W) return false;
  if (P.lengths) {
    const int len = P.lengths[b];
    if (len < 0 || len > P.min_tokens) return false;
  }
  return true;
}

template <bool kStaged>
__global__ void __launch_bounds__(kThreads, kStaged ? kStagedCtas : 2) reorder_kernel(const __grid_constant__ Params P) {
  __shared__ long long src[SV_BEAM_MAX_BEAMS], dst[SV_BEAM_MAX_BEAMS];
  __shared__ int s_moves;
  unsigned cta = blockIdx.x;
  if (cta < static_cast<unsigned>(P.status_ctas)) {
    const int b = static_cast<int>(cta) * kThreads + static_cast<int>(threadIdx.x);
    if (b < P.B) P.status[b] = sequence_ok(P, b) ? 0u : SV_SEQ_BAD_LAYOUT;
    return;
  }
  cta -= static_cast<unsigned>(P.status_ctas);
  int k = 0;
  while (k + 1 < P.n && cta >= P.s[k + 1].first) ++k;
  const State& S = P.s[k];
  cta -= S.first;
  const int chunk = static_cast<int>(cta % static_cast<unsigned>(S.chunks));
  cta /= static_cast<unsigned>(S.chunks);
  const int seg = static_cast<int>(cta % static_cast<unsigned>(S.segs));
  const int b = static_cast<int>(cta / static_cast<unsigned>(S.segs));

  const int len = S.timed ? P.lengths[b] : S.tokens;
  const long long lo = static_cast<long long>(chunk) * P.chunk_bytes;
  long long hi = static_cast<long long>(len) * S.token_bytes;
  if (hi > lo + P.chunk_bytes) hi = lo + P.chunk_bytes;
  if (lo >= hi) return;  // also a negative length
  // the sequence's moves, by the first warp
  if (threadIdx.x < 32) {
    int moves = 0;
    bool ok = !P.lengths || (P.lengths[b] >= 0 && P.lengths[b] <= P.min_tokens);
    for (int w0 = 0; w0 < P.W; w0 += 32) {
      const int w = w0 + static_cast<int>(threadIdx.x);
      const int p = w < P.W ? P.parents[b * P.W + w] : -1;
      const bool moving = p >= 0 && p != w;
      ok = ok && !__any_sync(0xFFFFFFFFu, p >= P.W);
      const unsigned mask = __ballot_sync(0xFFFFFFFFu, moving);
      if (moving) {
        const int at = moves + __popc(mask & ((1u << threadIdx.x) - 1u));
        src[at] = p * S.beam;
        dst[at] = w * S.beam;
      }
      moves += __popc(mask);
    }
    if (threadIdx.x == 0) s_moves = ok ? moves : 0;
  }
  __syncthreads();
  const int m = s_moves;
  if (m == 0) return;
  char* base = S.data + b * S.seq + seg * S.seg;
  if constexpr (kStaged)
    move_staged(base, src, dst, m, lo, hi, S.unit);
  else
    move_aligned(base, src, dst, m, lo, hi);
}

}  // namespace svb

extern "C" sv_status sv_beam_reorder(const sv_beam_state* states, int32_t n_states, const int32_t* parents,
                                     const int32_t* lengths, int32_t batch, int32_t beams, uint32_t* status,
                                     void* stream) {
  svh::clear_error();
  if (batch < 0) return svh::fail(SV_ERR_ARG, "batch (%d) must be >= 0", batch);
  if (beams < 1 || beams > SV_BEAM_MAX_BEAMS)
    return svh::fail(SV_ERR_ARG, "beams (%d) must be in [1, %d]", beams, SV_BEAM_MAX_BEAMS);
  if (n_states < 1 || !states) return svh::fail(SV_ERR_ARG, "at least one state is needed");
  if (static_cast<long long>(batch) * beams > 0x7FFFFFFFLL) return svh::fail(SV_ERR_ARG, "batch * beams too large");
  int min_tokens = 0x7FFFFFFF;
  const int status_ctas = static_cast<int>((static_cast<long long>(batch) + svb::kThreads - 1) / svb::kThreads);
  // what divides every address and extent of a state
  // (a timed state may end after any token, another one only at its end)
  auto unit_of = [&](const sv_beam_state& s) {
    unsigned long long any = reinterpret_cast<uintptr_t>(s.data) | 16u |
                             static_cast<unsigned long long>(s.timed ? s.token_bytes : s.tokens * s.token_bytes);
    if (batch > 1) any |= static_cast<unsigned long long>(s.seq_stride);
    if (beams > 1) any |= static_cast<unsigned long long>(s.beam_stride);
    if (s.segs > 1) any |= static_cast<unsigned long long>(s.seg_stride);
    return static_cast<int>(any & (~any + 1));
  };
  long long all_ctas = 0, aligned_ctas = 0;  // of a sequence, in chunks of kMinChunk
  for (int i = 0; i < n_states; ++i) {
    const sv_beam_state& s = states[i];
    if (s.segs < 0 || s.tokens < 0 || s.token_bytes < 0)
      return svh::fail(SV_ERR_ARG, "state %d: a size is negative", i);
    if (s.seq_stride < 0 || s.beam_stride < 0 || s.seg_stride < 0)
      return svh::fail(SV_ERR_ARG, "state %d: a stride is negative", i);
    if (s.token_bytes > 0 && s.tokens > (1LL << 46) / s.token_bytes)
      return svh::fail(SV_ERR_ARG, "state %d: a segment is too large", i);
    const long long bytes = s.tokens * s.token_bytes;
    if (batch > 0 && s.segs > 0 && bytes > 0) {
      if (!s.data) return svh::fail(SV_ERR_ARG, "state %d: data is NULL", i);
      if ((s.segs > 1 && s.seg_stride < bytes) || (beams > 1 && s.beam_stride < bytes))
        return svh::fail(SV_ERR_ARG, "state %d: a stride is shorter than a segment", i);
    }
    const long long chunks = (bytes + svb::kMinChunk - 1) / svb::kMinChunk;
    const long long ctas = s.segs == 0 ? 0 : chunks > 0x7FFFFFFFLL ? chunks : chunks * s.segs;
    all_ctas += ctas;
    if (all_ctas > 0x7FFFFFFFLL || (batch > 0 && all_ctas > (0x7FFFFFFFLL - status_ctas) / batch))
      return svh::fail(SV_ERR_UNSUPPORTED, "the states are too large for one call");
    if (unit_of(s) == 16) aligned_ctas += ctas;
    if (s.timed) {
      if (!lengths) return svh::fail(SV_ERR_ARG, "state %d is timed: lengths is NULL", i);
      if (s.tokens < min_tokens) min_tokens = s.tokens;
    }
  }
  if (batch == 0) return SV_OK;
  if (!parents || !status) return svh::fail(SV_ERR_ARG, "parents or status is NULL");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int aligned_chunk = svb::kMaxChunk;
  while (aligned_chunk > svb::kMinChunk && (aligned_chunk * beams > svb::kChunkOfAll ||
                                            aligned_ctas * batch * svb::kMinChunk < static_cast<long long>(svb::kSms) * aligned_chunk))
    aligned_chunk /= 2;
  svb::Params p;
  p.parents = parents;
  p.lengths = lengths;
  p.status = status;
  p.B = batch;
  p.W = beams;
  p.min_tokens = min_tokens;
  p.status_ctas = status_ctas;
  p.n = 0;
  long long ctas = 0;
  auto launch = [&](bool staged) -> sv_status {
    const long long grid = ctas + p.status_ctas;
    if (grid == 0) return SV_OK;
    if (staged) {  // the shared-memory opt-in, once per device
      static bool attr_set[64] = {};
      int dev = 0;
      if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
      if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(svb::reorder_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   svb::kStageBytes);
        if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        attr_set[dev] = true;
      }
      svb::reorder_kernel<true><<<static_cast<unsigned>(grid), svb::kThreads, svb::kStageBytes, st>>>(p);
    } else {
      svb::reorder_kernel<false><<<static_cast<unsigned>(grid), svb::kThreads, 0, st>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    p.status = nullptr;
    p.status_ctas = 0;
    p.n = 0;
    ctas = 0;
    return SV_OK;
  };
  for (int kind = 0; kind < 2; ++kind) {  // aligned states, then the others
    const int chunk = kind == 0 ? aligned_chunk : svb::kMinChunk;
    p.chunk_bytes = chunk;
    for (int i = 0; i < n_states; ++i) {
      const sv_beam_state& s = states[i];
      const long long bytes = s.tokens * s.token_bytes;
      if (s.segs == 0 || bytes == 0) continue;
      const int unit = unit_of(s);
      if ((unit < 16) != (kind == 1)) continue;
      svb::State& q = p.s[p.n++];
      q.data = static_cast<char*>(s.data);
      q.seq = s.seq_stride;
      q.beam = s.beam_stride;
      q.seg = s.seg_stride;
      q.token_bytes = s.token_bytes;
      q.segs = s.segs;
      q.tokens = s.tokens;
      q.timed = s.timed != 0;
      q.unit = unit;
      q.chunks = static_cast<int>((bytes + chunk - 1) / chunk);
      q.first = static_cast<unsigned>(ctas);
      ctas += static_cast<long long>(q.chunks) * s.segs * batch;
      if (p.n == svb::kStates) {
        const sv_status r = launch(kind == 1);
        if (r != SV_OK) return r;
      }
    }
    if (p.n || (kind == 1 && p.status_ctas)) {
      const sv_status r = launch(kind == 1 && p.n);
      if (r != SV_OK) return r;
    }
  }
  return SV_OK;
}
