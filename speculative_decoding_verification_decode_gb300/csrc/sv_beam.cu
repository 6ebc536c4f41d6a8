// Beam search's selection over beams and vocabulary (include/sv_beam.h).
//
// The n best of W x V scores c_w + l_wv - lse_w need every logit once for the
// logarithms of the sums, and nearly none of them a second time.  Two kernels:
//
// 1 rows_kernel, over (row, slice): a streaming pass that leaves, per slice,
//   the maximum M and s = sum 2^(l k - ceil(M k)) (k = log2 e in f32; the
//   subtrahend is an integer, so partial sums are joined by exact powers of
//   two), and per group of 64 16-byte vectors its maximum.
// 2 pick_kernel, one CTA per sequence: the logarithms; tau, a lower bound of
//   the n-th best of the groups' maxima in score terms (bisection over values
//   in registers, ended as soon as between n and 2n of them lie above): n
//   candidates lie at or above tau, so only groups whose maximum reaches it
//   are read again, about n of them, and of those the logits that reach it
//   are ranked.
//
// A small call (a launch and the host's time for it are what it costs) is one
// kernel instead: a cluster of eight CTAs per sequence, whose warps each stream
// a slice of a row; the first CTA goes on as the second kernel does.
//
// An f32 score of row w is off by the row's margin (its
//   logarithm's error and roundings at the size of c_w - lse_w); a row is held
//   against tau less the largest margin among the rows that reach tau and less
//   its own, so beams far below (kept alive at -1e9, or at the lowest f32)
//   widen nobody's threshold.
//
// Order.  Scores of one beam are ordered by its logits, exactly.  Between
// beams the logarithms' f32 errors count, so pairs of different beams that lie
// closer than their bound (eps each) send their rows through precise_lse: the
// sum in 64-bit fixed point from terms good to 2^-36, equal for rows that are
// permutations of one another, whatever the order.  All scores are then
// compared as doubles.
//
// eps, relative error of a row's sum (hence absolute error of its log), in
// units of 2^-24: an exponent's rounding, 1 per unit of its size, which is
// H - H_min <= 17 bits on average under the row's own weights (17 ln 2 = 12);
// k's representation, at most 3 for entropies up to 12 nats after dividing by
// the same k; the exponential, 8 (2^-21); the additions on a term's way, 3 in
// its vector, 3 to its batch, 8 batches of a warp, 5 + 3 + 6 in warp, CTA and
// row; the logarithm of a value in [1, 2), 2.  Together 53, taken as 64 (and
// one more for each doubling of the vocabulary beyond 2^17 and each 32 slices).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/sv_beam.h"
#include "sv_host.h"
#include "sv_ptx.cuh"

namespace svs {

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
constexpr int kPickThreads = 512, kPickWarps = kPickThreads / 32;
constexpr int kCluster = 8;      // CTAs of a small call's sequence
constexpr int kGroupVecs = 64;   // 16-byte vectors per group: two per lane of a warp
constexpr int kCap = 4096;       // candidate entries a CTA holds (power of two)
constexpr int kGroupList = 1024; // groups read again before the ordered pass takes over
constexpr int kUnits = 8192;     // maxima in the bisection
constexpr int kAhead = 12;        // of a row's maxima, loads per lane in flight
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMaxF32 = 3.4028234663852886e38f;
constexpr float kLarge = 1048576.f;  // |M| above this: the row's sum is taken precisely (l k - c would lose bits)
// A maximum below this (a stretch of masked logits) leaves no sum: its base is off
// by 64 and more, so terms could be infinite, and so that a join's power of two,
// 0, would make NaN of them.  Beside a larger maximum they are nothing; a row of
// such alone is taken precisely.
constexpr float kMasked = -1073741824.f;

struct Params {
  const void* logits;
  long long stride;
  const float* scores;
  const unsigned char* finished;
  int eos, B, W, V, n;
  int groups;  // per row
  int slices;  // CTAs per row
  int per_slice;  // groups per slice
  double eps;     // bound of a fast logarithm's error
  float2* part;   // [B W][slices]: (M, s); M NaN: bad value
  float* gmax;    // [B W][groups]
  float* out_s;
  int* out_p;
  int* out_t;
  unsigned* st;
};

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int E = 4;
  static __device__ float f32(float x) { return x; }
  static __device__ void unpack(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  // the maximum of a vector, NaN if it holds one
  static __device__ float max_of(uint4 v) {
    return svk::fmax_nan(svk::fmax_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                         svk::fmax_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static __device__ float max_of(uint4 a, uint4 b) { return svk::fmax_nan(max_of(a), max_of(b)); }
  static __device__ uint4 neg_inf() { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ float f32(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ void two(unsigned w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  }
  static __device__ void unpack(uint4 v, float (&x)[8]) {
    two(v.x, x[0], x[1]);
    two(v.y, x[2], x[3]);
    two(v.z, x[4], x[5]);
    two(v.w, x[6], x[7]);
  }
  static __device__ unsigned pack_max(uint4 v) {
    return svk::bf16x2_max_nan(svk::bf16x2_max_nan(v.x, v.y), svk::bf16x2_max_nan(v.z, v.w));
  }
  static __device__ float max_of(uint4 a, uint4 b) {
    float x, y;
    two(svk::bf16x2_max_nan(pack_max(a), pack_max(b)), x, y);
    return svk::fmax_nan(x, y);
  }
  static __device__ uint4 neg_inf() { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
};
template <>
struct Elem<__half> {
  static constexpr int E = 8;
  static __device__ float f32(__half x) { return __half2float(x); }
  static __device__ void two(unsigned w, float& a, float& b) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&w));
    a = f.x;
    b = f.y;
  }
  static __device__ void unpack(uint4 v, float (&x)[8]) {
    two(v.x, x[0], x[1]);
    two(v.y, x[2], x[3]);
    two(v.z, x[4], x[5]);
    two(v.w, x[6], x[7]);
  }
  static __device__ unsigned pack_max(uint4 v) {
    return svk::f16x2_max_nan(svk::f16x2_max_nan(v.x, v.y), svk::f16x2_max_nan(v.z, v.w));
  }
  static __device__ float max_of(uint4 a, uint4 b) {
    float x, y;
    two(svk::f16x2_max_nan(pack_max(a), pack_max(b)), x, y);
    return svk::fmax_nan(x, y);
  }
  static __device__ uint4 neg_inf() { return make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u); }
};

// A row as aligned 16-byte vectors: vector i holds elements i E - head ..,
// those outside [0, V) read as -inf and never touched in memory.
template <typename T>
struct Row {
  static constexpr int E = Elem<T>::E;
  const T* p;
  int head;  // elements of vector 0 before the row
  int V;
  __device__ Row(const T* row, int vocab)
      : p(row), head(static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T))), V(vocab) {}
  __device__ long long first(long long vec) const { return vec * E - head; }
  __device__ bool inside(long long v0, long long v1) const { return first(v0) >= 0 && first(v1) + E <= V; }
  __device__ uint4 whole(long long vec) const { return __ldg(reinterpret_cast<const uint4*>(p + first(vec))); }
  __device__ uint4 load(long long vec) const {
    const long long e = first(vec);
    if (e >= 0 && e + E <= V) return whole(vec);
    uint4 v = Elem<T>::neg_inf();
    T* x = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (e + i >= 0 && e + i < V) x[i] = p[e + i];
    return v;
  }
};

__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) x = svk::fmax_nan(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

// Sum of one vector's terms 2^(x k - c), a tree.
template <int E>
__device__ __forceinline__ float terms(const float (&x)[E], float c) {
  float e[E];
#pragma unroll
  for (int i = 0; i < E; ++i) e[i] = svk::ex2_ftz(fmaf(x[i], kLog2e, -c));
#pragma unroll
  for (int h = E / 2; h > 0; h /= 2)
#pragma unroll
    for (int i = 0; i < h; ++i) e[i] += e[i + h];
  return e[0];
}

// The integer that the exponents of a sum with maximum M are taken below.
__device__ __forceinline__ float base_of(float M) { return ceilf(M * kLog2e); }

// Joins (M, s) and (M2, s2): the scale factors are powers of two.
__device__ __forceinline__ void join(float& M, float& s, float M2, float s2) {
  const float m = svk::fmax_nan(M, M2);
  if (m == M2 && M == M2) {
    s += s2;
  } else if (m > kMasked && m < INFINITY) {
    const float c = base_of(m);
    s = (M > -INFINITY ? s * svk::ex2_ftz(base_of(M) - c) : 0.f) + (M2 > -INFINITY ? s2 * svk::ex2_ftz(base_of(M2) - c) : 0.f);
  }
  M = m;
}

// Groups g, g + 1, then `step` further on, up to `end` of a row by a warp: their
// maxima, and (M, s) of what the warp saw (s per lane).
template <typename T>
__device__ __forceinline__ void stream_groups(const Row<T>& row, float* gmax, int groups, int g, int end, int step, int lane,
                                              float& M, float& s) {
  constexpr int E = Elem<T>::E;
  for (; g < end; g += step) {
    const long long v0 = static_cast<long long>(g) * kGroupVecs + lane;
    uint4 q[4];
    if (row.inside(v0 - lane, v0 - lane + 2 * kGroupVecs - 1)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = row.whole(v0 + 32 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = row.load(v0 + 32 * i);
    }
    const float ma = warp_max_nan(Elem<T>::max_of(q[0], q[1])), mb = warp_max_nan(Elem<T>::max_of(q[2], q[3]));
    if (lane == 0) {
      gmax[g] = ma;
      if (g + 1 < groups) gmax[g + 1] = mb;
    }
    const float m = svk::fmax_nan(M, svk::fmax_nan(ma, mb));
    if (m > kMasked && m < INFINITY) {
      const float c = base_of(m);
      if (M > -INFINITY && M < m) s *= svk::ex2_ftz(base_of(M) - c);
      float t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[E];
        Elem<T>::unpack(q[i], x);
        t[i] = terms(x, c);
      }
      s += (t[0] + t[1]) + (t[2] + t[3]);
    }
    M = m;
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ Params P) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long r = blockIdx.x / static_cast<unsigned>(P.slices);
  const int slice = static_cast<int>(blockIdx.x % static_cast<unsigned>(P.slices));
  if ((P.finished && P.finished[r]) || P.scores[r] == -INFINITY) return;
  const Row<T> row(static_cast<const T*>(P.logits) + r * P.stride, P.V);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g_end = min(P.groups, (slice + 1) * P.per_slice);
  float M = -INFINITY, s = 0.f;
  stream_groups(row, P.gmax + r * P.groups, P.groups, slice * P.per_slice + 2 * warp, g_end, 2 * kRowWarps, lane, M, s);
  __shared__ float2 part[kRowWarps];
  if (lane == 0) part[warp] = make_float2(M, s);
  __syncthreads();
  if (warp == 0) {
    float2 a = lane < kRowWarps ? part[lane] : make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int o = kRowWarps / 2; o > 0; o /= 2) {
      const float M2 = __shfl_xor_sync(0xFFFFFFFFu, a.x, o), s2 = __shfl_xor_sync(0xFFFFFFFFu, a.y, o);
      join(a.x, a.y, M2, s2);
    }
    if (lane == 0) P.part[r * P.slices + slice] = a;
  }
}

// ---------------------------------------------------------------- the second kernel

struct Shared {
  double log_sum[SV_BEAM_MAX_BEAMS];  // the row's logarithm less its maximum: ln sum e^(l - M)
  double cum[SV_BEAM_MAX_BEAMS];
  float M[SV_BEAM_MAX_BEAMS];
  float whole[SV_BEAM_MAX_BEAMS], rest[SV_BEAM_MAX_BEAMS];  // the logarithm to base 2: an integer and log2 of [1, 2)
  float add[SV_BEAM_MAX_BEAMS];  // f32 score = logit + add; -inf: no candidates
  float margin[SV_BEAM_MAX_BEAMS];  // by which that score may be off
  float thr[SV_BEAM_MAX_BEAMS];     // f32 scores below are not among the n best
  unsigned char ended[SV_BEAM_MAX_BEAMS], precise[SV_BEAM_MAX_BEAMS], again[SV_BEAM_MAX_BEAMS];
  unsigned long long table[32];  // 2^(j / 32), units of 2^-61
  unsigned long long sum_hi[kPickWarps], sum_lo[kPickWarps];
  int cnt[2][kPickWarps];
  int n_groups, n_entries, redo, next;
  int order[SV_BEAM_MAX_CANDIDATES];
  int rank[kPickThreads];
  union {
    unsigned unit[kUnits];         // ordered bits of the units' best f32 scores (until the groups are listed)
    unsigned long long key[kCap];  // ordered bits of the entries' scores
  };
  int2 group[kGroupList];  // (row, group)
  int index[kCap];         // w V + v
  float logit[kCap];
  unsigned char row[kCap];  // w
};

__device__ __forceinline__ unsigned f32_key(float x) {
  const unsigned b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_f32(unsigned k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ unsigned long long f64_key(double x) {
  const unsigned long long b = __double_as_longlong(x);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_f64(unsigned long long k) {
  return __longlong_as_double(k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k);
}

// Sum over the CTA; `turn` alternates the slots, so one barrier is enough.
__device__ __forceinline__ int block_sum(Shared& sm, int x, int& turn) {
  x = __reduce_add_sync(0xFFFFFFFFu, x);
  if (threadIdx.x % 32 == 0) sm.cnt[turn][threadIdx.x / 32] = x;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kPickWarps; ++w) t += sm.cnt[turn][w];
  turn ^= 1;
  return t;
}

// The integer next to x scale (|x scale| < 2^22), from the low bits of a sum with
// 1.5 2^23; x keeps what is left, exactly.  (Conversions to 64-bit integers run
// at the rate of doubles here, a sixty-fourth: the sum of a row took 70 us with two.)
__device__ __forceinline__ int take_int(float& x, float scale, float unit) {
  const float u = fmaf(x, scale, 12582912.f);
  x = fmaf(__fsub_rn(u, 12582912.f), -unit, x);
  return __float_as_int(u) - 0x4B400000;
}

// e^(x - M) in units of 2^-60, within 2^-36 of it: x - M exactly as a sum of
// two floats; times log2 e likewise, as n + j / 32 + g; 2^(j/32) from the table,
// 2^g - 1 by the first terms of its series (g ln 2 <= 0.011, the fifth power's
// term is the last above 2^-40) to 2^-38 as an integer.
__device__ __forceinline__ unsigned long long precise_term(float x, float M, const unsigned long long* table) {
  constexpr double kL = 1.4426950408889634, kN = 0.6931471805599453;
  constexpr float L1 = static_cast<float>(kL), L2 = static_cast<float>(kL - static_cast<double>(L1));
  constexpr float N1 = static_cast<float>(kN), N2 = static_cast<float>(kN - static_cast<double>(N1));
  const float y = __fsub_rn(x, M);
  const bool counts = y > -42.f;  // (or it is below 2^-60: less than a unit; -inf)
  const float bb = __fsub_rn(y, x);
  const float yl = __fadd_rn(__fsub_rn(x, __fsub_rn(y, bb)), __fsub_rn(-M, bb));
  const float t = __fmul_rn(y, L1);
  const float tl = fmaf(yl, L1, fmaf(y, L2, fmaf(y, L1, -t)));
  float g = t;
  const int k = take_int(g, 32.f, 0.03125f);  // |t| <= 61 where it counts
  const float z = __fmul_rn(g, N1);
  const float zl = fmaf(tl, N1, fmaf(g, N2, fmaf(g, N1, -z)));
  const float a = z + zl;
  float w = fmaf(a * a, fmaf(a, fmaf(a, fmaf(a, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f), zl), zr = z;
  // z + w in units of 2^-37, from |z| < 0.0114 in units of 2^-28, |w| < 6.6e-5 of 2^-35, and what is left
  int Z = take_int(zr, 0x1p28f, 0x1p-28f) * 512;
  Z += take_int(w, 0x1p35f, 0x1p-35f) * 4;
  float left = zr + w;
  Z += take_int(left, 0x1p37f, 0x1p-37f);
  const long long e = static_cast<long long>(table[k & 31]);
  const int shift = 1 - (k >> 5);
  const unsigned long long q = static_cast<unsigned long long>(e + (static_cast<long long>(static_cast<int>(e >> 31)) * Z >> 6));
  return counts ? q >> (shift & 63) : 0ull;
}

// The row's logarithm less its maximum to better than 2^-35, by the whole CTA.
// (Their sum would keep that only up to |M| = 2^18.)
// (A call of 64 x 8 x 128256 with two equal beams in one sequence: 114 us, where
// 64-bit conversions, a branch per term and loads without a successor took 187.)
template <typename T>
__device__ __noinline__ void precise_lse(Shared& sm, const Params& P, int b, int w) {
  constexpr int E = Elem<T>::E;
  const Row<T> row(static_cast<const T*>(P.logits) + (static_cast<long long>(b) * P.W + w) * P.stride, P.V);
  if (threadIdx.x < 32) sm.table[threadIdx.x] = static_cast<unsigned long long>(exp2(threadIdx.x / 32.0) * 0x1p61);
  __syncthreads();
  const float M = sm.M[w];
  unsigned long long hi = 0, lo = 0;
  const long long vecs = (static_cast<long long>(row.head) + P.V + E - 1) / E;
  uint4 next = threadIdx.x < vecs ? row.load(threadIdx.x) : Elem<T>::neg_inf();
  for (long long v = threadIdx.x; v < vecs; v += kPickThreads) {
    float x[E];
    Elem<T>::unpack(next, x);
    if (v + kPickThreads < vecs) next = row.load(v + kPickThreads);
    unsigned long long q = 0;  // of eight terms up to 2^60 each
#pragma unroll
    for (int i = 0; i < E; ++i) q += precise_term(x[i], M, sm.table);
    hi += q >> 32;
    lo += q & 0xFFFFFFFFu;
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    hi += __shfl_xor_sync(0xFFFFFFFFu, hi, o);
    lo += __shfl_xor_sync(0xFFFFFFFFu, lo, o);
  }
  if (threadIdx.x % 32 == 0) {
    sm.sum_hi[threadIdx.x / 32] = hi;
    sm.sum_lo[threadIdx.x / 32] = lo;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    hi = lo = 0;
    for (int i = 0; i < kPickWarps; ++i) {
      hi += sm.sum_hi[i];
      lo += sm.sum_lo[i];
    }
    const double total = static_cast<double>(hi + (lo >> 32)) + static_cast<double>(lo & 0xFFFFFFFFu) * 0x1p-32;
    sm.log_sum[w] = log(total * 0x1p-28);
    sm.precise[w] = 1;
    sm.again[w] = 0;
  }
  __syncthreads();
}

__device__ __forceinline__ double score_of(const Shared& sm, int w, float l) {
  return sm.ended[w] ? sm.cum[w] : sm.cum[w] + ((static_cast<double>(l) - static_cast<double>(sm.M[w])) - sm.log_sum[w]);
}

__device__ __forceinline__ bool before(unsigned long long ka, int ia, unsigned long long kb, int ib) {
  return ka > kb || (ka == kb && ia < ib);
}

// order[0..min(L, most) - 1]: the entries' places, best first.
__device__ __forceinline__ void sort_entries(Shared& sm, int L, int most) {
  if (L <= kPickThreads) {  // by counting, each entry's rivals split over several threads
    int lanes = 32;
    while (lanes < L) lanes *= 2;
    const int i = threadIdx.x & (lanes - 1), parts = kPickThreads / lanes, part = threadIdx.x / lanes;
    sm.rank[threadIdx.x] = 0;
    __syncthreads();
    if (i < L) {
      const unsigned long long k = sm.key[i];
      const int x = sm.index[i];
      int rank = 0;
#pragma unroll 2
      for (int j = part; j < L; j += parts) rank += before(sm.key[j], sm.index[j], k, x);
      if (rank) atomicAdd(&sm.rank[i], rank);
    }
    __syncthreads();
    if (threadIdx.x < L && sm.rank[threadIdx.x] < most) sm.order[sm.rank[threadIdx.x]] = threadIdx.x;
    __syncthreads();
    return;
  }
  int size = kPickThreads;
  while (size < L) size *= 2;
  for (int i = L + threadIdx.x; i < size; i += kPickThreads) {
    sm.key[i] = 0;
    sm.index[i] = 0x7FFFFFFF;
  }
  __syncthreads();
  for (int k = 2; k <= size; k *= 2)
    for (int h = k / 2; h > 0; h /= 2) {
      for (int t = threadIdx.x; t < size / 2; t += kPickThreads) {
        const int i = (t & ~(h - 1)) * 2 + (t & (h - 1)), j = i + h;
        const bool up = (i & k) == 0;  // best first
        if (before(sm.key[j], sm.index[j], sm.key[i], sm.index[i]) == up) {
          const unsigned long long kk = sm.key[i];
          const int ii = sm.index[i];
          const float ll = sm.logit[i];
          const unsigned char rr = sm.row[i];
          sm.key[i] = sm.key[j];
          sm.index[i] = sm.index[j];
          sm.logit[i] = sm.logit[j];
          sm.row[i] = sm.row[j];
          sm.key[j] = kk;
          sm.index[j] = ii;
          sm.logit[j] = ll;
          sm.row[j] = rr;
        }
      }
      __syncthreads();
    }
  for (int i = threadIdx.x; i < most && i < L; i += kPickThreads) sm.order[i] = i;
  __syncthreads();
}

// Appends an entry; counts it even where the list is full.
__device__ __forceinline__ void append(Shared& sm, int V, int w, int token, float logit) {
  const int at = atomicAdd(&sm.n_entries, 1);
  if (at < kCap) {
    sm.index[at] = w * V + token;
    sm.row[at] = static_cast<unsigned char>(w);
    sm.logit[at] = logit;
  }
}

__device__ __forceinline__ void score_entries(Shared& sm, int from, int L) {
  for (int i = from + threadIdx.x; i < L; i += kPickThreads) sm.key[i] = f64_key(score_of(sm, sm.row[i], sm.logit[i]));
  __syncthreads();
}

// A row's f32 addend and margin from its score and its logarithm in f32.  An
// addend that leaves f32's range, at either end (a score of 1e32 on a row whose
// logits are all near the lowest f32), says nothing.
__device__ __forceinline__ float set_add(Shared& sm, int w, float c, float lse, double eps) {
  const float a = __fsub_rn(c, lse);
  const bool fits = fabsf(a) <= kMaxF32;
  const float add = fits ? a : copysignf(kMaxF32, a);
  sm.add[w] = add;
  sm.margin[w] = fits ? static_cast<float>(eps) + (fabsf(add) * 0x1p-22f + fabsf(c) * 0x1p-22f + fabsf(lse) * 0x1p-22f) : INFINITY;
  return add;
}

// More candidates than the lists hold (many equal logits, rows in ascending
// order): a pass over the tiles of the rows in index order that keeps the n
// best so far.  Later equals lose their ties, so a full list only admits
// strictly better entries.
template <typename T>
__device__ __noinline__ int ordered_pass(Shared& sm, const Params& P, int b) {
  constexpr int E = Elem<T>::E, kTileVecs = 256;  // 4 groups; at most 2048 entries
  constexpr int kTileGroups = kTileVecs / kGroupVecs;
  const int tiles = (P.groups + kTileGroups - 1) / kTileGroups;
  const long long all = static_cast<long long>(tiles) * P.W;
  int have = 0;                  // entries kept
  unsigned long long worst = 0;  // key of the n-th best once n are kept
  if (threadIdx.x == 0) sm.n_entries = 0;
  __syncthreads();
  for (long long t0 = 0; t0 < all;) {
    // the first tile at or after t0 that may hold better entries
    if (threadIdx.x == 0) sm.next = kPickThreads;
    __syncthreads();
    const long long mine = t0 + threadIdx.x;
    bool may = false;
    if (mine < all) {
      const int w = static_cast<int>(mine / tiles), tile = static_cast<int>(mine % tiles);
      if (sm.ended[w]) {
        may = tile == 0 && (have < P.n || f64_key(sm.cum[w]) > worst);
      } else if (sm.add[w] > -INFINITY) {
        const float* gm = P.gmax + (static_cast<long long>(b) * P.W + w) * P.groups;
        float m = -INFINITY;
        for (int g = tile * kTileGroups; g < min(P.groups, (tile + 1) * kTileGroups); ++g) m = fmaxf(m, gm[g]);
        may = m > -INFINITY && m + sm.add[w] >= sm.thr[w] && (have < P.n || f64_key(score_of(sm, w, m)) > worst);
      }
    }
    if (may) atomicMin(&sm.next, static_cast<int>(threadIdx.x));
    __syncthreads();
    const int found = sm.next;
    __syncthreads();
    if (found == kPickThreads) {
      t0 += kPickThreads;
      continue;
    }
    t0 += found;
    const int w = static_cast<int>(t0 / tiles), tile = static_cast<int>(t0 % tiles);
    ++t0;
    if (sm.ended[w]) {
      if (threadIdx.x == 0) append(sm, P.V, w, P.eos, 0.f);
    } else if (threadIdx.x < kTileVecs) {
      const Row<T> row(static_cast<const T*>(P.logits) + (static_cast<long long>(b) * P.W + w) * P.stride, P.V);
      const long long v = static_cast<long long>(tile) * kTileVecs + threadIdx.x;
      float x[E];
      Elem<T>::unpack(row.load(v), x);
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (x[i] > -INFINITY && (have < P.n || f64_key(score_of(sm, w, x[i])) > worst))
          append(sm, P.V, w, static_cast<int>(row.first(v) + i), x[i]);
    }
    __syncthreads();
    const int L = sm.n_entries;
    __syncthreads();
    if (L == have) continue;
    score_entries(sm, have, L);
    if (L >= P.n) {  // keep the n best, in order, at the front
      sort_entries(sm, L, P.n);
      unsigned long long k = 0;
      int x = 0;
      float l = 0.f;
      unsigned char w_of = 0;
      if (threadIdx.x < P.n) {
        const int i = sm.order[threadIdx.x];
        k = sm.key[i];
        x = sm.index[i];
        l = sm.logit[i];
        w_of = sm.row[i];
      }
      __syncthreads();
      if (threadIdx.x < P.n) {
        sm.key[threadIdx.x] = k;
        sm.index[threadIdx.x] = x;
        sm.logit[threadIdx.x] = l;
        sm.row[threadIdx.x] = w_of;
      }
      if (threadIdx.x == 0) sm.n_entries = P.n;
      __syncthreads();
      worst = sm.key[P.n - 1];
      have = P.n;
    } else {
      have = L;
    }
  }
  return have;
}

// A dozen short phases on a handful of values: what it takes is barriers, trips
// to L2 and the instructions of few warps, not their fetching (a second pass over
// the same takes as long).  So a warp takes a row's maxima and sums together, in
// one round of loads, and its logarithm in f32; the doubles of all rows are taken
// at once; groups' vectors without a candidate go by after one comparison; and
// nothing divides.  (16 x 152064 x 8 f16: 25.4 to 20.7 us with the first kernel.)
template <typename T, bool kOne>
__device__ __forceinline__ void pick(const Params& P, int b) {
  constexpr int E = Elem<T>::E;
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const long long r0 = static_cast<long long>(b) * P.W;
  if (tid == 0) sm.n_groups = sm.n_entries = sm.redo = 0;
  int q = 1;  // a unit of the bisection: q groups of a row
  while (static_cast<long long>((P.groups + q - 1) / q) * P.W > kUnits) ++q;
  const int units = q == 1 ? P.groups : (P.groups + q - 1) / q, total = units * P.W;
  const unsigned none = f32_key(-INFINITY);
  if constexpr (!kOne) asm volatile("griddepcontrol.wait;" ::: "memory");

  // the rows' logarithms, and the units' best scores
  unsigned top = 0, low = 0xFFFFFFFFu;
  int finite = 0;
  bool bad = false, large = false;
  auto put = [&](int at, float x) {
    const unsigned k = f32_key(x + 0.f);  // (-0 is 0)
    sm.unit[at] = k;
    if (k > none) {
      ++finite;
      top = max(top, k);
      low = min(low, k);
    }
  };
  auto unit_max = [&](int w, int u) {
    float x = -INFINITY;
    for (int g = u * q; g < min(P.groups, u * q + q); ++g) x = fmaxf(x, P.gmax[(r0 + w) * P.groups + g]);
    return x;
  };
#pragma unroll 1
  for (int w = warp; w < P.W; w += kPickWarps) {
    const float c = P.scores[r0 + w];
    const bool fin = P.finished && P.finished[r0 + w], live = !fin && c != -INFINITY, ended = fin && c > -INFINITY;
    float M = -INFINITY, s = 0.f, m[kAhead];
    const int ahead = q == 1 ? min(units, 32 * kAhead) : 0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) m[i] = live && lane + 32 * i < ahead ? P.gmax[(r0 + w) * P.groups + lane + 32 * i] : -INFINITY;
    if (live)
      for (int i = lane; i < P.slices; i += 32) {
        const float2 a = P.part[(r0 + w) * P.slices + i];
        join(M, s, a.x, a.y);
      }
#pragma unroll 1
    for (int o = 16; o > 0; o /= 2) {
      const float M2 = __shfl_xor_sync(0xFFFFFFFFu, M, o), s2 = __shfl_xor_sync(0xFFFFFFFFu, s, o);
      join(M, s, M2, s2);
    }
    float add = -INFINITY;
    if (lane == 0) {
      // log2 s = exponent + log2 of the significand; in f32 for the addend, the
      // doubles (a sixteenth of a warp at a time on this machine) all at once later
      const int e = static_cast<int>(__float_as_uint(s) >> 23) - 127;
      const float f = __uint_as_float((__float_as_uint(s) & 0x7FFFFFu) | 0x3F800000u);
      const float whole = base_of(M) + static_cast<float>(e), rest = log2f(f);
      sm.M[w] = M;
      sm.whole[w] = whole;
      sm.rest[w] = rest;
      sm.add[w] = -INFINITY;
      sm.margin[w] = 0.f;
      if (M > -INFINITY) add = set_add(sm, w, c, (whole + rest) * 0.6931471805599453f, P.eps);
      sm.ended[w] = ended;
      sm.precise[w] = 0;
      sm.again[w] = M > -INFINITY && fabsf(M) > kLarge;
    }
    bad |= isnan(c) || c == INFINITY || isnan(M) || M == INFINITY;
    large |= M > -INFINITY && fabsf(M) > kLarge;
    add = __shfl_sync(0xFFFFFFFFu, add, 0);
    if (ended && lane == 0) m[0] = c;
    const float plus = ended ? 0.f : add;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (lane + 32 * i < ahead) put(w * units + lane + 32 * i, m[i] + plus);
    for (int u = ahead + lane; u < units; u += 32) put(w * units + u, ended ? (u == 0 ? c : -INFINITY) : live ? unit_max(w, u) + plus : -INFINITY);
  }
  if (__syncthreads_or(bad)) {
    for (int k = tid; k < P.n; k += kPickThreads) {
      P.out_s[static_cast<long long>(b) * P.n + k] = -INFINITY;
      P.out_p[static_cast<long long>(b) * P.n + k] = -1;
      P.out_t[static_cast<long long>(b) * P.n + k] = -1;
    }
    if (tid == 0) P.st[b] = SV_SEQ_BAD_VALUE;
    return;
  }
  if (__syncthreads_or(large)) {  // rows whose fast sum says nothing: precisely, and their scores again
    top = 0;
    low = 0xFFFFFFFFu;
    finite = 0;
    for (int w = 0; w < P.W; ++w) {
      if (sm.again[w]) {
        precise_lse<T>(sm, P, b, w);
        if (tid == 0) set_add(sm, w, P.scores[r0 + w], static_cast<float>(static_cast<double>(sm.M[w]) + sm.log_sum[w]), P.eps);
        __syncthreads();
      }
      for (int u = tid; u < units; u += kPickThreads)
        put(w * units + u, sm.ended[w] ? (u == 0 ? P.scores[r0 + w] : -INFINITY)
                                       : sm.add[w] > -INFINITY ? unit_max(w, u) + sm.add[w] : -INFINITY);
    }
  }

  if (tid < P.W) {
    constexpr double kBack = 1.0 / static_cast<double>(kLog2e);
    sm.cum[tid] = P.scores[r0 + tid] + 0.f;  // (a score of -0 is one of 0)
    if (!sm.precise[tid])
      sm.log_sum[tid] = (static_cast<double>(sm.whole[tid]) + static_cast<double>(sm.rest[tid])) * kBack - static_cast<double>(sm.M[tid]);
  }

  // tau: at least n units reach it, and hardly more than 2 n.  Where there are
  // fewer units with candidates than that (one live beam, as in a search's first
  // step), all their groups are listed, and a second round takes smaller units of
  // those: without it 70 to 540 us went into the ordered pass.
  int turn = 0, n_groups = 0, in = total;
  bool finer = false;
  unsigned thr_key = none + 1;  // of the lowest threshold of a row
#pragma unroll 1
  for (;;) {
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    if (lane == 0) sm.sum_lo[warp] = static_cast<unsigned long long>(top) << 32 | low;
    const int all = block_sum(sm, finite, turn);
#pragma unroll 1
    for (int w = 0; w < kPickWarps; ++w) {
      top = max(top, static_cast<unsigned>(sm.sum_lo[w] >> 32));
      low = min(low, static_cast<unsigned>(sm.sum_lo[w]));
    }
    if (all >= P.n) {
      unsigned lo = low, hi = top + 1;  // at least n units >= lo, fewer than n >= hi
      int above = all;
#pragma unroll 1
      while (hi - lo > 1 && above > 2 * P.n) {
        const unsigned mid = lo + (hi - lo) / 2;
        int c = 0;
#pragma unroll 4
        for (int i = tid; i < in; i += kPickThreads) c += sm.unit[i] >= mid;
        c = block_sum(sm, c, turn);
        if (c >= P.n) {
          lo = mid;
          above = c;
        } else {
          hi = mid;
        }
      }
      const float tau = fminf(key_f32(lo), kMaxF32);  // (a sum may round past f32's range: its row's margin is as wide)
      // (every warp computes, and writes, the same)
      float widest = 0.f, all_widest = 0.f;
#pragma unroll 1
      for (int w = lane; w < P.W; w += 32) {
        const float best = sm.ended[w] ? P.scores[r0 + w] : sm.M[w] + sm.add[w];  // (-inf where it has none)
        if (best >= tau) widest = fmaxf(widest, sm.margin[w]);
        all_widest = fmaxf(all_widest, sm.margin[w]);
      }
      widest = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(widest)));
      all_widest = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(all_widest)));
      const float base = tau - fabsf(tau) * 0x1p-21f - widest;
#pragma unroll 1
      for (int w = lane; w < P.W; w += 32) sm.thr[w] = base - sm.margin[w];
      thr_key = max(thr_key, f32_key(base - all_widest));
    } else {
      for (int w = lane; w < P.W; w += 32) sm.thr[w] = -INFINITY;
    }
    __syncwarp();

    // the groups that reach it
    if (!finer) {
#pragma unroll 1
      for (int i = tid; i < total; i += kPickThreads)
        if (sm.unit[i] >= thr_key) {
          const int w = i / units, u = i - w * units;
          if (!(key_f32(sm.unit[i]) >= sm.thr[w])) continue;
          if (sm.ended[w]) {
            append(sm, P.V, w, P.eos, 0.f);
          } else {
#pragma unroll 1
            for (int g = u * q; g < min(P.groups, u * q + q); ++g)
              if (q == 1 || P.gmax[(r0 + w) * P.groups + g] + sm.add[w] >= sm.thr[w]) {
                const int at = atomicAdd(&sm.n_groups, 1);
                if (at < kGroupList) sm.group[at] = make_int2(w, g);
              }
          }
        }
    }
    __syncthreads();
    n_groups = sm.n_groups;
    if (finer || all >= P.n || n_groups == 0 || n_groups > kGroupList) break;
    finer = true;
    int sub = 64;  // units of a group
    while (n_groups * sub > kUnits) sub /= 2;
    in = n_groups * sub;
    top = 0;
    low = 0xFFFFFFFFu;
    finite = 0;
#pragma unroll 1
    for (int j = warp; j < n_groups; j += kPickWarps) {
      const int2 wg = sm.group[j];
      const Row<T> row(static_cast<const T*>(P.logits) + (r0 + wg.x) * P.stride, P.V);
      const long long v = static_cast<long long>(wg.y) * kGroupVecs + lane;
      const uint4 v0 = row.load(v), v1 = row.load(v + 32);
      const float add = sm.add[wg.x], m0 = Elem<T>::max_of(v0, v0), m1 = Elem<T>::max_of(v1, v1);
      if (sub == 64) {
        put(j * 64 + lane, m0 + add);
        put(j * 64 + 32 + lane, m1 + add);
      } else {
        float m = fmaxf(m0, m1);
        const int lanes = 32 / sub;
        for (int o = 1; o < lanes; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (lane % lanes == 0) put(j * sub + lane / lanes, m + add);
      }
    }
  }

  // their logits that do
  if (n_groups <= kGroupList) {
    // half a group at a time, four loads per lane in flight; most vectors have
    // nothing, which their maximum tells
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int j0 = warp; j0 < 2 * n_groups; j0 += kBatch * kPickWarps) {
      uint4 q[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = j0 + i * kPickWarps;
        q[i] = Elem<T>::neg_inf();
        if (j < 2 * n_groups) {
          const int2 wg = sm.group[j / 2];
          const Row<T> row(static_cast<const T*>(P.logits) + (r0 + wg.x) * P.stride, P.V);
          const long long v = static_cast<long long>(wg.y) * kGroupVecs + 32 * (j & 1) + lane;
          q[i] = row.inside(v, v) ? row.whole(v) : row.load(v);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = j0 + i * kPickWarps;
        if (j >= 2 * n_groups) break;
        const int2 wg = sm.group[j / 2];
        const float add = sm.add[wg.x], thr = sm.thr[wg.x], top_of = Elem<T>::max_of(q[i], q[i]);
        if (top_of > -INFINITY && top_of + add >= thr) {
          const Row<T> row(static_cast<const T*>(P.logits) + (r0 + wg.x) * P.stride, P.V);
          const int e = static_cast<int>(row.first(static_cast<long long>(wg.y) * kGroupVecs + 32 * (j & 1) + lane));
          float x[E];
          Elem<T>::unpack(q[i], x);
#pragma unroll
          for (int k = 0; k < E; ++k)
            if (x[k] > -INFINITY && x[k] + add >= thr) append(sm, P.V, wg.x, e + k, x[k]);
        }
      }
    }
  }
  __syncthreads();
  int L = sm.n_entries;
  if (L > kCap || n_groups > kGroupList) {
    // every row that may hold candidates, precisely; then the ordered pass
    if (finer) {
      for (int i = tid; i < n_groups; i += kPickThreads) sm.again[sm.group[i].x] = 1;
    } else {
      for (int i = tid; i < total; i += kPickThreads)
        if (sm.unit[i] >= thr_key) sm.again[i / units] = 1;
    }
    __syncthreads();
    for (int w = 0; w < P.W; ++w)
      if (sm.again[w] && !sm.ended[w] && !sm.precise[w]) precise_lse<T>(sm, P, b, w);
    L = ordered_pass<T>(sm, P, b);
    score_entries(sm, 0, L);
    sort_entries(sm, L, P.n);
  } else {
    score_entries(sm, 0, L);
    sort_entries(sm, L, P.n);
    // pairs of different beams that the logarithms' errors could swap: neighbours
    // among the n best, and whatever lies as near to the last of them
    auto flag = [&](int wi, int wj) {
      if (!sm.precise[wi] && !sm.ended[wi]) sm.again[wi] = sm.redo = 1;
      if (!sm.precise[wj] && !sm.ended[wj]) sm.again[wj] = sm.redo = 1;
    };
    if (tid + 1 < P.n && tid + 1 < L) {
      const int i = sm.order[tid], j = sm.order[tid + 1], wi = sm.row[i], wj = sm.row[j];
      if (wi != wj && key_f64(sm.key[i]) - key_f64(sm.key[j]) <= 2.0 * P.eps) flag(wi, wj);
    }
    if (L > P.n) {
      const int last = sm.order[P.n - 1], wl = sm.row[last];
      const unsigned long long k_hi = f64_key(key_f64(sm.key[last]) + 2.0 * P.eps),
                               k_lo = f64_key(key_f64(sm.key[last]) - 2.0 * P.eps);
#pragma unroll 1
      for (int i = tid; i < L; i += kPickThreads)
        if (sm.key[i] >= k_lo && sm.key[i] <= k_hi && sm.row[i] != wl) flag(sm.row[i], wl);
    }
    __syncthreads();
    if (sm.redo) {
      for (int w = 0; w < P.W; ++w)
        if (sm.again[w]) precise_lse<T>(sm, P, b, w);
      score_entries(sm, 0, L);
      sort_entries(sm, L, P.n);
    }
  }
  if (tid < P.n) {
    float s = -INFINITY;
    int p = -1, t = -1;
    if (tid < L) {
      const int i = sm.order[tid];
      s = static_cast<float>(key_f64(sm.key[i]));
      if (s > -INFINITY) {  // (or it lies below f32's range)
        p = sm.row[i];
        t = sm.index[i] - p * P.V;
      }
    }
    const long long o = static_cast<long long>(b) * P.n + tid;
    P.out_s[o] = s;
    P.out_p[o] = p;
    P.out_t[o] = t;
  }
  if (tid == 0) P.st[b] = 0u;
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads, 1)  // (without the block count 64 registers, and spills)
    pick_kernel(const __grid_constant__ Params P) {
  pick<T, false>(P, blockIdx.x);
}

template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPickThreads, 1) one_kernel(const __grid_constant__ Params P) {
  const int b = blockIdx.x / kCluster, rank = blockIdx.x % kCluster, lane = threadIdx.x % 32;
  for (int i = rank * kPickWarps + threadIdx.x / 32; i < P.W * P.slices; i += kCluster * kPickWarps) {
    const int w = i / P.slices, slice = i - w * P.slices;
    const long long r = static_cast<long long>(b) * P.W + w;
    if ((P.finished && P.finished[r]) || P.scores[r] == -INFINITY) continue;
    const Row<T> row(static_cast<const T*>(P.logits) + r * P.stride, P.V);
    float M = -INFINITY, s = 0.f;
    stream_groups(row, P.gmax + r * P.groups, P.groups, slice * P.per_slice, min(P.groups, (slice + 1) * P.per_slice), 2, lane, M, s);
    if (lane == 0) P.part[r * P.slices + slice] = make_float2(M, s);
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0) pick<T, true>(P, b);
}

// Sizes of a call: groups of a row at the worst alignment, slices, workspace.
struct Plan {
  int groups, per_slice, slices;
  bool one;  // one kernel
  size_t part_bytes, bytes;
};

Plan plan_of(int batch, int beams, int vocab, int elem) {
  Plan p;
  const long long E = 16 / elem;
  const long long vecs = (vocab + 2 * (E - 1)) / E;  // ceil((E - 1 + vocab) / E)
  p.groups = static_cast<int>((vecs + kGroupVecs - 1) / kGroupVecs);
  const long long rows = static_cast<long long>(batch) * beams;
  // groups per CTA: as many as leave four waves of five CTAs per SM, between
  // two per warp (one load round) and sixteen
  int per = 2 * kRowWarps;
  while (per < 16 * kRowWarps && rows * ((p.groups + per - 1) / per) > 152 * 5 * 4) per *= 2;
  // one kernel where a cluster streams a sequence in less than the host takes
  // to issue a call, and the clusters find room at once: calls one after
  // another take 21-23 us, with two kernels 25-27; on the device 10.6 against
  // 10.5 us (4 x 32000 bf16), at the largest 20.5 against 19.0 (19 sequences of
  // 8 x 98000) and 18.5 against 14.8 (one of 16 x 48000)
  p.one = batch <= 152 / kCluster && static_cast<long long>(beams) * vocab * elem <= kCluster * 196608;
  if (p.one) {
    const int s = kCluster * kPickWarps / beams;  // slices of a row: a warp each
    per = ((p.groups + s - 1) / s + 1) / 2 * 2;
  }
  p.per_slice = per;
  p.slices = (p.groups + per - 1) / per;
  p.part_bytes = (static_cast<size_t>(rows) * p.slices * sizeof(float2) + 15) / 16 * 16;
  p.bytes = p.part_bytes + (static_cast<size_t>(rows) * p.groups * sizeof(float) + 15) / 16 * 16;
  return p;
}

}  // namespace svs

extern "C" {

size_t sv_beam_select_workspace_size(int32_t batch, int32_t beams, int32_t vocab, int32_t n) {
  if (batch < 0 || beams < 1 || beams > SV_BEAM_MAX_BEAMS || vocab < 1 || n < 1 || n > SV_BEAM_MAX_CANDIDATES) return 0;
  const svs::Plan a = svs::plan_of(batch, beams, vocab, 4), b = svs::plan_of(batch, beams, vocab, 2);
  return a.bytes > b.bytes ? a.bytes : b.bytes;  // any dtype
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
  const svs::Plan plan = svs::plan_of(batch, beams, vocab, static_cast<int>(elem));
  const long long ctas = static_cast<long long>(batch) * beams * plan.slices;
  if (ctas > 0x7FFFFFFFLL) return svh::fail(SV_ERR_UNSUPPORTED, "batch * beams * vocab too large for one launch");
  svs::Params p;
  p.logits = logits;
  p.stride = row_stride;
  p.scores = scores;
  p.finished = finished;
  p.eos = eos;
  p.B = batch;
  p.W = beams;
  p.V = vocab;
  p.n = n;
  p.groups = plan.groups;
  p.slices = plan.slices;
  p.per_slice = plan.per_slice;
  int units = 64 + plan.slices / 32;
  for (long long v = 131072; v < vocab; v *= 2) ++units;
  p.eps = units / 16777216.0;
  p.part = static_cast<float2*>(workspace);
  p.gmax = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + plan.part_bytes);
  p.out_s = out_scores;
  p.out_p = out_parents;
  p.out_t = out_tokens;
  p.st = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // the shared-memory opt-in, once per (device, element type)
  static bool attr_set[64][3] = {};
  auto go = [&](void (*rows)(svs::Params), void (*pick)(svs::Params), void (*one)(svs::Params)) -> sv_status {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    if (!attr_set[dev][dtype]) {
      cudaError_t e = cudaFuncSetAttribute(pick, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(sizeof(svs::Shared)));
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(svs::Shared)));
      if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
      attr_set[dev][dtype] = true;
    }
    if (plan.one) {
      one<<<static_cast<unsigned>(batch * svs::kCluster), svs::kPickThreads, sizeof(svs::Shared), st>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
      return SV_OK;
    }
    rows<<<static_cast<unsigned>(ctas), svs::kRowThreads, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    // the second kernel is set up while the first one's last CTAs run; it
    // waits for them before it reads anything they wrote
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(batch));
    cfg.blockDim = dim3(svs::kPickThreads);
    cfg.dynamicSmemBytes = sizeof(svs::Shared);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, pick, p);
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return SV_OK;
  };
  switch (dtype) {
    case SV_F32: return go(svs::rows_kernel<float>, svs::pick_kernel<float>, svs::one_kernel<float>);
    case SV_BF16: return go(svs::rows_kernel<__nv_bfloat16>, svs::pick_kernel<__nv_bfloat16>, svs::one_kernel<__nv_bfloat16>);
    default: return go(svs::rows_kernel<__half>, svs::pick_kernel<__half>, svs::one_kernel<__half>);
  }
}

}  // extern "C"
