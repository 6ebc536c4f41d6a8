// The LM head with a projection in 4 bits (include/sv_lm_head_q4.h).
//
// Logits = H W^T with W[v][k] = s[v][k / g] (q[v][k] - z[v][k / g]).
//
// The projection's bytes bound the product up to some tens of rows: every
// weight is read once for up to 64 rows of states, and what has to be kept
// up with that stream is turning 4-bit codes into operands.  So:
//   - the weights are the A operand (128 vocabulary rows of an MMA), the
//     states the B operand (N rows).  A thread owns a vocabulary row: it takes
//     the row's codes from shared memory (TMA, 128-byte swizzle), makes the
//     integers q - z in 16 bits (exact), and stores them as its lane of tensor
//     memory, from where the MMA reads them: no round trip through shared
//     memory.
//   - one MMA chain per group; its f32 result, N columns of the thread's lane,
//     is read back and added to the thread's N f32 sums times the group's
//     scale.  No weight is rounded, and a scale is one register.
//   - operands and results go through a ring of buffers in tensor memory, so
//     the tensor cores work on some groups while the warps turn the next and
//     add the last.  A warp passes its turn with a single arrival: by then it
//     has read the result that the MMA will overwrite.
//   - two warpgroups share the rows: each turns half of a group's codes and
//     keeps half of the N sums, so an SM has sixteen warps to hide the steps'
//     latencies with.  Nothing else may wait in their way: scales come by
//     cp.async from warps of their own.
//   - each half has an MMA warp whose lanes all run the loop, so that
//     descriptors stay in uniform registers.  One thread that issued for both
//     halves took 1700 clocks per 128 columns and half, and all waited for it
//     (44 rows x 152064 x 4096, groups of 128: 177 us, now 135).
// A CTA has H halves of 128 rows (8 warps each), H warps that supply (the first
// also starts the copies) and H that issue.  Twenty warps per SM leave 96
// registers each; a twenty-first left 80 and spilled.  Its tiles have R <= 128 H
// rows, R chosen so that the vocabulary divides evenly over the CTAs (the MMA's
// idle rows cost nothing).
//
// Measured: 44 rows x 152064 x 4096 of bf16 states, groups of 32: 200 us (28% of
// the memory's rate), 64: 175, 128: 135.  Without the stores to tensor memory
// and the turning 127 / - / 89 us, with neither turning nor adding nor MMA 78 /
// - / 73: what the hand-overs and the stream itself take.  Measured and not
// taken: warps of their own for the adding (215 / 196 / 157 us), one polling
// warp per half with the others at a barrier (223 / 198 / 159), 64 columns per
// step with two buffers for groups of 32 and 64 (207 / 180), four chains of 64
// rows (254 against 214 then).
//
// Every wait is bounded; one that gives up sets bit 0 of *err.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "../../include/sv_lm_head_q4.h"
#include "sv_host.h"
#include "sv_ptx.cuh"

namespace svq {

using svk::mbar_arrive_expect_tx;
using svk::mbar_arrive_local;
using svk::mbar_init;
using svk::smem_u32;

constexpr int kStageK = 256;    // weights of a row per ring stage: 128 bytes
constexpr int kMaxStages = 6;
constexpr int kHalfCols = 256;  // tensor-memory columns of a half: `ring` operands of step / 2 columns and a result of N per group
constexpr int kMaxRing = 2;

__host__ __device__ constexpr int per_stage_of(int group) { return kStageK / group; }
// Columns of W that pass between the warps and the MMA at a time: a hand-over
// costs some 900 clocks whatever its size, so as many as the results of all
// their groups leave room for (groups of 32, 44 rows: 200 us with one buffer of
// 128 columns, 207 with two of 64).
__host__ __device__ constexpr int step_of(int group, int n) { return group == 32 && n == 64 ? 64 : 128; }
// Operand / result buffers that fit.
__host__ __device__ constexpr int ring_of(int group, int n) {
  return 2 * (step_of(group, n) / 2 + step_of(group, n) / group * n) <= kHalfCols ? 2 : 1;
}

struct Args {
  const void* scales;
  const unsigned char* zeros;
  float* out0;
  float* out1;
  unsigned* err;
  long long ld;
  int scale_dtype, G;         // G scales per row
  int rows0, rows1, split;    // virtual rows: rows0 from 0, rows1 from `split` (a multiple of 8)
  int blocks;                 // row blocks of N
  int V, d, R, tiles, nk, stages;
};

struct __align__(8) Bars {
  uint64_t full[kMaxStages];   // producer and scale warps -> all: the stage landed
  uint64_t empty[kMaxStages];  // warps (codes read) and MMA (states read) -> producer
  uint64_t a_full[2][kMaxRing];  // [half][buffer] warps -> MMA: operand written, result buffer free
  uint64_t d_full[2][kMaxRing];  // MMA -> warps: result ready, operand buffer free
  uint64_t done;               // every MMA has completed
  uint32_t tmem;
  volatile int abort;
};

// Shared-memory matrix descriptor of a K-major tile with 128-byte swizzle: low
// word the address in 16-byte units, high word the stride between 8-row groups
// (1024 bytes), version 1 and the swizzle.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | 1u << 16; }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  return static_cast<uint64_t>((1024u >> 4) | 1u << 14 | 2u << 29) << 32 | lo;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// D (tensor memory) (+)= A (tensor memory) x B (shared memory), K = 16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr));
}

// (a0, a1) += s (x0, x1), both in one instruction.
__device__ __forceinline__ void fma2(float& a0, float& a1, float s, float x0, float x1) {
  asm("{\n .reg .b64 a, x, s;\n mov.b64 a, {%0, %1};\n mov.b64 x, {%3, %4};\n mov.b64 s, {%2, %2};\n"
      " fma.rn.f32x2 a, s, x, a;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(a0), "+f"(a1)
      : "f"(s), "f"(x0), "f"(x1));
}

__device__ __forceinline__ void give_up(Bars& bars, unsigned* err) {
  bars.abort = 1;
  if (err) atomicOr(err, 1u);
}

// Some 512 polls of a phase, two instructions each: a warp that waits takes
// its polls' issue slots from the warps that work (a loop of ten instructions
// took half of all).
__device__ __forceinline__ bool poll(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, 128;\n"
      "again:\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n @p bra done;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n @p bra done;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n @p bra done;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n @p bra done;\n"
      " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra again;\n"
      "done:\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "n"(svk::kSuspendNs)
      : "memory");
  return ok != 0;
}

// A bounded wait that also gives up once another role has.
__device__ __forceinline__ bool wait_or_abort(Bars& bars, uint64_t* bar, uint32_t parity, unsigned* err) {
  for (uint32_t i = 0; i < svk::kWaitPolls / 512; ++i) {
    if (poll(bar, parity)) return true;
    if (bars.abort) return false;
  }
  give_up(bars, err);
  return false;
}

// The same for a warp.
__device__ __forceinline__ bool warp_wait(Bars& bars, uint64_t* bar, uint32_t parity, unsigned* err) {
  return __all_sync(0xFFFFFFFFu, wait_or_abort(bars, bar, parity, err));
}
__device__ __forceinline__ bool warp_wait_bounded(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, svk::mbar_wait_bounded(bar, parity));
}

// One lane of the warp, the same every time.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// Two codes as 16-bit integers in a word: base + code, where base is a power
// of two whose unit in the last place is 1, then minus (base + zero), exact.
template <typename T>
struct Code;
template <>
struct Code<__nv_bfloat16> {
  static constexpr uint32_t kBase = 0x43004300u;  // 128
  static __device__ uint32_t sub(uint32_t a, uint32_t z) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&z));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct Code<__half> {
  static constexpr uint32_t kBase = 0x64006400u;  // 1024
  static __device__ uint32_t sub(uint32_t a, uint32_t z) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&z));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

// Eight codes of a word to four words of two, in order.
template <typename T>
__device__ __forceinline__ void turn(uint32_t w, uint32_t z, uint32_t* a) {
  const uint32_t odd = w >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t both = __byte_perm(w, odd, j | j << 4 | (4 + j) << 8 | (4 + j) << 12);
    a[j] = Code<T>::sub((both & 0x000F000Fu) | Code<T>::kBase, z);
  }
}

// Shared memory by 32-bit address (a pointer that went through an integer, as
// aligned ones do, loads by the generic path).
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// A 16-bit scale's value.
__device__ __forceinline__ float scale16(uint32_t v, int dtype) {
  return dtype == SV_BF16 ? __uint_as_float(v << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
}

// One 32-bit word to shared memory; its arrival is counted by the barrier that
// cp_async_arrive names.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Words `from + 4 k` of every row of a tile to shared memory by `warps` warps,
// this the `first`: word k of row r for the lanes' (r, k), a lane's next rows
// 32 / kWords times `warps` on.  Those lie 4 apart or more, 8 for bytes, so
// their places within a word are alike.
template <int kWords>
__device__ __forceinline__ void fetch_words(uintptr_t from, long long row_bytes, int bytes, uint32_t* to, int stride,
                                            int rows, int lane, int warps, int first = 0) {
  constexpr int kRows = 32 / kWords;  // per load
  const int k = lane % kWords;
  int r = first * kRows + lane / kWords;
  const uintptr_t at = from + r * row_bytes;
  uintptr_t word = (at & ~static_cast<uintptr_t>(3)) + 4 * k;
  if (word >= at + bytes) return;
  uint32_t dst = smem_u32(to + r * stride + k);
#pragma unroll 4
  for (; r < rows; r += warps * kRows) {
    cp_async4(dst, reinterpret_cast<const void*>(word));
    word += warps * kRows * row_bytes;
    dst += warps * kRows * stride * 4;
  }
}

template <typename T, int N, int G, int H>
__global__ void __launch_bounds__(32 * 10 * H, H == 1 ? 2 : 1)
    q4_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap h0,
              const __grid_constant__ CUtensorMap h1, const __grid_constant__ CUtensorMap whole,
              const __grid_constant__ Args g) {
  constexpr int kWarps = 8 * H;  // that turn codes
  constexpr int kHelp = H;       // that fetch scales
  constexpr int kSWords = per_stage_of(G) + 1;  // 32-bit words of a row's scales in a stage (odd: no bank conflicts)
  const int z_words = g.zeros ? 3 : 0;          // and of its zeros
  constexpr bool kBf16 = Code<T>::kBase == 0x43004300u;
  // instruction descriptor: D f32, A and B bf16 / f16, both K-major, N / 8, M / 16
  constexpr uint32_t kIdesc = (1u << 4) | (kBf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t(N) >> 3) << 17) |
                              ((128u >> 4) << 24);
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  const int w_bytes = g.R * 128, stage_bytes = w_bytes + N * kStageK * 2;
  uint32_t* sbuf = reinterpret_cast<uint32_t*>(smem + g.stages * stage_bytes);  // [stage][128 H][s_words]
  uint32_t* zbuf = sbuf + g.stages * 128 * H * kSWords;                       // [stage][128 H][z_words]
  Bars& bars = *reinterpret_cast<Bars*>(zbuf + g.stages * 128 * H * z_words);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&bars.full[s], 1 + 32 * kHelp);
      mbar_init(&bars.empty[s], kWarps + H);
    }
    for (int h = 0; h < 2; ++h)
      for (int i = 0; i < kMaxRing; ++i) {
        mbar_init(&bars.a_full[h][i], 8);
        mbar_init(&bars.d_full[h][i], 1);
      }
    mbar_init(&bars.done, H);
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarps + kHelp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)),
                 "r"(H * kHalfCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = bars.tmem;
  constexpr int per_stage = per_stage_of(G), ring = ring_of(G, N);
  constexpr int kStep = step_of(G, N), kGroups = kStep / G, kSteps = kStageK / kStep;
  constexpr int a_cols = kStep / 2, d_cols = kGroups * N, d_at = ring * a_cols;  // a half's columns: operands, then results

  if (warp >= kWarps && warp < kWarps + kHelp) {
    // ---- supply: codes and states by TMA (one lane of the first warp), the
    // scales and zeros of 128 rows each as the 32-bit words that hold them
    const int base_row = (warp - kWarps) * 128;
    const int elem = g.scale_dtype == SV_F32 ? 4 : 2;
    const bool copies = warp == kWarps && elected();
    int s = 0, use = 0, issued = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < g.tiles; t += gridDim.x) {
      const long long v0 = static_cast<long long>(t) * g.R + base_row;
      const int rows = static_cast<int>(min(static_cast<long long>(min(128, g.R - base_row)), g.V - v0));
      for (int blk = 0; ok && blk < g.blocks; ++blk)
        for (int ks = 0; ok && ks < g.nk; ++ks) {
          if (use > 0) ok = warp_wait(bars, &bars.empty[s], (use - 1) & 1, g.err);
          if (!ok) break;
          if (copies) {
            const uint32_t dst = smem_u32(smem) + s * stage_bytes;
            mbar_arrive_expect_tx(&bars.full[s], stage_bytes);
            tma_load_2d(dst, &wmap, ks * 128, t * g.R, &bars.full[s]);
            if (blk * N + N <= g.split) {  // the first set's rows alone, in boxes of N
#pragma unroll
              for (int c = 0; c < kStageK / 64; ++c)
                tma_load_2d(dst + w_bytes + c * N * 128, &whole, ks * kStageK + c * 64, blk * N, &bars.full[s]);
            } else {
#pragma unroll 1
              for (int r = 0; r < N; r += 8) {  // 8 rows of one of the two row sets
                const int v = blk * N + r;
                const bool second = v >= g.split;
                const CUtensorMap* map = second ? &h1 : &h0;
                const int y = second ? v - g.split : v;
#pragma unroll
                for (int c = 0; c < kStageK / 64; ++c)
                  tma_load_2d(dst + w_bytes + c * N * 128 + r * 128, map, ks * kStageK + c * 64, y, &bars.full[s]);
              }
            }
          }
          ++issued;
          __syncwarp();
          const int j0 = ks * per_stage, n = min(per_stage, g.G - j0);
          fetch_words<per_stage>(reinterpret_cast<uintptr_t>(g.scales) + (v0 * g.G + j0) * elem,
                                 static_cast<long long>(g.G) * elem, n * elem, sbuf + (s * 128 * H + base_row) * kSWords,
                                 kSWords, rows, lane, 1);
          if (g.zeros)
            fetch_words<per_stage == 8 ? 4 : 2>(reinterpret_cast<uintptr_t>(g.zeros) + v0 * g.G + j0, g.G, n,
                                                zbuf + (s * 128 * H + base_row) * z_words, z_words, rows, lane, 1);
          cp_async_arrive(&bars.full[s]);
          if (++s == g.stages) {
            s = 0;
            ++use;
          }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // no copy may still be writing shared memory at exit; once a role has
    // given up, a stage may lack the other scale warp's arrivals for good
    if (copies)
      for (int k = issued - g.stages > 0 ? issued - g.stages : 0; k < issued; ++k)
        if (!svk::mbar_wait_bounded(&bars.full[k % g.stages], (k / g.stages) & 1)) give_up(bars, g.err);
    __syncwarp();
  } else if (warp >= kWarps + kHelp) {
    // ---- MMA: a warp per half; all its lanes run the loops, so that addresses
    // stay in uniform registers, and one issues
    const int h = warp - (kWarps + kHelp);
    const uint32_t a0 = tmem + h * kHalfCols, d0 = a0 + d_at;
    const bool issues = elected();
    int s = 0, use = 0, buf = 0, turn_no = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < g.tiles; t += gridDim.x)
      for (int blk = 0; ok && blk < g.blocks; ++blk)
        for (int ks = 0; ok && ks < g.nk; ++ks) {
          ok = warp_wait(bars, &bars.full[s], use & 1, g.err);
          const uint32_t b_lo = desc_lo(smem_u32(smem) + s * stage_bytes + w_bytes);
          const int n = min(per_stage, g.G - ks * per_stage);
#pragma unroll 1
          for (int i = 0; i < kSteps; ++i) {
            if (!ok || i * kGroups >= n) break;
            ok = warp_wait(bars, &bars.a_full[h][buf], turn_no & 1, g.err);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            constexpr uint32_t kChunk = N * 128 / 16;  // 64 columns of the states, in descriptor units
            const uint32_t a = a0 + buf * a_cols, dd = d0 + buf * d_cols, b = b_lo + i * (kStep / 64) * kChunk;
            if (issues) {
#pragma unroll
              for (int kk = 0; kk < kStep / 16; ++kk)
                mma_ts(dd + kk * 16 / G * N, a + kk * 8, desc_of(b + (kk * 16 / 64) * kChunk + (kk * 16 % 64) / 8), kIdesc,
                       kk * 16 % G ? 1u : 0u);
              mma_commit(&bars.d_full[h][buf]);
            }
            __syncwarp();
            if (++buf == ring) {
              buf = 0;
              ++turn_no;
            }
          }
          if (ok && issues) mma_commit(&bars.empty[s]);
          __syncwarp();
          if (++s == g.stages) {
            s = 0;
            ++use;
          }
        }
    if (issues) mma_commit(&bars.done);
    __syncwarp();
    if (!warp_wait_bounded(&bars.done, 0)) give_up(bars, g.err);
  } else {
    // ---- a thread per vocabulary row and warpgroup
    const int half = warp / 8, wg = warp / 4 % 2;
    const int in_tile = half * 128 + warp % 4 * 32 + lane;
    const int row = min(in_tile, g.R - 1);  // rows past the tile repeat its last one, unused
    const uint32_t ta = tmem + half * kHalfCols + (static_cast<uint32_t>(warp % 4 * 32) << 16) + wg * (a_cols / 2);
    const uint32_t td = tmem + half * kHalfCols + (static_cast<uint32_t>(warp % 4 * 32) << 16) + d_at + wg * (N / 2);
    constexpr int kLag = ring - 1;  // a step's results are added this many steps later
    int s = 0, use = 0, buf = 0, turn_no = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < g.tiles; t += gridDim.x) {
      const long long v = static_cast<long long>(t) * g.R + in_tile;
      // where the row's scales and zeros begin in their first words
      const long long first = (static_cast<long long>(t) * g.R + row) * g.G;
      const int s_off = g.scale_dtype == SV_F32 ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(g.scales) / 2 + first) & 1);
      const int z_off = static_cast<int>((reinterpret_cast<uintptr_t>(g.zeros) + first) & 3);
      for (int blk = 0; ok && blk < g.blocks; ++blk) {
        float acc[N / 2];
#pragma unroll
        for (int n = 0; n < N / 2; ++n) acc[n] = 0.f;
        float late[kGroups] = {};  // scales of the step whose results are still to be added
        int pending = 0, rbuf = buf, rturn = turn_no;
        auto add = [&](const float (&scale)[kGroups]) {
          if (!warp_wait(bars, &bars.d_full[half][rbuf], rturn & 1, g.err)) return false;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
          for (int p = 0; p < kGroups; ++p) {
            uint32_t d[N / 2];
#pragma unroll
            for (int n = 0; n < N / 2; n += 8) tmem_ld8(td + rbuf * d_cols + p * N + n, d + n);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int n = 0; n < N / 2; n += 2) fma2(acc[n], acc[n + 1], scale[p], __uint_as_float(d[n]), __uint_as_float(d[n + 1]));
          }
          if (++rbuf == ring) {
            rbuf = 0;
            ++rturn;
          }
          return true;
        };
        for (int ks = 0; ok && ks < g.nk; ++ks) {
          ok = warp_wait(bars, &bars.full[s], use & 1, g.err);
          const uint32_t codes = smem_u32(smem) + s * stage_bytes + row * 128;
          const uint32_t srow = smem_u32(sbuf) + (s * 128 * H + row) * kSWords * 4;
          const uint32_t zrow = smem_u32(zbuf) + (s * 128 * H + row) * z_words * 4 + ((z_off + ks * per_stage) & 3);
          const int n = min(per_stage, g.G - ks * per_stage);
#pragma unroll 1
          for (int i = 0; i < kSteps; ++i) {
            if (!ok || i * kGroups >= n) break;
            float scale[kGroups];
#pragma unroll
            for (int p = 0; p < kGroups; ++p) {
              const int j = i * kGroups + p;
              const float x = g.scale_dtype == SV_F32 ? __uint_as_float(lds32(srow + j * 4)) : scale16(lds16(srow + (s_off + j) * 2), g.scale_dtype);
              scale[p] = j < n ? x : 0.f;  // past the row's last group the codes are padding
            }
            const uint32_t dst = ta + buf * a_cols;
#pragma unroll
            for (int c = 0; c < kStep / 64; ++c) {  // 32 codes: 16 bytes
              const int at = i * kStep / 32 + wg * (kStep / 64) + c;
              const int j = i * kGroups + (G == 128 ? 0 : G == 64 ? (kStep == 128 ? wg : 0) : wg * (kStep / 64) + c);
              const uint32_t z0 = g.zeros ? lds8(zrow + j) & 15u : 8u;
              const uint32_t z = (z0 | z0 << 16) + Code<T>::kBase;
              const uint4 q = lds128(codes + ((at ^ (row & 7)) << 4));
              uint32_t a[16];
              turn<T>(q.x, z, a);
              turn<T>(q.y, z, a + 4);
              turn<T>(q.z, z, a + 8);
              turn<T>(q.w, z, a + 12);
              tmem_st16(dst + c * 16, a);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_local(&bars.a_full[half][buf]);
              if ((i + 1) * kGroups >= n) mbar_arrive_local(&bars.empty[s]);
            }
            if (++buf == ring) {
              buf = 0;
              ++turn_no;
            }
            if constexpr (kLag == 0) {
              ok = add(scale);
            } else {
              if (pending) ok = add(late);
              pending = 1;
#pragma unroll
              for (int p = 0; p < kGroups; ++p) late[p] = scale[p];
            }
          }
          if (++s == g.stages) {
            s = 0;
            ++use;
          }
        }
        if (ok && pending) ok = add(late);
        if (ok && in_tile < g.R && v < g.V) {
#pragma unroll
          for (int n = 0; n < N / 2; ++n) {
            const int r = blk * N + wg * (N / 2) + n;
            float* out = r >= g.split ? (r - g.split < g.rows1 ? g.out1 + (r - g.split) * g.ld : nullptr)
                                      : (r < g.rows0 ? g.out0 + r * g.ld : nullptr);
            if (out) out[v] = acc[n];
          }
        }
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kWarps + kHelp) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(H * kHalfCols) : "memory");
  }
}

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// A row-major matrix in boxes of `width` (64 or 128) bytes x box_rows, swizzled
// over that width; what lies outside reads 0.
inline bool encode(CUtensorMap* map, CUtensorMapDataType type, int elem, const void* base, long long rows,
                   long long cols, int box_rows, int width = 128) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * elem};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(width / elem), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t es[2] = {1, 1};
  return encoder()(map, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SMs of the current device, which it also names.
inline int sm_count(int* dev_out) {
  static int sms[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  if (!sms[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    sms[dev] = n;
  }
  *dev_out = dev;
  return sms[dev];
}

// Rows of states per block, CTAs per SM and ring of an instantiation.
template <typename T, int N, int G, int H>
sv_status start(Args g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t stream) {
  int dev = 0;
  const int sms = sm_count(&dev);
  constexpr int kCtas = H == 1 ? 2 : 1;
  constexpr int kBudget = (H == 1 ? 113 : 227) * 1024;  // shared memory per CTA
  constexpr int kFixed = 1024 + static_cast<int>(sizeof(Bars));
  constexpr int kWords = per_stage_of(G) + 1;
  // tile rows: as few rounds as 128 H rows per CTA allow, then rows spread evenly
  const long long slots = static_cast<long long>(sms) * kCtas;
  const long long rounds = (g.V + slots * 128 * H - 1) / (slots * 128 * H);
  g.R = static_cast<int>(((g.V + slots * rounds - 1) / (slots * rounds) + 7) / 8 * 8);
  g.tiles = (g.V + g.R - 1) / g.R;
  const int stage_bytes = g.R * 128 + N * kStageK * 2 + 128 * H * 4 * (kWords + (g.zeros ? 3 : 0));
  g.stages = (kBudget - kFixed) / stage_bytes;
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  g.nk = (g.d + kStageK - 1) / kStageK;
  CUtensorMap mw, m0, m1, mn;
  const CUtensorMapDataType type =
      Code<T>::kBase == 0x43004300u ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!encode(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, proj->packed, g.V, g.d / 2, g.R) ||
      !encode(&m0, type, 2, g.rows0 ? s0 : s1, g.rows0 ? g.rows0 : g.rows1, g.d, 8) ||
      !encode(&m1, type, 2, g.rows1 ? s1 : s0, g.rows1 ? g.rows1 : g.rows0, g.d, 8) ||
      !encode(&mn, type, 2, g.rows0 ? s0 : s1, g.rows0 ? g.rows0 : g.rows1, g.d, N))
    return svh::fail(SV_ERR_ARG, "tensor map encoding failed (alignment or size)");
  const int smem = kFixed + g.stages * stage_bytes;
  static bool attr_set[64] = {false};
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(q4_kernel<T, N, G, H>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBudget);
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set[dev] = true;
  }
  const unsigned grid = static_cast<unsigned>(g.tiles < slots ? g.tiles : slots);
  q4_kernel<T, N, G, H><<<grid, 32 * 10 * H, smem, stream>>>(mw, m0, m1, mn, g);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

// The instantiation for n rows of states per block (a multiple of 16, up to 64).
template <typename T, int G>
sv_status start_rows(const Args& g, int n, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  if (n <= 16) return start<T, 16, G, 1>(g, proj, s0, s1, st);
  if (n <= 32) return start<T, 32, G, 2>(g, proj, s0, s1, st);
  if (n <= 48) return start<T, 48, G, 2>(g, proj, s0, s1, st);
  return start<T, 64, G, 2>(g, proj, s0, s1, st);
}

template <typename T>
sv_status start_group(const Args& g, int n, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  if (proj->group == 32) return start_rows<T, 32>(g, n, proj, s0, s1, st);
  if (proj->group == 64) return start_rows<T, 64>(g, n, proj, s0, s1, st);
  return start_rows<T, 128>(g, n, proj, s0, s1, st);
}

}  // namespace svq
