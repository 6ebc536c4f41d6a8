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
//   - operands and results alternate between two buffers, so the tensor cores
//     work on one group while the warps turn the next and add the last.  A
//     warp passes its turn with a single arrival: by then it has read the
//     result that the MMA will overwrite.
// A CTA has H halves of 128 rows (4 warps each), a producer warp and an MMA
// warp.  Its tiles have R <= 128 H rows, R chosen so that the vocabulary
// divides evenly over the CTAs (the MMA's idle rows cost nothing).
//
// Every wait is bounded; one that gives up sets bit 0 of *err.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "../../include/sv_lm_head.h"
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
constexpr int kMaxScales = kStageK / 32;  // per row and stage
constexpr int kACols = 64;      // tensor-memory columns of one operand buffer: 128 16-bit pairs' worth
constexpr int kDCols = 64;      // and of one result buffer: up to 64 rows of states
constexpr int kHalfCols = 2 * (kACols + kDCols);

struct Args {
  const void* scales;
  const unsigned char* zeros;
  float* out0;
  float* out1;
  unsigned* err;
  long long ld;
  int scale_dtype, group, G;  // G scales per row
  int rows0, rows1, split;    // virtual rows: rows0 from 0, rows1 from `split` (a multiple of 8)
  int blocks;                 // row blocks of N
  int V, d, R, tiles, nk, stages;
};

struct __align__(8) Bars {
  uint64_t full[kMaxStages];   // producer -> all: the stage landed
  uint64_t empty[kMaxStages];  // warps (codes read) and MMA (states read) -> producer
  uint64_t a_full[2][2];       // [half][buffer] warps -> MMA: operand written, result buffer free
  uint64_t d_full[2][2];       // MMA -> warps: result ready, operand buffer free
  uint64_t done;               // every MMA has completed
  uint32_t tmem;
  volatile int abort;
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
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

// 16 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

__device__ __forceinline__ void give_up(Bars& bars, unsigned* err) {
  bars.abort = 1;
  if (err) atomicOr(err, 1u);
}

// A bounded wait that also gives up once another role has.
__device__ __forceinline__ bool wait_or_abort(Bars& bars, uint64_t* bar, uint32_t parity, unsigned* err) {
  for (uint32_t i = 0; i < svk::kWaitPolls; ++i) {
    if (svk::mbar_try_wait(bar, parity)) return true;
    if (bars.abort) return false;
  }
  give_up(bars, err);
  return false;
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

// 32 codes (16 bytes) to 16 words of two, in order.
template <typename T>
__device__ __forceinline__ void turn(uint4 q, uint32_t z, uint32_t (&a)[16]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t odd = w[i] >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t both = __byte_perm(w[i], odd, j | j << 4 | (4 + j) << 8 | (4 + j) << 12);
      a[4 * i + j] = Code<T>::sub((both & 0x000F000Fu) | Code<T>::kBase, z);
    }
  }
}

__device__ __forceinline__ float scale_at(const Args& g, long long i) {
  if (g.scale_dtype == SV_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(g.scales)[i]);
  if (g.scale_dtype == SV_F16) return __half2float(static_cast<const __half*>(g.scales)[i]);
  return static_cast<const float*>(g.scales)[i];
}

template <typename T, int N, int H>
__global__ void __launch_bounds__(128 * H + 64, H == 1 ? 2 : 1)
    q4_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap h0,
              const __grid_constant__ CUtensorMap h1, const __grid_constant__ Args g) {
  constexpr int kWarps = 4 * H;
  constexpr bool kBf16 = sizeof(T) == 2 && Code<T>::kBase == 0x43004300u;
  // instruction descriptor: D f32, A and B bf16 / f16, both K-major, N / 8, M / 16
  constexpr uint32_t kIdesc = (1u << 4) | (kBf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t(N) >> 3) << 17) |
                              ((128u >> 4) << 24);
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  const int w_bytes = g.R * 128, stage_bytes = w_bytes + N * kStageK * 2;
  float* sbuf = reinterpret_cast<float*>(smem + g.stages * stage_bytes);            // [warp][32][kMaxScales]
  uint32_t* zbuf = reinterpret_cast<uint32_t*>(sbuf + kWarps * 32 * kMaxScales);    // the same: base + zero, twice
  Bars& bars = *reinterpret_cast<Bars*>(zbuf + kWarps * 32 * kMaxScales);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], kWarps + 1);
    }
    for (int h = 0; h < 2; ++h)
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.a_full[h][i], 4);
        mbar_init(&bars.d_full[h][i], 1);
      }
    mbar_init(&bars.done, 1);
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)),
                 "r"(H * kHalfCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = bars.tmem;
  const int units = g.tiles * g.blocks;            // a CTA's units: all row blocks of its tiles
  const int steps = (g.d + g.group - 1) / g.group;  // groups of a row
  const int per_stage = kStageK / g.group;

  if (warp == kWarps) {
    // ---- producer: one thread
    if (lane == 0) {
      int gk = 0;  // stages issued so far
      for (int t = blockIdx.x; t < g.tiles && !bars.abort; t += gridDim.x)
        for (int blk = 0; blk < g.blocks && !bars.abort; ++blk)
          for (int ks = 0; ks < g.nk; ++ks, ++gk) {
            const int s = gk % g.stages;
            if (gk >= g.stages && !wait_or_abort(bars, &bars.empty[s], ((gk / g.stages) - 1) & 1, g.err)) break;
            const uint32_t dst = smem_u32(smem + s * stage_bytes);
            mbar_arrive_expect_tx(&bars.full[s], stage_bytes);
            tma_load_2d(dst, &wmap, ks * 128, t * g.R, &bars.full[s]);
            for (int r = 0; r < N; r += 8) {  // 8 rows of one of the two row sets
              const int v = blk * N + r;
              const bool second = v >= g.split;
              for (int c = 0; c < kStageK / 64; ++c)
                tma_load_2d(dst + w_bytes + c * N * 128 + r * 128, second ? &h1 : &h0, ks * kStageK + c * 64,
                            second ? v - g.split : v, &bars.full[s]);
            }
          }
      // no copy may still be writing shared memory at exit
      for (int k = gk - g.stages > 0 ? gk - g.stages : 0; k < gk; ++k)
        if (!svk::mbar_wait_bounded(&bars.full[k % g.stages], (k / g.stages) & 1)) give_up(bars, g.err);
    }
  } else if (warp == kWarps + 1) {
    // ---- MMA: one thread issues
    if (lane == 0) {
      int gk = 0, gs = 0;  // stages and groups so far
      bool ok = true;
      for (int u = blockIdx.x * g.blocks; ok && u < units; u += (u + 1) % g.blocks ? 1 : 1 + (gridDim.x - 1) * g.blocks)
        for (int ks = 0; ok && ks < g.nk; ++ks, ++gk) {
          const int s = gk % g.stages;
          ok = wait_or_abort(bars, &bars.full[s], (gk / g.stages) & 1, g.err);
          const uint32_t b0 = smem_u32(smem + s * stage_bytes) + w_bytes;
          for (int i = 0; ok && i < per_stage && ks * per_stage + i < steps; ++i, ++gs) {
            const int buf = gs & 1, k0 = i * g.group;
            for (int h = 0; ok && h < H; ++h) {
              ok = wait_or_abort(bars, &bars.a_full[h][buf], (gs >> 1) & 1, g.err);
              if (!ok) break;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
              const uint32_t a = tmem + h * kHalfCols + buf * kACols;
              const uint32_t dd = tmem + h * kHalfCols + 2 * kACols + buf * kDCols;
              for (int kk = 0; kk < g.group / 16; ++kk) {
                const int k = k0 + kk * 16;
                mma_ts(dd, a + kk * 8, desc_sw128(b0 + (k / 64) * N * 128 + (k % 64) * 2), kIdesc, kk ? 1u : 0u);
              }
              mma_commit(&bars.d_full[h][buf]);
            }
          }
          if (ok) mma_commit(&bars.empty[s]);
        }
      mma_commit(&bars.done);
      if (!svk::mbar_wait_bounded(&bars.done, 0)) give_up(bars, g.err);
    }
  } else {
    // ---- a thread per vocabulary row
    const int half = warp / 4;
    const int row = min(warp * 32 + lane, g.R - 1);  // rows past the tile repeat its last one, unused
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t ta = tmem + half * kHalfCols + lanes, td = ta + 2 * kACols;
    float* my_s = sbuf + warp * 32 * kMaxScales;
    uint32_t* my_z = zbuf + warp * 32 * kMaxScales;
    const int lg = per_stage == 8 ? 3 : per_stage == 4 ? 2 : 1;  // log2 of the scales per row and stage
    int gk = 0, gs = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < g.tiles; t += gridDim.x) {
      const int v0 = t * g.R + warp * 32;
      // scales (and zeros) of a stage, for this warp's rows: lanes take
      // neighbouring scales of a row, so a load touches few lines
      float sv[kMaxScales];
      uint32_t zv[kMaxScales];
      auto fetch = [&](int ks) {
#pragma unroll
        for (int i = 0; i < kMaxScales; ++i)
          if (i < per_stage) {
            const int e = i * 32 + lane, r = e >> lg, j = (ks << lg) + (e & (per_stage - 1));
            const bool in = warp * 32 + r < g.R && v0 + r < g.V && j < g.G;
            const long long at = static_cast<long long>(v0 + r) * g.G + j;
            sv[i] = in ? scale_at(g, at) : 0.f;
            zv[i] = in && g.zeros ? g.zeros[at] & 15u : 8u;
          }
      };
      fetch(0);
      for (int blk = 0; ok && blk < g.blocks; ++blk) {
        float acc[N];
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = 0.f;
        float s_last = 0.f;
        int left = 0;  // results not yet added: 0 or 1
        auto add_result = [&](int step, float s) {
          if (!__all_sync(0xFFFFFFFFu, wait_or_abort(bars, &bars.d_full[half][step & 1], (step >> 1) & 1, g.err)))
            return false;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          uint32_t d[N];
#pragma unroll
          for (int n = 0; n < N; n += 16) tmem_ld16(td + (step & 1) * kDCols + n, d + n);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int n = 0; n < N; ++n) acc[n] = fmaf(s, __uint_as_float(d[n]), acc[n]);
          return true;
        };
        for (int ks = 0; ok && ks < g.nk; ++ks, ++gk) {
          // this stage's scales to their rows, the next one's on their way
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kMaxScales; ++i)
            if (i < per_stage) {
              my_s[i * 32 + lane] = sv[i];
              my_z[i * 32 + lane] = (zv[i] | zv[i] << 16) + Code<T>::kBase;
            }
          __syncwarp();
          if (ks + 1 < g.nk)
            fetch(ks + 1);
          else if (blk + 1 < g.blocks)
            fetch(0);
          const int s = gk % g.stages;
          ok = __all_sync(0xFFFFFFFFu, wait_or_abort(bars, &bars.full[s], (gk / g.stages) & 1, g.err));
          const unsigned char* codes = smem + s * stage_bytes + row * 128;
          for (int i = 0; ok && i < per_stage && ks * per_stage + i < steps; ++i, ++gs) {
            const uint32_t z = my_z[(lane << lg) + i];
            const int c0 = i * g.group / 32;
            for (int c = 0; c < g.group / 32; ++c) {
              const uint4 q = *reinterpret_cast<const uint4*>(codes + (((c0 + c) ^ (row & 7)) << 4));
              uint32_t a[16];
              turn<T>(q, z, a);
              tmem_st16(ta + (gs & 1) * kACols + c * 16, a);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_local(&bars.a_full[half][gs & 1]);
              if (i + 1 == per_stage || ks * per_stage + i + 1 == steps) mbar_arrive_local(&bars.empty[s]);
            }
            if (left) ok = add_result(gs - 1, s_last);
            left = 1;
            s_last = my_s[(lane << lg) + i];
          }
        }
        if (ok && left) ok = add_result(gs - 1, s_last);
        if (ok && warp * 32 + lane < g.R && v0 + lane < g.V) {
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const int v = blk * N + n;
            float* out = v >= g.split ? (v - g.split < g.rows1 ? g.out1 + (v - g.split) * g.ld : nullptr)
                                      : (v < g.rows0 ? g.out0 + v * g.ld : nullptr);
            if (out) out[v0 + lane] = acc[n];
          }
        }
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kWarps + 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(H * kHalfCols) : "memory");
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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

// A row-major matrix in boxes of 128 bytes x box_rows, 128-byte swizzle;
// what lies outside reads 0.
bool encode(CUtensorMap* map, CUtensorMapDataType type, int elem, const void* base, long long rows, long long cols,
            int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * elem};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t es[2] = {1, 1};
  return encoder()(map, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

// Rows of states per block, CTAs per SM and ring of an instantiation.
template <typename T, int N, int H>
sv_status start(Args g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  static int sms[64] = {0};
  if (!sms[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    sms[dev] = n;
  }
  constexpr int kCtas = H == 1 ? 2 : 1;
  constexpr int kBudget = (H == 1 ? 113 : 227) * 1024;  // shared memory per CTA
  constexpr int kFixed = 1024 + 4 * H * 32 * kMaxScales * 8 + static_cast<int>(sizeof(Bars));
  // tile rows: as few rounds as 128 H rows per CTA allow, then rows spread evenly
  const long long slots = static_cast<long long>(sms[dev]) * kCtas;
  const long long rounds = (g.V + slots * 128 * H - 1) / (slots * 128 * H);
  g.R = static_cast<int>(((g.V + slots * rounds - 1) / (slots * rounds) + 7) / 8 * 8);
  g.tiles = (g.V + g.R - 1) / g.R;
  const int stage_bytes = g.R * 128 + N * kStageK * 2;
  g.stages = (kBudget - kFixed) / stage_bytes;
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  g.nk = (g.d + kStageK - 1) / kStageK;
  CUtensorMap mw, m0, m1;
  const CUtensorMapDataType type =
      Code<T>::kBase == 0x43004300u ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!encode(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, proj->packed, g.V, g.d / 2, g.R) ||
      !encode(&m0, type, 2, g.rows0 ? s0 : s1, g.rows0 ? g.rows0 : g.rows1, g.d, 8) ||
      !encode(&m1, type, 2, g.rows1 ? s1 : s0, g.rows1 ? g.rows1 : g.rows0, g.d, 8))
    return svh::fail(SV_ERR_ARG, "tensor map encoding failed (alignment or size)");
  const int smem = kFixed + g.stages * stage_bytes;
  static bool attr_set[64] = {false};
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(q4_kernel<T, N, H>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBudget);
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set[dev] = true;
  }
  const unsigned grid = static_cast<unsigned>(g.tiles < slots ? g.tiles : slots);
  q4_kernel<T, N, H><<<grid, 128 * H + 64, smem, stream>>>(mw, m0, m1, g);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

template <typename T>
sv_status start_rows(const Args& g, int n, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  if (n <= 16) return start<T, 16, 1>(g, proj, s0, s1, st);
  if (n <= 32) return start<T, 32, 2>(g, proj, s0, s1, st);
  if (n <= 48) return start<T, 48, 2>(g, proj, s0, s1, st);
  return start<T, 64, 2>(g, proj, s0, s1, st);
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
  g.group = proj->group;
  g.G = (dim + proj->group - 1) / proj->group;
  g.out0 = out0;
  g.out1 = out1;
  g.err = err;
  g.ld = ld;
  g.rows0 = rows0;
  g.rows1 = rows1;
  g.V = vocab;
  g.d = dim;
  const long long split = rows1 ? (static_cast<long long>(rows0) + 7) / 8 * 8 : 0x40000000LL;
  const long long all = rows1 ? split + rows1 : rows0;
  if (all > 0x3FFFFFFFLL) return svh::fail(SV_ERR_UNSUPPORTED, "too many rows");
  g.split = static_cast<int>(split);
  g.blocks = static_cast<int>((all + 63) / 64);
  const int n = static_cast<int>(((all + g.blocks - 1) / g.blocks + 15) / 16 * 16);
  g.blocks = static_cast<int>((all + n - 1) / n);
  return dtype == SV_BF16 ? start_rows<__nv_bfloat16>(g, n, proj, s0, s1, stream)
                          : start_rows<__half>(g, n, proj, s0, s1, stream);
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
