// The 4-bit LM head for up to 16 rows of states (include/sv_lm_head_q4.h).
//
// With so few rows the product is a stream of codes, and what must not stall
// it is the way from a code to an operand.  The tensor-memory kernel pays a
// store to tensor memory and two barrier trips per group on that way (61 us of
// its 150 at 11 rows, V = 128256, d = 4096 are left with the arithmetic taken
// out); here a code goes from a register straight into an mma.sync operand
// and nothing waits but on the stream itself.  mma.sync runs at 1006
// multiply-adds per clock and SM (measured): 16 rows use 16 per weight, and
// the memory delivers 45 weights per clock and SM, so it is fast enough up to
// here and not beyond.
//
//   - W rows are the MMA's 16 rows; a warp has 32 of them (two m tiles) and
//     one 64-column half of every 128-column stage, sixteen warps in all.
//   - Eight codes of a word make the pairs (0,4) (1,5) (2,6) (3,7) with one
//     mask each; the states are laid out in that order once, as operands, in
//     shared memory, where all of them stay.
//   - The sums of a group are f32 accumulators of their own, added to the
//     row's with the group's scale: no weight is rounded.
//   - Codes come by TMA, scales by cp.async from a warp of their own, in one
//     ring of stages.
//   - The two halves' sums are joined through shared memory at the tile's end,
//     in a fixed order.
// Every mbarrier wait is bounded; one that gives up sets bit 0 of *err, and
// the warps then run through their remaining barriers without computing.
#pragma once
#include "sv_lm_head_q4.cuh"

namespace svq {

constexpr int kFewK = 128;       // columns per stage: 64 bytes of a row
constexpr int kFewTile = 256;    // rows per tile at most
constexpr int kFewWarps = 16;    // that compute: 8 row groups x 2 halves of a stage
constexpr int kFewThreads = 32 * (kFewWarps + 2);
constexpr int kFewStages = 8;    // at most
constexpr int kFewBudget = 227 * 1024;

struct __align__(8) FewBars {
  uint64_t full[kFewStages], empty[kFewStages];
  volatile int abort;
};

__device__ __forceinline__ bool few_wait(FewBars& bars, uint64_t* bar, uint32_t parity, unsigned* err) {
  for (uint32_t i = 0; i < svk::kWaitPolls; ++i) {
    if (svk::mbar_try_wait(bar, parity)) return true;
    if (bars.abort) return false;
  }
  bars.abort = 1;
  if (err) atomicOr(err, 1u);
  return false;
}

template <int ID>
__device__ __forceinline__ void bar_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(32 * kFewWarps) : "memory");
}
template <int ID>
__device__ __forceinline__ void bar_arrive() {
  asm volatile("bar.arrive %0, %1;" ::"n"(ID), "n"(32 * kFewWarps) : "memory");
}

// A word's eight codes as the pairs (0,4) (1,5) (2,6) (3,7) of integers minus
// the zero.  In f16 a code four bits up is 16 times itself above 1024, which
// the subtraction's multiplier takes back (exact), so half the shifts go.
__device__ __forceinline__ void pairs_of(uint32_t w, uint32_t z, uint32_t (&p)[4], __nv_bfloat16) {
  using C = Code<__nv_bfloat16>;
  p[0] = C::sub((w & 0x000F000Fu) | C::kBase, z);
  p[1] = C::sub((w >> 4 & 0x000F000Fu) | C::kBase, z);
  p[2] = C::sub((w >> 8 & 0x000F000Fu) | C::kBase, z);
  p[3] = C::sub((w >> 12 & 0x000F000Fu) | C::kBase, z);
}
__device__ __forceinline__ void pairs_of(uint32_t w, uint32_t z, uint32_t (&p)[4], __half) {
  using C = Code<__half>;
  const __half2 sixteenth = __float2half2_rn(0.0625f), down = __float2half2_rn(960.f);  // 1024 - 64
  const __half2 z16 = __hsub2(down, *reinterpret_cast<__half2*>(&z));                   // -(64 + zero)
  auto high = [&](uint32_t x) {
    uint32_t y = (x & 0x00F000F0u) | C::kBase;
    const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&y), sixteenth, z16);
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  p[0] = C::sub((w & 0x000F000Fu) | C::kBase, z);
  p[1] = high(w);
  const uint32_t x = w >> 8;
  p[2] = C::sub((x & 0x000F000Fu) | C::kBase, z);
  p[3] = high(x);
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (Code<T>::kBase == 0x43004300u)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct FewArgs {
  Args g;
  const uint4* s0;
  const uint4* s1;
  int group;
};

// Words of a row's scales (zeros) looked at per stage of `n` groups, and the
// odd stride they lie at.
__host__ __device__ constexpr int few_stride(int n) { return n == 1 ? 1 : n + 1; }
__host__ __device__ constexpr int few_zstride(int n) { return n == 1 ? 1 : 3; }

// NT tiles of 8 states; SMALL: groups of 32 (two to a warp's half stage).
template <typename T, int NT, bool SMALL>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ CUtensorMap wmap,
                                                             const __grid_constant__ FewArgs f) {
  const Args& g = f.g;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  const int stage_bytes = g.R * 64, rows = g.rows0 + g.rows1, per_stage = kFewK / f.group;
  const int sstride = few_stride(per_stage), zstride = g.zeros ? few_zstride(per_stage) : 0;
  unsigned char* frag = smem + g.stages * stage_bytes;                             // [32-column block][row][4 x 16 bytes]
  float* red = reinterpret_cast<float*>(frag + g.nk * 4 * rows * 64);              // [row warp][8 NT][32]
  uint32_t* sbuf = reinterpret_cast<uint32_t*>(red + kFewWarps / 2 * 8 * NT * 32);  // [stage][tile row][sstride]
  uint32_t* zbuf = sbuf + g.stages * kFewTile * sstride;
  FewBars& bars = *reinterpret_cast<FewBars*>(zbuf + g.stages * kFewTile * zstride);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&bars.full[s], 1 + 32);
      mbar_init(&bars.empty[s], kFewWarps);
    }
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  if (warp == kFewWarps) {
    // ---- codes: one thread
    if (lane == 0) {
      int s = 0, use = 0, issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < g.tiles; t += gridDim.x)
        for (int ks = 0; ok && ks < g.nk; ++ks) {
          if (use > 0 && !few_wait(bars, &bars.empty[s], (use - 1) & 1, g.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars.full[s], stage_bytes);
          tma_load_2d(smem_u32(smem + s * stage_bytes), &wmap, ks * 64, t * g.R, &bars.full[s]);
          ++issued;
          if (++s == g.stages) {
            s = 0;
            ++use;
          }
        }
      // no copy may still be writing shared memory at exit
      for (int k = issued > g.stages ? issued - g.stages : 0; k < issued; ++k)
        if (!svk::mbar_wait_bounded(&bars.full[k % g.stages], (k / g.stages) & 1) && g.err) atomicOr(g.err, 1u);
    }
    return;
  }
  if (warp == kFewWarps + 1) {
    // ---- scales and zeros, as the 32-bit words that hold them
    const int elem = g.scale_dtype == SV_F32 ? 4 : 2;
    const int sw = per_stage == 4 ? 2 : per_stage == 2 ? 1 : 0, zw = per_stage == 1 ? 0 : 1;
    int s = 0, use = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < g.tiles; t += gridDim.x) {
      const long long v0 = static_cast<long long>(t) * g.R;
      const int n_rows = static_cast<int>(v0 + g.R <= g.V ? g.R : g.V - v0);
      for (int ks = 0; ok && ks < g.nk; ++ks) {
        if (use > 0) ok = __all_sync(0xFFFFFFFFu, few_wait(bars, &bars.empty[s], (use - 1) & 1, g.err));
        if (!ok) break;
        const int j0 = ks * per_stage, n = min(per_stage, g.G - j0);
        uint32_t* sd = sbuf + s * kFewTile * sstride;
#pragma unroll 4
        for (int e = lane; e < n_rows << sw; e += 32) {
          const int r = e >> sw, k = e & ((1 << sw) - 1);
          const uintptr_t at = reinterpret_cast<uintptr_t>(g.scales) + ((v0 + r) * g.G + j0) * elem;
          const uintptr_t word = (at & ~static_cast<uintptr_t>(3)) + 4 * k;
          if (word < at + n * elem) cp_async4(smem_u32(sd + r * sstride + k), reinterpret_cast<const void*>(word));
        }
        if (g.zeros) {
          uint32_t* zd = zbuf + s * kFewTile * zstride;
#pragma unroll 4
          for (int e = lane; e < n_rows << zw; e += 32) {
            const int r = e >> zw, k = e & ((1 << zw) - 1);
            const uintptr_t at = reinterpret_cast<uintptr_t>(g.zeros) + (v0 + r) * g.G + j0;
            const uintptr_t word = (at & ~static_cast<uintptr_t>(3)) + 4 * k;
            if (word < at + n) cp_async4(smem_u32(zd + r * zstride + k), reinterpret_cast<const void*>(word));
          }
        }
        cp_async_arrive(&bars.full[s]);
        if (++s == g.stages) {
          s = 0;
          ++use;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  // ---- the states as operands: block q, row n, quarter t holds columns
  // 32 q + 8 t .. + 7 as the pairs above; columns past dim are 0
  for (int e = threadIdx.x; e < rows * g.nk * 16; e += 32 * kFewWarps) {
    const int n = e / (g.nk * 16), j = e - n * (g.nk * 16);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (j < g.d / 8)
      x = __ldg((n < g.rows0 ? f.s0 + static_cast<long long>(n) * (g.d / 8) : f.s1 + static_cast<long long>(n - g.rows0) * (g.d / 8)) + j);
    uint4 y;
    y.x = __byte_perm(x.x, x.z, 0x5410);
    y.y = __byte_perm(x.x, x.z, 0x7632);
    y.z = __byte_perm(x.y, x.w, 0x5410);
    y.w = __byte_perm(x.y, x.w, 0x7632);
    *reinterpret_cast<uint4*>(frag + ((j / 4) * rows + n) * 64 + j % 4 * 16) = y;
  }
  bar_sync<1>();

  const int rw = warp % 8, kh = warp / 8, gq = lane / 4, t4 = lane % 4;
  const bool active = rw * 32 < g.R;
  const int code0 = (rw * 32 + gq) * 64 + t4 * 4, swz = gq >> 1 & 3;
  int s = 0, use = 0;
  bool ok = true, first_tile = true;
  for (int t = blockIdx.x; t < g.tiles; t += gridDim.x) {
    const long long v0 = static_cast<long long>(t) * g.R + rw * 32;
    // place of a row's first scale in its word; the rows of a lane lie 8 apart, so it is theirs all
    const int s_par = g.scale_dtype == SV_F32 ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(g.scales) / 2 + (v0 + gq) * g.G) & 1);
    const int z_par = static_cast<int>((reinterpret_cast<uintptr_t>(g.zeros) + (v0 + gq) * g.G) & 3);
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    for (int ks = 0; ks < g.nk; ++ks) {
      ok = __all_sync(0xFFFFFFFFu, ok && few_wait(bars, &bars.full[s], use & 1, g.err));
      if (ok && active) {
        const unsigned char* codes = smem + s * stage_bytes + code0;
        uint32_t w[2][2][2];  // [m tile][row half][32-column block]
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[m][h][i] = *reinterpret_cast<const uint32_t*>(codes + (m * 16 + h * 8) * 64 + (((2 * kh + i) ^ swz) << 4));
        const int j0 = ks * per_stage;
        const uint32_t* srow = sbuf + (s * kFewTile + rw * 32 + gq) * sstride;
        const unsigned char* zrow = reinterpret_cast<const unsigned char*>(zbuf + (s * kFewTile + rw * 32 + gq) * zstride) + (z_par + j0 & 3);
        const int s_at = s_par + j0 & 1;
        float part[2][NT][4];
        float scale[2][2];
        uint32_t z[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 0 || SMALL) {
            const int j = SMALL ? 2 * kh + i : f.group == 64 ? kh : 0;  // the group within the stage
            const bool in = j0 + j < g.G;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t* p = srow + (m * 16 + h * 8) * sstride;
                float x;
                if (g.scale_dtype == SV_F32)
                  x = __uint_as_float(p[j]);
                else if (g.scale_dtype == SV_BF16)
                  x = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(p)[s_at + j]) << 16);
                else
                  x = __half2float(reinterpret_cast<const __half*>(p)[s_at + j]);
                scale[m][h] = in ? x : 0.f;  // past the row's last group the codes are padding
                const uint32_t zero = g.zeros ? zrow[(m * 16 + h * 8) * zstride * 4 + j] & 15u : 8u;
                z[m][h] = (zero | zero << 16) + Code<T>::kBase;
              }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[m][n][e] = 0.f;
          }
          uint4 b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            b[n] = n * 8 + gq < rows ? *reinterpret_cast<const uint4*>(frag + (((ks * 4 + kh * 2 + i) * rows + n * 8 + gq) * 4 + t4) * 16)
                                     : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            uint32_t lo[4], hi[4];
            pairs_of(w[m][0][i], z[m][0], lo, T());
            pairs_of(w[m][1][i], z[m][1], hi, T());
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<T>(part[m][n], lo[0], hi[0], lo[1], hi[1], b[n].x, b[n].y);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<T>(part[m][n], lo[2], hi[2], lo[3], hi[3], b[n].z, b[n].w);
          }
          if (i == 1 || SMALL) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][n][e] = fmaf(scale[m][e / 2], part[m][n][e], acc[m][n][e]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_local(&bars.empty[s]);
      if (++s == g.stages) {
        s = 0;
        ++use;
      }
    }
    // join the halves; the first one's warps write the logits
    float* mine = red + rw * 8 * NT * 32 + lane;
    if (kh == 1) {
      if (!first_tile) bar_sync<3>();  // the last tile's sums have been read
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[((m * NT + n) * 4 + e) * 32] = acc[m][n][e];
      __syncwarp();
      bar_arrive<2>();
    } else {
      bar_sync<2>();
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][n][e] += mine[((m * NT + n) * 4 + e) * 32];
      __syncwarp();
      if (t + static_cast<int>(gridDim.x) < g.tiles) bar_arrive<3>();
      if (ok && active) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = n * 8 + 2 * t4 + e;
            if (r >= rows) continue;
            float* out = r < g.rows0 ? g.out0 + r * g.ld : g.out1 + (r - g.rows0) * g.ld;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int in = rw * 32 + m * 16 + h * 8 + gq;
                if (in < g.R && v0 + m * 16 + h * 8 + gq < g.V) out[v0 + m * 16 + h * 8 + gq] = acc[m][n][2 * h + e];
              }
          }
      }
    }
    first_tile = false;
  }
}

// Shared memory of a call with `stages` stages.
inline int few_smem(const Args& g, int group, int stages, int nt) {
  const int per = kFewK / group;
  return 1024 + stages * (g.R * 64 + kFewTile * 4 * (few_stride(per) + (g.zeros ? few_zstride(per) : 0))) +
         g.nk * 4 * (g.rows0 + g.rows1) * 64 + kFewWarps / 2 * 8 * nt * 32 * 4 + 8 + static_cast<int>(sizeof(FewBars));
}

// Launches the call here if its states fit beside a ring of four stages
// (SV_ERR_UNSUPPORTED otherwise, with nothing enqueued).
template <typename T, int NT, bool SMALL>
sv_status start_few(Args g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t stream) {
  int dev = 0;
  const int sms = sm_count(&dev);
  // tile rows: as few rounds as tiles of 256 allow, then spread evenly, in warps' 32 rows
  const long long rounds = (g.V + static_cast<long long>(sms) * kFewTile - 1) / (static_cast<long long>(sms) * kFewTile);
  g.R = static_cast<int>(((g.V + sms * rounds - 1) / (sms * rounds) + 31) / 32 * 32);
  g.tiles = (g.V + g.R - 1) / g.R;
  g.nk = (g.d + kFewK - 1) / kFewK;
  g.stages = kFewStages;
  while (g.stages >= 4 && few_smem(g, proj->group, g.stages, NT) > kFewBudget) --g.stages;
  if (g.stages < 4) return SV_ERR_UNSUPPORTED;
  CUtensorMap mw;
  if (!encode(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, proj->packed, g.V, g.d / 2, g.R, 64))
    return svh::fail(SV_ERR_ARG, "tensor map encoding failed (alignment or size)");
  static bool attr_set[64] = {false};
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(few_kernel<T, NT, SMALL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewBudget);
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set[dev] = true;
  }
  FewArgs f{g, static_cast<const uint4*>(s0), static_cast<const uint4*>(s1), proj->group};
  few_kernel<T, NT, SMALL><<<static_cast<unsigned>(g.tiles < sms ? g.tiles : sms), kFewThreads,
                             few_smem(g, proj->group, g.stages, NT), stream>>>(mw, f);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

template <typename T>
sv_status start_few_any(const Args& g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  const int rows = g.rows0 + g.rows1;
  if (rows > 16) return SV_ERR_UNSUPPORTED;
  if (proj->group == 32)
    return rows <= 8 ? start_few<T, 1, true>(g, proj, s0, s1, st) : start_few<T, 2, true>(g, proj, s0, s1, st);
  return rows <= 8 ? start_few<T, 1, false>(g, proj, s0, s1, st) : start_few<T, 2, false>(g, proj, s0, s1, st);
}

}  // namespace svq
