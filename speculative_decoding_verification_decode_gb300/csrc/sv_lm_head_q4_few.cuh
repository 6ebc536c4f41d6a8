// The 4-bit LM head for up to 16 rows of states (include/sv_lm_head_q4.h).
//
// With so few rows the product is a stream of codes, and what must not stall
// it is the way from a code to an operand.  The tensor-memory kernel pays a
// store to tensor memory and two barrier trips per 128 columns on that way (135
// us at 11 rows, V = 128256, d = 4096, groups of 128; here 79, and 60 to 62 up
// to 8 rows); here a code goes from a register straight into an mma.sync operand
// and nothing waits but on the stream itself.  mma.sync runs at 1006
// multiply-adds per clock and SM (measured): 16 rows use 16 per weight, and
// the memory delivers 45 weights per clock and SM, so it is fast enough up to
// here and not beyond.
//
//   - W rows are the MMA's 16 rows; a warp has 32 of them (two m tiles) of
//     every other 128-column stage, fourteen warps in all.  A warp reads the
//     codes of its next stage before it multiplies this one's.
//   - Eight codes of a word make the pairs (0,4) (1,5) (2,6) (3,7), by one
//     mask each and one shift: a code in the lowest bits of a half word IS a
//     subnormal number, q times the type's smallest, and four bits up 16 q
//     times it.  One packed multiply-add takes that to q - z in units of 1/64
//     (1/512 in f16), exact, a normal number: nine instructions for eight
//     weights.  The operands are of the states' own type, and the states go in
//     as they are, so every product is exact, and a state that meets a code
//     equal to its zero adds nothing, however large it is (8e-8 of the logits'
//     norm, with states of 30000 on such codes as without).  Codes as they lie,
//     with the zero as what a group's sum starts from, are four instructions
//     less (1 row 54.5 us where this takes 60; 11 rows 79 both; with groups of
//     32 142 where this takes 100), but q h and z h then cancel only as far as
//     either is rounded: a state of 1000 on such a code took logits off by more
//     than 2^-16 of sum |h W|.
//   - The states lie in shared memory as operands in the pairs' order, all of
//     them, for the kernel's life.
//   - The sums of a group are f32 accumulators of their own, added to the
//     row's with the group's scale: no weight is rounded.  A lane's codes of a
//     stage are those of whole groups (32, 16 or 8 in a row for groups of 128,
//     64, 32), so an MMA never mixes two.
//   - Codes come by TMA, scales by cp.async from a warp of their own, in
//     one ring of stages.
//   - The two stage parities' sums are joined through shared memory at the
//     tile's end, in a fixed order, pair by pair of warps.
// Every mbarrier wait is bounded; one that gives up sets bit 0 of *err, and
// the warps then run through their remaining barriers without computing.
#pragma once
#include "sv_lm_head_q4.cuh"

namespace svq {

constexpr int kFewK = 128;       // columns per stage: 64 bytes of a row
constexpr int kFewGroups = 7;    // row groups of a tile
constexpr int kFewTile = 32 * kFewGroups;  // rows per tile at most
constexpr int kFewWarps = 2 * kFewGroups;  // that compute: row groups x 2 stage parities
constexpr int kFewHelp = 1;      // that fetches scales; with the producer sixteen warps: 128 registers each
constexpr int kFewThreads = 32 * (kFewWarps + kFewHelp + 1);
constexpr int kFewStages = 8;    // at most
constexpr int kFewBudget = 227 * 1024;

struct __align__(8) FewBars {
  uint64_t full[kFewStages], empty[kFewStages];
  volatile int abort;
};

__device__ __forceinline__ bool few_wait(FewBars& bars, uint64_t* bar, uint32_t parity, unsigned* err) {
  for (uint32_t i = 0; i < svk::kWaitPolls / 512; ++i) {
    if (poll(bar, parity)) return true;
    if (bars.abort) return false;
  }
  bars.abort = 1;
  if (err) atomicOr(err, 1u);
  return false;
}

__device__ __forceinline__ void all_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory"); }
// The two warps of row group `rw`.
__device__ __forceinline__ void pair_sync(int rw) { asm volatile("bar.sync %0, 64;" ::"r"(rw + 2) : "memory"); }

// D += A x B, K = 16: bf16 or f16 operands.
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Operand words of codes less their zero, (q - z) / kUnit, exactly.  A code in
// the lowest bits of a half word is the number q u (u the type's smallest
// subnormal), four bits up 16 q u (of both types' numbers, those up to 255 u are
// evenly spaced): one multiply-add by a power of two and -z / kUnit.
template <bool BF>
struct Operand {
  static constexpr float kUnit = BF ? 64.f : 512.f;  // 2^127 u and 2^15 u, the largest powers that fit
  uint32_t zero;
  __device__ explicit Operand(uint32_t z) {
    const float f = -1.f / kUnit * static_cast<float>(z);
    if constexpr (BF) {
      const __nv_bfloat162 two = __float2bfloat162_rn(f);
      zero = *reinterpret_cast<const uint32_t*>(&two);
    } else {
      const __half2 two = __float2half2_rn(f);
      zero = *reinterpret_cast<const uint32_t*>(&two);
    }
  }
  // codes P and P + 4 of a word
  template <int P>
  __device__ uint32_t of(uint32_t w) const {
    const uint32_t at = (P < 2 ? w : w >> 8) & (P % 2 ? 0x00F000F0u : 0x000F000Fu);
    if constexpr (BF) {
      const uint32_t k = P % 2 ? 0x7D007D00u : 0x7F007F00u;
      const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&at), *reinterpret_cast<const __nv_bfloat162*>(&k),
                                       *reinterpret_cast<const __nv_bfloat162*>(&zero));
      return *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const uint32_t k = P % 2 ? 0x68006800u : 0x78007800u;
      const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&at), *reinterpret_cast<const __half2*>(&k),
                                *reinterpret_cast<const __half2*>(&zero));
      return *reinterpret_cast<const uint32_t*>(&r);
    }
  }
};

struct FewArgs {
  Args g;
  const uint4* s0;
  const uint4* s1;
};

// The odd stride at which a row's scales (zeros) of a stage of n groups lie, in words.
__host__ __device__ constexpr int few_stride(int n) { return n == 1 ? 1 : n + 1; }
__host__ __device__ constexpr int few_zstride(int n) { return n == 1 ? 1 : 3; }

// NT tiles of 8 states, groups of G, Z: zeros are given, BF: bf16 states (else f16).
template <int NT, int G, bool Z, bool BF>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ CUtensorMap wmap,
                                                             const __grid_constant__ FewArgs f) {
  constexpr int kPer = kFewK / G;       // groups per stage
  constexpr int kLen = G / 32;          // words of a lane in a group
  // chains of MMAs per m tile (V = 128256, d = 4096, groups of 128: 11 rows 78.6
  // us, with one 81.3; with zeros 16 rows 132 and 126, groups of 64 11 rows 117
  // and 111)
  constexpr int kChains = G == 128 && !Z ? 2 : 1;
  constexpr int kStride = few_stride(kPer);
  const Args& g = f.g;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  const int stage_bytes = g.R * 64, rows = g.rows0 + g.rows1;
  constexpr int kZStride = Z ? few_zstride(kPer) : 0;
  const int elem = g.scale_dtype == SV_F32 ? 4 : 2;
  const int frag_row = g.nk * 256 + 64;  // (64 more: neighbouring rows in other banks)
  unsigned char* frag = smem + g.stages * stage_bytes;                              // [row][stage][operand 0..3][4 x 16 bytes]
  float* red = reinterpret_cast<float*>(frag + rows * frag_row);                    // [row warp][parity][4 NT][32]
  uint32_t* sbuf = reinterpret_cast<uint32_t*>(red + kFewWarps * NT * 128);  // [slot][tile row][kStride]
  uint32_t* zbuf = sbuf + g.stages * kFewTile * kStride;
  FewBars& bars = *reinterpret_cast<FewBars*>(zbuf + g.stages * kFewTile * kZStride);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // The states' 8-column chunks, shared evenly by the computing threads (a half
  // warp stays in one row, its places 16 columns apart).  The first loads go out
  // before the codes' own.
  constexpr int kAhead = 8;
  const int chunks = g.d / 8, all_chunks = g.nk * 16;
  auto step = [&](int& r, int& j) {
    while (j >= all_chunks) {
      j -= all_chunks;
      ++r;
    }
  };
  uint4 raw[kAhead];
  auto load = [&](uint4 (&raw)[kAhead], int r, int j, int n) {  // the first n
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k >= n) break;
      const int in = min(r, rows - 1);
      const uint4* src = in < g.rows0 ? f.s0 + static_cast<long long>(in) * chunks
                                      : f.s1 + static_cast<long long>(in - g.rows0) * chunks;
      raw[k] = __ldg(src + min(j, chunks - 1));
      j += 32 * kFewWarps;
      step(r, j);
    }
  };
  const int turns = (rows * all_chunks + 32 * kFewWarps - 1) / (32 * kFewWarps);  // chunks of a thread, at most
  int row0 = 0, chunk0 = threadIdx.x;
  if (warp < kFewWarps) {
    step(row0, chunk0);
    load(raw, row0, chunk0, turns);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&bars.full[s], 1 + 32 * kFewHelp);
      mbar_init(&bars.empty[s], kFewWarps / 2);
    }
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  if (warp == kFewWarps + kFewHelp) {
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
  if (warp >= kFewWarps) {
    // ---- scales and zeros, as the 32-bit words that hold them
    int s = 0, use = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < g.tiles; t += gridDim.x) {
      const long long v0 = static_cast<long long>(t) * g.R;
      const int n_rows = static_cast<int>(v0 + g.R <= g.V ? g.R : g.V - v0);
      for (int ks = 0; ok && ks < g.nk; ++ks) {
        if (use > 0) ok = __all_sync(0xFFFFFFFFu, few_wait(bars, &bars.empty[s], (use - 1) & 1, g.err));
        if (!ok) break;
        const int n = min(kPer, g.G - ks * kPer);
        fetch_words<kPer>(reinterpret_cast<uintptr_t>(g.scales) + (v0 * g.G + ks * kPer) * elem,
                          static_cast<long long>(g.G) * elem, n * elem, sbuf + s * kFewTile * kStride, kStride, n_rows,
                          lane, kFewHelp, warp - kFewWarps);
        if constexpr (Z)
          fetch_words<kPer == 1 ? 1 : 2>(reinterpret_cast<uintptr_t>(g.zeros) + v0 * g.G + ks * kPer, g.G, n,
                                         zbuf + s * kFewTile * kZStride, kZStride, n_rows, lane, kFewHelp, warp - kFewWarps);
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

  // ---- the states as operands; columns past dim are 0.  Everything waits for
  // this: several loads are in flight.
  {
    const int c = lane % 16, quarter = G == 128 ? c / 4 : G == 64 ? c % 8 / 2 : c % 4,
              word = G == 128 ? c % 4 : G == 64 ? c / 8 * 2 + c % 2 : c / 4;
    // chunk c of a stage: which lane quarter multiplies it, and as its how manieth word
    const uint32_t my_frag = smem_u32(frag) + word * 64 + quarter * 16;
    int r = row0, j = chunk0;
    for (int i0 = 0; i0 < turns; i0 += kAhead) {
      const int left = turns - i0;
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k < left) {
          if (j >= chunks) raw[k] = make_uint4(0, 0, 0, 0);
          if (r < rows)
            sts128(my_frag + r * frag_row + j / 16 * 256,
                   make_uint4(__byte_perm(raw[k].x, raw[k].z, 0x5410), __byte_perm(raw[k].x, raw[k].z, 0x7632),
                              __byte_perm(raw[k].y, raw[k].w, 0x5410), __byte_perm(raw[k].y, raw[k].w, 0x7632)));
          j += 32 * kFewWarps;
          step(r, j);
        }
      if (left > kAhead) load(raw, r, j, left - kAhead);
    }
  }
  all_sync();

  const int rw = warp % kFewGroups, kh = warp / kFewGroups, gq = lane / 4, t4 = lane % 4;
  const bool active = rw * 32 < g.R;
  const int swz = gq >> 1 & 3;
  const uint32_t codes0 = smem_u32(smem) + (rw * 32 + gq) * 64;
  const uint32_t srow0 = smem_u32(sbuf) + (rw * 32 + gq) * kStride * 4, zrow0 = smem_u32(zbuf) + (rw * 32 + gq) * kZStride * 4;
  uint32_t frag0[NT];  // columns of an MMA past the last row repeat it, unused
#pragma unroll
  for (int n = 0; n < NT; ++n) frag0[n] = smem_u32(frag) + min(n * 8 + gq, rows - 1) * frag_row + t4 * 16;
  const int scale_dtype = g.scale_dtype, G_all = g.G, nk = g.nk, stages = g.stages;
  auto release = [&](int slot) {
    __syncwarp();
    if (lane == 0) mbar_arrive_local(&bars.empty[slot]);
  };
  bool ok = true;
  int tile_no = 0;
  for (int t = blockIdx.x; t < g.tiles; t += gridDim.x, ++tile_no) {
    const long long v0 = static_cast<long long>(t) * g.R + rw * 32;
    // place of a row's first scale in its word; the rows of a lane lie 8 apart, so it is theirs all
    const int s_par = scale_dtype == SV_F32 ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(g.scales) / 2 + (v0 + gq) * g.G) & 1);
    const int z_par = static_cast<int>((reinterpret_cast<uintptr_t>(g.zeros) + (v0 + gq) * g.G) & 3);
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    // stages go to the warp groups by the parity of their count since the
    // start, and the ring's length is even: a slot has one group for good, so
    // a group sees every phase of its slots (a parity wait that skips one
    // could pass on the phase before)
    const int odd = tile_no & nk & 1;
    const long long count = static_cast<long long>(tile_no) * nk + (kh ^ odd);
    int s = static_cast<int>(count % stages), use = static_cast<int>(count / stages & 1);
    const int my_stages = (nk - (kh ^ odd) + 1) / 2;
    uint32_t w[2][2][2][4];  // [this stage's, the next one's][m tile][row half][word]
    auto fetch = [&](uint32_t (&to)[2][2][4], int slot, int phase) {
      ok = __all_sync(0xFFFFFFFFu, ok && few_wait(bars, &bars.full[slot], phase, g.err));
      if (!ok || !active) return;
      const uint32_t codes = codes0 + slot * stage_bytes;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t p = codes + (m * 16 + h * 8) * 64;
          if constexpr (G == 128) {
            const uint4 q = lds128(p + ((t4 ^ swz) << 4));
            to[m][h][0] = q.x, to[m][h][1] = q.y, to[m][h][2] = q.z, to[m][h][3] = q.w;
          } else if constexpr (G == 64) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint2 q = lds64(p + (((2 * j + t4 / 2) ^ swz) << 4) + t4 % 2 * 8);
              to[m][h][2 * j] = q.x, to[m][h][2 * j + 1] = q.y;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) to[m][h][j] = lds32(p + ((j ^ swz) << 4) + t4 * 4);
          }
        }
    };
    auto multiply = [&](const uint32_t (&w)[2][2][4], int ks, int slot) {
      if (ok && active) {
        const uint32_t srow = srow0 + slot * (kFewTile * kStride * 4) + (scale_dtype == SV_F32 ? 0 : (s_par + ks * kPer & 1) * 2);
        const uint32_t zrow = zrow0 + slot * (kFewTile * kZStride * 4) + (z_par + ks * kPer & 3);
        const int n_groups = min(kPer, G_all - ks * kPer);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if (j >= n_groups) break;
          float scale[2][2];
          if (scale_dtype == SV_F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) scale[i / 2][i % 2] = __uint_as_float(lds32(srow + (i * 8 * kStride + j) * 4));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) scale[i / 2][i % 2] = scale16(lds16(srow + i * 8 * kStride * 4 + j * 2), scale_dtype);
          }
          // groups of 128: everything the warp needs of the slot is in registers
          if constexpr (kPer == 1 && !Z) release(slot);
          uint32_t z[2][2];  // of each m tile's row halves
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i / 2][i % 2] = Z ? lds8(zrow + i * 8 * kZStride * 4 + j) & 15u : 8u;
          float part[kChains][2][NT][4] = {};
#pragma unroll
          for (int i = 0; i < kLen; ++i) {
            uint4 b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = lds128(frag0[n] + ks * 256 + (j * kLen + i) * 64);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t lo = w[m][0][j * kLen + i], hi = w[m][1][j * kLen + i];
              const Operand<BF> z_lo(z[m][0]), z_hi(z[m][1]);
              const uint32_t a0 = z_lo.template of<0>(lo), a1 = z_hi.template of<0>(hi), a2 = z_lo.template of<1>(lo),
                             a3 = z_hi.template of<1>(hi);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<BF>(part[0][m][n], a0, a1, a2, a3, b[n].x, b[n].y);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t lo = w[m][0][j * kLen + i], hi = w[m][1][j * kLen + i];
              const Operand<BF> z_lo(z[m][0]), z_hi(z[m][1]);
              const uint32_t a0 = z_lo.template of<2>(lo), a1 = z_hi.template of<2>(hi), a2 = z_lo.template of<3>(lo),
                             a3 = z_hi.template of<3>(hi);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<BF>(part[kChains - 1][m][n], a0, a1, a2, a3, b[n].z, b[n].w);
            }
          }
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float sum = kChains == 2 ? part[0][m][n][e] + part[1][m][n][e] : part[0][m][n][e];
                acc[m][n][e] = fmaf(scale[m][e / 2], sum, acc[m][n][e]);
              }
        }
      }
      if (!(kPer == 1 && !Z && ok && active)) release(slot);
    };
    auto next = [&]() {
      s += 2;
      if (s >= stages) {
        s -= stages;
        use ^= 1;
      }
    };
    int ks = kh ^ odd;
    if (my_stages > 0) fetch(w[0], s, use);
    for (int i = 0; i < my_stages; i += 2) {
      int slot = s;
      next();
      if (i + 1 < my_stages) fetch(w[1], s, use);
      multiply(w[0], ks, slot);
      ks += 2;
      if (i + 1 >= my_stages) break;
      slot = s;
      next();
      if (i + 2 < my_stages) fetch(w[0], s, use);
      multiply(w[1], ks, slot);
      ks += 2;
    }
    // join the parities: each warp of a pair gives away one m tile's sums and
    // finishes the other
    float* theirs = red + (rw * 2 + 1 - kh) * NT * 128 + lane;
    const float* mine = red + (rw * 2 + kh) * NT * 128 + lane;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        theirs[(n * 4 + e) * 32] = kh ? acc[0][n][e] : acc[1][n][e];
        if (kh) acc[0][n][e] = acc[1][n][e];
      }
    pair_sync(rw);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[0][n][e] += mine[(n * 4 + e) * 32];
    pair_sync(rw);  // read before the next tile's are written
    if (ok && active) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = n * 8 + 2 * t4 + e;
          if (r >= rows) continue;
          float* out = r < g.rows0 ? g.out0 + r * g.ld : g.out1 + (r - g.rows0) * g.ld;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const long long v = v0 + kh * 16 + h * 8 + gq;
            if (v < g.V) out[v] = acc[0][n][2 * h + e] * Operand<BF>::kUnit;
          }
        }
    }
  }
}

// Shared memory of a call with `stages` stages.
inline long long few_smem(const Args& g, int group, int stages, int nt) {
  const int per = kFewK / group;
  return 1024LL + stages * (g.R * 64 + kFewTile * 4 * (few_stride(per) + (g.zeros ? few_zstride(per) : 0))) +
         (g.rows0 + g.rows1) * (g.nk * 256LL + 64) + kFewWarps * nt * 128 * 4 + static_cast<int>(sizeof(FewBars));
}

// Launches the call here if its states fit beside a ring of four stages
// (SV_ERR_UNSUPPORTED otherwise, with nothing enqueued).
template <int NT, int G, bool Z, bool BF>
sv_status start_few(Args g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t stream) {
  int dev = 0;
  const int sms = sm_count(&dev);
  // tile rows: as few rounds as tiles of kFewTile allow, then spread evenly, in warps' 32 rows
  const long long rounds = (g.V + static_cast<long long>(sms) * kFewTile - 1) / (static_cast<long long>(sms) * kFewTile);
  g.R = static_cast<int>(((g.V + sms * rounds - 1) / (sms * rounds) + 31) / 32 * 32);
  g.tiles = (g.V + g.R - 1) / g.R;
  g.nk = (g.d + kFewK - 1) / kFewK;
  g.stages = kFewStages;
  while (g.stages >= 4 && few_smem(g, G, g.stages, NT) > kFewBudget) g.stages -= 2;  // (even: see the kernel)
  if (g.stages < 4) return SV_ERR_UNSUPPORTED;
  CUtensorMap mw;
  if (!encode(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, proj->packed, g.V, g.d / 2, g.R, 64))
    return svh::fail(SV_ERR_ARG, "tensor map encoding failed (alignment or size)");
  static bool attr_set[64] = {false};
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(few_kernel<NT, G, Z, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewBudget);
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set[dev] = true;
  }
  FewArgs f{g, static_cast<const uint4*>(s0), static_cast<const uint4*>(s1)};
  few_kernel<NT, G, Z, BF><<<static_cast<unsigned>(g.tiles < sms ? g.tiles : sms), kFewThreads,
                         static_cast<size_t>(few_smem(g, G, g.stages, NT)), stream>>>(mw, f);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  return SV_OK;
}

template <int NT, int G, bool BF>
sv_status start_few_zeros(const Args& g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  return g.zeros ? start_few<NT, G, true, BF>(g, proj, s0, s1, st) : start_few<NT, G, false, BF>(g, proj, s0, s1, st);
}

template <int G, bool BF>
sv_status start_few_group(const Args& g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  return g.rows0 + g.rows1 <= 8 ? start_few_zeros<1, G, BF>(g, proj, s0, s1, st)
                                : start_few_zeros<2, G, BF>(g, proj, s0, s1, st);
}

template <bool BF>
sv_status start_few_any(const Args& g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  if (proj->group == 32) return start_few_group<32, BF>(g, proj, s0, s1, st);
  if (proj->group == 64) return start_few_group<64, BF>(g, proj, s0, s1, st);
  return start_few_group<128, BF>(g, proj, s0, s1, st);
}

}  // namespace svq
