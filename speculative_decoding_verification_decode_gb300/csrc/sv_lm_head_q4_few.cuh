// The 4-bit LM head for up to 16 rows of states (include/sv_lm_head_q4.h).
//
// With so few rows the product is a stream of codes, and what must not stall
// it is the way from a code to an operand.  The tensor-memory kernel pays a
// store to tensor memory and two barrier trips per 128 columns on that way (135
// us at 11 rows, V = 128256, d = 4096, groups of 128; here 80, and 56 to 62 up
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
//     mask each and one shift: a code in the lowest bits of a half word IS the
//     f16 number q 2^-24, four bits up q 2^-20 (subnormal; tensor cores take
//     them as they are).  The states that meet the second kind are kept 16
//     times smaller.  The zeros come in as what a group's sum starts from,
//     -z sum_k h, the sums kept from the beginning.  Five instructions for
//     eight weights, and every product is exact.
//     Codes that low lose bits of the products' ends (measured: as if the
//     MMA aligned every subnormal's products by 2^-14): nothing to speak of
//     with bf16's eight significant bits (3.4e-7 of the logits' norm, as much
//     as a sum in f32), but 8.5e-7 with f16's eleven.  With f16 states
//     all four pairs therefore stand four bits up, two more shifts per word.
//   - So the states are f16 under a power of two per row that takes the row's
//     largest to 2^14: exact for whatever is above 2^-24 of it, within 2^-35
//     of it below, far under the f32 sums' roundings; the logits take the
//     power back.  They lie in shared memory as operands in the pairs' order,
//     all of them, for the kernel's life.
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
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from c.
__device__ __forceinline__ void mma16816_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

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
  float* sums = reinterpret_cast<float*>(frag + rows * frag_row);                   // [group][NT][lane quarter][4]
  float* red = sums + g.nk * kPer * NT * 16;                                        // [row warp][parity][4 NT][32]
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
  if (threadIdx.x < 16) reinterpret_cast<uint32_t*>(red)[threadIdx.x] = 0;
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
  // this: several loads are in flight, and several chunks in the making.
  uint32_t* tops = reinterpret_cast<uint32_t*>(red);   // the rows' largest finite states
  int* shifts = reinterpret_cast<int*>(red) + 16;      // and their powers of two (both until the first tile ends)
  const int c = lane % 16, quarter = G == 128 ? c / 4 : G == 64 ? c % 8 / 2 : c % 4,
            word = G == 128 ? c % 4 : G == 64 ? c / 8 * 2 + c % 2 : c / 4;
  // chunk c of a stage: which lane quarter multiplies it, and as its how manieth word
  const uint32_t my_frag = smem_u32(frag) + word * 64 + quarter * 16;
  auto place = [&](int r, int j) { return my_frag + r * frag_row + j / 16 * 256; };
  {
    const uint32_t limit = BF ? 0x7F80u : 0x7C00u;
    int r = row0, j = chunk0, rows_of[kAhead];
    for (int i0 = 0; i0 < turns; i0 += kAhead) {
      const int left = turns - i0;
      uint32_t top[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        top[k] = 0;
        if (k < left) {
          if (j >= chunks) raw[k] = make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t lo = w[i] & 0x7FFFu, hi = w[i] >> 16 & 0x7FFFu;
            top[k] = max(top[k], max(lo < limit ? lo : 0u, hi < limit ? hi : 0u));
          }
          rows_of[k] = r;
          if (r < rows) sts128(place(r, j), raw[k]);
          j += 32 * kFewWarps;
          step(r, j);
        }
      }
#pragma unroll
      for (int o = 8; o > 0; o /= 2)
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (k < left) top[k] = max(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], o));
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k < left && lane % 16 == 0 && rows_of[k] < rows) atomicMax(&tops[rows_of[k]], top[k]);
      if (left > kAhead) load(raw, r, j, left - kAhead);
    }
  }
  all_sync();
  // the power of two that takes a row's largest finite state to 2^14
  if (threadIdx.x < 16) {
    const uint32_t t = tops[threadIdx.x];
    shifts[threadIdx.x] =
        t ? 14 - ilogbf(BF ? __uint_as_float(t << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(t)))) : 0;
  }
  all_sync();
  constexpr int kMake = 2;
  int r = row0, j = chunk0;
#pragma unroll 1
  for (int i0 = 0; i0 < turns; i0 += kMake) {
    uint4 x[kMake];
    int rr[kMake], jj[kMake], shift[kMake];
#pragma unroll
    for (int k = 0; k < kMake; ++k) {  // (past the last row: the last one again, unused)
      rr[k] = r, jj[k] = j;
      const int in = min(r, rows - 1);
      x[k] = lds128(place(in, j));
      shift[k] = shifts[in];
      j += 32 * kFewWarps;
      step(r, j);
    }
    float sum[kMake];
    uint4 y[kMake];
#pragma unroll
    for (int k = 0; k < kMake; ++k) {
      const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      float h[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF) {
          h[2 * i] = __uint_as_float(w[i] << 16);
          h[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
          const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          h[2 * i] = two.x;
          h[2 * i + 1] = two.y;
        }
      }
      int left = shift[k];
      if constexpr (BF)
        if (left > 126) {  // (tiny rows: two factors)
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] *= 0x1p40f;
          left -= 40;
        }
      const float up = power(left), up_odd = BF ? power(left - 4) : up;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] *= i % 2 ? up_odd : up;
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 two = __floats2half2_rn(h[i], h[i + 4]);
        p[i] = *reinterpret_cast<const uint32_t*>(&two);
      }
      y[k] = make_uint4(p[0], p[1], p[2], p[3]);
      sum[k] = fmaf(BF ? 16.f : 1.f, (h[1] + h[3]) + (h[5] + h[7]), (h[0] + h[2]) + (h[4] + h[6]));
    }
    // the groups' sums, in the units of the products, with the zero of 8 or 1
#pragma unroll
    for (int o = 1; o < G / 8; o *= 2)
#pragma unroll
      for (int k = 0; k < kMake; ++k) sum[k] += __shfl_xor_sync(0xFFFFFFFFu, sum[k], o);
#pragma unroll
    for (int k = 0; k < kMake; ++k)
      if (rr[k] < rows) {
        sts128(place(rr[k], jj[k]), y[k]);
        if (jj[k] % (G / 8) == 0) {
          const float total = sum[k] * (BF ? (Z ? -0x1p-24f : -0x1p-21f) : (Z ? -0x1p-20f : -0x1p-17f));
          float* to = sums + (jj[k] / (G / 8) * NT + rr[k] / 8) * 16 + rr[k] % 8 / 2 * 4 + rr[k] % 2;
          to[0] = total;
          to[2] = total;
        }
      }
  }
  all_sync();

  const int rw = warp % kFewGroups, kh = warp / kFewGroups, gq = lane / 4, t4 = lane % 4;
  const bool active = rw * 32 < g.R;
  int back[NT][2];  // the rows' powers of two, to take back
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = n * 8 + 2 * t4 + e;
      back[n][e] = r < rows ? (BF ? 24 : 20) - shifts[r] : 0;
    }
  all_sync();
  const int swz = gq >> 1 & 3;
  const uint32_t codes0 = smem_u32(smem) + (rw * 32 + gq) * 64;
  const uint32_t srow0 = smem_u32(sbuf) + (rw * 32 + gq) * kStride * 4, zrow0 = smem_u32(zbuf) + (rw * 32 + gq) * kZStride * 4;
  uint32_t frag0[NT];  // columns of an MMA past the last row repeat it, unused
#pragma unroll
  for (int n = 0; n < NT; ++n) frag0[n] = smem_u32(frag) + min(n * 8 + gq, rows - 1) * frag_row + t4 * 16;
  const int scale_dtype = g.scale_dtype, G_all = g.G, nk = g.nk, stages = g.stages;
  const uint32_t sums0 = smem_u32(sums) + t4 * 16;
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
          float from[NT][4];  // -(zero or 1) sum h
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 x = lds128(sums0 + ((ks * kPer + j) * NT + n) * 64);
            from[n][0] = __uint_as_float(x.x), from[n][1] = __uint_as_float(x.y);
            from[n][2] = __uint_as_float(x.z), from[n][3] = __uint_as_float(x.w);
          }
          // groups of 128: everything the warp needs of the slot is in registers
          if constexpr (kPer == 1 && !Z) release(slot);
          float part[2][NT][4];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if constexpr (Z) {
              float z[2];
#pragma unroll
              for (int h = 0; h < 2; ++h)  // small integers: 2^23 + z less 2^23
                z[h] = __uint_as_float(0x4B000000u | (lds8(zrow + (m * 16 + h * 8) * kZStride * 4 + j) & 15u)) - 8388608.f;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[m][n][e] = from[n][e] * z[e / 2];
            }
          }
#pragma unroll
          for (int i = 0; i < kLen; ++i) {
            uint4 b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = lds128(frag0[n] + ks * 256 + (j * kLen + i) * 64);
            // (a tile's two MMAs apart: the second waits for the first)
            constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u, kEven = BF ? kLow : kHigh;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t lo = w[m][0][j * kLen + i], hi = w[m][1][j * kLen + i];
              const uint32_t lo0 = BF ? lo : lo << 4, hi0 = BF ? hi : hi << 4;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                if (i == 0 && !Z)
                  mma16816_from(part[m][n], lo0 & kEven, hi0 & kEven, lo & kHigh, hi & kHigh, b[n].x, b[n].y, from[n]);
                else
                  mma16816(part[m][n], lo0 & kEven, hi0 & kEven, lo & kHigh, hi & kHigh, b[n].x, b[n].y);
              }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t lo = w[m][0][j * kLen + i] >> 8, hi = w[m][1][j * kLen + i] >> 8;
              const uint32_t lo2 = BF ? lo : w[m][0][j * kLen + i] >> 4, hi2 = BF ? hi : w[m][1][j * kLen + i] >> 4;
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816(part[m][n], lo2 & kEven, hi2 & kEven, lo & kHigh, hi & kHigh, b[n].z, b[n].w);
            }
          }
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[m][n][e] = fmaf(scale[m][e / 2], part[m][n][e], acc[m][n][e]);
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
          const float a = power(back[n][e] / 2), b = power(back[n][e] - back[n][e] / 2);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const long long v = v0 + kh * 16 + h * 8 + gq;
            if (v < g.V) out[v] = acc[0][n][2 * h + e] * a * b;
          }
        }
    }
  }
}

// Shared memory of a call with `stages` stages.
inline long long few_smem(const Args& g, int group, int stages, int nt) {
  const int per = kFewK / group;
  return 1024LL + stages * (g.R * 64 + kFewTile * 4 * (few_stride(per) + (g.zeros ? few_zstride(per) : 0))) +
         (g.rows0 + g.rows1) * (g.nk * 256LL + 64) + static_cast<long long>(g.nk) * per * nt * 64 + kFewWarps * nt * 128 * 4 + static_cast<int>(sizeof(FewBars));
}

// Launches the call here if its states fit beside a ring of four stages
// (SV_ERR_UNSUPPORTED otherwise, with nothing enqueued).
template <int NT, int G, bool Z, bool BF>
sv_status start_few(Args g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t stream) {
  int dev = 0;
  const int sms = sm_count(&dev);
  // tile rows: as few rounds as tiles of 256 allow, then spread evenly, in warps' 32 rows
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
