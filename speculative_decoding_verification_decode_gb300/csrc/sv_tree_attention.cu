// Attention of a tree of drafted tokens over a paged cache
// (include/sv_tree.h).
//
// One key head's queries of a sequence (its nodes times the query heads that
// share the key head) are rows of tiles of 128; a key tile is 128 tokens of the
// cache, or 128 of the nodes.  S = Q K^T and O += P V run on the tensor cores
// (tcgen05, f32 accumulators in tensor memory); a softmax thread owns a row, so
// its maximum and sum need no exchange.  Few rows leave the MMA's other rows
// idle, which costs nothing while the cache's bytes bound the call.
//
// A CTA, one per SM, has
//   warps 0-3, 4-7  two softmax streams, each with a score tile and an output
//                   tile in tensor memory (4 x 128 columns, all there are);
//   warp 8, 11      producers of keys, of queries and values: TMA loads, one box
//                   per page (or part of a page) and 64 elements, 128-byte
//                   swizzle, into rings of tiles;
//   warp 9          issues the MMAs;
//   warp 10         mends value tiles: zeros past the last key, and what is no
//                   finite number among the drafted values (below).
// The softmax warps take registers that the others have no use for.
// A step is one query tile against one key tile, step g on stream g % 2.  With
// one query tile to an item the streams take its key tiles in turn and their
// results are joined at the end; with two, each takes one, and a key tile is
// loaded once for both.  The MMA warp issues QK(g + 2) right behind PV(g), into
// the score tile that PV(g) has just read the weights from (they lie over the
// scores), so that the tensor cores work on one stream while the other's warps
// take exponentials.  A step takes 1600 to 1800 clocks (the products alone 1070):
// score, softmax (1550), weights and output follow one another in a stream.
//
// Measured (both kernels, calls in a graph on inputs in turn; a call from Python takes
// 30 us of host time by itself): 64 sequences of up to 32 nodes and 4096 tokens, 64 / 8
// heads of 128: 167 us (the bytes alone 125); 2 of 100000 tokens with chains of 6:
// 116 us (106), 6.2 TB/s; one tree of 60 after 8191 tokens 35 us, one token after 777
// 15 us, both of them latencies one after another and code that is not yet fetched.
//
// The weights are taken against a reference that follows the row's maximum: it
// moves when the maximum passes it by 8 (in powers of two), and only then the
// output is rescaled, which keeps that off the ordinary step (167 us, moved with
// every new maximum 171); weights up to 2^8 lose nothing in either type.
//
// The work is cut into one piece per CTA, so that ragged lengths balance and one
// long context uses every SM.  Either the items, sequence after sequence, are cut
// evenly by what their tiles and ends cost, wherever that falls; or, where that
// costs no more, each item is divided by itself, into pieces as short as the CTAs
// allow (an item's end inside a piece takes some 10000 clocks).  An item that a cut divides leaves its parts (f32
// outputs, maximum, sum) in the workspace, at most two per CTA, and a second
// kernel joins them in order: the result depends on the inputs and the number of
// CTAs only.
//
// The weights multiply the values in the inputs' type, off by at most half a step
// (2^-8 in bf16): both operands of an MMA have one type, and the values have that one.
// Their sum, which divides, has them in f32.  The result's own rounding is as large:
// against 64 bits the error is 0.0018 to 0.0023 (bf16) and 0.00025 to 0.00029 (f16) of
// the outputs' norm, where weights in f32 leave 0.0016 to 0.0017 and 0.00021.  Weights
// in two halves (what the rounding leaves in the score tile's second half, the product
// with the values twice) would remove that; measured, with spilled registers: the full
// batch 251 us instead of 168, one tree 40.7 (35.0), a small batch 28.8 (24.1), long
// contexts 124.4 (115.5), one token 16.9 (15.3).
//
// What a node must not see may hold anything: scores are masked by selection,
// the values past a length are set to 0 before the MMA, and a drafted value that
// is no finite number is replaced by 0 and added to the rows that see it at
// the end (it is inf or NaN times a positive weight, so the weight's size does
// not matter).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>

#include "../../include/sv_tree.h"
#include "sv_host.h"
#include "sv_ptx.cuh"

namespace sva {

using svk::mbar_arrive_expect_tx;
using svk::mbar_arrive_local;
using svk::mbar_init;
using svk::smem_u32;

constexpr int kThreads = 384, kSoftWarps = 8;
// Registers a thread: 384 of 168 are 64512 at launch; 256 of 200 and 128 of 96 are 63488.
constexpr int kSoftRegs = 200, kOtherRegs = 96;
constexpr int kTile = 128;     // rows of a query tile, keys of a key tile
constexpr int kMaxCtas = 152;  // one per SM
constexpr int kFinishThreads = 256;
constexpr int kFinishRows = 32;  // rows that a CTA of the second kernel joins
constexpr float kSlack = 8.0f;   // how far the maximum may pass the reference, powers of two

__host__ __device__ constexpr int tile_bytes(int dp) { return kTile * dp * 2; }
// Slots of the rings of keys and values: with two query tiles they fill the
// shared memory.
__host__ __device__ constexpr int k_slots(int dp) { return dp == 128 ? 3 : 5; }
__host__ __device__ constexpr int v_slots(int dp) { return dp == 128 ? 2 : 5; }

// What a CTA leaves for the second kernel: the item whose first part, but not
// whole, it had.  A record per item (`pairs` > 0) is not written where its CTA gave
// up before it: the second kernel knows such an item from its own place, and what
// else it takes from the record only chooses among the parts.
struct __align__(16) Join {
  int parts;  // the CTAs behind it that have the others; 0: no such item
  int slot;   // of its part
  int cta;
  int b, head, pair;
  int nodes;     // of the sequence
  unsigned err;  // a wait gave up
};

struct Args {
  int G, per_tile;  // query heads per key head; nodes per query tile
  uint32_t G_inv;         // floor(2^32 / G) + 1: row / G is exact for the rows of a tile
  uint32_t per_pair_inv;  // ceil(2^32 / (nodes per pair of query tiles)): exact for as few nodes as there are
  int Hkv, D, page, box, tree_box;  // keys per box (a power of two), of the cache and of the nodes
  int box_shift;
  int batch, n, total, pages;
  long long max_pages, table_stride;
  const int* table;
  const int* lengths;
  const int* parents;
  const int* cu;
  const void* v;
  long long v_row, v_head;
  void* out;
  long long out_row, out_head;
  float* lse;
  int q_heads;
  bool wide;        // out in 32-byte stores
  float c;          // scale in powers of two, not negative
  bool flip;        // the scores' sign is turned (a negative scale)
  bool expire;      // testing aid: waits for a segment's outputs give up at once
  float* part;      // [2 CTAs][dp / 4][256 rows][4]: a warp, a row per lane, writes and reads whole lines
  float2* part_ml;  // [2 CTAs][256]: maximum (powers of two), sum
  struct Join* join;  // [CTAs], then one per item where `pairs` > 0
  int pairs;          // pairs of query tiles per key head, 0: more items than CTAs
  unsigned* status;
};

// ------------------------------------------------------------------ the plan

struct Sequence {
  int first, N, len;
  int cached, tiles, items;  // key tiles of the cache, all key tiles of an item, items (pairs of query tiles) per key head
};

// Sequence b; N = 0 where it has nothing to do or its offsets or length are bad.
__device__ __forceinline__ Sequence sequence(const Args& A, int b) {
  Sequence s;
  s.first = b * A.n;
  s.N = A.n;
  if (A.cu) {
    s.first = A.cu[b];
    const int end = A.cu[b + 1];
    s.N = s.first >= 0 && end >= s.first && end <= A.total && end - s.first <= A.n ? end - s.first : 0;
  }
  s.len = A.lengths[b];
  if (s.len < 0 || s.len > A.max_pages * A.page) s.N = 0;
  s.cached = (s.len + kTile - 1) / kTile;
  s.tiles = s.cached + (s.N + kTile - 1) / kTile;
  s.items = static_cast<int>(__umulhi(static_cast<uint32_t>(s.N + 2 * A.per_tile - 1), A.per_pair_inv));
  return s;
}

// Row r of a query tile is query head row_head of the tile's node row_node.
__device__ __forceinline__ int row_node(const Args& A, int r) {
  return A.G == 1 ? r : static_cast<int>(__umulhi(static_cast<uint32_t>(r), A.G_inv));
}
__device__ __forceinline__ int row_head(const Args& A, int r) { return r - row_node(A, r) * A.G; }

// What a key tile costs: five units for a pair of query tiles (two steps), three
// for a single one; and what an item costs beside its tiles (the pipeline's filling
// and the end).  Fitted to the CTAs' clocks on 64 ragged sequences of up to 4096
// tokens and 32 nodes: 3221, 1904, and 8000 to 10200 an item; with 4, 3 and 8 the
// slowest CTA took 14% longer than the mean.  (Fitted on that batch alone.)
constexpr int kPairCost = 5, kSingleCost = 3, kItemCost = 15;
// Units of one key head; the last pair of a sequence may lack its second tile.
__device__ __forceinline__ int units_of_head(const Args& A, const Sequence& s) {
  const bool odd = s.N <= (2 * s.items - 1) * A.per_tile;
  return s.tiles * (kPairCost * s.items - (odd ? kPairCost - kSingleCost : 0)) + kItemCost * s.items;
}
__device__ __forceinline__ long long units_of(const Args& A, const Sequence& s) {
  return s.N > 0 ? static_cast<long long>(units_of_head(A, s)) * A.Hkv : 0;
}

// W units over CTAs 0 .. ctas - 1, the first `more` of which take one more than
// `each`.
struct Cut {
  long long each;
  int more, ctas;
  __device__ __forceinline__ long long begin(int c) const { return each * c + (c < more ? c : more); }
  __device__ __forceinline__ long long count(int c) const { return c < ctas ? each + (c < more ? 1 : 0) : 0; }
  // the CTA that has unit u
  __device__ __forceinline__ int owner(long long u) const {
    const long long wide = (each + 1) * more;
    if (u < wide) return divide(u, each + 1);
    return more + divide(u - wide, each);
  }
  // (a division of 64 bits is some hundred instructions)
  static __device__ __forceinline__ int divide(long long a, long long b) {
    if ((a | b) >> 32) return static_cast<int>(a / b);
    return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
  }
};

// A run of key tiles of one item, on this CTA.
struct Segment {
  Sequence q;
  int b, head, pair;  // item: key head, pair of query tiles
  int t0, t1;         // key tiles
  bool two;           // both query tiles of the pair exist
  bool whole;         // all key tiles of the item
  int steps;
};

struct Walk {
  int b;
  long long off, left;
  int count;     // segments so far
  int rest;      // units of the last one's item behind it

  __device__ __forceinline__ bool next(const Args& A, Segment& s) {
    if (left <= 0) return false;
    for (;; ++b, off = 0) {
      if (b >= A.batch) return false;
      s.q = sequence(A, b);
      if (off < units_of(A, s.q)) break;
    }
    cut(A, s);
    return s.steps > 0;  // (part of a key tile at the end of a piece is none)
  }
  // The next segment, in sequence s.q; a cut inside a key tile leaves the tile to
  // the piece behind it.
  __device__ __forceinline__ void cut(const Args& A, Segment& s) {
    const int per_head = units_of_head(A, s.q);
    s.head = off < per_head ? 0 : Cut::divide(off, per_head);
    const int in_head = static_cast<int>(off - static_cast<long long>(s.head) * per_head), per_pair = kItemCost + kPairCost * s.q.tiles;
    s.pair = in_head < per_pair ? 0 : in_head / per_pair;
    const int in = in_head - s.pair * per_pair;
    s.b = b;
    s.two = s.q.N > (2 * s.pair + 1) * A.per_tile;
    const int all = s.two ? per_pair : kItemCost + kSingleCost * s.q.tiles, end = all - in < left ? all : in + static_cast<int>(left);
    const int from = in > kItemCost ? in - kItemCost : 0, to = end > kItemCost ? end - kItemCost : 0;
    s.t0 = s.two ? from / kPairCost : from / kSingleCost;
    s.t1 = s.two ? to / kPairCost : to / kSingleCost;
    s.whole = s.t0 == 0 && s.t1 == s.q.tiles;
    s.steps = (s.t1 - s.t0) * (s.two ? 2 : 1);
    rest = all - end;
    off += end - in;
    left -= end - in;
    ++count;
  }
};

struct PlanScratch {
  long long warp_sums[kThreads / 32];
  int warp_counts[kThreads / 32];
};
struct PlanMem {
  Cut cut;
  Walk w;     // after the CTA's first segment
  Segment s;  // that
  int any;    // there is one
  int parts;  // where items are divided by themselves: the parts behind this one; else -1
};

// Pieces of at most `limit` steps that the sequence's items are divided into:
// those of a pair of query tiles, of a last single one, of a key head.
struct Pieces {
  int pair, single, head;
};
__device__ __forceinline__ Pieces pieces_of(const Args& A, const Sequence& s, int limit) {
  Pieces p;
  const bool odd = s.N <= (2 * s.items - 1) * A.per_tile;
  const int tiles = limit < 2 ? 1 : limit / 2;  // of a pair
  p.pair = (s.tiles + tiles - 1) / tiles;
  p.single = (s.tiles + limit - 1) / limit;
  p.head = p.pair * (s.items - (odd ? 1 : 0)) + (odd ? p.single : 0);
  return p;
}

constexpr int kFewSequences = 32;  // worked out by every warp for itself (one tree 35.0 us, by the CTA 36.9)
constexpr int kLaneSequences = 8, kLaneSteps = 256;

// How the units are cut over C CTAs, and CTA c's first segment: by all of the
// CTA's threads, or by every warp for itself (few sequences: all write the same
// words, and none waits for another).
template <bool kWarp>
__device__ __forceinline__ void make_plan(const Args& A, int C, int c, PlanMem& m, PlanScratch& scratch) {
  constexpr int T = kWarp ? 32 : kThreads;
  const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5), t = kWarp ? lane : static_cast<int>(threadIdx.x);
  auto sync = [] {
    if (kWarp)
      __syncwarp();
    else
      __syncthreads();
  };
  const int per = A.batch <= T ? 1 : (A.batch + T - 1) / T;
  const int lo = t * per < A.batch ? t * per : A.batch, hi = lo + per < A.batch ? lo + per : A.batch;
  long long mine = 0;
  Sequence q{};
  for (int b = lo; b < hi; ++b) {
    q = sequence(A, b);
    mine += units_of(A, q);
  }
  long long x = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  long long before = x - mine, W = 0;
  if (kWarp) {
    W = __shfl_sync(0xFFFFFFFFu, x, 31);
  } else {
    if (lane == 31) scratch.warp_sums[warp] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const long long v = scratch.warp_sums[w];
      if (w < warp) before += v;
      W += v;
    }
  }
  // Each item by itself, in the shortest pieces that C CTAs can take, if the longest
  // of them (three units a step) costs no more than an even cut and the item's end
  // inside a piece, which that has.  2 sequences of 100000 tokens, 16 items in 9
  // pieces each: 116 us, cut evenly 120; 8 items of 8 tiles 14.8 and 20.6; of 65
  // tiles, two query tiles, 35 both ways.
  const long long longest = (Cut::divide(W, C) + kItemCost) / kSingleCost;
  const int most = longest < 1 << 20 ? static_cast<int>(longest) : 1 << 20;
  if (A.pairs && A.batch <= T) {  // (no more items than CTAs)
    // (by bisection, the longest first; a piece has a key tile, of three units or more)
    int lo = 1, hi = most;
    if (kWarp && A.batch <= kLaneSequences && most <= kLaneSteps) {
      // (few sequences: a lane per length, all looked at together; one tree after
      // 8191 tokens: 34.4 us, by bisection 37.1)
      unsigned fit = 0;
      for (int base = 0; base < most && !fit; base += 32) {
        int all = 0;
        for (int b = 0; b < A.batch; ++b) {
          Sequence o;
          o.N = __shfl_sync(0xFFFFFFFFu, q.N, b);
          o.tiles = __shfl_sync(0xFFFFFFFFu, q.tiles, b);
          o.items = __shfl_sync(0xFFFFFFFFu, q.items, b);
          if (o.N > 0) all += pieces_of(A, o, base + lane + 1).head * A.Hkv;
        }
        fit = __ballot_sync(0xFFFFFFFFu, all <= C && base + lane < most);
        if (fit) lo = hi = base + __ffs(fit);
      }
    }
    // (at most 22 turns halve 2^20 lengths; whatever the counts, the search ends)
    for (int turn = 0, limit = hi; turn < 24 && lo <= hi; ++turn) {
      const Pieces p = t < A.batch && q.N > 0 ? pieces_of(A, q, limit) : Pieces{0, 0, 0};
      const int count = p.head * A.Hkv;  // (of at most as many items as CTAs, 2^20 tiles each)
      int y = count;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int z = __shfl_up_sync(0xFFFFFFFFu, y, d);
        if (lane >= d) y += z;
      }
      int ahead = y - count, all = 0;
      if (kWarp) {
        all = __shfl_sync(0xFFFFFFFFu, y, 31);
      } else {
        if (lane == 31) scratch.warp_counts[warp] = y;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
          const int v = scratch.warp_counts[w];
          if (w < warp) ahead += v;
          all += v;
        }
      }
      if (all > C) {
        if (limit == most) break;
        lo = limit + 1;
      } else {
        hi = limit;
      }
      if (all <= C && lo == hi) {
        if (c >= ahead && c < ahead + count) {
          Segment s;
          s.q = q;
          s.b = t;
          const int i = c - ahead;
          s.head = i / p.head;
          const int in = i - s.head * p.head;
          s.pair = in / p.pair < q.items ? in / p.pair : q.items - 1;
          s.two = q.N > (2 * s.pair + 1) * A.per_tile;
          const int piece = in - s.pair * p.pair, n = s.two ? p.pair : p.single;
          s.t0 = static_cast<int>(static_cast<long long>(q.tiles) * piece / n);
          s.t1 = static_cast<int>(static_cast<long long>(q.tiles) * (piece + 1) / n);
          s.whole = n == 1;
          s.steps = (s.t1 - s.t0) * (s.two ? 2 : 1);
          m.s = s;
          m.w.b = t;
          m.w.off = m.w.left = 0;
          m.w.count = 1;
          m.any = 1;
          m.parts = n - 1 - piece;
        }
        sync();
        return;
      }
      limit = (lo + hi) / 2;
      sync();  // the counts have been read
    }
    sync();
  }
  Cut cut;  // (at least what an item and a key tile cost: a smaller piece may hold the end of no tile)
  constexpr int kLeast = kItemCost + kPairCost;
  cut.ctas = W >= static_cast<long long>(kLeast) * C ? C : W >= kLeast ? static_cast<int>(W / kLeast) : 1;
  cut.each = Cut::divide(W, cut.ctas);
  cut.more = static_cast<int>(W - cut.each * cut.ctas);
  const long long u = cut.begin(c);
  if (t == 0) m.cut = cut;
  if (u >= before && u < before + mine && cut.count(c) > 0) {
    int b = lo;
    if (per > 1)
      for (;; ++b) {
        q = sequence(A, b);
        const long long k = units_of(A, q);
        if (u < before + k || b + 1 >= hi) break;
        before += k;
      }
    Walk w;
    Segment s;
    w.b = b;
    w.off = u - before;
    w.left = cut.count(c);
    w.count = 0;
    s.q = q;
    w.cut(A, s);
    m.w = w;
    m.s = s;
    m.any = s.steps > 0;
  }
  sync();
}

// Keys of tile t that exist.
__device__ __forceinline__ int keys_of(const Segment& s, int t) {
  const int left = t < s.q.cached ? s.q.len - t * kTile : s.q.N - (t - s.q.cached) * kTile;
  return left < kTile ? left : kTile;
}

// ------------------------------------------------------------------ instructions

template <typename T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  static constexpr uint32_t kType = 1, kExp = 0x7F80;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
};
template <>
struct Num<__half> {
  static constexpr uint32_t kType = 0, kExp = 0x7C00;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float value(uint16_t x) { return __half2float(__ushort_as_half(x)); }
};

// Descriptors of tiles with 128-byte swizzle, panels of 64 elements (128-byte
// rows): low word the address in 16-byte units and the leading stride, high
// word the stride of 8 rows (1024 bytes), version 1 and the swizzle.  Query and
// key tiles are K-major; value tiles are N-major, their leading stride is that
// of the panels.
// Instruction descriptor: D f32, A and B of the type, M = 128, N; B N-major.
// kNegateA turns A's sign.
constexpr uint32_t kNegateA = 1u << 13;
template <typename T>
__host__ __device__ constexpr uint32_t idesc(int N, bool n_major) {
  return (1u << 4) | (Num<T>::kType << 7) | (Num<T>::kType << 10) | (n_major ? 1u << 16 : 0u) |
         ((static_cast<uint32_t>(N) >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

#define SVA_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define SVA_W8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// 32 consecutive columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : SVA_R8(v, 0), SVA_R8(v, 8), SVA_R8(v, 16), SVA_R8(v, 24)
      : "r"(taddr)
      : "memory");
}
// 128 of them: four loads in flight, one wait.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SVA_R8(v, 0), SVA_R8(v, 8), SVA_R8(v, 16), SVA_R8(v, 24)
      : "r"(taddr)
      : "memory");
}
#define SVA_RW8(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7])
__device__ __forceinline__ void tmem_ld32_wait(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SVA_RW8(v, 0), SVA_RW8(v, 8), SVA_RW8(v, 16), SVA_RW8(v, 24)::"memory");
}
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, uint32_t* v) {
#pragma unroll
  for (int i = 0; i < 128; i += 32) tmem_ld32_issue(taddr + i, v + i);
#pragma unroll
  for (int i = 0; i < 128; i += 32) tmem_ld32_wait(v + i);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15};" ::SVA_W8(v, 0),
      SVA_W8(v, 8), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::SVA_W8(v, 0),
      SVA_W8(v, 8), SVA_W8(v, 16), SVA_W8(v, 24), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// (x0, x1) = (x0, x1) * (c, c) + (a, a)
__device__ __forceinline__ void fma2(float& x0, float& x1, float c, float a) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mov.b64 z, {%3, %3};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1)
      : "f"(c), "f"(a));
}
__device__ __forceinline__ void add2(float& a0, float& a1, float x0, float x1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(a0), "+f"(a1)
      : "f"(x0), "f"(x1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ------------------------------------------------------------------ the kernel

// The segments of a CTA are worked out once, by the keys' producer, and handed to
// the MMA and softmax warps in a ring: segment i + 1, and whether there is one,
// stand there before segment i's last key tile has landed.  The producer is at
// most k_slots tiles ahead of the scores, those two steps of the softmax, that
// one segment of its epilogue, and one segment is written ahead: k_slots + 4 at
// most.
struct Entry {
  Segment s;
  int rest;  // Walk::rest
  int more;  // there is a segment behind this one
};

template <int DP>
struct __align__(16) Shared {
  static constexpr int kQueue = k_slots(DP) + 6;
  uint64_t k_full[k_slots(DP)], k_empty[k_slots(DP)];  // keys: producer -> MMA, MMA -> producer
  uint64_t v_full[v_slots(DP)], v_empty[v_slots(DP)];  // values: producer -> MMA and mender, both -> producer
  uint64_t v_mended[v_slots(DP)];    // mender -> MMA
  uint64_t q_full[2], q_empty[2];    // query tiles
  uint64_t s_full[2];                // MMA -> softmax: the stream's scores
  uint64_t p_full[2];                // softmax -> MMA: its weights
  uint64_t o_full, o_empty;          // MMA -> softmax: a segment's outputs; softmax -> MMA: read
  uint64_t done;                     // every MMA has completed
  uint32_t tmem;
  volatile int abort;
  Join join;
  PlanMem plan;
  Entry queue[kQueue];               // segments behind the first, by number
  uint32_t v_odd[v_slots(DP)][4];    // keys of a value tile of nodes whose values are no finite numbers
  uint32_t odd[8];                   // the segment's nodes with such values
  union {
    float2 ex[2][kTile];             // [stream]: maximum, sum of each row
    PlanScratch scratch;             // (before that)
  };
};

// Segment i (0: the plan's), and what the queue says of it.
template <class S>
__device__ __forceinline__ const Segment& segment(const S& sm, int i) {
  return i ? sm.queue[i % S::kQueue].s : sm.plan.s;
}

// Steps of a CTA one after another.
struct Steps {
  int i;  // segment
  Segment s;
  int k;  // step of the segment
  bool ok;

  template <class S>
  __device__ __forceinline__ void start(const S& sm) {
    i = 0;
    s = sm.plan.s;
    k = 0;
    ok = sm.plan.any != 0;
  }
  // (the segment's last key tile has landed)
  template <class S>
  __device__ __forceinline__ void advance(const S& sm) {
    if (++k == s.steps) {
      k = 0;
      ok = sm.queue[i % S::kQueue].more != 0;
      ++i;
      if (ok) s = segment(sm, i);
    }
  }
  __device__ __forceinline__ int tile() const { return s.t0 + (s.two ? k >> 1 : k); }
  __device__ __forceinline__ bool fresh() const { return !s.two || !(k & 1); }  // the first step with its key tile
  __device__ __forceinline__ bool last() const { return !s.two || (k & 1); }    // and the last
};

template <class S>
__device__ __forceinline__ bool wait(S& sm, uint64_t* bar, uint32_t parity, uint32_t polls = svk::kWaitPolls) {
  for (uint32_t i = 0; i < polls; ++i) {
    if (svk::mbar_try_wait(bar, parity)) return true;
    if (sm.abort) return false;
  }
  sm.abort = 1;
  return false;
}
template <class S>
__device__ __forceinline__ bool warp_wait(S& sm, uint64_t* bar, uint32_t parity, uint32_t polls = svk::kWaitPolls) {
  return __all_sync(0xFFFFFFFFu, wait(sm, bar, parity, polls));
}
__device__ __forceinline__ void bar_soft() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory"); }

__device__ __forceinline__ bool all_soft(bool mine) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n selp.s32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<int>(mine)), "n"(32 * kSoftWarps)
      : "memory");
  return r != 0;
}

template <int DP>
__host__ __device__ constexpr int smem_bytes() {
  return (2 + k_slots(DP) + v_slots(DP)) * tile_bytes(DP) + static_cast<int>(sizeof(Shared<DP>));
}

static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "a CTA's shared memory");

// One lane of the warp, the same every time.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// The page of this lane's box of key tile t (looked up before the slot that the
// tile waits for is free), and its first token there.
struct Box {
  int id, at;
};
template <int DP>
__device__ __forceinline__ Box look_up(const Args& A, const Segment& s, int t, int lane) {
  constexpr int kPanels = DP / 64;
  Box x = {0, 0};
  if (t < s.q.cached && (lane / kPanels) << A.box_shift < keys_of(s, t)) {  // (at most 16 boxes of a panel)
    const int at = t * kTile + ((lane / kPanels) << A.box_shift), p = at / A.page;
    x.id = A.table[s.b * A.table_stride + p];
    x.at = at - p * A.page;
  }
  return x;
}

// Tile t of keys or values to shared memory at `dst`: every lane its box.
template <int DP>
__device__ __forceinline__ void load_tile(const Args& A, const Segment& s, int t, const Box& x, const CUtensorMap* cache,
                                          const CUtensorMap* own, uint32_t dst, uint64_t* bar, int lane) {
  constexpr int kPanels = DP / 64;
  if (t < s.q.cached) {
    const int boxes = (keys_of(s, t) + A.box - 1) >> A.box_shift;
    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * A.box * 128 * kPanels));
    __syncwarp();
    if (lane < boxes * kPanels)
      tma_4d(dst + (lane % kPanels) * (kTile * 128) + (lane / kPanels) * A.box * 128, cache, (lane % kPanels) * 64, x.at, s.head, x.id,
             bar);
  } else {
    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(A.tree_box * 128 * kPanels));
    __syncwarp();
    if (lane < kPanels)
      tma_3d(dst + lane * (kTile * 128), own, lane * 64, s.q.first + (t - s.q.cached) * kTile, s.head, bar);
  }
  __syncwarp();
}

template <int DP>
__device__ __forceinline__ void produce_keys(const Args& A, Shared<DP>& sm, uint32_t ring, const CUtensorMap* km, const CUtensorMap* kcm) {
  constexpr int kSlots = k_slots(DP);
  const int lane = static_cast<int>(threadIdx.x & 31);
  Walk w = sm.plan.w;
  Segment s = sm.plan.s;
  uint32_t slot = 0, turn = 0, loads = 0;
  bool alive = true;
  int i = 0;
  for (bool go = sm.plan.any; alive && go; ++i) {
    Segment behind;
    bool more = false;
    auto hand_over = [&]() {
      more = w.next(A, behind);
      if (lane == 0) {
        if (more) {
          sm.queue[(i + 1) % Shared<DP>::kQueue].s = behind;
          sm.queue[(i + 1) % Shared<DP>::kQueue].rest = w.rest;
        }
        sm.queue[i % Shared<DP>::kQueue].more = more;
      }
      __syncwarp();
    };
    if (s.t1 - s.t0 == 1) hand_over();
    for (int t = s.t0; alive && t < s.t1; ++t) {
      const Box x = look_up<DP>(A, s, t, lane);
      if (turn) alive = warp_wait(sm, &sm.k_empty[slot], (turn - 1) & 1);
      if (!alive) break;
      load_tile<DP>(A, s, t, x, kcm, km, ring + slot * tile_bytes(DP), &sm.k_full[slot], lane);
      ++loads;
      if (++slot == kSlots) slot = 0, ++turn;
      if (t == s.t0 && s.t1 - s.t0 > 1) hand_over();
    }
    s = behind;
    go = more;
  }
  // no copy may still be writing shared memory at exit
  for (uint32_t i = loads > kSlots ? loads - kSlots : 0; i < loads; ++i) svk::mbar_wait_bounded(&sm.k_full[i % kSlots], (i / kSlots) & 1);
}

// Queries and values (a query tile waits for a buffer that the segment before
// gives back; the keys behind it must not wait with it).
template <int DP>
__device__ __forceinline__ void produce_values(const Args& A, Shared<DP>& sm, uint32_t q_smem, uint32_t ring, const CUtensorMap* qm,
                                               const CUtensorMap* vm, const CUtensorMap* vcm) {
  constexpr int kSlots = v_slots(DP), kPanels = DP / 64;
  uint32_t qs = 0;
  const int lane = static_cast<int>(threadIdx.x & 31);
  Walk w = sm.plan.w;
  Segment s = sm.plan.s;
  uint32_t slot = 0, turn = 0, loads = 0;
  bool alive = true;
  for (bool go = sm.plan.any; alive && go; go = w.next(A, s)) {
    for (int j = 0; alive && j < (s.two ? 2 : 1); ++j, ++qs) {
      const uint32_t buf = qs & 1;
      if (qs >= 2) alive = warp_wait(sm, &sm.q_empty[buf], ((qs >> 1) - 1) & 1);
      if (!alive) break;
      if (lane == 0) mbar_arrive_expect_tx(&sm.q_full[buf], static_cast<uint32_t>(A.per_tile * A.G * 128 * kPanels));
      __syncwarp();
      if (lane < kPanels)
        tma_3d(q_smem + buf * tile_bytes(DP) + lane * (kTile * 128), qm, lane * 64, s.head * A.G,
               s.q.first + (2 * s.pair + j) * A.per_tile, &sm.q_full[buf]);
    }
    for (int t = s.t0; alive && t < s.t1; ++t) {
      const Box x = look_up<DP>(A, s, t, lane);
      if (turn) alive = warp_wait(sm, &sm.v_empty[slot], (turn - 1) & 1);
      if (!alive) break;
      load_tile<DP>(A, s, t, x, vcm, vm, ring + slot * tile_bytes(DP), &sm.v_full[slot], lane);
      ++loads;
      if (++slot == kSlots) slot = 0, ++turn;
    }
  }
  for (uint32_t i = loads > kSlots ? loads - kSlots : 0; i < loads; ++i) svk::mbar_wait_bounded(&sm.v_full[i % kSlots], (i / kSlots) & 1);
  for (uint32_t i = qs > 2 ? qs - 2 : 0; i < qs; ++i) svk::mbar_wait_bounded(&sm.q_full[i & 1], (i >> 1) & 1);
}

// Whether a value tile is mended before it is used.
__device__ __forceinline__ bool mends(const Segment& s, int t, int keys) { return t >= s.q.cached || keys % 16; }

template <typename T, int DP>
__device__ __forceinline__ void mend(const Args& A, Shared<DP>& sm, unsigned char* ring) {
  constexpr int kPanels = DP / 64, kSlots = v_slots(DP);
  const int lane = static_cast<int>(threadIdx.x & 31);
  Walk w = sm.plan.w;
  Segment s = sm.plan.s;
  uint32_t slot = 0, turn = 0;
  bool alive = true;
  for (bool go = sm.plan.any; alive && go; go = w.next(A, s)) {
    for (int t = s.t0; alive && t < s.t1; ++t) {
      alive = warp_wait(sm, &sm.v_full[slot], turn & 1);
      if (!alive) break;
      const int keys = keys_of(s, t);
      if (mends(s, t, keys)) {
        unsigned char* v = ring + slot * tile_bytes(DP);
        if (t >= s.q.cached) {
          if (lane < 4) sm.v_odd[slot][lane] = 0;
          __syncwarp();
          constexpr uint32_t kE = Num<T>::kExp;
          for (int i = lane; i < keys * 8 * kPanels; i += 32) {
            const int r = i / (8 * kPanels), x = i % (8 * kPanels);
            uint4* p = reinterpret_cast<uint4*>(v + (x / 8) * (kTile * 128) + r * 128 + (x % 8) * 16);
            uint4 u = *p;
            uint32_t* e = reinterpret_cast<uint32_t*>(&u);
            bool odd = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if ((e[j] & kE) == kE) e[j] &= 0xFFFF0000u, odd = true;
              if ((e[j] >> 16 & kE) == kE) e[j] &= 0xFFFFu, odd = true;
            }
            if (odd) {
              *p = u;
              atomicOr(&sm.v_odd[slot][r / 32], 1u << (r % 32));
            }
          }
        }
        for (int i = keys * 8 * kPanels + lane; i < (keys + 15) / 16 * 16 * 8 * kPanels; i += 32) {
          const int r = i / (8 * kPanels), x = i % (8 * kPanels);
          *reinterpret_cast<uint4*>(v + (x / 8) * (kTile * 128) + r * 128 + (x % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      if (lane == 0) {
        mbar_arrive_local(&sm.v_mended[slot]);
        mbar_arrive_local(&sm.v_empty[slot]);
      }
      __syncwarp();
      if (++slot == kSlots) slot = 0, ++turn;
    }
  }
}

template <typename T, int DP>
__device__ __forceinline__ void issue(const Args& A, Shared<DP>& sm, uint32_t q_smem, uint32_t k_ring, uint32_t v_ring, uint32_t tmem) {
  constexpr uint32_t kUnits = tile_bytes(DP) / 16;  // of the descriptors' addresses
  constexpr uint32_t kHi = (1024u >> 4) | 1u << 14 | 2u << 29;
  const bool leads = elected();
  const int lane = static_cast<int>(threadIdx.x & 31);
  // (all lanes run the loops, so that addresses stay in uniform registers)
  const uint32_t q_lo = ((q_smem & 0x3FFFFu) >> 4) | 1u << 16, k_lo = ((k_ring & 0x3FFFFu) >> 4) | 1u << 16;
  const uint32_t v_lo = ((v_ring & 0x3FFFFu) >> 4) | (kTile * 128 / 16) << 16;
  const uint32_t qk_desc = idesc<T>(kTile, false) | (A.flip ? kNegateA : 0u);  // (scores of a negative scale)
  auto full = [](uint32_t lo) { return static_cast<uint64_t>(kHi) << 32 | lo; };
  Steps qk = {}, pv;
  qk.start(sm);
  pv = qk;
  uint32_t k_slot = 0, k_turn = 0, v_slot = 0, v_turn = 0, qs = 0, q_first = 0, gq = 0, gp = 0;
  auto scores = [&]() {
    if (!qk.ok) return true;
    const bool two = qk.s.two;
    const uint32_t j = two ? qk.k & 1 : 0;
    if (qk.k == 0) q_first = qs;
    if (qk.k <= (two ? 1 : 0)) {
      if (!warp_wait(sm, &sm.q_full[qs & 1], (qs >> 1) & 1)) return false;
      ++qs;
    }
    if (j == 0 && !warp_wait(sm, &sm.k_full[k_slot], k_turn & 1)) return false;
    fence_after();
    const bool last = j == 1 || !two;
    const uint32_t buf = (q_first + j) & 1;
    const uint32_t a = q_lo + buf * kUnits, b = k_lo + k_slot * kUnits, d = tmem + (gq & 1) * kTile;
    if (leads) {
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        const uint32_t at = (i / 4) * (kTile * 128 / 16) + (i % 4) * 2;
        mma_ss(d, full(a + at), full(b + at), qk_desc, i > 0);
      }
      mma_commit(&sm.s_full[gq & 1]);
      if (last) mma_commit(&sm.k_empty[k_slot]);
      if (qk.k >= qk.s.steps - (two ? 2 : 1)) mma_commit(&sm.q_empty[buf]);
    }
    __syncwarp();
    if (last && ++k_slot == k_slots(DP)) k_slot = 0, ++k_turn;
    ++gq;
    qk.advance(sm);
    return true;
  };
  bool alive = scores() && scores();
  uint32_t segments = 0;
  while (alive && pv.ok) {
    if (pv.k == 0) {  // the outputs of the segment before have been read
      if (segments && !warp_wait(sm, &sm.o_empty, (segments - 1) & 1)) break;
      ++segments;
      if (lane < 8) sm.odd[lane] = 0;
      __syncwarp();
    }
    // steps whose scores-to-come are of the segment too: PV(k) and QK(k + 2) at a time
    if (qk.ok && qk.i == pv.i && pv.k < pv.s.steps - 2) {
      const bool two = pv.s.two;
      const int steps = pv.s.steps, whole = pv.s.q.len / kTile, cached = pv.s.q.cached;
      const int gives_back = steps - (two ? 2 : 1);  // the last scores against a query tile
      int keys = kTile;
      for (int k = pv.k; alive && k < steps - 2; ++k) {
        const uint32_t st = gp & 1, j = two ? k & 1 : 0;
        const bool fresh = j == 0, last = j == 1 || !two;
        bool ok = true;
        if (fresh) {
          const int t = pv.s.t0 + (two ? k >> 1 : k);
          uint64_t* bar = &sm.v_full[v_slot];
          keys = kTile;
          if (t >= whole) {
            keys = keys_of(pv.s, t);
            if (mends(pv.s, t, keys)) bar = &sm.v_mended[v_slot];
          }
          ok = wait(sm, bar, v_turn & 1);
          if (t >= cached && lane < 4) sm.odd[(t - cached) * 4 + lane] = sm.v_odd[v_slot][lane];
        }
        ok = wait(sm, &sm.p_full[st], (gp >> 1) & 1) && ok;
        alive = __all_sync(0xFFFFFFFFu, ok);
        fence_after();
        const uint32_t v = v_lo + v_slot * kUnits, kk = k_lo + k_slot * kUnits, buf = (q_first + j) & 1, q = q_lo + buf * kUnits;
        const uint32_t s = tmem + st * kTile, o = tmem + 256 + st * 128, acc = k >= 2 ? 1u : 0u;
        if (leads && alive) {
          if (keys > kTile - 16) {
#pragma unroll
            for (int i = 0; i < kTile / 16; ++i) mma_ts(o, s + i * 8, full(v + i * 128), idesc<T>(DP, true), i > 0 ? 1u : acc);
          } else {
#pragma unroll 1
            for (int i = 0; i * 16 < keys; ++i) mma_ts(o, s + i * 8, full(v + i * 128), idesc<T>(DP, true), i > 0 ? 1u : acc);
          }
          if (last) mma_commit(&sm.v_empty[v_slot]);
        }
        if (fresh) alive = __all_sync(0xFFFFFFFFu, wait(sm, &sm.k_full[k_slot], k_turn & 1)) && alive;
        if (leads && alive) {
#pragma unroll
          for (int i = 0; i < DP / 16; ++i) {
            const uint32_t at = (i / 4) * (kTile * 128 / 16) + (i % 4) * 2;
            mma_ss(s, full(q + at), full(kk + at), qk_desc, i > 0);
          }
          mma_commit(&sm.s_full[st]);
          if (last) mma_commit(&sm.k_empty[k_slot]);
          if (k + 2 >= gives_back) mma_commit(&sm.q_empty[buf]);
        }
        __syncwarp();
        if (last) {
          if (++v_slot == v_slots(DP)) v_slot = 0, ++v_turn;
          if (++k_slot == k_slots(DP)) k_slot = 0, ++k_turn;
        }
        ++gp;
      }
      if (!alive) break;
      gq += static_cast<uint32_t>(steps - 2 - pv.k);
      pv.k = steps - 2;
      qk.k = steps - 1;
      qk.advance(sm);
    }
    // the last two: the scores behind them are the next segment's
    const uint32_t st = gp & 1;
    const int t = pv.tile(), keys = keys_of(pv.s, t);
    if (pv.fresh() && !warp_wait(sm, mends(pv.s, t, keys) ? &sm.v_mended[v_slot] : &sm.v_full[v_slot], v_turn & 1)) break;
    if (t >= pv.s.q.cached && lane < 4) sm.odd[(t - pv.s.q.cached) * 4 + lane] = sm.v_odd[v_slot][lane];
    const bool last = pv.last(), end = pv.k == pv.s.steps - 1;
    const uint32_t b = v_lo + v_slot * kUnits, d = tmem + 256 + st * 128, a = tmem + st * kTile;
    const uint32_t acc = pv.k >= 2 ? 1u : 0u;
    if (!warp_wait(sm, &sm.p_full[st], (gp >> 1) & 1)) break;
    fence_after();
    if (leads) {
      if (keys > kTile - 16) {
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i) mma_ts(d, a + i * 8, full(b + i * 128), idesc<T>(DP, true), i > 0 ? 1u : acc);
      } else {
#pragma unroll 1
        for (int i = 0; i * 16 < keys; ++i) mma_ts(d, a + i * 8, full(b + i * 128), idesc<T>(DP, true), i > 0 ? 1u : acc);
      }
      if (last) mma_commit(&sm.v_empty[v_slot]);
      if (end) mma_commit(&sm.o_full);
    }
    __syncwarp();
    if (last && ++v_slot == v_slots(DP)) v_slot = 0, ++v_turn;
    ++gp;
    pv.advance(sm);
    alive = scores();
  }
  if (leads) mma_commit(&sm.done);
  __syncwarp();
  svk::mbar_wait_bounded(&sm.done, 0);
}

// Bits of the nodes of tree tile j that node i sees.
__device__ __forceinline__ uint4 seen_bits(const Args& A, int first, int i, int j) {
  uint32_t w[4] = {0, 0, 0, 0};
  auto set = [&](int k) {
    k -= j * kTile;
    if (k >= 0 && k < kTile) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (k >> 5 == x) w[x] |= 1u << (k & 31);
    }
  };
  if (!A.parents) {  // 0 .. i
    const int k = i - j * kTile;
#pragma unroll
    for (int x = 0; x < 4; ++x) w[x] = k >= 32 * x + 31 ? 0xFFFFFFFFu : k >= 32 * x ? (2u << (k & 31)) - 1u : 0u;
  } else {
    set(i);
    for (int p = A.parents[first + i], was = i; p >= 0 && p < was;) {
      set(p);
      was = p;
      p = A.parents[first + p];
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ void store_out(T* dst, const float* o, float f) {
  uint4 u;
  u.x = Num<T>::pack(o[0] * f, o[1] * f);
  u.y = Num<T>::pack(o[2] * f, o[3] * f);
  u.z = Num<T>::pack(o[4] * f, o[5] * f);
  u.w = Num<T>::pack(o[6] * f, o[7] * f);
  *reinterpret_cast<uint4*>(dst) = u;
}

// 32 bytes, a whole sector.
template <typename T>
__device__ __forceinline__ void store_out16(T* dst, const float* o, float f) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = Num<T>::pack(o[2 * i] * f, o[2 * i + 1] * f);
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), SVA_W8(u, 0) : "memory");
}

// A softmax warp.
template <typename T, int DP>
__device__ __forceinline__ void soften(const Args& A, Shared<DP>& sm, uint32_t tmem, int c) {
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int stream = warp >> 2, row = (warp & 3) * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t s_col = tmem + lanes + stream * kTile, o_col = tmem + lanes + 256;
  uint32_t g = 0;          // steps before the segment, both streams
  uint32_t turns = 0;      // of this stream
  // (a scale of 0 as one that makes every finite score 0 too, and -inf still -inf)
  const float c2 = A.c > 0 ? A.c : 1e-45f;
  bool alive = true;
  Segment s = sm.plan.s;
  int number = 0;
  for (bool go = sm.plan.any; go; ++number) {
    // this stream's steps of the segment: k = k0, k0 + 2, ...
    const int k0 = static_cast<int>((stream ^ g) & 1);
    const int query = 2 * s.pair + (s.two ? k0 : 0);
    const int rows = (s.q.N - query * A.per_tile < A.per_tile ? s.q.N - query * A.per_tile : A.per_tile) * A.G;
    const bool busy = (warp & 3) * 32 < rows;  // the warp has a row
    const int node = query * A.per_tile + row_node(A, row);
    float ref = -INFINITY, sum = 0;
    for (int k = k0; k < s.steps; k += 2) {
      const int t = s.t0 + (s.two ? k >> 1 : k);
      const int keys = keys_of(s, t);
      const bool tree = t >= s.q.cached;
      uint32_t bits[4] = {0, 0, 0, 0};
      if (busy && tree && row < rows) {
        const uint4 seen = seen_bits(A, s.q.first, node, t - s.q.cached);
        bits[0] = seen.x, bits[1] = seen.y, bits[2] = seen.z, bits[3] = seen.w;
      }
      if (alive) alive = warp_wait(sm, &sm.s_full[stream], turns & 1);
      ++turns;
      fence_after();
      if (busy && alive) {
        const bool masked = tree || keys < kTile;
        if (masked && !tree) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = keys - 32 * i;
            bits[i] = n >= 32 ? 0xFFFFFFFFu : n > 0 ? (1u << n) - 1u : 0u;
          }
        }
        // what the row does not see becomes -inf, in tensor memory: few tiles need
        // it, and the code of the others stays short
        if (masked) {
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            uint32_t u[32];
            tmem_ld32(s_col + i * 32, u);
            const uint32_t bit = i == 0 ? bits[0] : i == 1 ? bits[1] : i == 2 ? bits[2] : bits[3];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(bit >> j & 1)) u[j] = 0xFF800000u;
            tmem_st32(s_col + i * 32, u);
          }
          tmem_st_wait();
        }
        uint32_t u[kTile];
        tmem_ld128(s_col, u);
        float* x = reinterpret_cast<float*>(u);
        float m0 = x[0], m1 = x[1], m2 = x[2], m3 = x[3];
#pragma unroll
        for (int j = 4; j < kTile - 4; j += 8) {
          m0 = max3(m0, x[j], x[j + 1]);
          m1 = max3(m1, x[j + 2], x[j + 3]);
          m2 = max3(m2, x[j + 4], x[j + 5]);
          m3 = max3(m3, x[j + 6], x[j + 7]);
        }
        m0 = max3(m0, x[kTile - 4], x[kTile - 3]);
        m1 = max3(m1, x[kTile - 2], x[kTile - 1]);
        float top = max3(fmaxf(m0, m1), m2, m3);
        top *= c2;
        const bool move = top > ref + kSlack || (ref == -INFINITY && top > -INFINITY);
        if (__any_sync(0xFFFFFFFFu, move)) {
          const float to = move ? top : ref;
          const float f = ref == -INFINITY ? 0.0f : svk::ex2_ftz(ref - to);
          ref = to;
          sum *= f;
          if (k >= 2) {
#pragma unroll 1
            for (int i = 0; i < DP / 32; ++i) {
              uint32_t o[32];
              tmem_ld32(o_col + stream * 128 + i * 32, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st32(o_col + stream * 128 + i * 32, o);
            }
          }
        }
        const float minus = ref == -INFINITY ? 0.0f : -ref;
        float a0 = 0, a1 = 0, b0 = 0, b1 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[16];
#pragma unroll
          for (int j = i * 32; j < i * 32 + 32; j += 4) {
            fma2(x[j], x[j + 1], c2, minus);
            fma2(x[j + 2], x[j + 3], c2, minus);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j + e] = svk::ex2_ftz(x[j + e]);
            add2(a0, a1, x[j], x[j + 1]);
            add2(b0, b1, x[j + 2], x[j + 3]);
            p[(j - i * 32) / 2] = Num<T>::pack(x[j], x[j + 1]);
            p[(j - i * 32) / 2 + 1] = Num<T>::pack(x[j + 2], x[j + 3]);
          }
          tmem_st16(s_col + i * 16, p);  // (over scores that have been read)
        }
        sum += (a0 + a1) + (b0 + b1);
        tmem_st_wait();
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_local(&sm.p_full[stream]);
    }
    // ---- the segment's end
    // what this stream's output and the other's are multiplied by; the step that
    // comes first is this stream's where k0 is 0
    float keep = 1.0f, keep_other = 0.0f;
    const bool have = s.two || k0 == 0 || s.steps > 1, have_other = !s.two && (k0 == 1 || s.steps > 1);
    if (!s.two) {
      sm.ex[stream][row] = make_float2(ref, sum);
      bar_soft();
      const float2 other = sm.ex[stream ^ 1][row];
      bar_soft();
      const float m = fmaxf(ref, other.x);
      const float mine = ref == -INFINITY ? 0.0f : svk::ex2_ftz(ref - m);
      const float theirs = other.x == -INFINITY ? 0.0f : svk::ex2_ftz(other.x - m);
      sum = sum * mine + other.y * theirs;
      ref = m;
      keep = mine;
      keep_other = theirs;
    }
    if (alive) alive = warp_wait(sm, &sm.o_full, number & 1, A.expire ? 0u : svk::kWaitPolls);
    fence_after();
    const int begin = s.two ? 0 : stream * (DP / 2), width = s.two ? DP : DP / 2;
    const bool mine = alive && busy && row < rows;
    const long long at = static_cast<long long>(s.q.first) + node;
    const int qh = s.head * A.G + row_head(A, row);
    const int slot = 2 * c + (number ? 1 : 0);
    float* part = A.part + static_cast<long long>(slot) * 256 * DP + ((s.two ? k0 * kTile : 0) + row) * 4;
    const float inv = sum > 0 || sum != sum ? 1.0f / sum : 0.0f;
    uint32_t odd_any = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) odd_any |= sm.odd[i];
    if (busy && alive) {
      for (int col = begin; col < begin + width; col += 32) {
        float o[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0;
        if (have) {
          uint32_t u[32];
          tmem_ld32(o_col + stream * 128 + col, u);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(u[j]) * keep;
        }
        if (have_other) {
          uint32_t u[32];
          tmem_ld32(o_col + (stream ^ 1) * 128 + col, u);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = fmaf(__uint_as_float(u[j]), keep_other, o[j]);
        }
        if (odd_any && row < rows) {  // drafted values that are no finite numbers, of the nodes this one sees
          for (int tt = 0; tt < 2; ++tt) {
            if (s.q.cached + tt < s.t0 || s.q.cached + tt >= s.t1) continue;
            const uint4 seen = seen_bits(A, s.q.first, node, tt);
#pragma unroll 1
            for (int x = 0; x < 4; ++x)
              for (uint32_t left = (x == 0 ? seen.x : x == 1 ? seen.y : x == 2 ? seen.z : seen.w) & sm.odd[tt * 4 + x]; left; left &= left - 1) {
                const int k = tt * kTile + x * 32 + __ffs(left) - 1;
                const uint16_t* v = static_cast<const uint16_t*>(A.v) + (static_cast<long long>(s.q.first) + k) * A.v_row + s.head * A.v_head;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (col + j < A.D && (v[col + j] & Num<T>::kExp) == Num<T>::kExp) o[j] += Num<T>::value(v[col + j]);
              }
          }
        }
        if (mine && s.whole) {
          T* dst = static_cast<T*>(A.out) + at * A.out_row + static_cast<long long>(qh) * A.out_head + col;
          if (A.wide) {
#pragma unroll
            for (int j = 0; j < 32; j += 16)
              if (col + j < A.D) store_out16<T>(dst + j, o + j, inv);
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              if (col + j < A.D) store_out<T>(dst + j, o + j, inv);
          }
        } else if (mine) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(part + (col + j) * 256) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        }
      }
    }
    if (s.t0 == 0 && threadIdx.x == 0 && (!s.whole || A.pairs)) {
      Join j;
      j.parts = s.whole ? 0 : sm.plan.parts;
      if (j.parts < 0) {  // up to the CTA that has the item's last unit
        j.parts = sm.plan.cut.owner(sm.plan.cut.begin(c + 1) + (number ? sm.queue[number % Shared<DP>::kQueue].rest : sm.plan.w.rest) - 1) - c;
      }
      j.slot = slot;
      j.cta = c;
      j.b = s.b;
      j.head = s.head;
      j.pair = s.pair;
      j.nodes = s.q.N;
      j.err = 0;
      if (A.pairs)
        A.join[gridDim.x + (s.b * A.Hkv + s.head) * A.pairs + s.pair] = j;
      else
        sm.join = j;
    }
    if (mine && (s.two || stream == 0)) {
      if (!s.whole)
        A.part_ml[slot * 256 + (s.two ? k0 * kTile : 0) + row] = make_float2(ref, sum);
      else if (A.lse)
        A.lse[at * A.q_heads + qh] = (ref + log2f(sum)) * 0.69314718055994531f;
    }
    fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_local(&sm.o_empty);
    g += static_cast<uint32_t>(s.steps);
    // (all warps go on or none, or one would wait for the others at a barrier; a
    // producer that gave up has not said whether there is more)
    go = all_soft(alive) && sm.queue[number % Shared<DP>::kQueue].more != 0;
    if (go) s = segment(sm, number + 1);
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ Args A, const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                  const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap kcm,
                  const __grid_constant__ CUtensorMap vcm) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = smem_raw;  // (the swizzle wants 1024 bytes, and there is no room to move up)
  if (smem_u32(base) & 1023) {
    if (threadIdx.x == 0) A.join[blockIdx.x].parts = 0, A.join[blockIdx.x].err = 1u;
    return;
  }
  unsigned char* v_ptr = base + (2 + k_slots(DP)) * tile_bytes(DP);
  Shared<DP>& sm = *reinterpret_cast<Shared<DP>*>(v_ptr + v_slots(DP) * tile_bytes(DP));
  const uint32_t q_smem = smem_u32(base), k_ring = q_smem + 2 * tile_bytes(DP), v_ring = smem_u32(v_ptr);
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int C = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < k_slots(DP); ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < v_slots(DP); ++i) {
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 2);
      mbar_init(&sm.v_mended[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, kSoftWarps);
    mbar_init(&sm.done, 1);
    sm.abort = 0;
    sm.join.parts = 0;
    sm.plan.any = 0;
    sm.plan.parts = -1;
    svk::fence_mbar_init_cluster();
  }
  if (warp == 8 && (threadIdx.x & 31) == 0)
    for (const CUtensorMap* m : {&qm, &km, &vm, &kcm, &vcm}) asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (A.batch <= kFewSequences)
    make_plan<true>(A, C, c, sm.plan, sm.scratch);
  else
    make_plan<false>(A, C, c, sm.plan, sm.scratch);
  const uint32_t tmem = sm.tmem;
  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8)
      produce_keys<DP>(A, sm, k_ring, &km, &kcm);
    else if (warp == 9)
      issue<T, DP>(A, sm, q_smem, k_ring, v_ring, tmem);
    else if (warp == 10)
      mend<T, DP>(A, sm, v_ptr);
    else
      produce_values<DP>(A, sm, q_smem, v_ring, &qm, &vm, &vcm);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    soften<T, DP>(A, sm, tmem, c);
  }
  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
  if (threadIdx.x == 0) {
    Join j = sm.join;
    j.err = sm.abort ? 1u : 0u;
    A.join[c] = j;
  }
}

// Whether what thread t of T looks at of sequence b's layout is bad.
__device__ __forceinline__ bool bad_layout(const Args& A, int b, int t, int T) {
  int first = b * A.n, N = A.n;
  if (A.cu) {
    first = A.cu[b];
    const int end = A.cu[b + 1];
    N = end - first;
    if (first < 0 || end < first || end > A.total || N > A.n) return true;
  }
  const int len = A.lengths[b];
  if (len < 0 || len > A.max_pages * A.page) return true;
  const int used = (len + A.page - 1) / A.page;
  const int* row = A.table + b * A.table_stride;
  bool bad = false;
#pragma unroll 8
  for (int j = t; j < used; j += T) {
    const int p = row[j];
    bad |= p < 0 || p >= A.pages;
  }
  if (A.parents && t < N) {  // (T is not less than the most nodes)
    const int p = A.parents[first + t];
    bad |= p < -1 || p >= t;
  }
  return bad;
}
static_assert(kFinishThreads >= SV_TREE_MAX_NODES, "a thread per node");

// Joins the parts of items that several CTAs had, 32 rows to a CTA, and writes the
// statuses.
// kWide parts at a time, all their loads in flight, and kCols columns of a
// thread (a lane per row): eight of eight where few items are in many parts, two
// of sixteen where most CTAs leave an item in two.
template <typename T, int DP, int kWide, int kCols>
__global__ void __launch_bounds__(kFinishThreads, kWide > 2 ? 2 : 4) finish_kernel(const __grid_constant__ Args A, int C, int chunks) {
  const int t = static_cast<int>(threadIdx.x);
  if (static_cast<int>(blockIdx.x) < A.batch) {  // a sequence's status
    const int b = static_cast<int>(blockIdx.x);
    const bool bad = __syncthreads_or(bad_layout(A, b, t, kFinishThreads));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool late = __syncthreads_or(t < C && A.join[t].err != 0);
    if (t == 0) A.status[b] = (bad ? SV_SEQ_BAD_LAYOUT : 0u) | (late ? SV_SEQ_TIMEOUT : 0u);
    if (!bad) return;
    int first = b * A.n, N = A.n;
    if (A.cu) {
      first = A.cu[b];
      const int end = A.cu[b + 1];
      N = end - first;
      if (first < 0 || end < first || end > A.total || N > A.n) return;
    }
    for (int i = t / 16; i < N * A.q_heads; i += kFinishThreads / 16) {
      const int r = i / A.q_heads, h = i % A.q_heads, d = t % 16;
      T* o = static_cast<T*>(A.out) + static_cast<long long>(first + r) * A.out_row + static_cast<long long>(h) * A.out_head;
      if (8 * d < A.D) *reinterpret_cast<uint4*>(o + 8 * d) = make_uint4(0, 0, 0, 0);
      if (A.lse && d == 0) A.lse[static_cast<long long>(first + r) * A.q_heads + h] = -INFINITY;
    }
    return;
  }
  const int id = static_cast<int>(blockIdx.x) - A.batch, which = id / chunks, k = id % chunks;
  constexpr int kColBlocks = DP / (8 * kCols);  // chunks of a row's columns
  const int r = k / kColBlocks * kFinishRows + (t & 31);
  const int col = (k % kColBlocks) * (8 * kCols) + (t >> 5) * kCols;
  bool bad = false;
  Sequence q;
  int b = 0, head = 0, pair = 0;
  if (A.pairs) {  // the item is known before its parts are there (and from its place: the record may be what the workspace held)
    const int item = which / A.pairs;
    pair = which - item * A.pairs;
    b = item / A.Hkv;
    head = item - b * A.Hkv;
    q = sequence(A, b);
    if (q.N <= 0 || pair >= q.items) return;
    bad = __syncthreads_or(bad_layout(A, b, t, kFinishThreads));
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Join j = A.join[A.pairs ? C + which : which];
  if (j.parts <= 0 || j.cta < 0 || j.parts >= C - j.cta || j.slot < 0 || j.slot >= 2 * C) return;
  int nodes = q.N;
  if (!A.pairs) {
    if (j.b < 0 || j.b >= A.batch) return;
    b = j.b, head = j.head, pair = j.pair, nodes = j.nodes;
    q = sequence(A, b);  // (needed at the end: its loads are in flight with the parts')
  }
  const int query = 2 * pair + (r >= kTile ? 1 : 0), rr = r % kTile;
  const int node = query * A.per_tile + row_node(A, rr);
  const bool mine = rr < A.per_tile * A.G && node < nodes && col < A.D;
  float m = -INFINITY, sum = 0, o[kCols] = {};
  if (mine) {
    // the first part is the last segment of its CTA, the others are their CTAs' first
    const float2* ml = A.part_ml + r;
    const float* part = A.part + (col / 4 * 256 + r) * 4;
    for (int x0 = 0; x0 <= j.parts; x0 += kWide) {
      float2 e[kWide];
      float4 v[kWide][kCols / 4];
#pragma unroll
      for (int x = 0; x < kWide; ++x) {
        const long long slot = x0 + x == 0 ? j.slot : 2LL * (j.cta + (x0 + x <= j.parts ? x0 + x : j.parts));
        e[x] = ml[slot * 256];
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) v[x][i] = *reinterpret_cast<const float4*>(part + slot * 256 * DP + i * 1024);
      }
      float top = m;
#pragma unroll
      for (int x = 0; x < kWide; ++x)
        if (x0 + x <= j.parts) top = fmaxf(top, e[x].x);
      const float f = m == -INFINITY ? 0.0f : svk::ex2_ftz(m - top);
      m = top;
      sum *= f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) o[i] *= f;
#pragma unroll
      for (int x = 0; x < kWide; ++x)
        if (x0 + x <= j.parts) {
          const float w = e[x].x == -INFINITY ? 0.0f : svk::ex2_ftz(e[x].x - top);
          sum = fmaf(e[x].y, w, sum);
#pragma unroll
          for (int i = 0; i < kCols / 4; ++i) {
            o[4 * i] = fmaf(v[x][i].x, w, o[4 * i]);
            o[4 * i + 1] = fmaf(v[x][i].y, w, o[4 * i + 1]);
            o[4 * i + 2] = fmaf(v[x][i].z, w, o[4 * i + 2]);
            o[4 * i + 3] = fmaf(v[x][i].w, w, o[4 * i + 3]);
          }
        }
    }
  }
  if (!A.pairs) bad = __syncthreads_or(bad_layout(A, b, t, kFinishThreads));
  if (bad || !mine || node >= q.N) return;  // (a bad sequence's rows are written where its status is)
  const float inv = 1.0f / sum;
  const int qh = head * A.G + row_head(A, rr);
  const long long at = static_cast<long long>(q.first) + node;
  T* dst = static_cast<T*>(A.out) + at * A.out_row + static_cast<long long>(qh) * A.out_head;
#pragma unroll
  for (int i = 0; i < kCols; i += 8)
    if (col + i < A.D) store_out<T>(dst + col + i, o + i, inv);
  if (A.lse && col == 0) A.lse[at * A.q_heads + qh] = (m + log2f(sum)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<void*> fn{nullptr};  // (threads that ask at once find the same)
  void* p = fn.load(std::memory_order_acquire);
  if (!p) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(p, std::memory_order_release);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
}

// Dimensions innermost first; strides in elements of all but the first.  A
// dimension of one entry may have any stride: one that the encoding takes is put
// in (the others' are not 0).
bool encode(CUtensorMap* map, int64_t dtype, const void* data, int dims, const int64_t* size, const int64_t* stride,
            const int* box) {
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], e[4] = {1, 1, 1, 1};
  for (int i = 0; i < dims; ++i) {
    d[i] = static_cast<cuuint64_t>(size[i]);
    b[i] = static_cast<cuuint32_t>(box[i]);
    if (i) s[i - 1] = static_cast<cuuint64_t>(stride[i - 1] > 0 ? stride[i - 1] * 2 : 16);
  }
  return encoder()(map, dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                   static_cast<cuuint32_t>(dims), const_cast<void*>(data), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether [total, heads, dim] elements of 2 bytes have places of their own: heads
// within a row, or rows within a head's stretch.
bool rows_apart(int64_t total, int64_t heads, int64_t dim, int64_t row, int64_t head) {
  if (total <= 1) return heads <= 1 || head >= dim;
  if (heads <= 1) return row >= dim;
  return (head >= dim && row >= (heads - 1) * head + dim) || (row >= dim && head >= (total - 1) * row + dim);
}

// The array of the call that out shares memory with, NULL: none.  An array lies
// between its first and its last element; two of rows of the same stride may lie in one
// another's gaps (columns of one projection).
const char* shares_with_out(const sv_tree_attn& a) {
  using Big = __int128;  // (strides and sizes of 31 bits and more)
  const auto at = [](const void* p) { return static_cast<Big>(reinterpret_cast<uintptr_t>(p)); };
  const Big out = at(a.out), row_span = static_cast<Big>(a.q_heads - 1) * a.out_head + a.dim;  // (elements)
  const Big out_end = out + 2 * (static_cast<Big>(a.total - 1) * a.out_row + row_span);
  const auto meets = [&](const void* p, Big bytes) { return p && bytes > 0 && at(p) < out_end && out < at(p) + bytes; };
  const struct {
    const char* name;
    const void* p;
    int64_t row, head, heads;
  } rows[] = {{"q", a.q, a.q_row, a.q_head, a.q_heads}, {"k", a.k, a.k_row, a.k_head, a.kv_heads}, {"v", a.v, a.v_row, a.v_head, a.kv_heads}};
  for (const auto& x : rows) {
    const Big span = static_cast<Big>(x.heads - 1) * x.head + a.dim;
    if (!meets(x.p, 2 * (static_cast<Big>(a.total - 1) * x.row + span))) continue;
    if (x.row == a.out_row && row_span <= x.row && span <= x.row) {
      const Big d = ((at(x.p) - out) / 2 % x.row + x.row) % x.row;  // of its rows' places behind out's
      if (d >= row_span && d + span <= x.row) continue;
    }
    return x.name;
  }
  const auto pool = [&](int64_t page, int64_t token, int64_t head) {
    return 2 * (static_cast<Big>(a.pages - 1) * page + static_cast<Big>(a.page_size - 1) * token + static_cast<Big>(a.kv_heads - 1) * head + a.dim);
  };
  if (meets(a.k_cache, pool(a.kc_page, a.kc_token, a.kc_head))) return "k_cache";
  if (meets(a.v_cache, pool(a.vc_page, a.vc_token, a.vc_head))) return "v_cache";
  if (a.max_pages > 0 && meets(a.table, 4 * (static_cast<Big>(a.batch - 1) * a.table_stride + a.max_pages))) return "table";
  if (meets(a.lengths, 4 * a.batch)) return "lengths";
  if (meets(a.parents, 4 * a.total)) return "parents";
  if (meets(a.cu_nodes, 4 * (a.batch + 1))) return "cu_nodes";
  if (meets(a.lse, 4 * static_cast<Big>(a.total) * a.q_heads)) return "lse";
  return meets(a.status, 4 * a.batch) ? "status" : nullptr;
}

size_t workspace_bytes_of(int dim) {
  const size_t rows = 2 * kMaxCtas * 256;
  return rows * (dim <= 64 ? 64 : 128) * 4 + rows * 8 + 2 * kMaxCtas * sizeof(Join);
}

template <typename T, int DP>
sv_status launch(const sv_tree_attn& a, float scale, uint32_t flags, unsigned char* ws, cudaStream_t st) {
  if (!encoder()) return svh::fail(SV_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  Args A;
  A.G = static_cast<int>(a.q_heads / a.kv_heads);
  A.per_tile = kTile / A.G;
  A.G_inv = A.G == 1 ? 0u : static_cast<uint32_t>((1ULL << 32) / A.G + 1);
  A.per_pair_inv = static_cast<uint32_t>((1ULL << 32) / (2 * A.per_tile) + 1);
  A.Hkv = static_cast<int>(a.kv_heads);
  A.D = static_cast<int>(a.dim);
  A.page = static_cast<int>(a.page_size);
  A.box = 8;
  A.box_shift = 3;
  while (A.box < kTile && A.page % (2 * A.box) == 0) A.box *= 2, ++A.box_shift;
  A.tree_box = 8;
  while (A.tree_box < kTile && A.tree_box < a.n) A.tree_box *= 2;
  A.batch = static_cast<int>(a.batch);
  A.n = a.total > 0 ? static_cast<int>(a.n) : 0;
  A.total = static_cast<int>(a.total);
  A.pages = static_cast<int>(a.pages);
  A.max_pages = a.max_pages;
  A.table_stride = a.table_stride;
  A.table = a.table;
  A.lengths = a.lengths;
  A.parents = a.parents;
  A.cu = a.cu_nodes;
  A.v = a.v;
  A.v_row = a.v_row;
  A.v_head = a.v_head;
  A.out = a.out;
  A.out_row = a.out_row;
  A.out_head = a.out_head;
  A.lse = a.lse;
  A.q_heads = static_cast<int>(a.q_heads);
  A.wide = !((reinterpret_cast<uintptr_t>(a.out) & 31) | ((a.out_row | a.out_head | a.dim) & 15));
  A.c = (scale < 0 ? -scale : scale) * 1.4426950408889634f;
  A.flip = scale < 0;
  A.expire = (flags & SV_FLAG_EXPIRE_EXCHANGE) != 0;
  const size_t rows = 2 * kMaxCtas * 256;
  A.part = reinterpret_cast<float*>(ws);
  A.part_ml = reinterpret_cast<float2*>(ws + rows * DP * 4);
  A.join = reinterpret_cast<Join*>(ws + rows * DP * 4 + rows * 8);
  A.status = a.status;
  CUtensorMap qm, km, vm, kcm, vcm;
  if (a.total > 0) {
    const int64_t qd[] = {a.dim, a.q_heads, a.total}, qs[] = {a.q_head, a.q_row};
    const int64_t kd[] = {a.dim, a.total, a.kv_heads}, ks[] = {a.k_row, a.k_head}, vs[] = {a.v_row, a.v_head};
    const int64_t cd[] = {a.dim, a.page_size, a.kv_heads, a.pages}, kcs[] = {a.kc_token, a.kc_head, a.kc_page},
                  vcs[] = {a.vc_token, a.vc_head, a.vc_page};
    const int qb[] = {64, A.G, A.per_tile}, kb[] = {64, A.tree_box, 1}, cb[] = {64, A.box, 1, 1};
    if (!encode(&qm, a.dtype, a.q, 3, qd, qs, qb) || !encode(&km, a.dtype, a.k, 3, kd, ks, kb) ||
        !encode(&vm, a.dtype, a.v, 3, kd, vs, kb) || !encode(&kcm, a.dtype, a.k_cache, 4, cd, kcs, cb) ||
        !encode(&vcm, a.dtype, a.v_cache, 4, cd, vcs, cb))
      return svh::fail(SV_ERR_ARG, "tensor map encoding failed (a stride or size is out of range)");
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  // CTAs per device, 0: the kernels' attributes are not set yet.  One word, so that
  // another thread's first call sees both or neither.
  static std::atomic<int> ctas[64] = {};
  int C = ctas[dev].load(std::memory_order_acquire);
  if (!C) {
    const cudaError_t e = cudaFuncSetAttribute(attend_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<DP>());
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    // (the same split of the SM's memory as the first kernel's: no change between the two)
    cudaFuncSetAttribute(finish_kernel<T, DP, 2, DP / 8>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    cudaFuncSetAttribute(finish_kernel<T, DP, 8, 8>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (cudaDeviceGetAttribute(&C, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || C <= 0 || C > kMaxCtas) C = kMaxCtas;
    ctas[dev].store(C, std::memory_order_release);
  }
  const long long pairs = (a.n + 2 * A.per_tile - 1) / (2 * A.per_tile);
  A.pairs = a.batch <= C && a.batch * a.kv_heads * pairs <= C ? static_cast<int>(pairs) : 0;
  if (a.total > 0) {
    attend_kernel<T, DP><<<C, kThreads, smem_bytes<DP>(), st>>>(A, qm, km, vm, kcm, vcm);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  }
  // rows of a pair of query tiles, the second's from kTile on
  const int most = static_cast<int>(a.n > A.per_tile ? kTile + (a.n - A.per_tile < A.per_tile ? a.n - A.per_tile : A.per_tile) * A.G
                                                     : a.n * A.G);
  const int chunks = (most + kFinishRows - 1) / kFinishRows * (A.pairs ? DP / 64 : 1);
  const int join = a.total == 0 ? 0 : (A.pairs ? static_cast<int>(a.batch) * A.Hkv * A.pairs : C) * chunks;
  if (a.batch > 0x7FFFFFFF - join) return svh::fail(SV_ERR_UNSUPPORTED, "batch too large");
  const int grid = join + static_cast<int>(a.batch);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kFinishThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = a.total > 0 ? 1 : 0;
  const cudaError_t e = A.pairs ? cudaLaunchKernelEx(&cfg, finish_kernel<T, DP, 8, 8>, A, a.total > 0 ? C : 0, chunks)
                                : cudaLaunchKernelEx(&cfg, finish_kernel<T, DP, 2, DP / 8>, A, a.total > 0 ? C : 0, chunks);
  return e == cudaSuccess ? SV_OK : svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
}

}  // namespace sva

extern "C" {

size_t sv_tree_attention_workspace_size(int32_t dim) {
  return dim < 1 ? 0 : sva::workspace_bytes_of(dim);
}

sv_status sv_tree_attention(const sv_tree_attn* args, float scale, void* workspace, size_t workspace_bytes,
                            void* stream) {
  return sv_tree_attention_flagged(args, scale, 0, workspace, workspace_bytes, stream);
}

sv_status sv_tree_attention_flagged(const sv_tree_attn* args, float scale, uint32_t flags, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  svh::clear_error();
  if (flags & ~static_cast<uint32_t>(SV_FLAG_EXPIRE_EXCHANGE)) return svh::fail(SV_ERR_ARG, "unknown flag (%u)", flags);
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
  if (a.max_pages > 0 && a.page_size > SV_TREE_MAX_TOKENS / a.max_pages)
    return svh::fail(SV_ERR_UNSUPPORTED, "max_pages * page_size is more than %d tokens", SV_TREE_MAX_TOKENS);
  if (a.table_stride < a.max_pages && a.batch > 1) return svh::fail(SV_ERR_ARG, "table_stride (%lld) is less than max_pages", (long long)a.table_stride);
  const float c = scale * 1.4426950408889634f;  // (in powers of two)
  if (!(c == c) || c - c != 0) return svh::fail(SV_ERR_ARG, "scale must be finite");
  if (a.batch == 0) return SV_OK;
  if (!a.status || !a.lengths || (!a.table && a.max_pages > 0)) return svh::fail(SV_ERR_ARG, "status, lengths or table is NULL");
  if (a.total > 0 && (!a.q || !a.k || !a.v || !a.out)) return svh::fail(SV_ERR_ARG, "q, k, v or out is NULL");
  if (!a.k_cache || !a.v_cache) return svh::fail(SV_ERR_ARG, "a cache is NULL");
  const int64_t strides[] = {a.q_row, a.q_head, a.k_row, a.k_head, a.v_row, a.v_head, a.kc_page, a.kc_token,
                             a.kc_head, a.vc_page, a.vc_token, a.vc_head, a.out_row, a.out_head};
  for (const int64_t x : strides)
    if (x < 0 || x % 8) return svh::fail(SV_ERR_ARG, "strides must be multiples of 8 elements, not negative");
  const struct {
    const char* name;
    int64_t stride, size;
  } steps[] = {{"q_row", a.q_row, a.total},      {"q_head", a.q_head, a.q_heads},    {"k_row", a.k_row, a.total},
               {"k_head", a.k_head, a.kv_heads}, {"v_row", a.v_row, a.total},        {"v_head", a.v_head, a.kv_heads},
               {"kc_page", a.kc_page, a.pages},  {"kc_token", a.kc_token, a.page_size}, {"kc_head", a.kc_head, a.kv_heads},
               {"vc_page", a.vc_page, a.pages},  {"vc_token", a.vc_token, a.page_size}, {"vc_head", a.vc_head, a.kv_heads}};
  for (const auto& x : steps)
    if (x.stride == 0 && x.size > 1 && a.total > 0)
      return svh::fail(SV_ERR_ARG, "%s: a stride of 0 along a dimension of %lld (a broadcast view)", x.name, (long long)x.size);
  if (!sva::rows_apart(a.total, a.q_heads, a.dim, a.out_row, a.out_head)) return svh::fail(SV_ERR_ARG, "rows of out overlap");
  for (const void* p : {a.q, a.k, a.v, a.k_cache, a.v_cache, static_cast<const void*>(a.out)})
    if (reinterpret_cast<uintptr_t>(p) & 15) return svh::fail(SV_ERR_ARG, "q, k, v, the caches and out must be 16-byte aligned");
  const size_t need = sva::workspace_bytes_of(static_cast<int>(a.dim));
  if (!workspace || workspace_bytes < need)
    return svh::fail(SV_ERR_ARG, "workspace_bytes (%zu) < the %zu bytes sv_tree_attention_workspace_size() asks for",
                     workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return svh::fail(SV_ERR_ARG, "workspace must be 16-byte aligned");
  if (a.total > 0)
    if (const char* name = sva::shares_with_out(a)) return svh::fail(SV_ERR_ARG, "out shares memory with %s", name);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.dtype == SV_BF16)
    return a.dim <= 64 ? sva::launch<__nv_bfloat16, 64>(a, scale, flags, ws, st) : sva::launch<__nv_bfloat16, 128>(a, scale, flags, ws, st);
  return a.dim <= 64 ? sva::launch<__half, 64>(a, scale, flags, ws, st) : sva::launch<__half, 128>(a, scale, flags, ws, st);
}

}  // extern "C"
