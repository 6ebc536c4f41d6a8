// Pages of paged key/value caches: appending, sharing, giving up
// (include/sv_cache.h).
//
// Appending takes two kernels.  The first decides, in one CTA: a thread per
// sequence looks at its last page and what it needs, a prefix sum over the
// sequences says which of the free pages are its own, and the free pages come
// from a scan of the counts, lowest first, that ends where enough are found.  So
// which page goes where depends on the tables alone, not on the order of
// threads.  The second moves the rows of all pools, shared last pages first
// copied to their new ones.
//
// The second starts while the first still runs (a programmatic dependency).  Calls in
// a graph: 64
// paths of 32 nodes into 16 layers, then back: 15.7 us with four pools to a CTA,
// 18.7 with one, 16.6 with two, 16.0 with eight; the bytes alone are 3.  24 x 8 beams,
// 12 layers: 31 us for sharing, appending and giving up, of which the one CTA that
// deals out pages takes 9: a chain of dependent reads, which is what bounds these
// calls on the device.  From Python they take 74 to 88 us, most of it the host's: a
// launch each, and questions to every layer's tensors, which is what this interface (a
// list of tensors per layer) costs and not what the work needs.
//
// Sharing (fork) reads the table entries that a group's slots hold, lets every
// slot take its parent's, and corrects the pages' counts where an entry
// changed: beams that share a prefix change a few entries at the end.  The
// counts are sums of +1 and -1, so the order of the atomics does not matter.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sv_cache.h"
#include "sv_host.h"
#include "sv_ptx.cuh"

namespace svc {

constexpr int kPlanThreads = 1024;
constexpr int kScan = 16;  // pages that a thread looks at in a round
constexpr int kCopyThreads = 256;
constexpr int kGroup = 4;    // pools that a CTA copies side by side
constexpr int kPools = 64;  // per launch: their addresses are kernel parameters

struct Pages {
  int* table;
  long long stride, max_pages;
  int* lengths;
  int* refs;
  int pages, page, S;
};

// What the first kernel tells the second (and itself) of a sequence.
struct __align__(16) Seq {
  int start;   // length before
  int count;   // tokens to append; 0: nothing to do (or refused)
  int from;    // page to copy from, -1: none
  int need;    // new pages
  int offset;  // of its pages in the list of free ones
  int last;    // partly filled last page that others hold too, -1: none
  int first;   // table entry of its first new page
  int row;     // first of its rows
};

struct Plan {
  Pages c;
  const int* counts;
  const int* path;
  const int* cu;
  int n, total, cap;
  unsigned* status;
  Seq* seq;
  int* list;
};

// Sum over the CTA's threads of what precedes this one's `v`; the whole sum in
// `all`.
__device__ __forceinline__ int block_scan(int v, int& all, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the last round's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int w = warp_sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, w, d);
    if (lane >= d) w += y;
  }
  all = __shfl_sync(0xFFFFFFFFu, w, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, w, warp > 0 ? warp - 1 : 0);
  return x - v + (warp > 0 ? before : 0);
}

__device__ __forceinline__ int pages_of(long long tokens, int page) { return static_cast<int>((tokens + page - 1) / page); }

// Sequence b's request: status bits, and what it would take if no page were shared.
__device__ __forceinline__ unsigned request(const Plan& P, int b, Seq& q) {
  const Pages& c = P.c;
  q = Seq{0, 0, -1, 0, 0, -1, 0, 0};
  int lo = b * P.n, rows = P.n;
  if (P.cu) {
    lo = P.cu[b];
    const int hi = P.cu[b + 1];
    if (lo < 0 || hi < lo || hi > P.total || hi - lo > P.n) return SV_SEQ_BAD_LAYOUT;
    rows = hi - lo;
  }
  const int len = c.lengths[b], count = P.counts ? P.counts[b] : rows;
  if (count < 0 || count > rows || len < 0 || len > c.max_pages * c.page) return SV_SEQ_BAD_LAYOUT;
  if (P.path) {
    bool ok = true;
    for (int j = 0; j < count; ++j) {
      const int node = P.path[static_cast<long long>(b) * P.n + j];
      ok = ok && node >= 0 && node < rows;
    }
    if (!ok) return SV_SEQ_BAD_LAYOUT;
  }
  if (count == 0) return 0;
  if (static_cast<long long>(len) + count > c.max_pages * c.page || static_cast<long long>(len) + count > 0x7FFFFFFFLL)
    return SV_SEQ_NO_PAGES;
  if (len % c.page) {
    const int last = c.table[b * c.stride + len / c.page];
    if (last < 0 || last >= c.pages) return SV_SEQ_BAD_LAYOUT;
    if (c.refs[last] > 1) q.last = last;
  }
  q.start = len;
  q.count = count;
  q.row = lo;
  q.first = pages_of(len, c.page);
  q.need = pages_of(static_cast<long long>(len) + count, c.page) - q.first;
  return 0;
}

__device__ __forceinline__ void take_copy(Seq& q) {
  q.from = q.last;
  q.first -= 1;
  q.need += 1;
}

__device__ __forceinline__ void assign(const Plan& P, int b, const Seq& q) {
  const Pages& c = P.c;
  for (int j = 0; j < q.need; ++j) {
    const int p = P.list[q.offset + j];
    c.table[b * c.stride + q.first + j] = p;
    c.refs[p] = 1;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ Plan P) {
  __shared__ int warp_sums[32];
  __shared__ __align__(16) int s_last[kPlanThreads];
  __shared__ int s_start[kPlanThreads];
  const Pages& c = P.c;
  const int t = static_cast<int>(threadIdx.x);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // requests
  int any = 0;
  for (int b = t; b < c.S; b += kPlanThreads) {
    Seq q;
    P.status[b] = request(P, b, q);
    P.seq[b] = q;
    any |= q.last >= 0;
  }
  // of the sequences that share a last page the first refs - 1 copy it, and the
  // last too where its tokens would go among those that another still reads
  if (__syncthreads_or(any)) {
    for (int b0 = 0; b0 < c.S; b0 += kPlanThreads) {
      const int b = b0 + t;
      const int mine = b < c.S ? P.seq[b].last : -1, start = b < c.S ? P.seq[b].start : 0;
      int before = 0;
      bool further = false;
      for (int a0 = 0; a0 <= b0; a0 += kPlanThreads) {
        s_last[t] = a0 + t < c.S ? P.seq[a0 + t].last : -1;
        s_start[t] = a0 + t < c.S ? P.seq[a0 + t].start % c.page : 0;
        __syncthreads();
        const int end = a0 == b0 ? t : kPlanThreads;
        if (mine >= 0)
          for (int a = 0; a < end; a += 4) {
            const int4 four = *reinterpret_cast<const int4*>(s_last + a);
            const bool same[4] = {four.x == mine, four.y == mine, four.z == mine, four.w == mine};
            if (same[0] | same[1] | same[2] | same[3])
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (same[j] && a + j < end) {
                  ++before;
                  further = further || s_start[a + j] > start % c.page;
                }
          }
        __syncthreads();
      }
      if (mine >= 0 && (c.refs[mine] - before > 1 || further)) take_copy(P.seq[b]);  // (counts change further down)
    }
    __syncthreads();
  }
  // whose pages are where in the list
  int want = 0;
  for (int b0 = 0; b0 < c.S; b0 += kPlanThreads) {
    const int b = b0 + t;
    int all;
    const int at = block_scan(b < c.S ? P.seq[b].need : 0, all, warp_sums);
    if (b < c.S) P.seq[b].offset = want + at;
    want += all;
  }
  // the lowest free pages, 16 per thread and round
  int found = 0;
  const bool vec = (reinterpret_cast<uintptr_t>(c.refs) & 15) == 0;
  for (long long p0 = 0; p0 < c.pages && found < want; p0 += kScan * kPlanThreads) {
    const long long p = p0 + kScan * t;
    unsigned free = 0;
    if (vec && p + kScan <= c.pages) {
      int4 r[kScan / 4];
#pragma unroll
      for (int j = 0; j < kScan / 4; ++j) r[j] = *reinterpret_cast<const int4*>(c.refs + p + 4 * j);
#pragma unroll
      for (int j = 0; j < kScan / 4; ++j)
        free |= ((r[j].x == 0) | (r[j].y == 0) << 1 | (r[j].z == 0) << 2 | (r[j].w == 0) << 3) << (4 * j);
    } else {
      for (int j = 0; j < kScan; ++j) free |= p + j < c.pages && c.refs[p + j] == 0 ? 1u << j : 0u;
    }
    int all;
    int at = found + block_scan(__popc(free), all, warp_sums);
    for (; free && at < P.cap; free &= free - 1) P.list[at++] = static_cast<int>(p) + __ffs(free) - 1;
    found += all;
  }
  __syncthreads();
  if (found >= want) {
    for (int b = t; b < c.S; b += kPlanThreads) {
      const Seq q = P.seq[b];
      if (q.count == 0) continue;
      assign(P, b, q);
      if (q.from >= 0) atomicSub(c.refs + q.from, 1);
      c.lengths[b] = q.start + q.count;
    }
  } else {  // too few: one sequence after another, on what those before have left
    const int have = found < P.cap ? found : P.cap;
    int used = 0;
    for (int b = 0; b < c.S; ++b) {
      Seq q = P.seq[b];
      if (q.count == 0) continue;
      if (q.from >= 0) {  // (decided as if every one got its pages)
        q.from = -1;
        q.first += 1;
        q.need -= 1;
      }
      if (q.last >= 0) {
        bool copy = c.refs[q.last] > 1;
        if (!copy) {
          for (int a = t; a < b; a += kPlanThreads)
            copy = copy || (P.seq[a].from == q.last && P.seq[a].start % c.page > q.start % c.page);
          copy = __syncthreads_or(copy);
        }
        if (copy) take_copy(q);
      }
      __syncthreads();  // refs[last] and seq[b] have been read
      const bool served = q.need <= have - used;
      if (t == 0) {
        if (served) {
          q.offset = used;
          assign(P, b, q);
          if (q.from >= 0) c.refs[q.from] -= 1;
          c.lengths[b] = q.start + q.count;
        } else {
          P.status[b] = SV_SEQ_NO_PAGES;
          q.count = 0;
          q.from = -1;
        }
        P.seq[b] = q;
      }
      if (served) used += q.need;
      __syncthreads();
    }
  }
}

struct Copy {
  char* pool[kPools];
  const char* rows[kPools];
  const Seq* seq;
  const int* path;
  const int* table;
  long long table_stride;
  long long page_stride, token_stride, head_stride, row_stride, row_head_stride;
  int heads, units, page, n, pools;
  unsigned groups, splits;
};

// A CTA takes a share of a sequence's rows in up to kGroup pools: units of U,
// consecutive threads on consecutive units of a row, the group's loads in flight
// together.
template <typename U>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ Copy P) {
  unsigned cta = blockIdx.x;
  const int g = static_cast<int>(cta % P.groups) * kGroup;
  cta /= P.groups;
  const int split = static_cast<int>(cta % P.splits), b = static_cast<int>(cta / P.splits);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Seq q = P.seq[b];
  if (q.count == 0) return;
  const int part = q.from >= 0 ? q.start % P.page : 0;
  const int* table = P.table + b * P.table_stride;
  const int n = P.pools - g < kGroup ? P.pools - g : kGroup;
  // (fewer than 2^31 units in a token, and the tokens' product in 64 bits)
  const int per_token = P.heads * P.units;
  const long long items = static_cast<long long>(q.count + part) * per_token;
  for (long long i = static_cast<long long>(split) * kCopyThreads + threadIdx.x; i < items;
       i += static_cast<long long>(P.splits) * kCopyThreads) {
    const int t = items < 0x7FFFFFFF ? static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(per_token))
                                     : static_cast<int>(i / per_token);
    const int r = static_cast<int>(i - static_cast<long long>(t) * per_token);
    const int h = r / P.units, x = r - h * P.units;
    long long src, dst;
    const bool fresh = t < q.count;
    if (fresh) {
      const int node = P.path ? P.path[static_cast<long long>(b) * P.n + t] : t;
      const int pos = q.start + t;
      src = (static_cast<long long>(q.row) + node) * P.row_stride + h * P.row_head_stride;
      dst = table[pos / P.page] * P.page_stride + (pos % P.page) * P.token_stride + h * P.head_stride;
    } else {
      const long long in = (t - q.count) * P.token_stride + h * P.head_stride;
      src = q.from * P.page_stride + in;
      dst = table[q.start / P.page] * P.page_stride + in;
    }
    src += x * static_cast<long long>(sizeof(U));
    dst += x * static_cast<long long>(sizeof(U));
    U v[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k)
      if (k < n) v[k] = *reinterpret_cast<const U*>((fresh ? P.rows[g + k] : P.pool[g + k]) + src);
#pragma unroll
    for (int k = 0; k < kGroup; ++k)
      if (k < n) *reinterpret_cast<U*>(P.pool[g + k] + dst) = v[k];
  }
}

__global__ void __launch_bounds__(128) truncate_kernel(const __grid_constant__ Pages c, const int* to_, unsigned* status) {
  const int b = static_cast<int>(blockIdx.x);
  const int len = c.lengths[b], to = to_[b];
  bool ok = to >= 0 && to <= len && len <= c.max_pages * c.page;
  const int lo = ok ? pages_of(to, c.page) : 0, hi = ok ? pages_of(len, c.page) : 0;
  const int* row = c.table + b * c.stride;
  for (int j = lo + static_cast<int>(threadIdx.x); j < hi; j += 128) ok = ok && row[j] >= 0 && row[j] < c.pages;
  ok = __syncthreads_and(ok);
  if (ok)
    for (int j = lo + static_cast<int>(threadIdx.x); j < hi; j += 128) atomicSub(c.refs + row[j], 1);
  if (threadIdx.x == 0) {
    status[b] = ok ? 0u : SV_SEQ_BAD_LAYOUT;
    if (ok) c.lengths[b] = to;
  }
}

constexpr int kForkThreads = 512;
constexpr int kStaged = 8192;  // table entries that a CTA holds at a time

// A cluster per group; its CTAs share the columns of the table.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const __grid_constant__ Pages c, const int* parents, int W,
                                                             unsigned* status) {
  __shared__ int s_len[SV_CACHE_MAX_WIDTH], s_parent[SV_CACHE_MAX_WIDTH];
  __shared__ int s_held[kStaged];
  __shared__ unsigned char s_used[SV_CACHE_MAX_WIDTH];  // the slot moves, or another takes what it has
  __shared__ int s_bad[8], s_most;
  const int rank = static_cast<int>(svk::cluster_rank()), size = static_cast<int>(svk::cluster_size());
  const int group = static_cast<int>(blockIdx.x) / size;
  const long long slot0 = static_cast<long long>(group) * W;
  int* const table = c.table + slot0 * c.stride;
  const int t = static_cast<int>(threadIdx.x);
  if (t == 0) s_most = 0;
  svk::cluster_sync_all();  // every CTA runs before another writes to it
  bool ok = true;
  for (int w = t; w < W; w += kForkThreads) {
    int p = parents[slot0 + w];
    ok = ok && p < W;
    if (p < 0 || p >= W) p = w;
    s_parent[w] = p;
    s_len[w] = c.lengths[slot0 + w];
    s_used[w] = 0;
  }
  __syncthreads();
  // slots that take part: those that move and their parents
  for (int w = t; w < W; w += kForkThreads) {
    const int p = s_parent[w];
    if (p == w) continue;
    s_used[w] = s_used[p] = 1;
    const int a = s_len[w], d = s_len[p];
    const bool good = a >= 0 && d >= 0 && a <= c.max_pages * c.page && d <= c.max_pages * c.page;
    ok = ok && good;
    if (good) atomicMax(&s_most, pages_of(a > d ? a : d, c.page));
  }
  ok = __syncthreads_and(ok);
  const int most = s_most;
  const int cols = kStaged / W;
  // columns j0 .. j0 + k - 1 of every slot to shared memory, -1 past its length;
  // false: a page that would be counted does not exist
  auto stage = [&](int j0, int k) {
    bool good = true;
    for (int i = t; i < W * k; i += kForkThreads) {
      const int w = i / k, j = j0 + i % k;
      int e = -1;
      if (j < pages_of(s_len[w], c.page)) {
        e = table[w * c.stride + j];
        if (s_used[w]) good = good && e >= 0 && e < c.pages;
      }
      s_held[i] = e;
    }
    return good;
  };
  auto width_of = [&](int j0) { return most - j0 < cols ? most - j0 : cols; };
  const bool once = most <= size * cols;  // every CTA holds all its columns at a time
  const int j_own = rank * cols;
  if (ok) {  // every page that would be counted exists
    if (once) {
      if (j_own < most) ok = stage(j_own, width_of(j_own));
    } else {
      for (int j0 = j_own; j0 < most; j0 += size * cols) {
        const int k = width_of(j0);
        for (int i = t; i < W * k; i += kForkThreads) {
          const int w = i / k, j = j0 + i % k;
          if (s_used[w] && j < pages_of(s_len[w], c.page)) {
            const int e = table[w * c.stride + j];
            ok = ok && e >= 0 && e < c.pages;
          }
        }
      }
    }
  }
  ok = __syncthreads_and(ok);
  if (t < size) svk::dsmem_st_u32(svk::dsmem_addr(&s_bad[rank], t), ok ? 0u : 1u);
  svk::cluster_sync_all();  // and every CTA has read the lengths
  for (int r = 0; r < size; ++r) ok = ok && s_bad[r] == 0;
  if (rank == 0 && t == 0) status[group] = ok ? 0u : SV_SEQ_BAD_LAYOUT;
  if (!ok) return;
  for (int j0 = j_own; j0 < most; j0 += size * cols) {
    const int k = width_of(j0);
    if (!once) {
      stage(j0, k);
      __syncthreads();
    }
    for (int i = t; i < W * k; i += kForkThreads) {
      const int w = i / k, j = i % k, p = s_parent[w];
      if (p == w) continue;
      const int was = s_held[i], is = s_held[p * k + j];
      if (was == is) continue;
      if (was >= 0) atomicSub(c.refs + was, 1);
      if (is >= 0) {
        atomicAdd(c.refs + is, 1);
        table[w * c.stride + j0 + j] = is;
      }
    }
    __syncthreads();
  }
  if (rank == 0)
    for (int w = t; w < W; w += kForkThreads)
      if (s_parent[w] != w) c.lengths[slot0 + w] = s_len[s_parent[w]];
}

sv_status check(const sv_cache_pages* c, Pages& p) {
  if (!c) return svh::fail(SV_ERR_ARG, "cache is NULL");
  if (c->sequences < 0 || c->sequences > 0x7FFFFFFFLL) return svh::fail(SV_ERR_ARG, "sequences (%lld) out of range", (long long)c->sequences);
  if (c->pages < 1 || c->pages > 0x7FFFFFFFLL) return svh::fail(SV_ERR_ARG, "pages (%lld) out of range", (long long)c->pages);
  if (c->page_size < 1 || c->page_size > 0x7FFFFFFFLL) return svh::fail(SV_ERR_ARG, "page_size (%lld) out of range", (long long)c->page_size);
  if (c->max_pages < 0 || c->max_pages > 0x7FFFFFFFLL) return svh::fail(SV_ERR_ARG, "max_pages (%lld) out of range", (long long)c->max_pages);
  if (c->table_stride < c->max_pages && c->sequences > 1)
    return svh::fail(SV_ERR_ARG, "table_stride (%lld) is less than max_pages", (long long)c->table_stride);
  if (c->sequences > 0 && (!c->lengths || !c->refs || (!c->table && c->max_pages > 0)))
    return svh::fail(SV_ERR_ARG, "table, lengths or refs is NULL");
  p.table = c->table;
  p.stride = c->table_stride;
  p.max_pages = c->max_pages;
  p.lengths = c->lengths;
  p.refs = c->refs;
  p.pages = static_cast<int>(c->pages);
  p.page = static_cast<int>(c->page_size);
  p.S = static_cast<int>(c->sequences);
  return SV_OK;
}

sv_status launched() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SV_OK : svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
}

// Most pages that one call can take.
long long list_cap(long long sequences, long long n, long long pages, long long page) {
  const long long most = sequences * ((n + page - 1) / page + 1);
  return most < pages ? most : pages;
}

}  // namespace svc

extern "C" {

size_t sv_cache_append_workspace_size(int32_t sequences, int32_t n, int32_t pages, int32_t page_size) {
  if (sequences < 0 || n < 0 || pages < 1 || page_size < 1) return 0;
  return sizeof(svc::Seq) * static_cast<size_t>(sequences) + (4 * static_cast<size_t>(svc::list_cap(sequences, n, pages, page_size)) + 15) / 16 * 16;
}

sv_status sv_cache_append(const sv_cache_pages* cache, const sv_cache_rows* layout, void* const* pools,
                          const void* const* rows, int32_t n_pools, const int32_t* counts, const int32_t* path,
                          const int32_t* cu_nodes, int32_t n, int32_t total, uint32_t* status, void* workspace,
                          size_t workspace_bytes, void* stream) {
  svh::clear_error();
  svc::Plan P;
  sv_status s = svc::check(cache, P.c);
  if (s != SV_OK) return s;
  const int S = P.c.S;
  if (n < 0 || total < 0) return svh::fail(SV_ERR_ARG, "n (%d) and total (%d) must be >= 0", n, total);
  if (!cu_nodes && static_cast<long long>(S) * n != total)
    return svh::fail(SV_ERR_ARG, "without cu_nodes, total must equal sequences * n");
  if (n_pools < 1 || !pools || !rows || !layout) return svh::fail(SV_ERR_ARG, "at least one pool is needed");
  if (layout->heads < 0 || layout->row_bytes < 0 || layout->heads > 0x7FFFFFFFLL || layout->row_bytes > 0x7FFFFFFFLL ||
      layout->heads * layout->row_bytes > 0x7FFFFFFFLL)
    return svh::fail(SV_ERR_ARG, "heads or row_bytes out of range");
  if (layout->page_stride < 0 || layout->token_stride < 0 || layout->head_stride < 0 || layout->row_stride < 0 ||
      layout->row_head_stride < 0)
    return svh::fail(SV_ERR_ARG, "a stride is negative");
  if (S == 0) return SV_OK;
  if (!status) return svh::fail(SV_ERR_ARG, "status is NULL");
  const bool some = layout->heads > 0 && layout->row_bytes > 0 && n > 0;
  unsigned long long any = static_cast<unsigned long long>(layout->page_stride | layout->token_stride | layout->row_stride |
                                                           layout->row_bytes | 16);
  if (layout->heads > 1) any |= static_cast<unsigned long long>(layout->head_stride | layout->row_head_stride);
  for (int i = 0; i < n_pools && some; ++i) {
    if (!pools[i] || (!rows[i] && total > 0)) return svh::fail(SV_ERR_ARG, "pool %d or its rows: NULL", i);
    any |= reinterpret_cast<uintptr_t>(pools[i]) | reinterpret_cast<uintptr_t>(rows[i]);
  }
  const size_t need = sv_cache_append_workspace_size(S, n, P.c.pages, P.c.page);
  if (!workspace || workspace_bytes < need)
    return svh::fail(SV_ERR_ARG, "workspace_bytes (%zu) < the %zu bytes sv_cache_append_workspace_size() asks for",
                     workspace_bytes, need);
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return svh::fail(SV_ERR_ARG, "workspace must be 16-byte aligned");
  const long long splits = static_cast<long long>(n > P.c.page ? n : P.c.page) / 64 + 1;
  if (splits * S > 0x7FFFFFFFLL / svc::kPools || (static_cast<long long>(n) / P.c.page + 2) * S > 1LL << 30)
    return svh::fail(SV_ERR_UNSUPPORTED, "too many sequences and rows for one call");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  P.counts = counts;
  P.path = path;
  P.cu = cu_nodes;
  P.n = n;
  P.total = total;
  P.cap = static_cast<int>(svc::list_cap(S, n, P.c.pages, P.c.page));
  P.status = status;
  P.seq = static_cast<svc::Seq*>(workspace);
  P.list = reinterpret_cast<int*>(P.seq + S);
  svc::plan_kernel<<<1, svc::kPlanThreads, 0, st>>>(P);
  s = svc::launched();
  if (s != SV_OK || !some) return s;
  const int unit = static_cast<int>(any & (~any + 1));
  svc::Copy C;
  C.seq = P.seq;
  C.path = path;
  C.table = P.c.table;
  C.table_stride = P.c.stride;
  C.page_stride = layout->page_stride;
  C.token_stride = layout->token_stride;
  C.head_stride = layout->head_stride;
  C.row_stride = layout->row_stride;
  C.row_head_stride = layout->row_head_stride;
  C.heads = static_cast<int>(layout->heads);
  C.units = static_cast<int>(layout->row_bytes / unit);
  C.page = P.c.page;
  C.n = n;
  C.splits = static_cast<unsigned>(splits);
  for (int i = 0; i < n_pools; i += svc::kPools) {
    C.pools = n_pools - i < svc::kPools ? n_pools - i : svc::kPools;
    for (int k = 0; k < C.pools; ++k) {
      C.pool[k] = static_cast<char*>(pools[i + k]);
      C.rows[k] = static_cast<const char*>(rows[i + k]);
    }
    C.groups = static_cast<unsigned>((C.pools + svc::kGroup - 1) / svc::kGroup);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(C.groups * static_cast<unsigned>(splits * S));
    cfg.blockDim = dim3(svc::kCopyThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = i == 0 ? 1 : 0;  // (behind the first kernel; a later launch waits for all before it)
    cudaError_t e;
    if (unit == 16)
      e = cudaLaunchKernelEx(&cfg, svc::copy_kernel<uint4>, C);
    else if (unit == 8)
      e = cudaLaunchKernelEx(&cfg, svc::copy_kernel<uint2>, C);
    else if (unit == 4)
      e = cudaLaunchKernelEx(&cfg, svc::copy_kernel<unsigned>, C);
    else if (unit == 2)
      e = cudaLaunchKernelEx(&cfg, svc::copy_kernel<unsigned short>, C);
    else
      e = cudaLaunchKernelEx(&cfg, svc::copy_kernel<unsigned char>, C);
    if (e != cudaSuccess) return svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  }
  return SV_OK;
}

sv_status sv_cache_truncate(const sv_cache_pages* cache, const int32_t* to, uint32_t* status, void* stream) {
  svh::clear_error();
  svc::Pages c;
  const sv_status s = svc::check(cache, c);
  if (s != SV_OK || c.S == 0) return s;
  if (!to || !status) return svh::fail(SV_ERR_ARG, "to or status is NULL");
  svc::truncate_kernel<<<static_cast<unsigned>(c.S), 128, 0, static_cast<cudaStream_t>(stream)>>>(c, to, status);
  return svc::launched();
}

sv_status sv_cache_fork(const sv_cache_pages* cache, const int32_t* parents, int32_t width, uint32_t* status,
                        void* stream) {
  svh::clear_error();
  svc::Pages c;
  const sv_status s = svc::check(cache, c);
  if (s != SV_OK) return s;
  if (width < 1 || width > SV_CACHE_MAX_WIDTH)
    return svh::fail(SV_ERR_ARG, "width (%d) must be in [1, %d]", width, SV_CACHE_MAX_WIDTH);
  if (c.S % width) return svh::fail(SV_ERR_ARG, "sequences (%d) must be a multiple of width (%d)", c.S, width);
  if (c.S == 0) return SV_OK;
  if (!parents || !status) return svh::fail(SV_ERR_ARG, "parents or status is NULL");
  const unsigned groups = static_cast<unsigned>(c.S / width);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  // (a group of few slots and pages is one CTA's work: 64 groups of 8 x 512 entries
  // 12 us, with eight CTAs each 20; one group of 64 x 2048 entries 274 us, with eight 41)
  const long long entries = c.max_pages * width;
  const unsigned size = entries > 4 * svc::kStaged ? 8 : entries > svc::kStaged ? 4 : 1;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  if (groups > 0x7FFFFFFFu / 8) return svh::fail(SV_ERR_UNSUPPORTED, "too many groups for one call");
  cfg.gridDim = dim3(groups * size);
  cfg.blockDim = dim3(svc::kForkThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, svc::fork_kernel, c, parents, static_cast<int>(width), status);
  return e == cudaSuccess ? SV_OK : svh::fail(SV_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
