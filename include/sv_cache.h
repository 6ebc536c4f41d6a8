/*
 * sv_cache.h - the pages of paged key/value caches: appending, sharing and
 * giving up (part of libsv.so).
 *
 * A model's caches are `n_pools` pools (keys and values of every layer) of
 * `pages` pages of `page_size` tokens.  One page table serves all of them:
 * sequence b holds lengths[b] tokens, token t at position t % page_size of
 * page table[b][t / page_size]; entries past the length mean nothing and keep
 * what they hold.  refs[p] counts the table entries in use that name page p; a
 * page with 0 is free.  The calls below keep that so; a caller that starts
 * with lengths and refs all 0 needs nothing else.
 * The conventions of sv.h apply: device pointers owned by the caller,
 * stream-ordered, no host synchronisation, host-detectable errors as sv_status
 * with sv_last_error(), data-dependent ones as status bits per sequence,
 * results a pure function of the inputs.
 */
#ifndef SV_CACHE_H
#define SV_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "sv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_SEQ_NO_PAGES 128u /* not enough free pages, or no room in the table row */

/* The page table and what goes with it. */
typedef struct {
  int32_t* table; /* [sequences, max_pages], rows table_stride apart */
  int64_t table_stride, max_pages;
  int32_t* lengths; /* [sequences] */
  int32_t* refs;    /* [pages] */
  int64_t pages, page_size, sequences;
} sv_cache_pages;

/* Where the pools and the new rows lie: strides in BYTES, a row is one head's
 * vector of one token. */
typedef struct {
  int64_t page_stride, token_stride, head_stride; /* of every pool */
  int64_t row_stride, row_head_stride;            /* of every array of new rows */
  int64_t heads, row_bytes;
} sv_cache_rows;

/*
 * Appends counts[b] tokens to every sequence: token j of sequence b is row
 * cu_nodes[b] + path[b][j] of every array of new rows (without path: row
 * cu_nodes[b] + j), written at position lengths[b] + j of the pool of the same
 * index; then lengths[b] += counts[b].
 *   The sequences take pages one after another, b = 0 first: a sequence that
 *   needs k new pages gets the k lowest-numbered free ones (free before the
 *   call, and not given to an earlier sequence), for rising positions.  A
 *   last page that is partly filled is not written, its tokens go to a new page
 *   first, in every pool, and its refs drop by one, where its refs are above 1
 *   (earlier sequences of the call that copied it no longer count), or where an
 *   earlier sequence of the call copied it and holds more of it.
 * pools, rows  host arrays of n_pools device pointers (copied by the call): the
 *          pools, and the [total, heads] new rows for each.
 * counts   [sequences], or NULL: all of a sequence's rows.
 * path     [sequences, n] int32, or NULL (as sv_verify_tree_greedy writes it,
 *          with counts = n_accepted + 1).
 * cu_nodes [sequences + 1], or NULL: sequence b has rows b * n .. b * n + n - 1
 *          (total = sequences * n).  n: the most rows of a sequence, any number.
 * status   [sequences]: 0; SV_SEQ_BAD_LAYOUT (offsets, count, path, length or a
 *          last page out of range); SV_SEQ_NO_PAGES.  Such a sequence and its
 *          pages stay as they are.
 * No pool may share memory with another array of the call.
 * workspace: sv_cache_append_workspace_size() bytes, 16-byte aligned, no
 *          initial contents needed.  Calls that share one must not overlap on
 *          the GPU.
 * One launch for the pages and one per 64 pools.
 */
size_t sv_cache_append_workspace_size(int32_t sequences, int32_t n, int32_t pages, int32_t page_size);
sv_status sv_cache_append(const sv_cache_pages* cache, const sv_cache_rows* layout, void* const* pools,
                          const void* const* rows, int32_t n_pools, const int32_t* counts, const int32_t* path,
                          const int32_t* cu_nodes, int32_t n, int32_t total, uint32_t* status, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * Takes every sequence back to to[b] tokens: the pages past them are given up
 * (refs drop by one); 0 gives up the whole sequence.  to[b] outside
 * [0, lengths[b]], a length or a page to be given up out of range: status[b] is
 * SV_SEQ_BAD_LAYOUT, and the sequence stays as it is.  One launch.
 */
sv_status sv_cache_truncate(const sv_cache_pages* cache, const int32_t* to, uint32_t* status, void* stream);

/*
 * The sequences in groups of `width`: slot w of a group takes the pages and
 * the length that slot parents[w] of its group held before the call, sharing
 * them (refs count up), and gives up its own.  A negative parent, or its own,
 * leaves a slot as it is.
 * parents  [sequences].  status [sequences / width], one word per group: 0, or
 *          SV_SEQ_BAD_LAYOUT (a parent >= width, or a length or page of a slot
 *          that takes part out of range): nothing of that group changes.
 * One launch.  1 <= width <= SV_CACHE_MAX_WIDTH, a divisor of sequences.
 */
#define SV_CACHE_MAX_WIDTH 1024
sv_status sv_cache_fork(const sv_cache_pages* cache, const int32_t* parents, int32_t width, uint32_t* status,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SV_CACHE_H */
