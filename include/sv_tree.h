/*
 * sv_tree.h - verification of a drafted tree, and the attention that scores
 * its tokens over a paged key/value cache (part of libsv.so).
 *
 * A round drafts a tree instead of a chain: node 0 of a sequence is its last
 * committed token, every other node continues an earlier one (its parent).
 * The target scores all nodes in one pass, each seeing the cached tokens and
 * its own ancestors (sv_tree_attention); the accepted tokens are those of the
 * path from node 0 that follows the target's choices as far as the tree goes,
 * to the lowest node where siblings carry the same token
 * (sv_verify_tree_greedy, sv_verify_tree).  The path's keys and values then go
 * into the cache (sv_cache.h); the others were never written there.
 * The conventions of sv.h apply: device pointers owned by the caller,
 * stream-ordered, no host synchronisation, host-detectable errors as sv_status
 * with sv_last_error(), data-dependent ones as status bits per sequence,
 * results a pure function of the inputs.
 *
 * Layout of the nodes: sequence b has N_b nodes, rows cu_nodes[b] ..
 * cu_nodes[b + 1] - 1 of every array of `total` rows; without cu_nodes
 * (NULL) each has n, and total = batch * n.  N_b <= n <= SV_TREE_MAX_NODES; 0
 * is a sequence that takes no part.  parents[row of node i] is in [-1, i): the
 * node i continues, within its sequence; -1: none.  parents NULL: a chain,
 * node i continues node i - 1.
 * Offsets that are negative, decrease, pass `total` or leave more than n
 * nodes, and parents out of range, are the sequence's SV_SEQ_BAD_LAYOUT.
 */
#ifndef SV_TREE_H
#define SV_TREE_H

#include <stddef.h>
#include <stdint.h>

#include "sv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_TREE_MAX_NODES 256         /* nodes per sequence */
#define SV_TREE_MAX_TOKENS 134217728  /* tokens that a row of a page table holds */

/*
 * Greedy verification of a tree.
 *   c(i) = argmax of target row i (ties to the lowest index; NaN never wins, it
 *   ranks below -Inf).  From node 0: while a child of the node has the token
 *   c(node), go to the lowest such child.  The nodes after node 0 are accepted,
 *   the next token is c(the last one).
 * target   [total] rows of `dtype`, `row_stride` elements apart (any element
 *          alignment): the distribution (probabilities or logits) after each
 *          node.  Only rows that the path may reach are needed.
 * tokens   [total]: the nodes' tokens (node 0's is not looked at).  An id
 *          outside [0, vocab) is never followed; a child of a node on the path
 *          with such an id sets SV_SEQ_BAD_TOKEN.
 * n_accepted, next_token, status [batch]; path [batch, n]: the nodes of the
 *          path, node 0 first, n_accepted + 1 of them, then -1.
 * A NaN in a row on the path sets SV_SEQ_BAD_VALUE (an all-NaN row's choice is
 * 0).  A sequence with no nodes, or with SV_SEQ_BAD_LAYOUT, has 0, -1 and an
 * empty path.  One launch.
 */
sv_status sv_verify_tree_greedy(const void* target, sv_dtype dtype, int64_t row_stride, const int32_t* tokens,
                                const int32_t* parents, const int32_t* cu_nodes, int32_t batch, int32_t n,
                                int32_t total, int32_t vocab, int32_t* n_accepted, int32_t* next_token,
                                int32_t* path, uint32_t* status, void* stream);

/*
 * The same for choices that the caller has drawn: choices[row] is the
 * target's token after that node (sampling: sv_accept_from_logits on the rows
 * with K_b = 0 draws them, and what is emitted follows the target's law). A
 * negative choice (a row that could not be drawn from) ends the path: the next
 * token is then -1.  One launch.
 */
sv_status sv_verify_tree(const int32_t* choices, const int32_t* tokens, const int32_t* parents,
                         const int32_t* cu_nodes, int32_t batch, int32_t n, int32_t total, int32_t* n_accepted,
                         int32_t* next_token, int32_t* path, uint32_t* status, void* stream);

/*
 * Attention of the nodes over their sequence's cached tokens and their own
 * ancestors.  For node i and query head h (key head h / (q_heads / kv_heads)):
 *   s_j = scale * q . k_j over the lengths[b] cached tokens j and over node i
 *   and its ancestors;  out = sum_j softmax(s)_j v_j;  lse = ln sum_j exp(s_j).
 * The cache of sequence b is in pages: token t at position t % page_size of
 * page table[b][t / page_size].  Cached tokens past the length and nodes that
 * are not ancestors take no part, whatever they hold.
 * Everything in `dtype` (SV_BF16 or SV_F16) except lse (f32).  Products and
 * sums in f32 (a row with a score past f32's range, or with values whose weighted
 * sum passes it before the division, weights being up to 2^8, has no defined
 * result); the weights are rounded to `dtype` before they multiply the values, each
 * off by at most half a step, 2^-8 (bf16) or 2^-11 (f16) of itself.
 * All strides in ELEMENTS; the head dimension has unit stride.  Addresses and
 * strides of q, k, v, out and the caches are multiples of 16 bytes, and no stride is
 * 0 along a dimension of more than one entry; out shares no memory with another
 * array.
 * status [batch]: 0, or SV_SEQ_BAD_LAYOUT (offsets or parents as above, a
 *   length outside [0, max_pages * page_size], a page outside [0, pages)): the
 *   rows of such a sequence (where its offsets are good) are 0, their lse -Inf.
 *   SV_SEQ_TIMEOUT: a bounded device wait gave up, the rows are invalid.
 * Rows of out and lse past the last sequence are left as they are.
 * workspace: sv_tree_attention_workspace_size() bytes, 16-byte aligned, no
 *   initial contents needed.  Calls that share one must not overlap on the GPU.
 * dim a multiple of 8 up to 128; page_size a multiple of 8; max_pages *
 * page_size at most SV_TREE_MAX_TOKENS; q_heads a multiple of kv_heads, at most
 * 128 times as many.
 */
typedef struct {
  int64_t dtype, q_heads, kv_heads, dim;
  const void *q, *k, *v; /* [total, q_heads, dim], [total, kv_heads, dim] */
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;
  const void *k_cache, *v_cache; /* [pages, page_size, kv_heads, dim] */
  int64_t kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  int64_t pages, page_size;
  const int32_t* table; /* [batch, max_pages], rows table_stride apart */
  int64_t table_stride, max_pages;
  const int32_t *lengths, *parents, *cu_nodes;
  int64_t batch, n, total;
  void* out; /* [total, q_heads, dim] */
  int64_t out_row, out_head;
  float* lse; /* [total, q_heads], or NULL */
  uint32_t* status;
} sv_tree_attn;

size_t sv_tree_attention_workspace_size(int32_t dim);
sv_status sv_tree_attention(const sv_tree_attn* args, float scale, void* workspace, size_t workspace_bytes,
                            void* stream);
/* The same with flags: 0, or SV_FLAG_EXPIRE_EXCHANGE (sv.h; a testing aid), with
 * which every wait for outputs of the tensor cores gives up at once: where there is a
 * row, all sequences end with SV_SEQ_TIMEOUT, their rows hold anything, and nothing
 * else is written. */
sv_status sv_tree_attention_flagged(const sv_tree_attn* args, float scale, uint32_t flags, void* workspace,
                                    size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SV_TREE_H */
