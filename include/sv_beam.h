/*
 * sv_beam.h - beam search: selection over beams and vocabulary, and the
 * reordering of the beams' states that follows it (part of libsv.so).
 *
 * A beam-search step extends W partial sequences of each of B requests by one
 * token: the n best pairs (beam, token) by accumulated log-probability become
 * the next candidates (sv_beam_select), and everything a model keeps per beam
 * (key / value caches, recurrent states, token histories) moves from the
 * chosen parents' slots to the new ones (sv_beam_reorder).  The conventions of
 * sv.h apply: device pointers owned by the caller, stream-ordered, no host
 * synchronisation, host-detectable errors as sv_status with sv_last_error(),
 * data-dependent ones as status bits per sequence, results a pure function of
 * the inputs.
 */
#ifndef SV_BEAM_H
#define SV_BEAM_H

#include <stddef.h>
#include <stdint.h>

#include "sv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_BEAM_MAX_BEAMS 64       /* beams per sequence */
#define SV_BEAM_MAX_CANDIDATES 128 /* candidates per sequence (twice the beams, so that
                                      every beam may end and W live ones remain) */

/*
 * Bytes of workspace sv_beam_select needs for these sizes (0 for sizes it
 * refuses).
 */
size_t sv_beam_select_workspace_size(int32_t batch, int32_t beams, int32_t vocab, int32_t n);

/*
 * The n best continuations of every sequence.
 *   score(w, v) = scores[w] + logits[w][v] - ln sum_u exp(logits[w][u])
 *   best first; equal scores by the lower beam, then the lower token.  The
 *   order is that of the scores in 64 bits, not of the rounded f32 outputs:
 *   scores[w] + ((logits[w][v] - the row's maximum) - the logarithm of the sum
 *   below that maximum), the logarithm to better than 2^-34 and the two sums
 *   rounded once each.  Candidates of two beams whose scores differ by less
 *   than 2^-34, or 2^-52 of the larger of |scores[w]| and |score|, may come out
 *   in either order.
 * logits   [batch * beams] rows of `dtype`, `row_stride` elements apart
 *          (any element alignment); beam w of sequence b is row b * beams + w.
 * scores   [batch, beams] f32: the beams' accumulated log-probabilities; a
 *          beam at -Inf is dead: no candidates, its row is not read.
 * finished [batch, beams] bytes, or NULL: a beam marked nonzero has ended; its
 *          one candidate is (eos, its score unchanged) and its row is not read.
 * A logit of -Inf (a masked token) is no candidate; a row of nothing else has
 * none; nor is a score below f32's range one (a beam and a token both at the
 * lowest finite value).  A sequence with fewer than n candidates gets score -Inf, parent -1,
 * token -1 in the places left over.
 * out_scores, out_parents, out_tokens [batch, n].
 * status   [batch]: 0, or SV_SEQ_BAD_VALUE (NaN or +Inf among the logits of a
 *          live beam, or a score that is NaN or +Inf): every candidate of the
 *          sequence is then -Inf, -1, -1.
 * workspace: sv_beam_select_workspace_size() bytes, 16-byte aligned, no
 *          initial contents needed.  Calls that share one must not overlap on
 *          the GPU.
 * One or two launches; nothing is enqueued when the call is refused.
 * 1 <= beams <= SV_BEAM_MAX_BEAMS, 1 <= n <= SV_BEAM_MAX_CANDIDATES,
 * beams * vocab < 2^31.
 */
sv_status sv_beam_select(const void* logits, sv_dtype dtype, int64_t row_stride, const float* scores,
                         const uint8_t* finished, int32_t eos, int32_t batch, int32_t beams,
                         int32_t vocab, int32_t n, float* out_scores, int32_t* out_parents,
                         int32_t* out_tokens, uint32_t* status, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * One state tensor [batch, beams, segs, tokens, token_bytes].  Strides are in
 * BYTES; the tokens of a segment are contiguous.  `timed` != 0: only the first
 * lengths[b] tokens of each segment are in use and move; 0: all of them.
 */
typedef struct {
  void* data;
  int64_t seq_stride;  /* between sequences */
  int64_t beam_stride; /* between the beams of a sequence */
  int64_t seg_stride;  /* between the segments of a beam (heads, layers) */
  int64_t token_bytes;
  int32_t segs;
  int32_t tokens;
  int32_t timed;
  int32_t reserved; /* 0 */
} sv_beam_state;

/*
 * In place, for every state, sequence b and slot w with p = parents[b][w]:
 *   state[b][w][.][:len] = (the state before the call)[b][p][.][:len]
 * with len = lengths[b] for a timed state.  A slot that is its own parent, or
 * whose parent is negative (no candidate), keeps its contents, and so does
 * everything past the length.
 * states   host array of n_states descriptions (copied by the call).  Two
 *          states must not share memory, nor two beams of one, nor a state
 *          with parents, lengths or status.
 * parents  [batch, beams] int32; lengths [batch] int32, or NULL when no state
 *          is timed.
 * status   [batch]: 0, or SV_SEQ_BAD_LAYOUT (a parent >= beams, or a length
 *          outside [0, tokens of the shortest timed state]): nothing of that
 *          sequence moves.
 * One launch per 48 states, those whose addresses, strides and extents are
 * multiples of 16 bytes apart from the others.  1 <= beams <= SV_BEAM_MAX_BEAMS.
 */
sv_status sv_beam_reorder(const sv_beam_state* states, int32_t n_states, const int32_t* parents,
                          const int32_t* lengths, int32_t batch, int32_t beams, uint32_t* status,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SV_BEAM_H */
