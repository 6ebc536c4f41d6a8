/*
 * sv_lm_head_q4.h - the LM head with a projection held in 4 bits (part of
 * libsv.so).
 *
 * For a few rows of hidden states (one token of one request, the K + 1
 * positions of a verification, the beams of a search) the LM head is bound by
 * the bytes of its projection; in 4 bits with a scale per group of weights it
 * has a quarter of them.  The calls stand beside those of sv_lm_head.h (same
 * layouts of states and logits, same conventions).
 *
 * The projection W [vocab, dim]:
 *   W[v][k] = scale[v][k / group] * (q[v][k] - zero[v][k / group])
 *   packed  [vocab, dim / 2] bytes: byte j of a row holds q[2j] in its low
 *           four bits and q[2j + 1] in its high four;
 *   scales  [vocab, ceil(dim / group)] of scale_dtype;
 *   zeros   [vocab, ceil(dim / group)] bytes in 0..15, or NULL for 8
 *           everywhere.
 * The logits are those of these weights: products of the states with the
 * integers q - zero, summed in f32 within a group, then scaled and summed over
 * the groups in f32 (no weight is rounded to 16 bits on the way, no state to
 * fewer bits than it has; a state that meets a code equal to its zero adds
 * nothing).  A group's sum is taken before its scale, so it stays in f32's range
 * for states below 2^116.
 * Every 64 rows are a pass over the projection: past 64 rows the bf16 projection
 * of sv_lm_head.h is the faster one (128256 x 4096, groups of 128: 64 rows 148
 * against 193 us, 96 rows 266 against 205).
 * Requirements: dim a multiple of 32 (16-byte rows), group 32, 64 or 128 (the
 * last group may be cut by dim), states and packed 16-byte aligned.
 */
#ifndef SV_LM_HEAD_Q4_H
#define SV_LM_HEAD_Q4_H

#include <stddef.h>
#include <stdint.h>

#include "sv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A projection in 4 bits: device pointers, owned by the caller. */
typedef struct {
  const void* packed;
  const void* scales;
  const uint8_t* zeros;
  sv_dtype scale_dtype; /* SV_F32, SV_BF16 or SV_F16 */
  int32_t group;        /* weights per scale: 32, 64 or 128 */
} sv_q4_proj;

/*
 * logits[r][v] = sum_k states[r][k] W[v][k] in f32.
 * states [rows, dim] SV_BF16 or SV_F16, rows `dim` elements apart; logits
 * [rows, ld] f32, ld >= vocab; `err`, optional device word: bit 0 is OR-ed in
 * if a bounded device wait of the kernel gave up (the logits are then
 * invalid); the caller zeroes it.  One launch.
 * A row of states with an infinity or a NaN in it has logits that are not
 * finite (infinite or NaN); the other rows' are as they would be without it.
 */
sv_status sv_lm_head_q4_logits(const void* states, sv_dtype dtype, const sv_q4_proj* proj, int32_t rows,
                               int32_t vocab, int32_t dim, float* logits, int64_t ld, uint32_t* err,
                               void* stream);

/*
 * sv_lm_head_verify (sv_lm_head.h) on a 4-bit projection: the target and
 * draft rows' logits, then the mixed greedy / sampled verification of them.
 * Arguments, results and the workspace (sv_lm_head_workspace_size() bytes) as
 * there; `dtype` is the states'.
 */
sv_status sv_lm_head_q4_verify(const void* target_states, const void* draft_states, sv_dtype dtype,
                               const sv_q4_proj* proj, int32_t dim, const float* temperature,
                               const int32_t* draft_tokens, const float* uniforms, const int32_t* cu_k,
                               int32_t batch, int32_t k, int32_t sum_k, int32_t vocab,
                               int32_t* n_accepted, int32_t* next_token, uint32_t* status,
                               void* workspace, size_t workspace_bytes, uint32_t flags, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SV_LM_HEAD_Q4_H */
