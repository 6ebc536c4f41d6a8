// The 4-bit LM head's kernels for few rows of bf16 states (a translation unit of
// its own: they compile in parallel).
#include "sv_lm_head_q4_few.cuh"

namespace svq {

sv_status start_few_bf16(const Args& g, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  return start_few_any<true>(g, proj, s0, s1, st);
}

}  // namespace svq
