// The 4-bit LM head's kernels for few rows (a translation unit of its own:
// they compile in parallel).
#include "sv_lm_head_q4_few.cuh"

namespace svq {

sv_status start_few_any(const Args& g, bool bf16, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  if (proj->group == 32) return start_few_group<32>(g, bf16, proj, s0, s1, st);
  if (proj->group == 64) return start_few_group<64>(g, bf16, proj, s0, s1, st);
  return start_few_group<128>(g, bf16, proj, s0, s1, st);
}

}  // namespace svq
