// The 4-bit LM head's kernels for few rows (a translation unit of its own:
// they compile in parallel).
#include "sv_lm_head_q4_few.cuh"

namespace svq {

sv_status start_few_any(const Args& g, bool bf16, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  if (proj->scale_dtype == SV_F32) return start_few_scale<SV_F32>(g, bf16, proj, s0, s1, st);
  if (proj->scale_dtype == SV_BF16) return start_few_scale<SV_BF16>(g, bf16, proj, s0, s1, st);
  return start_few_scale<SV_F16>(g, bf16, proj, s0, s1, st);
}

}  // namespace svq
