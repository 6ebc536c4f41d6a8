// The 4-bit LM head's tensor-memory kernels for bf16 states (a translation unit
// of its own: they compile in parallel).
#include "sv_lm_head_q4.cuh"

namespace svq {

sv_status start_bf16(const Args& g, int n, const sv_q4_proj* proj, const void* s0, const void* s1, cudaStream_t st) {
  return start_group<__nv_bfloat16>(g, n, proj, s0, s1, st);
}

}  // namespace svq
