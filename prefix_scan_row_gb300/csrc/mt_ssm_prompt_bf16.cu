// mt_ssm_prompt_bf16.cu -- the selective scan of prompts, its segments' carries in
// both directions, and the single-token form, for bf16 activations.
#include "mt_ssm_prompt.cuh"

namespace mt {

cudaError_t ssm_prompt_bf16(const SsmArgs &a, const Launch &L) { return prompt_states<__nv_bfloat16>(a, L); }
cudaError_t ssm_adjoint_carries_bf16(const SsmArgs &a, const Launch &L) { return adjoint_carries<__nv_bfloat16>(a, L); }
cudaError_t ssm_step_bf16(const SsmArgs &a, const Launch &L) { return step_states<__nv_bfloat16>(a, L); }

}  // namespace mt
