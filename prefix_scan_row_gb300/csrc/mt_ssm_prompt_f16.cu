// mt_ssm_prompt_f16.cu -- the selective scan of prompts, its segments' carries in
// both directions, and the single-token form, for f16 activations.
#include "mt_ssm_prompt.cuh"

namespace mt {

cudaError_t ssm_prompt_f16(const SsmArgs &a, const Launch &L) { return prompt_states<__half>(a, L); }
cudaError_t ssm_adjoint_carries_f16(const SsmArgs &a, const Launch &L) { return adjoint_carries<__half>(a, L); }
cudaError_t ssm_step_f16(const SsmArgs &a, const Launch &L) { return step_states<__half>(a, L); }

}  // namespace mt
