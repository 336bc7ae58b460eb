// mt_ssm_prompt_f32.cu -- the selective scan of prompts, its segments' carries in
// both directions, and the single-token form, for f32 activations.
#include "mt_ssm_prompt.cuh"

namespace mt {

cudaError_t ssm_prompt_f32(const SsmArgs &a, const Launch &L) { return prompt_states<float>(a, L); }
cudaError_t ssm_adjoint_carries_f32(const SsmArgs &a, const Launch &L) { return adjoint_carries<float>(a, L); }
cudaError_t ssm_step_f32(const SsmArgs &a, const Launch &L) { return step_states<float>(a, L); }

}  // namespace mt
