// mt_ssm_grad_f32.cu -- the selective scan's gradient for f32 activations.
#include "mt_ssm_grad.cuh"

namespace mt {

cudaError_t ssm_grad_f32(const SsmArgs &a, const Launch &L) { return grad_states<float>(a, L); }

}  // namespace mt
