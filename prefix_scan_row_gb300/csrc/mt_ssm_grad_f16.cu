// mt_ssm_grad_f16.cu -- the selective scan's gradient for f16 activations.
#include "mt_ssm_grad.cuh"

namespace mt {

cudaError_t ssm_grad_f16(const SsmArgs &a, const Launch &L) { return grad_states<__half>(a, L); }

}  // namespace mt
