// mt_ssm_grad_bf16.cu -- the selective scan's gradient for bf16 activations.
#include "mt_ssm_grad.cuh"

namespace mt {

cudaError_t ssm_grad_bf16(const SsmArgs &a, const Launch &L) { return grad_states<__nv_bfloat16>(a, L); }

}  // namespace mt
