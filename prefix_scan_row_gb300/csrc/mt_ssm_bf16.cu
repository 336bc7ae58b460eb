// mt_ssm_bf16.cu -- the selective state space scan's kernels for bf16 activations.
#include "mt_ssm_launch.cuh"

namespace mt {

cudaError_t ssm_bf16(const SsmArgs &a, SsmWhat what, const Launch &L) { return ssm_type<__nv_bfloat16>(a, what, L); }

}  // namespace mt
