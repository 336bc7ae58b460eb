// mt_ssm_f16.cu -- the selective state space scan's kernels for f16 activations.
#include "mt_ssm_launch.cuh"

namespace mt {

cudaError_t ssm_f16(const SsmArgs &a, SsmWhat what, const Launch &L) { return ssm_type<__half>(a, what, L); }

}  // namespace mt
