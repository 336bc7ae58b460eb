// mt_ssm_f32.cu -- the selective state space scan's kernels for f32 activations.
#include "mt_ssm_launch.cuh"

namespace mt {

cudaError_t ssm_f32(const SsmArgs &a, SsmWhat what, const Launch &L) { return ssm_type<float>(a, what, L); }

}  // namespace mt
