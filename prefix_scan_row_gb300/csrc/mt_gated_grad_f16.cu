// mt_gated_grad_f16.cu -- the gated scan's gradient for f16 activations.
#include "mt_gated.cuh"

namespace mt {
MT_GATED_GRAD_TYPE(f16, __half)
}  // namespace mt
