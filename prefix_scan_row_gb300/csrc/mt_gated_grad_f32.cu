// mt_gated_grad_f32.cu -- the gated scan's gradient for f32 activations.
#include "mt_gated.cuh"

namespace mt {
MT_GATED_GRAD_TYPE(f32, float)
}  // namespace mt
