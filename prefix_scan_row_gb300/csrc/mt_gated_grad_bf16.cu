// mt_gated_grad_bf16.cu -- the gated scan's gradient for bf16 activations.
#include "mt_gated.cuh"

namespace mt {
MT_GATED_GRAD_TYPE(bf16, __nv_bfloat16)
}  // namespace mt
