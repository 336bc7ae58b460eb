// mt_gated_bf16.cu -- the gated scan's kernels for bf16 activations: prompts and single tokens.
#include "mt_gated.cuh"

namespace mt {
MT_GATED_TYPE(bf16, __nv_bfloat16)
}  // namespace mt
