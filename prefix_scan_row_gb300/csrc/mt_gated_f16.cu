// mt_gated_f16.cu -- the gated scan's kernels for f16 activations: prompts and single tokens.
#include "mt_gated.cuh"

namespace mt {
MT_GATED_TYPE(f16, __half)
}  // namespace mt
