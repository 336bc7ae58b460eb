// mt_gated_f32.cu -- the gated scan's kernels for f32 activations: prompts and single tokens.
#include "mt_gated.cuh"

namespace mt {
MT_GATED_TYPE(f32, float)
}  // namespace mt
