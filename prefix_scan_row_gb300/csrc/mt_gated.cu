// mt_gated.cu -- launches of the gated scan.
#include "mt_gated.cuh"

namespace mt {

int64_t gated_scratch_slots(int64_t batch, int64_t, int64_t dim) { return (batch * dim + 1) / 2; }

template <class S> static cudaError_t forward(const mt_gated_args &p, int64_t tokens, const Launch &L) {
    const unsigned grid = (unsigned)((p.dim + 127) / 128 * p.batch);
    note_launch();
    return p.rate ? launch_pdl(k_gated_plain<S, true>, grid, 128, 0, L.stream, p, tokens)
                  : launch_pdl(k_gated_plain<S, false>, grid, 128, 0, L.stream, p, tokens);
}
template <class S> static cudaError_t gradient(const mt_gated_args &p, const Launch &L) {
    const unsigned cols = (unsigned)((p.dim + 127) / 128);
    if (p.batch > 0) {
        note_launch();
        const cudaError_t e = p.rate ? launch_pdl(k_gated_grad_plain<S, true>, (unsigned)(cols * p.batch), 128, 0, L.stream, p)
                                     : launch_pdl(k_gated_grad_plain<S, false>, (unsigned)(cols * p.batch), 128, 0, L.stream, p);
        if (e != cudaSuccess || p.drate == nullptr)
            return e;
    }
    if (p.drate == nullptr)
        return cudaSuccess;
    note_launch();
    return launch_pdl(k_gated_rate_join, cols, 128, 0, L.stream, (const float *)p.scratch, p.drate, p.batch, p.dim);
}
#define MT_BY_TYPE(f, ...)                                   \
    switch (p.dtype) {                                       \
    case MT_F32: return f<float>(__VA_ARGS__);               \
    case MT_BF16: return f<__nv_bfloat16>(__VA_ARGS__);      \
    case MT_F16: return f<__half>(__VA_ARGS__);              \
    default: return cudaErrorInvalidValue;                   \
    }
cudaError_t gated_launch(const mt_gated_args &p, const Launch &L) { MT_BY_TYPE(forward, p, 0, L) }
cudaError_t gated_step_launch(const mt_gated_args &p, const Launch &L) { MT_BY_TYPE(forward, p, -1, L) }
cudaError_t gated_grad_launch(const mt_gated_args &p, const Launch &L) { MT_BY_TYPE(gradient, p, L) }
#undef MT_BY_TYPE

}  // namespace mt
