// mt_ssm_launch.cuh -- launches of the selective scan's kernels for one activation type.
#pragma once

#include "mt_ssm_grad.cuh"

namespace mt {

template <class K> static cudaError_t ssm_smem(K kernel, size_t bytes) {
    return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) : cudaSuccess;
}

// The prompt kernels: K states a lane, P lanes a channel pair.
template <class S, int K, int P, bool REV> static cudaError_t carry_go(const SsmArgs &a, const Launch &L) {
    SsmArgs c = a;
    c.plan.ctiles = (a.gdim + 64 / P - 1) / (64 / P);
    const int64_t warps = a.p.batch * a.p.groups * c.plan.ctiles * (a.plan.segments - 1);
    const int64_t grid = (warps + kSsmWarps - 1) / kSsmWarps;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    const size_t smem = kSsmWarps * PromptSmem<S, K, P, 1>::kBytes;
    const cudaError_t e = ssm_smem(k_ssm_carry<S, K, P, REV>, smem);
    if (e != cudaSuccess)
        return e;
    note_launch();
    const cudaError_t r = launch_pdl(k_ssm_carry<S, K, P, REV>, (unsigned)grid, kSsmThreads, smem, L.stream, c, warps);
    if (r != cudaSuccess)
        return r;
    const int64_t chain = (a.p.batch * a.p.dim * a.p.nstate + 255) / 256;
    if (chain > INT32_MAX)
        return cudaErrorInvalidValue;
    note_launch();
    return launch_pdl(k_ssm_chain<REV>, (unsigned)chain, 256, 0, L.stream, a);
}
template <class S, int K, int P> static cudaError_t prompt_go(const SsmArgs &a, const Launch &L) {
    cudaError_t e;
    if (a.plan.segments > 1 && (e = carry_go<S, K, P, false>(a, L)) != cudaSuccess)
        return e;
    const int64_t warps = a.p.batch * a.p.groups * a.plan.ctiles * a.plan.segments;
    const int64_t grid = (warps + kSsmWarps - 1) / kSsmWarps;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    const size_t smem = kSsmWarps * PromptSmem<S, K, P, 2>::kBytes;
    if ((e = ssm_smem(k_ssm<S, K, P>, smem)) != cudaSuccess)
        return e;
    note_launch();
    return launch_pdl(k_ssm<S, K, P>, (unsigned)grid, kSsmThreads, smem, L.stream, a, warps);
}

template <class S, int P> static cudaError_t step_go(const SsmArgs &a, const Launch &L) {
    const int64_t grid = (a.p.batch * a.p.dim * P + 255) / 256;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    note_launch();
    return launch_pdl(k_ssm_step<S, P>, (unsigned)grid, 256, 0, L.stream, a);
}

template <class S, int P> static cudaError_t grad_go(const SsmArgs &a, const Launch &L) {
    cudaError_t e;
    const int64_t grid = a.p.batch * a.p.groups * a.plan.ctiles * a.plan.segments;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    if (grid > 0) {
        const size_t smem = GradSmem<S, P>::kBytes;
        if ((e = ssm_smem(k_ssm_grad<S, P>, smem)) != cudaSuccess)
            return e;
        note_launch();
        if ((e = launch_pdl(k_ssm_grad<S, P>, (unsigned)grid, kSsmThreads, smem, L.stream, a)) != cudaSuccess)
            return e;
    }
    const int64_t items = a.p.batch * a.p.len * a.p.groups * 2 * a.p.nstate + a.p.dim * a.p.nstate + a.p.dim;
    int64_t jgrid = (items + 255) / 256;
    if (jgrid > 16 * (int64_t)L.sm_count)
        jgrid = 16 * (int64_t)L.sm_count;
    note_launch();
    return launch_pdl(k_ssm_grad_join<S>, (unsigned)jgrid, 256, 0, L.stream, a, 4 * P);
}

// by the number of states, rounded up to what a lane holds
#define MT_BY_STATES(n, f)              \
    if ((n) <= 4) return f(4, 1);       \
    if ((n) <= 8) return f(8, 1);       \
    if ((n) <= 16) return f(16, 1);     \
    if ((n) <= 32) return f(16, 2);     \
    if ((n) <= 64) return f(16, 4);     \
    return f(16, 8)
template <class S> static cudaError_t prompt_states(const SsmArgs &a, const Launch &L) {
#define MT_GO(K, P) prompt_go<S, K, P>(a, L)
    MT_BY_STATES(a.p.nstate, MT_GO);
#undef MT_GO
}
template <class S> static cudaError_t carry_states(const SsmArgs &a, const Launch &L) {
#define MT_GO(K, P) carry_go<S, K, P, true>(a, L)
    MT_BY_STATES(a.p.nstate, MT_GO);
#undef MT_GO
}
#undef MT_BY_STATES

template <class S> static cudaError_t ssm_type(const SsmArgs &a, SsmWhat what, const Launch &L) {
    if (what == kSsmForward)
        return prompt_states<S>(a, L);
    if (what == kSsmGrad && a.plan.segments > 1) {
        const cudaError_t e = carry_states<S>(a, L);
        if (e != cudaSuccess)
            return e;
    }
#define MT_LANES(P) \
    case P: return what == kSsmStep ? step_go<S, P>(a, L) : grad_go<S, P>(a, L)
    switch (a.plan.lanes) {
        MT_LANES(2);
        MT_LANES(4);
        MT_LANES(8);
        MT_LANES(16);
        MT_LANES(32);
    default: return cudaErrorInvalidValue;
    }
#undef MT_LANES
}

}  // namespace mt
