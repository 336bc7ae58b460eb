// mt_ssm.cu -- plans of the selective state space scan: how many lanes share a
// channel, into how many segments the tokens are cut, and the scratch's parts.
#include "mt_ssm.cuh"

namespace mt {

// Warps that keep an SM's arithmetic busy: a lane has 16 independent
// recurrences, so a few warps a scheduler suffice. The plan must not ask the
// device (scratch is sized on the host), so it counts GB300's 152 SMs.
constexpr int64_t kSsmSms = 152;
constexpr int64_t kEnoughWarps = kSsmSms * 5;   // from here on the tokens are not cut
constexpr int64_t kTargetWarps = kSsmSms * 24;  // what a cut aims at
constexpr int64_t kTargetCtas = kSsmSms * 9;    // the same for the gradient's CTAs
constexpr int64_t kLeastSegment = 16;           // tokens: a warp alone takes as long for a token as the chain of carries does

SsmPlan ssm_plan(int64_t batch, int64_t len, int64_t dim, int64_t nstate, int64_t groups, bool grad) {
    SsmPlan p;
    p.lanes = 2;
    while (p.lanes < 32 && 4 * p.lanes < nstate)
        p.lanes *= 2;
    const int64_t gdim = dim / groups;
    // gradient: a CTA's channels; forward: a warp's, 64 until more than 16 states share them out
    const int64_t channels = grad ? 128 / p.lanes * kSsmWarps : nstate <= 16 ? 64 : nstate <= 32 ? 32 : nstate <= 64 ? 16 : 8;
    p.ctiles = (gdim + channels - 1) / channels;
    const int64_t units = batch * groups * p.ctiles;  // warps or CTAs of one segment
    const int64_t enough = grad ? kSsmSms * 3 : kEnoughWarps, target = grad ? kTargetCtas : kTargetWarps;
    p.segments = 1;
    p.seg_len = len > 0 ? (len + 15) / 16 * 16 : 16;
    if (units > 0 && units < enough && len > kLeastSegment) {
        int64_t s = target / units;
        const int64_t most = len / kLeastSegment;
        if (s > most)
            s = most;
        if (s > 1) {
            p.seg_len = ((len + s - 1) / s + 15) / 16 * 16;
            p.segments = (len + p.seg_len - 1) / p.seg_len;
        }
    }
    const int64_t cut = p.segments > 1 ? batch * p.segments * dim : 0;
    p.carry_slots = (cut * nstate + 3) / 4 * 2;
    p.decay_slots = (cut + 3) / 4 * 2;
    p.shared_slots = p.param_slots = 0;
    if (grad) {
        p.shared_slots = groups * p.ctiles * batch * len * (4 * p.lanes);  // 2 x 4 lanes values of f32
        p.param_slots = (batch * p.segments * dim * (nstate + 2) + 3) / 4 * 2;
    }
    return p;
}

static bool fits(const void *p, int64_t a, int64_t b, int64_t bytes, int64_t values = 4) {
    return (uintptr_t)p % bytes == 0 && a % values == 0 && b % values == 0;
}
// whether `values` neighbouring channels of every tensor of the call can be moved as one
static bool channels_fit(const mt_ssm_args &p, bool grad, int64_t gdim, int64_t values) {
    const int64_t v = values * (p.dtype == MT_F32 ? 4 : 2);
    const bool in = gdim % values == 0 && fits(p.u, p.u_batch, p.u_token, v, values) &&
                    fits(p.delta, p.delta_batch, p.delta_token, v, values) && fits(p.z, p.z_batch, p.z_token, v, values);
    if (!grad)
        return in && fits(p.out, p.out_batch, p.out_token, v, values);
    return in && fits(p.dout, p.dout_batch, p.dout_token, v, values) && fits(p.du, p.du_batch, p.du_token, v, values) &&
           fits(p.ddelta, p.ddelta_batch, p.ddelta_token, v, values) && fits(p.dz, p.dz_batch, p.dz_token, v, values);
}

// The kernels' arguments of a call: what its plan and its addresses allow.
static SsmArgs ssm_args(const mt_ssm_args &p, bool grad) {
    SsmArgs a;
    a.p = p;
    a.plan = ssm_plan(p.batch, p.len, p.dim, p.nstate, p.groups, grad);
    a.ntiles = (p.len + kSsmTile - 1) / kSsmTile;
    a.gdim = p.dim / p.groups;
    const int64_t v = p.dtype == MT_F32 ? 16 : 8;  // bytes of four values
    a.nvec = p.nstate % 4 == 0 && fits(p.A, 0, 0, 16) && fits(p.state, 0, 0, 16) && fits(p.checkpoints, 0, 0, 16) &&
             fits(p.dfinal, 0, 0, 16) && fits(p.dinit, 0, 0, 16);
    a.bvec = p.nstate % 4 == 0 && fits(p.B, p.B_batch, p.B_token, v) && fits(p.C, p.C_batch, p.C_token, v);
    a.aligned = a.nvec && a.bvec && channels_fit(p, grad, a.gdim, p.dtype == MT_F32 ? 4 : 8);
    uint64_t *s = static_cast<uint64_t *>(p.scratch);
    a.carry = a.decay = a.shared = a.dA_part = a.dD_part = a.dbias_part = nullptr;
    if (s != nullptr) {
        a.carry = reinterpret_cast<float *>(s);
        s += a.plan.carry_slots;
        a.decay = reinterpret_cast<float *>(s);
        s += a.plan.decay_slots;
        a.shared = reinterpret_cast<float *>(s);
        s += a.plan.shared_slots;
        a.dA_part = reinterpret_cast<float *>(s);
        a.dD_part = a.dA_part + p.batch * a.plan.segments * p.dim * p.nstate;
        a.dbias_part = a.dD_part + p.batch * a.plan.segments * p.dim;
    }
    return a;
}

#define MT_BY_TYPE(f)                          \
    switch (p.dtype) {                         \
    case MT_F32: return f##_f32(a, L);         \
    case MT_BF16: return f##_bf16(a, L);       \
    case MT_F16: return f##_f16(a, L);         \
    default: return cudaErrorInvalidValue;     \
    }
cudaError_t ssm_launch(const mt_ssm_args &p, const Launch &L) {
    const SsmArgs a = ssm_args(p, false);
    MT_BY_TYPE(ssm_prompt)
}
cudaError_t ssm_step_launch(const mt_ssm_args &p, const Launch &L) {
    const SsmArgs a = ssm_args(p, false);
    MT_BY_TYPE(ssm_step)
}
static cudaError_t carries(const mt_ssm_args &p, const SsmArgs &a, const Launch &L) { MT_BY_TYPE(ssm_adjoint_carries) }
cudaError_t ssm_grad_launch(const mt_ssm_args &p, const Launch &L) {
    const SsmArgs a = ssm_args(p, true);
    if (a.plan.segments > 1) {
        const cudaError_t e = carries(p, a, L);
        if (e != cudaSuccess)
            return e;
    }
    MT_BY_TYPE(ssm_grad)
}
#undef MT_BY_TYPE

}  // namespace mt
