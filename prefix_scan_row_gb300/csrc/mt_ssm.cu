// mt_ssm.cu -- plans of the selective state space scan: how many lanes share a
// channel, into how many segments the tokens are cut, and the scratch's parts.
#include "mt_ssm.cuh"

namespace mt {

// The tokens are cut where the uncut work would leave SMs with less than it takes to keep
// their arithmetic busy: a lane has 32 independent recurrences, so that is little. Three
// CTAs of an SM run at once. The plan must not ask the device (scratch is sized on the host), so it
// counts GB300's 152 SMs.
// Both sides of the two lines, us, bf16, 4096 channels x 16 states, every plan forced uncut / left to ssm_segment:
//   sequences (warps of a prompt, CTAs of a gradient)   8 (512, 256)   12 (768, 384)   16 (1024, 512)   24 (1536, 768)   32 (2048, 1024)
//   prompt, 512 tokens                                   108 / 126       161 / 178       221 / 229        228 / 327        309 / 388
//   prompt, 2048 tokens                                  411 / 449       621 / 631       859 / 835        886 / 1201      1206 / 1455
//   the same with checkpoints                            524 / 503       751 / 710      1022 / 945       1053 / 1356      1463 / 1667
//   gradient, 512 tokens                                 511 / 381       524 / 546       779 / 733       1024 / 1042      1253 / 1253
//   gradient, 2048 tokens                               2001 / 1434     2061 / 2071     3055 / 2820      4044 / 4045      4934 / 4934
// A single line is right at both ends and not between: it costs prompts up to 18 % at 8 sequences (cut) and, where the
// last wave is half empty, up to 8 % at 16 (uncut).
constexpr int64_t kSsmSms = 152;
constexpr int64_t kEnoughWarps = kSsmSms * 5;  // from here on the tokens are not cut
constexpr int64_t kEnoughCtas = kSsmSms * 3;   // the same for the gradient's CTAs
constexpr int64_t kResident = 3, kMostCtas = 12;  // CTAs of an SM: at once, and all that a cut aims at
constexpr int64_t kLeastSegment = 16;  // tokens: at least 64 measured 100 us where 16 take 30 (2 x 700 tokens, 301 channels)
constexpr int64_t kSegmentStart = 8;   // tokens' time that a segment's first loads and its carry take

// Tokens of a segment, `units` / per_cta CTAs working on one. The time is that of the SM with the
// most CTAs, so of the cuts into 3 to 12 CTAs an SM the one is taken that makes it the least. Where
// lengths differ, CTAs end at any time and half a segment is left at the end, which favours short ones.
// 8 x 1027 tokens x 4096 channels: ragged, 80 tokens 189 us and 152 195; full, 241 and 240. A gradient over
// 4 x 2048 tokens x 4096 channels: 80 tokens in its forward pass 1000 us, 296 981; 16384 tokens x 2048: 288 229, 144 234.
static int64_t ssm_segment(int64_t len, int64_t units, int64_t per_cta, bool lens) {
    const int64_t wave = kSsmSms * per_cta;
    int64_t best = len, least = INT64_MAX;
    for (int64_t r = kResident; r <= kMostCtas; ++r) {
        const int64_t s = r * wave / units;
        int64_t seg = s > 0 ? ((len + s - 1) / s + kSsmTile - 1) / kSsmTile * kSsmTile : len;
        seg = seg < kLeastSegment ? kLeastSegment : seg;
        const int64_t busy = (units * ((len + seg - 1) / seg) + wave - 1) / wave;
        const int64_t cost = (busy < kResident ? kResident : busy) * (seg + kSegmentStart) + (lens ? seg / 2 : 0);
        if (cost < least) {
            least = cost;
            best = seg;
        }
    }
    return best;
}

SsmPlan ssm_plan(int64_t batch, int64_t len, int64_t dim, int64_t nstate, int64_t groups, bool grad, bool lens) {
    SsmPlan p;
    p.lanes = 2;
    while (p.lanes < 32 && 4 * p.lanes < nstate)
        p.lanes *= 2;
    const int64_t gdim = dim / groups;
    // gradient: a CTA's channels; forward: a warp's, 64 until more than 16 states share them out
    const int64_t channels = grad ? 128 / p.lanes * kSsmWarps : nstate <= 16 ? 64 : nstate <= 32 ? 32 : nstate <= 64 ? 16 : 8;
    p.ctiles = (gdim + channels - 1) / channels;
    const int64_t units = batch * groups * p.ctiles;  // warps or CTAs of one segment
    p.segments = 1;
    p.seg_len = len > 0 ? (len + kSsmTile - 1) / kSsmTile * kSsmTile : kSsmTile;
    if (units > 0 && units < (grad ? kEnoughCtas : kEnoughWarps) && len > kLeastSegment) {
        const int64_t seg = ssm_segment(len, units, grad ? 1 : kSsmWarps, lens);
        if (seg < len) {
            p.seg_len = seg;
            p.segments = (len + seg - 1) / seg;
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
    a.plan = ssm_plan(p.batch, p.len, p.dim, p.nstate, p.groups, grad, p.lens != nullptr);
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
