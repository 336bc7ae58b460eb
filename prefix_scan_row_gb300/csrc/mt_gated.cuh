// mt_gated.cuh -- the gated scan's mathematics, and its kernels per activation type (mt_gated_*.cu).
//
//   s = sigma(r);  a = exp(-rate s), w = sqrt(1 - a^2)  or, without rate,  a = 1 - s, w = s
//   h_t = a_t h_{t-1} + w_t v_t,  v = sigma(i) x or x,  out = h or h z sigma(z)
//
// Gradient, with g_t the gradient by h_t (from out_t, and from h_{t+1} through a_{t+1}):
//   dh = dout z sigma(z),  g_t = dh_t + a_{t+1} g_{t+1},  dz = dout h sigma(z) (1 + z (1 - sigma(z)))
//   dx = g w sigma(i),  di = g w v (1 - sigma(i))
//   rate: with u = rate s, da/du = -a and dw/du = a^2 / w, so e = g (v a^2 / w - h_{t-1} a) s,
//         dr = e rate (1 - s), drate = sum of e;  no rate: dr = g (v - h_{t-1}) s (1 - s)
#pragma once

#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

__device__ __forceinline__ int64_t gated_len(const mt_gated_args &p, int64_t b) {
    const int64_t n = p.lens != nullptr ? (int64_t)p.lens[b] : p.len;
    return n < 0 ? 0 : n > p.len ? p.len : n;
}
__device__ __forceinline__ int64_t gated_slot(const mt_gated_args &p, int64_t b) {
    const int64_t s = p.slots != nullptr ? (int64_t)p.slots[b] : b;
    return s >= 0 && s < p.nslots ? s : -1;
}

// sigma(x) and 1 - sigma(x), each to f32's relative precision: e = exp(-|x|) is at most 1, so nothing overflows.
__device__ __forceinline__ void sigmoid_both(float x, float &s, float &c) {
    const float e = ex2f(-kLog2e * fabsf(x));
    const float q = rcpf(1.0f + e);
    const float eq = e * q;
    s = x >= 0.0f ? q : eq;
    c = x >= 0.0f ? eq : q;
}

// 1 - exp(-u) = u (1 - u/2 (1 - u/3 (...))), Taylor's series of the exponential, for u below 1/2: the first
// term left out is below 2e-9 of the sum. The decay next to 1 is 1 minus this, so that a long memory's
// decays keep f32's precision and w = sqrt(1 - a^2) its relative one, which 1 - a * a does not.
__device__ __forceinline__ float one_minus_exp_small(float u) {
    float p = fmaf(u, -1.0f / 9.0f, 1.0f);
    p = fmaf(u * p, -1.0f / 8.0f, 1.0f);
    p = fmaf(u * p, -1.0f / 7.0f, 1.0f);
    p = fmaf(u * p, -1.0f / 6.0f, 1.0f);
    p = fmaf(u * p, -1.0f / 5.0f, 1.0f);
    p = fmaf(u * p, -1.0f / 4.0f, 1.0f);
    p = fmaf(u * p, -1.0f / 3.0f, 1.0f);
    p = fmaf(u * p, -1.0f / 2.0f, 1.0f);
    return u * p;
}

// One token's gate: decay a, weight w, and (rate) 1 / w, 0 where w is.
template <bool RATE> struct Gate {
    float s, c, a, w, rw;
    __device__ __forceinline__ void open(float r, float rate) {
        sigmoid_both(r, s, c);
        if constexpr (RATE) {
            const float u = rate * s;
            const float small = one_minus_exp_small(u), big = ex2f(-kLog2e * u);
            const bool near = u < 0.5f;
            a = near ? 1.0f - small : big;
            const float d = near ? small : 1.0f - big;
            const float q = d * (2.0f - d);  // 1 - a^2 = (1 - a) (1 + a)
            float y;
            asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(q));
            rw = q < 1.2e-38f ? 0.0f : y;
            w = q * rw;
        } else {
            a = c;
            w = s;
            rw = 0.0f;
        }
    }
};

// --- the plain kernels: a thread a channel, token after token ---------------------------------
template <class S, bool RATE> __global__ void k_gated_plain(mt_gated_args p, int64_t tokens) {
    pdl_prologue();
    const int64_t cols = (p.dim + blockDim.x - 1) / blockDim.x, b = blockIdx.x / cols;
    const int64_t d = (blockIdx.x - b * cols) * blockDim.x + threadIdx.x;
    if (d >= p.dim)
        return;
    const bool step = tokens < 0;
    const int64_t slot = gated_slot(p, b);
    const bool active = slot >= 0 || p.state == nullptr;
    const int64_t len = !active ? 0 : step ? 1 : gated_len(p, b), total = step ? 1 : p.len;
    float h = 0.0f;
    if (active && p.state != nullptr && (step || p.carry_in))
        h = p.state[slot * p.dim + d];
    const float rate = RATE ? p.rate[d] : 0.0f;
    const S *x = (const S *)p.x + b * p.x_batch + d, *r = (const S *)p.r + b * p.r_batch + d;
    const S *i = p.i ? (const S *)p.i + b * p.i_batch + d : nullptr, *z = p.z ? (const S *)p.z + b * p.z_batch + d : nullptr;
    S *out = (S *)p.out + b * p.out_batch + d;
    const int64_t ntiles = (p.len + kGatedTile - 1) / kGatedTile;
    for (int64_t t = 0; t < total; ++t) {
        if (!step && p.checkpoints != nullptr && t % kGatedTile == 0)
            p.checkpoints[(b * ntiles + t / kGatedTile) * p.dim + d] = h;
        float y = 0.0f;
        if (t < len) {
            Gate<RATE> g;
            g.open(Codec<S>::load1(r + t * p.r_token), rate);
            float v = Codec<S>::load1(x + t * p.x_token);
            if (i) {
                float s, c;
                sigmoid_both(Codec<S>::load1(i + t * p.i_token), s, c);
                v *= s;
            }
            h = fmaf(g.a, h, g.w * v);
            y = h;
            if (z) {
                float s, c;
                const float zz = Codec<S>::load1(z + t * p.z_token);
                sigmoid_both(zz, s, c);
                y = h * (zz * s);
            }
        }
        Codec<S>::store1(out + t * p.out_token, y);
    }
    if (active && p.state != nullptr)
        p.state[slot * p.dim + d] = h;
}

template <class S, bool RATE> __global__ void k_gated_grad_plain(mt_gated_args p) {
    pdl_prologue();
    const int64_t cols = (p.dim + blockDim.x - 1) / blockDim.x, b = blockIdx.x / cols;
    const int64_t d = (blockIdx.x - b * cols) * blockDim.x + threadIdx.x;
    if (d >= p.dim)
        return;
    const int64_t len = gated_len(p, b);
    const int64_t ntiles = (p.len + kGatedTile - 1) / kGatedTile;
    const float rate = RATE ? p.rate[d] : 0.0f;
    const S *x = (const S *)p.x + b * p.x_batch + d, *r = (const S *)p.r + b * p.r_batch + d;
    const S *i = p.i ? (const S *)p.i + b * p.i_batch + d : nullptr, *z = p.z ? (const S *)p.z + b * p.z_batch + d : nullptr;
    const S *dout = (const S *)p.dout + b * p.dout_batch + d;
    S *dx = (S *)p.dx + b * p.dx_batch + d, *dr = (S *)p.dr + b * p.dr_batch + d;
    S *di = (S *)p.di + b * p.di_batch + d, *dz = (S *)p.dz + b * p.dz_batch + d;
    for (int64_t t = len; t < p.len; ++t) {
        Codec<S>::store1(dx + t * p.dx_token, 0.0f);
        Codec<S>::store1(dr + t * p.dr_token, 0.0f);
        if (i)
            Codec<S>::store1(di + t * p.di_token, 0.0f);
        if (z)
            Codec<S>::store1(dz + t * p.dz_token, 0.0f);
    }
    float carry = p.dfinal ? p.dfinal[b * p.dim + d] : 0.0f, drate = 0.0f;
    for (int64_t tile = (len + kGatedTile - 1) / kGatedTile - 1; tile >= 0; --tile) {
        float before[kGatedTile];
        float h = p.checkpoints[(b * ntiles + tile) * p.dim + d];
        const int64_t t0 = tile * kGatedTile;
        const int n = (int)(len - t0 < kGatedTile ? len - t0 : kGatedTile);
        for (int k = 0; k < n; ++k) {
            Gate<RATE> g;
            g.open(Codec<S>::load1(r + (t0 + k) * p.r_token), rate);
            float v = Codec<S>::load1(x + (t0 + k) * p.x_token), s = 1.0f, c;
            if (i)
                sigmoid_both(Codec<S>::load1(i + (t0 + k) * p.i_token), s, c);
            before[k] = h;
            h = fmaf(g.a, h, g.w * (v * s));
        }
        for (int k = n - 1; k >= 0; --k) {
            const int64_t t = t0 + k;
            Gate<RATE> g;
            g.open(Codec<S>::load1(r + t * p.r_token), rate);
            const float xx = Codec<S>::load1(x + t * p.x_token), hp = before[k];
            float si = 1.0f, ci = 0.0f;
            if (i)
                sigmoid_both(Codec<S>::load1(i + t * p.i_token), si, ci);
            const float v = xx * si, dy = Codec<S>::load1(dout + t * p.dout_token);
            float gh = dy;
            if (z) {
                float s, c;
                const float zz = Codec<S>::load1(z + t * p.z_token);
                sigmoid_both(zz, s, c);
                gh = dy * (zz * s);
                Codec<S>::store1(dz + t * p.dz_token, dy * fmaf(g.a, hp, g.w * v) * (s * fmaf(zz, c, 1.0f)));
            }
            gh += carry;
            carry = gh * g.a;
            const float dv = gh * g.w;
            Codec<S>::store1(dx + t * p.dx_token, dv * si);
            if (i)
                Codec<S>::store1(di + t * p.di_token, dv * v * ci);
            if constexpr (RATE) {
                const float e = gh * (v * (g.a * g.a) * (g.s * g.rw) - hp * g.a * g.s);
                drate += e;
                Codec<S>::store1(dr + t * p.dr_token, e * rate * g.c);
            } else {
                Codec<S>::store1(dr + t * p.dr_token, gh * (v - hp) * (g.s * g.c));
            }
        }
    }
    if (p.dinit != nullptr)
        p.dinit[b * p.dim + d] = carry;
    if (RATE && p.drate != nullptr)
        reinterpret_cast<float *>(p.scratch)[b * p.dim + d] = drate;
}

static __global__ void k_gated_rate_join(const float *part, float *drate, int64_t rows, int64_t dim) {
    pdl_prologue();
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= dim)
        return;
    float s = 0.0f;
    for (int64_t k = 0; k < rows; ++k)
        s += part[k * dim + d];
    drate[d] = s;
}

}  // namespace mt
