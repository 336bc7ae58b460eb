// mt_ssm.cuh -- the selective state space scan: what its kernels share, and the
// single-token kernel, instantiated per activation type (mt_ssm_*.cu).
//
//   Delta = softplus(delta + delta_bias),  a_t[d,n] = exp(Delta_t[d] A[d,n])
//   h_t[d,n] = a_t[d,n] h_{t-1}[d,n] + Delta_t[d] u_t[d] B_t[n]
//   y_t[d] = sum_n C_t[n] h_t[d,n] + D[d] u_t[d],  out = y * z * sigmoid(z)
//
// The recurrence is a scan with the operator (a, b) o (a', b') = (a a', a' b + b'),
// whose products of a are exp(A * sum of Delta): the carry of a span of tokens is
// one state and one sum of steps per channel.
//
// Bound: per (token, channel, state) one exponential and four multiply-adds
// (Delta*A, the input, the recurrence, the output). The exponentials run at 30.5 and
// packed multiply-adds at up to 128 a clock and SM, so a token of 64 channels x 16 states
// takes 34 clocks of an SM against 24 of HBM traffic at 16-bit storage (8 bytes a channel),
// and in the carry pass as many again against 12: arithmetic, not bandwidth. With one token a
// sequence the states themselves are read and written, and bytes count again.
//
// Few channels do not fill the GPU: the tokens are then cut into segments that
// run side by side, after a pass that computes each segment's carry (a state
// from zero, and the sum of steps); a segment's first state is the combination of
// the carries before it.
//
// Here are the parts that prompts and gradients share, and the single-token kernel; the
// other kernels say how they split their work.
#pragma once

#include <type_traits>

#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

constexpr int kSsmWarps = 4;
constexpr int kSsmThreads = 32 * kSsmWarps;

struct SsmArgs {
    mt_ssm_args p;
    SsmPlan plan;
    int64_t ntiles;  // of the whole token axis
    int64_t gdim;    // channels per group
    int aligned;     // 16 bytes of channels, 4 states, and 4 values of B and C, may be moved as one
    int nvec, bvec;  // 4 states, or 4 values of B and C, may be
    float *carry, *decay, *shared, *dA_part, *dD_part, *dbias_part;
};

__device__ __forceinline__ int64_t ssm_len(const SsmArgs &a, int64_t b) {
    const int64_t n = a.p.lens != nullptr ? (int64_t)a.p.lens[b] : a.p.len;
    return n < 0 ? 0 : n > a.p.len ? a.p.len : n;
}
__device__ __forceinline__ int64_t ssm_slot(const SsmArgs &a, int64_t b) {
    const int64_t s = a.p.slots != nullptr ? (int64_t)a.p.slots[b] : b;
    return s >= 0 && s < a.p.nslots ? s : -1;
}

// The (channel, state) pairs of one lane, two neighbouring states a register pair.
struct Pairs {
    f32x2 v[4][2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c][0] = v[c][1] = 0ull;
    }
    // rows of nstate f32, one per channel; states from n0 on, `cl` channels
    __device__ __forceinline__ void load(const float *rows, int64_t nstate, int n0, int cl, bool vec, float scale = 1.0f) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (c < cl) {
                const float *r = rows + c * nstate + n0;
                if (vec) {
                    if (n0 < nstate) {
                        const float4 w = *reinterpret_cast<const float4 *>(r);
                        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (n0 + k < nstate)
                            x[k] = r[k];
                }
            }
            v[c][0] = pack2f(x[0] * scale, x[1] * scale);
            v[c][1] = pack2f(x[2] * scale, x[3] * scale);
        }
    }
    __device__ __forceinline__ void store(float *rows, int64_t nstate, int n0, int cl, bool vec) const {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c < cl) {
                float x[4];
                unpack2f(v[c][0], x[0], x[1]);
                unpack2f(v[c][1], x[2], x[3]);
                float *r = rows + c * nstate + n0;
                if (vec) {
                    if (n0 < nstate)
                        *reinterpret_cast<float4 *>(r) = make_float4(x[0], x[1], x[2], x[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (n0 + k < nstate)
                            r[k] = x[k];
                }
            }
        }
    }
};

// Four values over the P lanes of a channel group, summed: lane p is left with
// the sums of channels first..first+count-1.
template <int P> struct SumOut {
    static constexpr int kCount = P >= 4 ? 1 : 4 / P;  // P is 2 or more
};
template <int P> __device__ __forceinline__ void sum_lanes(const float (&v)[4], int p, float (&o)[SumOut<P>::kCount]) {
    if constexpr (P == 2) {
        const bool up = p & 1;
        const float s0 = up ? v[0] : v[2], s1 = up ? v[1] : v[3];
        o[0] = (up ? v[2] : v[0]) + __shfl_xor_sync(kFull, s0, 1);
        o[1] = (up ? v[3] : v[1]) + __shfl_xor_sync(kFull, s1, 1);
    } else {
        const bool up2 = p & 2, up1 = p & 1;
        const float s0 = up2 ? v[0] : v[2], s1 = up2 ? v[1] : v[3];
        const float r0 = (up2 ? v[2] : v[0]) + __shfl_xor_sync(kFull, s0, 2);
        const float r1 = (up2 ? v[3] : v[1]) + __shfl_xor_sync(kFull, s1, 2);
        float r = (up1 ? r1 : r0) + __shfl_xor_sync(kFull, up1 ? r0 : r1, 1);
#pragma unroll
        for (int d = 4; d < P; d <<= 1)
            r += __shfl_xor_sync(kFull, r, d);
        o[0] = r;
    }
}
// Writes them beside each other: row[4 g + channel].
template <int P> __device__ __forceinline__ void put_sums(float *row, int g, int p, const float (&o)[SumOut<P>::kCount]) {
    if constexpr (P == 2)
        *reinterpret_cast<float2 *>(row + 4 * g + 2 * p) = make_float2(o[0], o[1]);
    else if (P == 4 || p < 4)
        row[4 * g + p] = o[0];
}

// Shape of a warp's tile.
template <int P> struct SsmShape {
    static constexpr int CW = 128 / P;                 // channels of a warp
    static constexpr int NP = 4 * P;                   // states, rounded up
};

// h = exp2(dt A) h + du B for one token; A holds A * log2(e).
__device__ __forceinline__ void advance(Pairs &h, const Pairs &A, const float (&dt)[4], const float (&du)[4], f32x2 b0, f32x2 b1) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const f32x2 d2 = pack2f(dt[c], dt[c]), x2 = pack2f(du[c], du[c]);
        h.v[c][0] = fma2f(ex2_2f(exponent2f(d2, A.v[c][0])), h.v[c][0], mul2f(x2, b0));
        h.v[c][1] = fma2f(ex2_2f(exponent2f(d2, A.v[c][1])), h.v[c][1], mul2f(x2, b1));
    }
}
__device__ __forceinline__ void lds4(const float *p, float (&x)[4]) {
    const float4 w = *reinterpret_cast<const float4 *>(p);
    x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
}
__device__ __forceinline__ void lds_pairs(const float *p, f32x2 &a, f32x2 &b) {
    const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(p);
    a = w.x;
    b = w.y;
}
// Where a warp's work lies.
template <int P> struct SsmPlace {
    int64_t b, s, g, c0, ch;  // sequence, segment, group; first channel of the warp in its group; of the lane, absolute
    int n0, cl;               // first state of the lane, its live channels
    __device__ __forceinline__ void set(const SsmArgs &a, int64_t b_, int64_t s_, int64_t g_, int64_t ct, int lane) {
        b = b_; s = s_; g = g_;
        c0 = ct * SsmShape<P>::CW;
        const int cw = (lane / P) * 4;
        const int64_t left = a.gdim - c0 - cw;
        n0 = (lane % P) * 4;
        cl = left <= 0 ? 0 : left >= 4 ? 4 : (int)left;
        ch = g * a.gdim + c0 + cw;
    }
};

// ---- one token of each sequence --------------------------------------------------------
// P lanes share a channel, four states each: the state is read and written once
// (8 bytes a pair) and everything else is small beside it. A lane takes its channel of SEQ sequences, so A
// and the parameters are read once for them and their states are in flight together. 64 sequences of 4096 channels x 16
// states, 36 MB, take 10.7 us in a CUDA graph (states of 16 batches in turn; 8.8 for one that stays in L2): 3.4 TB/s, half of
// the copy's rate. 16 sequences take 4.2 us (2.2 TB/s), 128 take 18.8 (3.8): what is left is the latency of short CTAs
// that each load, compute and store once (27 warps an SM, issue 62 %), not the bytes.
// ALL: every sequence has a state and all values move as vectors, so that nothing stands between the loads.
template <class S, int P, int SEQ, bool ALL>
__device__ __forceinline__ void step_lane(const SsmArgs &a, int64_t b0, int64_t ch, int p, float *const (&sp)[SEQ], bool vec, int live) {
    const int64_t N = a.p.nstate, g = ch / a.gdim;
    const int n0 = 4 * p;
    float h[SEQ][4], A[4] = {0.0f, 0.0f, 0.0f, 0.0f}, y[SEQ], u[SEQ], d[SEQ], z[SEQ];
    Raw4<S> rb[SEQ], rc[SEQ];
#pragma unroll
    for (int s = 0; s < SEQ; ++s) {
        const int64_t b = b0 + s;
        y[s] = u[s] = d[s] = z[s] = 0.0f;
        if (!ALL) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                h[s][k] = 0.0f;
        }
        if (ALL || sp[s] != nullptr) {
            if (ALL || vec) {
                lds4(sp[s], h[s]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < live)
                        h[s][k] = sp[s][k];
            }
            u[s] = Codec<S>::load1(static_cast<const S *>(a.p.u) + b * a.p.u_batch + ch);
            d[s] = Codec<S>::load1(static_cast<const S *>(a.p.delta) + b * a.p.delta_batch + ch);
            rb[s].load(static_cast<const S *>(a.p.B) + b * a.p.B_batch + g * N + n0, ALL || a.bvec, ALL ? 4 : live);
            rc[s].load(static_cast<const S *>(a.p.C) + b * a.p.C_batch + g * N + n0, ALL || a.bvec, ALL ? 4 : live);
            if (a.p.z != nullptr)
                z[s] = Codec<S>::load1(static_cast<const S *>(a.p.z) + b * a.p.z_batch + ch);
        }
    }
    const float *ap = a.p.A + ch * N + n0;
    if (ALL || vec) {
        lds4(ap, A);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < live)
                A[k] = ap[k];
    }
    const float bias = a.p.delta_bias != nullptr ? a.p.delta_bias[ch] : 0.0f, skip = a.p.D != nullptr ? a.p.D[ch] : 0.0f;
#pragma unroll
    for (int s = 0; s < SEQ; ++s) {
        if (ALL || sp[s] != nullptr) {
            float bb[4], cc[4];
            rb[s].widen(bb);
            rc[s].widen(cc);
            d[s] += bias;
            if (a.p.softplus)
                d[s] = softplusf(d[s]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[s][k] = fmaf(ex2f(fmaf(d[s], A[k] * kLog2e, kExponentLow)), h[s][k], d[s] * u[s] * bb[k]);
                y[s] = fmaf(cc[k], h[s][k], y[s]);
            }
            if (ALL || vec) {
                *reinterpret_cast<float4 *>(sp[s]) = make_float4(h[s][0], h[s][1], h[s][2], h[s][3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < live)
                        sp[s][k] = h[s][k];
            }
            y[s] = p == 0 ? fmaf(skip, u[s], y[s]) : y[s];
        }
    }
    // the sums over states, by all lanes of the channel
    const unsigned with = P == 32 ? kFull : ((1u << (P % 32)) - 1u) << ((threadIdx.x & 31) / P * P);
#pragma unroll
    for (int s = 0; s < SEQ; ++s) {
#pragma unroll
        for (int m = 1; m < P; m <<= 1)
            y[s] += __shfl_xor_sync(with, y[s], m);
        const int64_t b = b0 + s;
        if (p == 0 && (ALL || b < a.p.batch)) {
            if (a.p.z != nullptr)
                y[s] *= z[s] * sigmoidf(z[s]);
            Codec<S>::store1(static_cast<S *>(a.p.out) + b * a.p.out_batch + ch, ALL || sp[s] != nullptr ? y[s] : 0.0f);
        }
    }
}

template <class S, int P, int SEQ>
__global__ void __launch_bounds__(256) k_ssm_step(const __grid_constant__ SsmArgs a) {
    pdl_prologue();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int p = (int)(i % P);
    const int64_t ch = (i / P) % a.p.dim, b0 = i / P / a.p.dim * SEQ;
    const int64_t left = a.p.nstate - 4 * p;
    const int live = left < 0 ? 0 : left > 4 ? 4 : (int)left;
    float *sp[SEQ];
    bool all = a.nvec && a.bvec && a.p.nstate == 4 * P;  // the same for all lanes of a channel
#pragma unroll
    for (int s = 0; s < SEQ; ++s) {
        const int64_t slot = b0 + s < a.p.batch ? ssm_slot(a, b0 + s) : -1;
        sp[s] = slot >= 0 ? a.p.state + (slot * a.p.dim + ch) * a.p.nstate + 4 * p : nullptr;
        all = all && slot >= 0;
    }
    if (all)
        step_lane<S, P, SEQ, true>(a, b0, ch, p, sp, true, 4);
    else
        step_lane<S, P, SEQ, false>(a, b0, ch, p, sp, a.nvec && live == 4, live);
}

template <class S, int P, int SEQ> static cudaError_t step_seq(const SsmArgs &a, const Launch &L) {
    const int64_t grid = ((a.p.batch + SEQ - 1) / SEQ * a.p.dim * P + 255) / 256;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    note_launch();
    return launch_pdl(k_ssm_step<S, P, SEQ>, (unsigned)grid, 256, 0, L.stream, a);
}
// two sequences a lane where that still fills the SMs (one measured 11.2 us there, four 11.8)
template <class S, int P> static cudaError_t step_go(const SsmArgs &a, const Launch &L) {
    return a.p.batch * a.p.dim * P >= 2 * 2048 * (int64_t)L.sm_count ? step_seq<S, P, 2>(a, L) : step_seq<S, P, 1>(a, L);
}
template <class S> static cudaError_t step_states(const SsmArgs &a, const Launch &L) {
    switch (a.plan.lanes) {
    case 2: return step_go<S, 2>(a, L);
    case 4: return step_go<S, 4>(a, L);
    case 8: return step_go<S, 8>(a, L);
    case 16: return step_go<S, 16>(a, L);
    case 32: return step_go<S, 32>(a, L);
    default: return cudaErrorInvalidValue;
    }
}

// One translation unit per kernel family and activation type (mt_ssm_*.cu).
#define MT_SSM_LAUNCHES(t)                                                                                    \
    cudaError_t ssm_prompt_##t(const SsmArgs &a, const Launch &L);                                            \
    cudaError_t ssm_adjoint_carries_##t(const SsmArgs &a, const Launch &L);                                   \
    cudaError_t ssm_grad_##t(const SsmArgs &a, const Launch &L);                                              \
    cudaError_t ssm_step_##t(const SsmArgs &a, const Launch &L);
MT_SSM_LAUNCHES(f32)
MT_SSM_LAUNCHES(bf16)
MT_SSM_LAUNCHES(f16)
#undef MT_SSM_LAUNCHES

}  // namespace mt
