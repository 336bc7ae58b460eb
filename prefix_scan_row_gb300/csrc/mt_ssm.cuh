// mt_ssm.cuh -- the selective state space scan: forward, gradient and
// single-token kernels, instantiated per activation type (mt_ssm_*.cu).
//
//   Delta = softplus(delta + delta_bias),  a_t[d,n] = exp(Delta_t[d] A[d,n])
//   h_t[d,n] = a_t[d,n] h_{t-1}[d,n] + Delta_t[d] u_t[d] B_t[n]
//   y_t[d] = sum_n C_t[n] h_t[d,n] + D[d] u_t[d],  out = y * z * sigmoid(z)
//
// The recurrence is a scan with the operator (a, b) o (a', b') = (a a', a' b + b'),
// whose products of a are exp(A * sum of Delta): the carry of a span of tokens is
// one state and one sum of steps per channel.
//
// Work split. A lane keeps 4 channels x 4 states in registers, P lanes share
// a channel group (4P states), so a warp holds 128/P channels. Per token
// a lane reads Delta and Delta*u of its 4 channels and B and C of its 4 states from
// shared memory, four 16-byte reads for 16 (channel, state) pairs: fewer
// channels a lane would make the reads, more would make the registers, the
// limit. The sum over states is 4 values over P lanes, exchanged so that every
// step halves the values that are left. A warp works through tiles of 16
// tokens on its own: it widens u and delta of the tile into shared memory, walks
// the 16 tokens, and gates and stores the tile.
//
// Bound: per (token, channel, state) one exponential and four multiply-adds
// (Delta*A, the input, the recurrence, the output); the exponentials run at 32
// and packed multiply-adds at 128 a clock and SM, so at 16 states a warp's token
// costs 16 clocks of either against 8 bytes per channel of HBM traffic
// (4.8 clocks at 16-bit storage): arithmetic, not bandwidth.
//
// Few channels do not fill the GPU: the tokens are then cut into segments that
// run side by side, after a pass that computes each segment's carry (a state
// from zero, and the sum of steps); a segment's first state is the combination of
// the carries before it.
#pragma once

#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

constexpr int kSsmWarps = 4;
constexpr int kSsmThreads = 32 * kSsmWarps;
constexpr int T16 = kSsmTile;

struct SsmArgs {
    mt_ssm_args p;
    SsmPlan plan;
    int64_t ntiles;  // of the whole token axis
    int64_t gdim;    // channels per group
    int cvec, nvec, bvec;  // 4 neighbouring channels / states / values of B and C may be moved as a vector
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
    static constexpr int kCount = P >= 4 ? 1 : 4 / P;
};
template <int P> __device__ __forceinline__ void sum_lanes(const float (&v)[4], int p, float (&o)[SumOut<P>::kCount]) {
    if constexpr (P == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = v[k];
    } else if constexpr (P == 2) {
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
    if constexpr (P == 1)
        *reinterpret_cast<float4 *>(row + 4 * g) = make_float4(o[0], o[1], o[2], o[3]);
    else if constexpr (P == 2)
        *reinterpret_cast<float2 *>(row + 4 * g + 2 * p) = make_float2(o[0], o[1]);
    else if (P == 4 || p < 4)
        row[4 * g + p] = o[0];
}

// Shape of a warp's tile.
template <int P> struct SsmShape {
    static constexpr int CW = 128 / P;                 // channels of a warp
    static constexpr int NP = 4 * P;                   // states, rounded up
    static constexpr int CV = CW / 4;                  // 4-channel vectors per token
    static constexpr int NV = (T16 * CV + 31) / 32;    // of a tile, per lane
    static constexpr int NB = (T16 * P + 31) / 32;     // 4-state vectors of a tile's B or C, per lane
};

// A lane's part of a tile of a [tokens, channels] tensor in storage form:
// vector i is token (32 i + lane) / CV, channels 4 ((32 i + lane) % CV); the channels are the same for every i.
template <class S, int P> struct TileRaw {
    Raw4<S> w[SsmShape<P>::NV];
    __device__ __forceinline__ void load(const S *base, int64_t token_stride, int64_t t0, int64_t n, int lane, int cl,
                                         bool vec) {
#pragma unroll
        for (int i = 0; i < SsmShape<P>::NV; ++i) {
            const int v = 32 * i + lane, t = v / SsmShape<P>::CV, c = (v % SsmShape<P>::CV) * 4;
            const bool in = t < T16 && t0 + t < n;
            w[i].load(base + (t0 + t) * token_stride + c, vec, in ? cl : 0);
        }
    }
};
// B or C of a tile into shared memory as f32, zeros past the sequence and the states.
template <class S, int P, int LANES>
__device__ __forceinline__ void load_shared(float *to, const S *base, int64_t token_stride, int64_t t0, int64_t n,
                                            int nstate, int tid, bool vec) {
    constexpr int kPer = (T16 * P + LANES - 1) / LANES;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int v = LANES * i + tid, t = v / P, s = (v % P) * 4;
        if (t < T16) {
            const int left = nstate - s;
            Raw4<S> w;
            w.load(base + (t0 + t) * token_stride + s, vec, t0 + t < n ? (left > 4 ? 4 : left) : 0);
            float x[4];
            w.widen(x);
            *reinterpret_cast<float4 *>(to + t * (4 * P) + s) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
}

// Delta of four raw values.
__device__ __forceinline__ void steps4(float (&x)[4], const float (&bias)[4], bool softplus) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[k] += bias[k];
        if (softplus)
            x[k] = softplusf(x[k]);
    }
}
__device__ __forceinline__ void load_param4(float (&x)[4], const float *p, int64_t c, int cl) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        x[k] = p != nullptr && k < cl ? p[c + k] : 0.0f;
}

// h = exp2(dt A) h + du B for one token; A holds A * log2(e).
template <bool OUT>
__device__ __forceinline__ void advance(Pairs &h, const Pairs &A, const float (&dt)[4], const float (&du)[4], f32x2 b0,
                                        f32x2 b1, f32x2 c0, f32x2 c1, float (&y)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const f32x2 d2 = pack2f(dt[c], dt[c]), x2 = pack2f(du[c], du[c]);
        h.v[c][0] = fma2f(ex2_2f(mul2f(d2, A.v[c][0])), h.v[c][0], mul2f(x2, b0));
        h.v[c][1] = fma2f(ex2_2f(mul2f(d2, A.v[c][1])), h.v[c][1], mul2f(x2, b1));
        if (OUT) {
            float lo, hi;
            unpack2f(fma2f(c1, h.v[c][1], mul2f(c0, h.v[c][0])), lo, hi);
            y[c] = lo + hi;
        }
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
// h = exp2(A * sum) h + more
__device__ __forceinline__ void combine(Pairs &h, const Pairs &A, const float (&sum)[4], const Pairs &more) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const f32x2 s2 = pack2f(sum[c], sum[c]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            h.v[c][k] = fma2f(ex2_2f(mul2f(s2, A.v[c][k])), h.v[c][k], more.v[c][k]);
    }
}

// Where a warp's work lies.
template <int P> struct SsmPlace {
    int64_t b, s, g, c0, ch;  // sequence, segment, group; first channel of the warp in its group; of the lane, absolute
    int n0, cl, vl;           // first state of the lane; its live channels in the walk, and in the tile's vectors
    int64_t vch;              // absolute first channel of the lane's tile vectors
    __device__ __forceinline__ void set(const SsmArgs &a, int64_t b_, int64_t s_, int64_t g_, int64_t ct, int lane) {
        b = b_; s = s_; g = g_;
        c0 = ct * SsmShape<P>::CW;
        const int64_t left = a.gdim - c0;
        const int cw = (lane / P) * 4, cv = (lane % SsmShape<P>::CV) * 4;
        n0 = (lane % P) * 4;
        cl = left - cw <= 0 ? 0 : left - cw >= 4 ? 4 : (int)(left - cw);
        vl = left - cv <= 0 ? 0 : left - cv >= 4 ? 4 : (int)(left - cv);
        ch = g * a.gdim + c0 + cw;
        vch = g * a.gdim + c0 + cv;
    }
};

// ---- carries of the segments -----------------------------------------------------
// Forward: the state that a segment leaves from zero (segment 0: from the
// first state). REV: the same of the adjoint, r = a (r + C g) from the last token
// down. One exponential and three multiply-adds a pair; no output.
template <class S, int P, bool REV>
__global__ void __launch_bounds__(kSsmThreads, 4) k_ssm_carry(const __grid_constant__ SsmArgs a, int64_t warps) {
    extern __shared__ float4 smem4[];
    using H = SsmShape<P>;
    constexpr int kFloats = T16 * (2 * H::CW + H::NP);
    const int lane = threadIdx.x & 31;
    float *dt = reinterpret_cast<float *>(smem4) + (threadIdx.x >> 5) * kFloats, *du = dt + T16 * H::CW, *sb = du + T16 * H::CW;
    pdl_prologue();
    int64_t w = (int64_t)blockIdx.x * kSsmWarps + (threadIdx.x >> 5);
    if (w >= warps)
        return;
    // forward: the last segment's carry goes nowhere; adjoint: the first's
    const int64_t active = a.plan.segments - 1;
    SsmPlace<P> at;
    const int64_t ct = w % a.plan.ctiles;
    w /= a.plan.ctiles;
    const int64_t g = w % a.p.groups;
    w /= a.p.groups;
    at.set(a, w / active, w % active + (REV ? 1 : 0), g, ct, lane);
    const int64_t n = ssm_len(a, at.b), N = a.p.nstate;
    const int64_t begin = at.s * a.plan.seg_len;
    int64_t end = begin + a.plan.seg_len < n ? begin + a.plan.seg_len : n;
    Pairs A, h;
    A.load(a.p.A + at.ch * N, N, at.n0, at.cl, a.nvec, kLog2e);
    h.zero();
    const int64_t row = (at.b * a.plan.segments + at.s) * a.p.dim + at.ch;
    if (!REV && at.s == 0) {
        const int64_t slot = ssm_slot(a, at.b);
        if (a.p.carry_in && a.p.state != nullptr && slot >= 0)
            h.load(a.p.state + (slot * a.p.dim + at.ch) * N, N, at.n0, at.cl, a.nvec);
        // the state is written by the next launch's last segment while its first
        // one starts: that one reads this copy, in the place of the last carry
        const int64_t spare = (at.b * a.plan.segments + a.plan.segments - 1) * a.p.dim + at.ch;
        h.store(a.carry + spare * N, N, at.n0, at.cl, a.nvec);
    }
    float bias[4], sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, none[4];
    load_param4(bias, a.p.delta_bias, at.vch, at.vl);
    const S *dp = static_cast<const S *>(a.p.delta) + at.b * a.p.delta_batch + at.g * a.gdim + at.c0;
    const S *xp = static_cast<const S *>(REV ? a.p.dout : a.p.u) + at.b * (REV ? a.p.dout_batch : a.p.u_batch) + at.g * a.gdim + at.c0;
    const int64_t xt = REV ? a.p.dout_token : a.p.u_token;
    const S *zp = static_cast<const S *>(a.p.z) + at.b * a.p.z_batch + at.g * a.gdim + at.c0;
    const S *bp = static_cast<const S *>(REV ? a.p.C : a.p.B) + at.b * (REV ? a.p.C_batch : a.p.B_batch) + at.g * N;
    const int64_t bt = REV ? a.p.C_token : a.p.B_token;
    const int64_t tiles = end > begin ? (end - begin + T16 - 1) / T16 : 0;
    for (int64_t k = 0; k < tiles; ++k) {
        const int64_t t0 = begin + (REV ? tiles - 1 - k : k) * T16;
        TileRaw<S, P> rd, rx, rz;
        rd.load(dp, a.p.delta_token, t0, end, lane, at.vl, a.cvec);
        rx.load(xp, xt, t0, end, lane, at.vl, a.cvec);
        if (REV && a.p.z != nullptr)
            rz.load(zp, a.p.z_token, t0, end, lane, at.vl, a.cvec);
        load_shared<S, P, 32>(sb, bp, bt, t0, end, (int)N, lane, a.bvec);
#pragma unroll
        for (int i = 0; i < H::NV; ++i) {
            const int v = 32 * i + lane, t = v / H::CV, c = (v % H::CV) * 4;
            if (t < T16) {
                float d[4], x[4];
                rd.w[i].widen(d);
                rx.w[i].widen(x);
                steps4(d, bias, a.p.softplus);
                if (REV && a.p.z != nullptr) {
                    float z[4];
                    rz.w[i].widen(z);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] *= z[e] * sigmoidf(z[e]);
                }
                const bool in = t0 + t < end;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d[e] = in && e < at.vl ? d[e] : 0.0f;
                    x[e] = in && e < at.vl ? (REV ? x[e] : d[e] * x[e]) : 0.0f;
                }
                *reinterpret_cast<float4 *>(dt + t * H::CW + c) = make_float4(d[0], d[1], d[2], d[3]);
                *reinterpret_cast<float4 *>(du + t * H::CW + c) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
        __syncwarp();
#pragma unroll 2
        for (int j = 0; j < T16; ++j) {
            const int t = REV ? T16 - 1 - j : j;
            float d[4], x[4];
            f32x2 b0, b1;
            lds4(dt + t * H::CW + (lane / P) * 4, d);
            lds4(du + t * H::CW + (lane / P) * 4, x);
            lds_pairs(sb + t * H::NP + (lane % P) * 4, b0, b1);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sum[c] += d[c];
            if (!REV) {
                advance<false>(h, A, d, x, b0, b1, 0ull, 0ull, none);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const f32x2 d2 = pack2f(d[c], d[c]), x2 = pack2f(x[c], x[c]);
                    h.v[c][0] = mul2f(ex2_2f(mul2f(d2, A.v[c][0])), fma2f(x2, b0, h.v[c][0]));
                    h.v[c][1] = mul2f(ex2_2f(mul2f(d2, A.v[c][1])), fma2f(x2, b1, h.v[c][1]));
                }
            }
        }
        __syncwarp();
    }
    // with two segments the copy of the first state and no carry meet: slots differ since segments - 1 >= 1
    h.store(a.carry + row * N, N, at.n0, at.cl, a.nvec);
    if (lane % P == 0)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < at.cl)
                a.decay[row + c] = sum[c];
}

// The state before segment s, from the carries before it.
template <int P> __device__ __forceinline__ void first_state(const SsmArgs &a, const SsmPlace<P> &at, const Pairs &A, Pairs &h) {
    const int64_t N = a.p.nstate, S = a.plan.segments;
    const int64_t row0 = at.b * S * a.p.dim + at.ch;
    h.load(a.carry + (row0 + (at.s == 0 ? S - 1 : 0) * a.p.dim) * N, N, at.n0, at.cl, a.nvec);
    for (int64_t j = 1; j < at.s; ++j) {
        Pairs more;
        float sum[4];
        more.load(a.carry + (row0 + j * a.p.dim) * N, N, at.n0, at.cl, a.nvec);
        load_param4(sum, a.decay, row0 + j * a.p.dim, at.cl);
        combine(h, A, sum, more);
    }
}

// ---- forward -------------------------------------------------------------------------
template <class S, int P>
__global__ void __launch_bounds__(kSsmThreads, 4) k_ssm(const __grid_constant__ SsmArgs a, int64_t warps) {
    extern __shared__ float4 smem4[];
    using H = SsmShape<P>;
    constexpr int kFloats = T16 * (2 * H::CW + 2 * H::NP);
    const int lane = threadIdx.x & 31;
    float *dt = reinterpret_cast<float *>(smem4) + (threadIdx.x >> 5) * kFloats, *du = dt + T16 * H::CW;
    float *sb = du + T16 * H::CW, *sc = sb + T16 * H::NP;
    pdl_prologue();
    int64_t w = (int64_t)blockIdx.x * kSsmWarps + (threadIdx.x >> 5);
    if (w >= warps)
        return;
    SsmPlace<P> at;
    const int64_t ct = w % a.plan.ctiles;
    w /= a.plan.ctiles;
    const int64_t g = w % a.p.groups;
    w /= a.p.groups;
    at.set(a, w / a.plan.segments, w % a.plan.segments, g, ct, lane);
    const int64_t N = a.p.nstate;
    const int64_t slot = ssm_slot(a, at.b);
    const bool active = slot >= 0 || a.p.state == nullptr;
    const int64_t n = active ? ssm_len(a, at.b) : 0;
    const int64_t begin = at.s * a.plan.seg_len;
    const int64_t stop = begin + a.plan.seg_len < a.p.len ? begin + a.plan.seg_len : a.p.len;
    float *state = a.p.state != nullptr && active ? a.p.state + (slot * a.p.dim + at.ch) * N : nullptr;
    Pairs A, h;
    A.load(a.p.A + at.ch * N, N, at.n0, at.cl, a.nvec, kLog2e);
    h.zero();
    if (a.plan.segments > 1)
        first_state<P>(a, at, A, h);
    else if (a.p.carry_in && state != nullptr)
        h.load(state, N, at.n0, at.cl, a.nvec);
    float bias[4], skip[4];
    load_param4(bias, a.p.delta_bias, at.vch, at.vl);
    load_param4(skip, a.p.D, at.vch, at.vl);
    const int64_t cb = at.g * a.gdim + at.c0;
    const S *dp = static_cast<const S *>(a.p.delta) + at.b * a.p.delta_batch + cb;
    const S *up = static_cast<const S *>(a.p.u) + at.b * a.p.u_batch + cb;
    const S *zp = static_cast<const S *>(a.p.z) + at.b * a.p.z_batch + cb;
    const S *bp = static_cast<const S *>(a.p.B) + at.b * a.p.B_batch + at.g * N;
    const S *cp = static_cast<const S *>(a.p.C) + at.b * a.p.C_batch + at.g * N;
    S *op = static_cast<S *>(a.p.out) + at.b * a.p.out_batch + cb;
    for (int64_t t0 = begin; t0 < stop; t0 += T16) {
        const bool any = t0 < n;
        TileRaw<S, P> ru, rz;
        if (any) {
            if (a.p.checkpoints != nullptr)
                h.store(a.p.checkpoints + ((at.b * a.ntiles + t0 / T16) * a.p.dim + at.ch) * N, N, at.n0, at.cl, a.nvec);
            TileRaw<S, P> rd;
            rd.load(dp, a.p.delta_token, t0, n, lane, at.vl, a.cvec);
            ru.load(up, a.p.u_token, t0, n, lane, at.vl, a.cvec);
            load_shared<S, P, 32>(sb, bp, a.p.B_token, t0, n, (int)N, lane, a.bvec);
            load_shared<S, P, 32>(sc, cp, a.p.C_token, t0, n, (int)N, lane, a.bvec);
            if (a.p.z != nullptr)
                rz.load(zp, a.p.z_token, t0, n, lane, at.vl, a.cvec);
#pragma unroll
            for (int i = 0; i < H::NV; ++i) {
                const int v = 32 * i + lane, t = v / H::CV, c = (v % H::CV) * 4;
                if (t < T16) {
                    float d[4], x[4];
                    rd.w[i].widen(d);
                    ru.w[i].widen(x);
                    steps4(d, bias, a.p.softplus);
                    const bool in = t0 + t < n;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        d[e] = in && e < at.vl ? d[e] : 0.0f;
                        x[e] = in && e < at.vl ? d[e] * x[e] : 0.0f;
                    }
                    *reinterpret_cast<float4 *>(dt + t * H::CW + c) = make_float4(d[0], d[1], d[2], d[3]);
                    *reinterpret_cast<float4 *>(du + t * H::CW + c) = make_float4(x[0], x[1], x[2], x[3]);
                }
            }
            __syncwarp();
#pragma unroll 2
            for (int t = 0; t < T16; ++t) {
                float d[4], x[4], y[4], o[SumOut<P>::kCount];
                f32x2 b0, b1, c0, c1;
                lds4(dt + t * H::CW + (lane / P) * 4, d);
                lds4(du + t * H::CW + (lane / P) * 4, x);
                lds_pairs(sb + t * H::NP + (lane % P) * 4, b0, b1);
                lds_pairs(sc + t * H::NP + (lane % P) * 4, c0, c1);
                advance<true>(h, A, d, x, b0, b1, c0, c1, y);
                sum_lanes<P>(y, lane % P, o);
                __syncwarp();
                put_sums<P>(du + t * H::CW, lane / P, lane % P, o);
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < H::NV; ++i) {
            const int v = 32 * i + lane, t = v / H::CV, c = (v % H::CV) * 4;
            if (t < T16 && t0 + t < stop) {
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (t0 + t < n) {
                    float x[4], z[4];
                    lds4(du + t * H::CW + c, y);
                    ru.w[i].widen(x);
                    if (a.p.z != nullptr)
                        rz.w[i].widen(z);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = fmaf(skip[e], x[e], y[e]);
                        if (a.p.z != nullptr)
                            y[e] *= z[e] * sigmoidf(z[e]);
                    }
                }
                store4<S>(op + (t0 + t) * a.p.out_token + c, y, a.cvec, at.vl);
            }
        }
        __syncwarp();
    }
    if (state != nullptr && at.s == a.plan.segments - 1)
        h.store(state, N, at.n0, at.cl, a.nvec);
}

// ---- one token of each sequence --------------------------------------------------------
// P lanes share a channel, four states each: the state is read and written once
// (8 bytes a pair) and everything else is small beside it; bound by bytes.
template <class S, int P>
__global__ void __launch_bounds__(256) k_ssm_step(const __grid_constant__ SsmArgs a) {
    pdl_prologue();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int p = (int)(i % P);
    const int64_t ch = (i / P) % a.p.dim, b = i / P / a.p.dim;
    const bool on = b < a.p.batch;
    const int64_t slot = on ? ssm_slot(a, b) : -1;
    const int64_t N = a.p.nstate;
    const int n0 = 4 * p;
    const int live = N - n0 < 0 ? 0 : N - n0 > 4 ? 4 : (int)(N - n0);
    float y = 0.0f, u = 0.0f;
    if (slot >= 0) {
        const int64_t g = ch / a.gdim;
        u = Codec<S>::load1(static_cast<const S *>(a.p.u) + b * a.p.u_batch + ch);
        float d = Codec<S>::load1(static_cast<const S *>(a.p.delta) + b * a.p.delta_batch + ch);
        float *sp = a.p.state + (slot * a.p.dim + ch) * N + n0;
        const float *ap = a.p.A + ch * N + n0;
        float h[4] = {0.0f, 0.0f, 0.0f, 0.0f}, A[4] = {0.0f, 0.0f, 0.0f, 0.0f}, bb[4], cc[4];
        if (a.nvec && live == 4) {
            lds4(sp, h);
            lds4(ap, A);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < live) {
                    h[k] = sp[k];
                    A[k] = ap[k];
                }
        }
        Raw4<S> rb, rc;
        rb.load(static_cast<const S *>(a.p.B) + b * a.p.B_batch + g * N + n0, a.bvec, live);
        rc.load(static_cast<const S *>(a.p.C) + b * a.p.C_batch + g * N + n0, a.bvec, live);
        rb.widen(bb);
        rc.widen(cc);
        if (a.p.delta_bias != nullptr)
            d += a.p.delta_bias[ch];
        if (a.p.softplus)
            d = softplusf(d);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = fmaf(ex2f(d * (A[k] * kLog2e)), h[k], d * u * bb[k]);
            y = fmaf(cc[k], h[k], y);
        }
        if (a.nvec && live == 4)
            *reinterpret_cast<float4 *>(sp) = make_float4(h[0], h[1], h[2], h[3]);
        else
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < live)
                    sp[k] = h[k];
    }
#pragma unroll
    for (int d = 1; d < P; d <<= 1)
        y += __shfl_xor_sync(kFull, y, d);
    if (on && p == 0) {
        if (slot >= 0) {
            if (a.p.D != nullptr)
                y = fmaf(a.p.D[ch], u, y);
            if (a.p.z != nullptr) {
                const float z = Codec<S>::load1(static_cast<const S *>(a.p.z) + b * a.p.z_batch + ch);
                y *= z * sigmoidf(z);
            }
        }
        Codec<S>::store1(static_cast<S *>(a.p.out) + b * a.p.out_batch + ch, y);
    }
}

// ---- gradient ------------------------------------------------------------------------------
// With g = dout * silu(z) and r_t = a_{t+1} dh_{t+1} coming from the right (at the last token: dfinal):
//   dh_t = C_t g_t + r_t,   r_{t-1} = a_t dh_t,   q = r_{t-1} h_{t-1}
//   dC_t = sum_d g h_t,  dB_t = sum_d Delta u dh_t,  dA = sum_t q Delta,
//   dDelta = sum_n (q A + dh B) u..., du = D g + Delta sum_n dh B, dz = dout y silu'(z).
// The states are not kept by the forward pass but every 16 tokens: a tile walks
// forward from its checkpoint, leaving the states before tokens 0, 4, 8 and 12 in
// shared memory, then takes its four quarters from the last to the first,
// each forward once more with its four states in registers and back. Storing every state would take 64
// bytes a (token, channel) at 16 states where the walk costs 12/16 of a forward.
//
// A CTA's four warps hold neighbouring channels of one group and share B and
// C; their sums over channels for dB and dC meet in shared memory and leave as one
// f32 row per token and CTA, which k_ssm_grad_join adds over the CTAs in order
// (no atomics, so the same bits every time). dA, dD and the bias's gradient stay in registers over a
// segment and are added over sequences and segments by the same kernel.
template <int P> struct GradShape : SsmShape<P> {
    using H = SsmShape<P>;
    static constexpr int kMarks = 4 * 16 * 32;                                // states before the quarters, a warp
    static constexpr int kRows = T16 * 2 * H::NP;                             // dB and dC of the tile, a warp
    static constexpr int kWarpFloats = 3 * T16 * H::CW + kMarks + kRows;
    static constexpr int kFloats = kSsmWarps * kWarpFloats + 2 * T16 * H::NP;
};

__device__ __forceinline__ void mark_store(float4 *m, int lane, const Pairs &h) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float x[4];
        unpack2f(h.v[c][0], x[0], x[1]);
        unpack2f(h.v[c][1], x[2], x[3]);
        m[c * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
    }
}
__device__ __forceinline__ void mark_load(const float4 *m, int lane, Pairs &h) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        lds_pairs(reinterpret_cast<const float *>(m + c * 32 + lane), h.v[c][0], h.v[c][1]);
}

// Eight values (dB and dC of a lane's four states) summed over the channel groups of the warp.
template <int P> __device__ __forceinline__ void put_rows(float *row, int lane, const f32x2 (&s)[4]) {
    constexpr int NP = 4 * P;
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        unpack2f(s[k], v[2 * k], v[2 * k + 1]);
    float *to = row + (lane % P) * 4;
    if constexpr (P == 32) {
        *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(to + NP) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        const bool b1 = lane & P;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float give = b1 ? v[k] : v[k + 4];
            v[k] = (b1 ? v[k + 4] : v[k]) + __shfl_xor_sync(kFull, give, P);
        }
        to += b1 ? NP : 0;
        if constexpr (P == 16) {
            *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            const bool b2 = lane & (2 * P);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float give = b2 ? v[k] : v[k + 2];
                v[k] = (b2 ? v[k + 2] : v[k]) + __shfl_xor_sync(kFull, give, 2 * P);
            }
            to += b2 ? 2 : 0;
            if constexpr (P == 8) {
                *reinterpret_cast<float2 *>(to) = make_float2(v[0], v[1]);
            } else {
                const bool b3 = lane & (4 * P);
                float x = (b3 ? v[1] : v[0]) + __shfl_xor_sync(kFull, b3 ? v[0] : v[1], 4 * P);
                to += b3 ? 1 : 0;
#pragma unroll
                for (int d = 8 * P; d < 32; d <<= 1)
                    x += __shfl_xor_sync(kFull, x, d);
                if (lane < 8 * P)
                    *to = x;
            }
        }
    }
}

template <class S, int P>
__global__ void __launch_bounds__(kSsmThreads, 2) k_ssm_grad(const __grid_constant__ SsmArgs a) {
    extern __shared__ float4 smem4[];
    using H = GradShape<P>;
    constexpr int CW = H::CW, NP = H::NP, CV = H::CV;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *sb = reinterpret_cast<float *>(smem4), *sc = sb + T16 * NP;
    float *rows0 = sc + T16 * NP;                                            // [warps][16][2 NP]
    float *dt = rows0 + kSsmWarps * H::kRows + warp * (3 * T16 * CW), *du = dt + T16 * CW, *sg = du + T16 * CW;
    float4 *marks = reinterpret_cast<float4 *>(rows0 + kSsmWarps * (H::kRows + 3 * T16 * CW) + warp * H::kMarks);
    pdl_prologue();
    int64_t w = blockIdx.x;
    SsmPlace<P> at;
    const int64_t ct = w % a.plan.ctiles;
    w /= a.plan.ctiles;
    const int64_t g = w % a.p.groups;
    w /= a.p.groups;
    const int64_t SEG = a.plan.segments;
    at.set(a, w / SEG, w % SEG, g, ct * kSsmWarps + warp, lane);
    const int64_t N = a.p.nstate, n = ssm_len(a, at.b);
    const int64_t begin = at.s * a.plan.seg_len;
    const int64_t stop = begin + a.plan.seg_len < a.p.len ? begin + a.plan.seg_len : a.p.len;
    Pairs A, r, dA;
    A.load(a.p.A + at.ch * N, N, at.n0, at.cl, a.nvec, kLog2e);
    dA.zero();
    r.zero();
    if (a.p.dfinal != nullptr)
        r.load(a.p.dfinal + (at.b * a.p.dim + at.ch) * N, N, at.n0, at.cl, a.nvec);
    for (int64_t j = SEG - 1; j > at.s; --j) {
        Pairs more;
        float sum[4];
        const int64_t row = (at.b * SEG + j) * a.p.dim + at.ch;
        more.load(a.carry + row * N, N, at.n0, at.cl, a.nvec);
        load_param4(sum, a.decay, row, at.cl);
        combine(r, A, sum, more);
    }
    float bias[4], skip[4], dskip[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dbias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    load_param4(bias, a.p.delta_bias, at.vch, at.vl);
    load_param4(skip, a.p.D, at.vch, at.vl);
    const int64_t cb = at.g * a.gdim + at.c0;
    const S *dp = static_cast<const S *>(a.p.delta) + at.b * a.p.delta_batch + cb;
    const S *up = static_cast<const S *>(a.p.u) + at.b * a.p.u_batch + cb;
    const S *zp = static_cast<const S *>(a.p.z) + at.b * a.p.z_batch + cb;
    const S *gp = static_cast<const S *>(a.p.dout) + at.b * a.p.dout_batch + cb;
    const S *bp = static_cast<const S *>(a.p.B) + at.b * a.p.B_batch + at.g * N;
    const S *cp = static_cast<const S *>(a.p.C) + at.b * a.p.C_batch + at.g * N;
    S *odu = static_cast<S *>(a.p.du) + at.b * a.p.du_batch + cb;
    S *odd = static_cast<S *>(a.p.ddelta) + at.b * a.p.ddelta_batch + cb;
    S *odz = static_cast<S *>(a.p.dz) + at.b * a.p.dz_batch + cb;
    const bool gated = a.p.z != nullptr;
    float *share = a.shared + ((at.g * a.plan.ctiles + ct) * a.p.batch + at.b) * a.p.len * (2 * NP);
    const int64_t tiles = stop > begin ? (stop - begin + T16 - 1) / T16 : 0;
    for (int64_t k = tiles - 1; k >= 0; --k) {
        const int64_t t0 = begin + k * T16;
        const bool any = t0 < n;  // the same for the whole CTA
        if (any) {
            load_shared<S, P, kSsmThreads>(sb, bp, a.p.B_token, t0, n, (int)N, threadIdx.x, a.bvec);
            load_shared<S, P, kSsmThreads>(sc, cp, a.p.C_token, t0, n, (int)N, threadIdx.x, a.bvec);
            {
                TileRaw<S, P> rd, ru, rz, rg;
                rd.load(dp, a.p.delta_token, t0, n, lane, at.vl, a.cvec);
                ru.load(up, a.p.u_token, t0, n, lane, at.vl, a.cvec);
                rg.load(gp, a.p.dout_token, t0, n, lane, at.vl, a.cvec);
                if (gated)
                    rz.load(zp, a.p.z_token, t0, n, lane, at.vl, a.cvec);
#pragma unroll
                for (int i = 0; i < H::NV; ++i) {
                    const int v = 32 * i + lane, t = v / CV, c = (v % CV) * 4;
                    if (t < T16) {
                        float d[4], x[4], o[4];
                        rd.w[i].widen(d);
                        ru.w[i].widen(x);
                        rg.w[i].widen(o);
                        steps4(d, bias, a.p.softplus);
                        if (gated) {
                            float z[4];
                            rz.w[i].widen(z);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[e] *= z[e] * sigmoidf(z[e]);
                        }
                        const bool in = t0 + t < n;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool live = in && e < at.vl;
                            d[e] = live ? d[e] : 0.0f;
                            x[e] = live ? d[e] * x[e] : 0.0f;
                            o[e] = live ? o[e] : 0.0f;
                        }
                        *reinterpret_cast<float4 *>(dt + t * CW + c) = make_float4(d[0], d[1], d[2], d[3]);
                        *reinterpret_cast<float4 *>(du + t * CW + c) = make_float4(x[0], x[1], x[2], x[3]);
                        *reinterpret_cast<float4 *>(sg + t * CW + c) = make_float4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            Pairs h;
            h.load(a.p.checkpoints + ((at.b * a.ntiles + t0 / T16) * a.p.dim + at.ch) * N, N, at.n0, at.cl, a.nvec);
            mark_store(marks, lane, h);
            __syncthreads();
            const int wo = (lane / P) * 4, no = (lane % P) * 4;
#pragma unroll 1
            for (int qt = 0; qt < 3; ++qt) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = 4 * qt + j;
                    float d[4], x[4], none[4];
                    f32x2 b0, b1;
                    lds4(dt + t * CW + wo, d);
                    lds4(du + t * CW + wo, x);
                    lds_pairs(sb + t * NP + no, b0, b1);
                    advance<false>(h, A, d, x, b0, b1, 0ull, 0ull, none);
                }
                mark_store(marks + (qt + 1) * 128, lane, h);
            }
#pragma unroll 1
            for (int qt = 3; qt >= 0; --qt) {
                Pairs hs[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = 4 * qt + j;
                    float d[4], x[4], none[4];
                    f32x2 b0, b1;
                    if (j == 0)
                        mark_load(marks + qt * 128, lane, hs[0]);
                    else
                        hs[j] = hs[j - 1];
                    lds4(dt + t * CW + wo, d);
                    lds4(du + t * CW + wo, x);
                    lds_pairs(sb + t * NP + no, b0, b1);
                    advance<false>(hs[j], A, d, x, b0, b1, 0ull, 0ull, none);
                }
#pragma unroll
                for (int j = 3; j >= 0; --j) {
                    const int t = 4 * qt + j;
                    float d[4], x[4], gg[4], y[4], hb[4], qa[4];
                    f32x2 b[2], c[2], rows[4] = {0ull, 0ull, 0ull, 0ull};
                    lds4(dt + t * CW + wo, d);
                    lds4(du + t * CW + wo, x);
                    lds4(sg + t * CW + wo, gg);
                    lds_pairs(sb + t * NP + no, b[0], b[1]);
                    lds_pairs(sc + t * NP + no, c[0], c[1]);
                    Pairs hp;
                    if (j == 0)
                        mark_load(marks + qt * 128, lane, hp);
                    else
                        hp = hs[j - 1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f32x2 d2 = pack2f(d[e], d[e]), x2 = pack2f(x[e], x[e]), g2 = pack2f(gg[e], gg[e]);
                        f32x2 y2 = 0ull, hb2 = 0ull, qa2 = 0ull;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const f32x2 dh = fma2f(c[s], g2, r.v[e][s]);
                            rows[s] = fma2f(x2, dh, rows[s]);
                            rows[2 + s] = fma2f(g2, hs[j].v[e][s], rows[2 + s]);
                            y2 = fma2f(c[s], hs[j].v[e][s], y2);
                            hb2 = fma2f(b[s], dh, hb2);
                            r.v[e][s] = mul2f(ex2_2f(mul2f(d2, A.v[e][s])), dh);
                            const f32x2 q = mul2f(r.v[e][s], hp.v[e][s]);
                            qa2 = fma2f(q, A.v[e][s], qa2);
                            dA.v[e][s] = fma2f(q, d2, dA.v[e][s]);
                        }
                        float lo, hi;
                        unpack2f(y2, lo, hi);
                        y[e] = lo + hi;
                        unpack2f(hb2, lo, hi);
                        hb[e] = lo + hi;
                        unpack2f(qa2, lo, hi);
                        qa[e] = lo + hi;
                    }
                    float o0[SumOut<P>::kCount], o1[SumOut<P>::kCount], o2[SumOut<P>::kCount];
                    sum_lanes<P>(y, lane % P, o0);
                    sum_lanes<P>(hb, lane % P, o1);
                    sum_lanes<P>(qa, lane % P, o2);
                    put_rows<P>(rows0 + warp * H::kRows + t * (2 * NP), lane, rows);
                    __syncwarp();  // every lane has read token t's row
                    put_sums<P>(dt + t * CW, lane / P, lane % P, o0);
                    put_sums<P>(du + t * CW, lane / P, lane % P, o1);
                    put_sums<P>(sg + t * CW, lane / P, lane % P, o2);
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < H::kRows; i += kSsmThreads) {
                const int t = i / (2 * NP);
                if (t0 + t < n) {
                    float s = rows0[i];
#pragma unroll
                    for (int v = 1; v < kSsmWarps; ++v)
                        s += rows0[v * H::kRows + i];
                    share[t0 * (2 * NP) + i] = s;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < H::NV; ++i) {
            const int v = 32 * i + lane, t = v / CV, c = (v % CV) * 4;
            if (t < T16 && t0 + t < stop) {
                float xu[4] = {0.0f, 0.0f, 0.0f, 0.0f}, xd[4] = {0.0f, 0.0f, 0.0f, 0.0f}, xz[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (t0 + t < n) {
                    Raw4<S> rd, ru, rz, rg;
                    float y[4], hb[4], qa[4], d[4], u[4], z[4], o[4];
                    rd.load(dp + (t0 + t) * a.p.delta_token + c, a.cvec, at.vl);
                    ru.load(up + (t0 + t) * a.p.u_token + c, a.cvec, at.vl);
                    rg.load(gp + (t0 + t) * a.p.dout_token + c, a.cvec, at.vl);
                    if (gated)
                        rz.load(zp + (t0 + t) * a.p.z_token + c, a.cvec, at.vl);
                    lds4(dt + t * CW + c, y);
                    lds4(du + t * CW + c, hb);
                    lds4(sg + t * CW + c, qa);
                    rd.widen(d);
                    ru.widen(u);
                    rg.widen(o);
                    if (gated)
                        rz.widen(z);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (e < at.vl) {
                            const float raw = d[e] + bias[e];
                            const float step = a.p.softplus ? softplusf(raw) : raw;
                            const float slope = a.p.softplus ? sigmoidf(raw) : 1.0f;
                            float gy = o[e];
                            if (gated) {
                                const float s = sigmoidf(z[e]);
                                gy = o[e] * (z[e] * s);
                                xz[e] = o[e] * fmaf(skip[e], u[e], y[e]) * (s * fmaf(z[e], 1.0f - s, 1.0f));
                            }
                            xu[e] = fmaf(skip[e], gy, step * hb[e]);
                            // A came with log2(e), so its product is put back
                            xd[e] = fmaf(qa[e], kLn2, hb[e] * u[e]) * slope;
                            dskip[e] = fmaf(gy, u[e], dskip[e]);
                            dbias[e] += xd[e];
                        }
                    }
                }
                store4<S>(odu + (t0 + t) * a.p.du_token + c, xu, a.cvec, at.vl);
                store4<S>(odd + (t0 + t) * a.p.ddelta_token + c, xd, a.cvec, at.vl);
                if (gated)
                    store4<S>(odz + (t0 + t) * a.p.dz_token + c, xz, a.cvec, at.vl);
            }
        }
        __syncthreads();
    }
    if (at.s == 0 && a.p.dinit != nullptr)
        r.store(a.p.dinit + (at.b * a.p.dim + at.ch) * N, N, at.n0, at.cl, a.nvec);
    const int64_t part = at.b * SEG + at.s;
    dA.store(a.dA_part + (part * a.p.dim + at.ch) * N, N, at.n0, at.cl, a.nvec);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int d = CV; d < 32; d <<= 1) {
            dskip[e] += __shfl_xor_sync(kFull, dskip[e], d);
            dbias[e] += __shfl_xor_sync(kFull, dbias[e], d);
        }
        if (lane < CV && e < at.vl) {
            a.dD_part[part * a.p.dim + at.vch + e] = dskip[e];
            a.dbias_part[part * a.p.dim + at.vch + e] = dbias[e];
        }
    }
}

// The sums over CTAs of dB and dC (rounded once, here), and over sequences and
// segments of dA, dD and the bias's gradient, each in a fixed order.
template <class S>
__global__ void __launch_bounds__(256) k_ssm_grad_join(const __grid_constant__ SsmArgs a, int np) {
    pdl_prologue();
    const int64_t N = a.p.nstate, D = a.p.dim, L = a.p.len, B = a.p.batch, G = a.p.groups;
    const int64_t shared = B * L * G * 2 * N, params = D * N;
    const int64_t parts = B * a.plan.segments;
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < shared + params + D; i += stride) {
        if (i < shared) {
            const int64_t s = i % N;
            int64_t q = i / N;
            const int64_t which = q & 1;
            q >>= 1;
            const int64_t g = q % G;
            q /= G;
            const int64_t t = q % L, b = q / L;
            float v = 0.0f;
            if (t < ssm_len(a, b)) {
                const float *p = a.shared + ((g * a.plan.ctiles * B + b) * L + t) * (2 * np) + which * np + s;
#pragma unroll 8
                for (int64_t k = 0; k < a.plan.ctiles; ++k)
                    v += p[k * B * L * (2 * np)];
            }
            S *to = which ? static_cast<S *>(a.p.dC) + b * a.p.dC_batch + t * a.p.dC_token
                          : static_cast<S *>(a.p.dB) + b * a.p.dB_batch + t * a.p.dB_token;
            Codec<S>::store1(to + g * N + s, v);
        } else if (i < shared + params) {
            const int64_t j = i - shared;
            float v = 0.0f;
#pragma unroll 4
            for (int64_t k = 0; k < parts; ++k)
                v += a.dA_part[k * params + j];
            a.p.dA[j] = v;
        } else {
            const int64_t j = i - shared - params;
            float v = 0.0f, w = 0.0f;
#pragma unroll 4
            for (int64_t k = 0; k < parts; ++k) {
                v += a.dD_part[k * D + j];
                w += a.dbias_part[k * D + j];
            }
            if (a.p.dD != nullptr)
                a.p.dD[j] = v;
            if (a.p.ddelta_bias != nullptr)
                a.p.ddelta_bias[j] = w;
        }
    }
}

// ---- launches --------------------------------------------------------------------------------
enum SsmWhat { kSsmForward, kSsmGrad, kSsmStep };

template <class K> static cudaError_t ssm_smem(K kernel, size_t bytes) {
    return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) : cudaSuccess;
}

template <class S, int P> static cudaError_t ssm_go(const SsmArgs &a, SsmWhat what, const Launch &L) {
    using H = SsmShape<P>;
    cudaError_t e;
    if (what == kSsmStep) {
        const int64_t grid = (a.p.batch * a.p.dim * P + 255) / 256;
        if (grid > INT32_MAX)
            return cudaErrorInvalidValue;
        note_launch();
        return launch_pdl(k_ssm_step<S, P>, (unsigned)grid, 256, 0, L.stream, a);
    }
    const size_t carry_smem = sizeof(float) * kSsmWarps * T16 * (2 * H::CW + H::NP);
    const int64_t per_segment = a.p.batch * a.p.groups * a.plan.ctiles;
    if (what == kSsmForward) {
        const size_t smem = sizeof(float) * kSsmWarps * T16 * (2 * H::CW + 2 * H::NP);
        if (a.plan.segments > 1) {
            const int64_t warps = per_segment * (a.plan.segments - 1), grid = (warps + kSsmWarps - 1) / kSsmWarps;
            if (grid > INT32_MAX)
                return cudaErrorInvalidValue;
            if ((e = ssm_smem(k_ssm_carry<S, P, false>, carry_smem)) != cudaSuccess)
                return e;
            note_launch();
            if ((e = launch_pdl(k_ssm_carry<S, P, false>, (unsigned)grid, kSsmThreads, carry_smem, L.stream, a, warps)) != cudaSuccess)
                return e;
        }
        const int64_t warps = per_segment * a.plan.segments, grid = (warps + kSsmWarps - 1) / kSsmWarps;
        if (grid > INT32_MAX)
            return cudaErrorInvalidValue;
        if ((e = ssm_smem(k_ssm<S, P>, smem)) != cudaSuccess)
            return e;
        note_launch();
        return launch_pdl(k_ssm<S, P>, (unsigned)grid, kSsmThreads, smem, L.stream, a, warps);
    }
    if (a.plan.segments > 1) {
        SsmArgs c = a;  // the carries' warps are placed one by one: as many tiles of a warp's channels
        c.plan.ctiles = (a.gdim + H::CW - 1) / H::CW;
        const int64_t warps = a.p.batch * a.p.groups * c.plan.ctiles * (a.plan.segments - 1);
        const int64_t grid = (warps + kSsmWarps - 1) / kSsmWarps;
        if (grid > INT32_MAX)
            return cudaErrorInvalidValue;
        if ((e = ssm_smem(k_ssm_carry<S, P, true>, carry_smem)) != cudaSuccess)
            return e;
        note_launch();
        if ((e = launch_pdl(k_ssm_carry<S, P, true>, (unsigned)grid, kSsmThreads, carry_smem, L.stream, c, warps)) != cudaSuccess)
            return e;
    }
    const int64_t grid = per_segment * a.plan.segments;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    const size_t smem = sizeof(float) * GradShape<P>::kFloats;
    if (grid > 0) {
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
    return launch_pdl(k_ssm_grad_join<S>, (unsigned)jgrid, 256, 0, L.stream, a, (int)H::NP);
}

template <class S> static cudaError_t ssm_type(const SsmArgs &a, SsmWhat what, const Launch &L) {
    switch (a.plan.lanes) {
    case 2: return ssm_go<S, 2>(a, what, L);
    case 4: return ssm_go<S, 4>(a, what, L);
    case 8: return ssm_go<S, 8>(a, what, L);
    case 16: return ssm_go<S, 16>(a, what, L);
    case 32: return ssm_go<S, 32>(a, what, L);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t ssm_f32(const SsmArgs &a, SsmWhat what, const Launch &L);   // mt_ssm_f32.cu
cudaError_t ssm_bf16(const SsmArgs &a, SsmWhat what, const Launch &L);  // mt_ssm_bf16.cu
cudaError_t ssm_f16(const SsmArgs &a, SsmWhat what, const Launch &L);   // mt_ssm_f16.cu

}  // namespace mt
