// mt_ssm_grad.cuh -- the gradient of the selective state space scan.
//
// With g = dout * silu(z) and r_t = a_{t+1} dh_{t+1} coming from the right (at the last token: dfinal):
//   dh_t = C_t g_t + r_t,   r_{t-1} = a_t dh_t,   q = r_{t-1} h_{t-1}
//   dC_t = sum_d g h_t,  dB_t = sum_d Delta u dh_t,  dA = sum_t q Delta,
//   dDelta = sum_n q A + u sum_n dh B, du = D g + Delta sum_n dh B, dz = dout y silu'(z).
//
// The forward pass keeps the states every 8 tokens (4 bytes a state, 8 a (token, channel) at 16
// states). A tile of 8 tokens walks forward from its checkpoint and leaves
// the states before tokens 0, 2, 4 and 6 in shared memory, then takes its four pairs of
// tokens from the last to the first: each forward once more, its states and
// decays in registers, and back. Keeping every state instead would take 64 bytes a
// (token, channel), where the walk costs 6/8 of a forward.
//
// A lane keeps 4 channels x 4 states, which makes the sums across lanes fewest:
// three sums over states (4 values over P lanes each) and two over channels (8
// values over 32/P lanes) take 16 shuffles a token, where one channel x 16 states a
// lane takes 31. The elementwise parts before and after the walk are made for two
// neighbouring channels at a time, and each is made once: the walk leaves Delta and g where they are.
//
// A CTA's four warps hold neighbouring channels of one group and share B and
// C; their sums over channels for dB and dC meet in shared memory and leave as one
// f32 row per token and CTA, which k_ssm_grad_join adds over the CTAs in order
// (no atomics, so the same bits every time). dA, dD and the bias's gradient stay in registers over a
// segment and are added over sequences and segments by the same kernel.
//
// 390 warp instructions a token of 32 channels at 16 states, of which the recurrences are 143 packed multiply-adds. 310 us
// of 4 x 1024 tokens x 4096 channels, bf16 (a tile of 16 tokens with 8 x 2 tokens' states and decays made twice: 481; channel pairs
// for state pairs: 316). Issue is 55 % busy, FMA 46, XU 20, DRAM 15: bound by how far 11 warps an SM (168 registers, 75 KB a CTA)
// cover an instruction's wait for the one before (1.0 of a warp's cycles between two instructions; shared memory 0.65, math pipes 0.5).
#pragma once

#include "mt_ssm_prompt.cuh"

namespace mt {

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

// Shared memory of a CTA.
template <class S, int P> struct GradSmem {
    using H = SsmShape<P>;
    using R = Rows8<S, H::CW>;
    using St = States8<S, H::NP>;
    static constexpr int kMarks = 4 * 16 * 32 * 4;              // states before the pairs of tokens
    static constexpr int kArray = kStep * H::CW * 4;            // Delta, Delta u (then sum q A), g
    static constexpr int kLast = 4 * H::CW * 4;                 // y and sum dh B of the last pair
    static constexpr int kRowFloats = kStep * 2 * H::NP;        // dB and dC of the tile
    static constexpr int kStage = 4 * R::kBytes;                // delta, u, dout, z
    static constexpr int kWarp = kMarks + 3 * kArray + kLast + 4 * kRowFloats + 2 * kStage;
    static constexpr int kShared = 2 * (2 * kStep * H::NP * 4) + 2 * (2 * St::kBytes);  // B and C, widened and as stored
    static constexpr int kBytes = kSsmWarps * kWarp + kShared;
};

template <class S, int P, bool ALN>
__global__ void __launch_bounds__(kSsmThreads, sizeof(S) == 2 && P <= 8 ? 3 : 2) k_ssm_grad(const __grid_constant__ SsmArgs a) {
    extern __shared__ float4 smem4[];
    using M = GradSmem<S, P>;
    using R = typename M::R;
    using St = typename M::St;
    constexpr int CW = M::H::CW, NP = M::H::NP;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    char *base = reinterpret_cast<char *>(smem4);
    // the CTA's: rows of all warps side by side, B and C of two tiles widened and as stored
    float *rows0 = reinterpret_cast<float *>(base);
    float *wide = rows0 + kSsmWarps * M::kRowFloats;  // [2][B, C][8][NP]
    char *kept = reinterpret_cast<char *>(wide + 2 * 2 * kStep * NP);
    // the warp's
    char *mine = kept + 2 * 2 * St::kBytes + warp * (M::kWarp - 4 * M::kRowFloats);
    float4 *marks = reinterpret_cast<float4 *>(mine);
    float *dt = reinterpret_cast<float *>(mine + M::kMarks), *du = dt + kStep * CW, *sg = du + kStep * CW, *last = sg + kStep * CW;
    char *stages = reinterpret_cast<char *>(last + 4 * CW);
    // y (which = 0) and sum dh B (1) of token t lie over the marks that the pair of tokens after it has used
    const auto result = [&](int t, int which) {
        float *p = t >= kStep - 2 ? last : reinterpret_cast<float *>(marks + (t / 2 + 1) * 128);
        return p + (2 * which + (t & 1)) * CW;
    };
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
    const int64_t end = n < stop ? n : stop;
    Pairs A, r, dA;
    A.load(a.p.A + at.ch * N, N, at.n0, at.cl, ALN || a.nvec, kLog2e);
    dA.zero();
    r.zero();
    if (SEG > 1)
        r.load(a.carry + ((at.b * SEG + at.s) * a.p.dim + at.ch) * N, N, at.n0, at.cl, ALN || a.nvec);
    else if (a.p.dfinal != nullptr)
        r.load(a.p.dfinal + (at.b * a.p.dim + at.ch) * N, N, at.n0, at.cl, ALN || a.nvec);
    // the elementwise parts: a lane has a channel pair, and every kTok-th token
    constexpr int kPairs = CW / 2 < 32 ? CW / 2 : 32, kTok = 32 / kPairs;
    const int ec = lane % kPairs * 2, et = lane / kPairs;
    const int64_t left_c = a.gdim - at.c0 - ec;
    const int el = left_c <= 0 ? 0 : left_c >= 2 ? 2 : 1;
    const int64_t cb = at.g * a.gdim + at.c0;  // the warp's first channel in a token's row
    const f32x2 bias = pair_of(a.p.delta_bias, cb + ec, el), skip = pair_of(a.p.D, cb + ec, el);
    f32x2 dskip = 0ull, dbias = 0ull;
    const bool gated = a.p.z != nullptr, softplus = a.p.softplus;
    const int channels = a.gdim - at.c0 <= 0 ? 0 : a.gdim - at.c0 < CW ? (int)(a.gdim - at.c0) : CW;
    const bool in = R::chunk(lane) < channels;
    const int64_t cs = cb + (in ? R::chunk(lane) : 0);
    const S *bp = static_cast<const S *>(a.p.B) + at.b * a.p.B_batch + at.g * N;
    const S *cp = static_cast<const S *>(a.p.C) + at.b * a.p.C_batch + at.g * N;
    float *share = a.shared + ((at.g * a.plan.ctiles + ct) * a.p.batch + at.b) * a.p.len * (2 * NP);
    const int tiles = end > begin ? (int)((end - begin + kStep - 1) / kStep) : 0;
    const auto fetch = [&](int k) {
        const int64_t t0 = begin + (int64_t)k * kStep, tl = t0 + R::token(lane);
        const int left = end - t0 < kStep ? (int)(end - t0) : kStep;
        const uint32_t to = smem_addr(stages) + (k & 1) * M::kStage;
        const S *dp = static_cast<const S *>(a.p.delta) + at.b * a.p.delta_batch, *up = static_cast<const S *>(a.p.u) + at.b * a.p.u_batch;
        const S *gp = static_cast<const S *>(a.p.dout) + at.b * a.p.dout_batch, *zp = static_cast<const S *>(a.p.z) + at.b * a.p.z_batch;
        if (ALN) {
            R::fetch16(to, dp + tl * a.p.delta_token + cs, a.p.delta_token, left, in, lane);
            R::fetch16(to + R::kBytes, up + tl * a.p.u_token + cs, a.p.u_token, left, in, lane);
            R::fetch16(to + 2 * R::kBytes, gp + tl * a.p.dout_token + cs, a.p.dout_token, left, in, lane);
            if (gated)
                R::fetch16(to + 3 * R::kBytes, zp + tl * a.p.z_token + cs, a.p.z_token, left, in, lane);
        } else {
            R::fetch_words(to, dp + cb, a.p.delta_token, t0, left, channels, lane);
            R::fetch_words(to + R::kBytes, up + cb, a.p.u_token, t0, left, channels, lane);
            R::fetch_words(to + 2 * R::kBytes, gp + cb, a.p.dout_token, t0, left, channels, lane);
            if (gated)
                R::fetch_words(to + 3 * R::kBytes, zp + cb, a.p.z_token, t0, left, channels, lane);
        }
        if (warp < 2) {  // warp 0 brings B, warp 1 C
            const uint32_t ks = smem_addr(kept) + ((k & 1) * 2 + warp) * St::kBytes;
            St::fetch(ks, warp == 0 ? bp : cp, warp == 0 ? a.p.B_token : a.p.C_token, t0, left, (int)N, lane, ALN || a.bvec);
        }
        cp_async_commit();
    };
    const auto widen = [&](int k) {
        const int64_t t0 = begin + (int64_t)k * kStep;
        const int left = end - t0 < kStep ? (int)(end - t0) : kStep;
        if (warp < 2)
            St::widen(wide + ((k & 1) * 2 + warp) * (kStep * NP), kept + ((k & 1) * 2 + warp) * St::kBytes, warp == 0 ? bp : cp,
                      warp == 0 ? a.p.B_token : a.p.C_token, t0, left, (int)N, lane, ALN || a.bvec);
    };
    if (tiles > 0) {
        fetch(tiles - 1);
        cp_async_wait_all();
        __syncwarp();
        widen(tiles - 1);  // a warp widens what it copied
        __syncthreads();
    }
    for (int k = tiles - 1; k >= 0; --k) {
        const int64_t t0 = begin + (int64_t)k * kStep;
        const int left = end - t0 < kStep ? (int)(end - t0) : kStep;
        char *raw = stages + (k & 1) * M::kStage;
        const float *sb = wide + (k & 1) * (2 * kStep * NP), *sc = sb + kStep * NP;
        if (k > 0)
            fetch(k - 1);
        if (!ALN) {
            const S *dp = static_cast<const S *>(a.p.delta) + at.b * a.p.delta_batch, *up = static_cast<const S *>(a.p.u) + at.b * a.p.u_batch;
            const S *gp = static_cast<const S *>(a.p.dout) + at.b * a.p.dout_batch, *zp = static_cast<const S *>(a.p.z) + at.b * a.p.z_batch;
            R::settle(raw, dp + cb, a.p.delta_token, t0, left, channels, lane);
            R::settle(raw + R::kBytes, up + cb, a.p.u_token, t0, left, channels, lane);
            R::settle(raw + 2 * R::kBytes, gp + cb, a.p.dout_token, t0, left, channels, lane);
            if (gated)
                R::settle(raw + 3 * R::kBytes, zp + cb, a.p.z_token, t0, left, channels, lane);
            __syncwarp();
        }
        if (left < kStep)
            R::no_steps(raw, left, lane);
        Pairs h;
        h.load(a.p.checkpoints + ((at.b * a.ntiles + t0 / kStep) * a.p.dim + at.ch) * N, N, at.n0, at.cl, ALN || a.nvec);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < (kStep + kTok - 1) / kTok; ++i) {
            const int t = et + i * kTok;
            if (kTok <= kStep || t < kStep) {
                f32x2 d = add2f(R::read(raw, t, ec), bias);
                if (softplus || t >= left)
                    d = softplus_2f(d);
                const f32x2 u = R::read(raw + R::kBytes, t, ec);
                f32x2 o = R::read(raw + 2 * R::kBytes, t, ec);
                if (gated) {
                    const f32x2 z = R::read(raw + 3 * R::kBytes, t, ec);
                    o = mul2f(o, mul2f(z, sigmoid_2f(z)));
                }
                *reinterpret_cast<f32x2 *>(dt + t * CW + ec) = d;
                *reinterpret_cast<f32x2 *>(du + t * CW + ec) = mul2f(d, u);
                *reinterpret_cast<f32x2 *>(sg + t * CW + ec) = o;
            }
        }
        mark_store(marks, lane, h);
        __syncwarp();
        const int wo = (lane / P) * 4, no = (lane % P) * 4;
#pragma unroll 1
        for (int qt = 0; qt < 3; ++qt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = 2 * qt + j;
                float d[4], x[4];
                f32x2 b0, b1;
                lds4(dt + t * CW + wo, d);
                lds4(du + t * CW + wo, x);
                lds_pairs(sb + t * NP + no, b0, b1);
                advance(h, A, d, x, b0, b1);
            }
            mark_store(marks + (qt + 1) * 128, lane, h);
        }
#pragma unroll 1
        for (int qt = 3; qt >= 0; --qt) {
            Pairs hs[2], dec[2];  // after each of the two tokens; their decays
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = 2 * qt + j;
                float d[4], x[4];
                f32x2 b[2];
                if (j == 0)
                    mark_load(marks + qt * 128, lane, hs[0]);
                else
                    hs[1] = hs[0];
                lds4(dt + t * CW + wo, d);
                lds4(du + t * CW + wo, x);
                lds_pairs(sb + t * NP + no, b[0], b[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 d2 = both(d[e]), x2 = both(x[e]);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        dec[j].v[e][s] = ex2_2f(exponent2f(d2, A.v[e][s]));
                        hs[j].v[e][s] = fma2f(dec[j].v[e][s], hs[j].v[e][s], mul2f(x2, b[s]));
                    }
                }
            }
#pragma unroll
            for (int j = 1; j >= 0; --j) {
                const int t = 2 * qt + j;
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
                    hp = hs[0];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x2 d2 = both(d[e]), x2 = both(x[e]), g2 = both(gg[e]);
                    f32x2 y2 = 0ull, hb2 = 0ull, qa2 = 0ull;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const f32x2 dh = fma2f(c[s], g2, r.v[e][s]);
                        rows[s] = fma2f(x2, dh, rows[s]);
                        rows[2 + s] = fma2f(g2, hs[j].v[e][s], rows[2 + s]);
                        y2 = fma2f(c[s], hs[j].v[e][s], y2);
                        hb2 = fma2f(b[s], dh, hb2);
                        r.v[e][s] = mul2f(dec[j].v[e][s], dh);
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
                put_rows<P>(rows0 + warp * M::kRowFloats + t * (2 * NP), lane, rows);
                __syncwarp();  // every lane has read what these take the place of
                put_sums<P>(result(t, 0), lane / P, lane % P, o0);
                put_sums<P>(result(t, 1), lane / P, lane % P, o1);
                put_sums<P>(du + t * CW, lane / P, lane % P, o2);
            }
        }
        cp_async_wait_all();
        __syncthreads();  // all warps' rows; the next tile's B and C as stored
        for (int i = threadIdx.x; i < left * 2 * NP; i += kSsmThreads) {
            float s = rows0[i];
#pragma unroll
            for (int v = 1; v < kSsmWarps; ++v)
                s += rows0[v * M::kRowFloats + i];
            share[t0 * (2 * NP) + i] = s;
        }
        if (k > 0)
            widen(k - 1);
        f32x2 tskip = 0ull, tbias = 0ull;  // of the tile: added to the segment's as one, which halves their rounding
#pragma unroll
        for (int i = 0; i < (kStep + kTok - 1) / kTok; ++i) {
            const int t = et + i * kTok;
            if (kTok <= kStep || t < kStep) {
                const f32x2 step = *reinterpret_cast<const f32x2 *>(dt + t * CW + ec), qa = *reinterpret_cast<const f32x2 *>(du + t * CW + ec);
                const f32x2 gy = *reinterpret_cast<const f32x2 *>(sg + t * CW + ec);
                const f32x2 y = *reinterpret_cast<const f32x2 *>(result(t, 0) + ec), hb = *reinterpret_cast<const f32x2 *>(result(t, 1) + ec);
                const f32x2 u = R::read(raw + R::kBytes, t, ec);
                R::write(raw + R::kBytes, t, ec, fma2f(skip, gy, mul2f(step, hb)));
                // A came with log2(e), so its product is put back
                f32x2 xd = fma2f(qa, both(kLn2), mul2f(hb, u));
                if (softplus)
                    xd = mul2f(xd, sigmoid_2f(add2f(R::read(raw, t, ec), bias)));
                R::write(raw, t, ec, xd);
                if (t < left) {
                    tskip = fma2f(gy, u, tskip);
                    tbias = add2f(tbias, xd);
                }
                if (gated) {
                    const f32x2 z = R::read(raw + 3 * R::kBytes, t, ec), o = R::read(raw + 2 * R::kBytes, t, ec), s = sigmoid_2f(z);
                    const f32x2 slope = mul2f(s, fma2f(z, add2f(both(1.0f), mul2f(both(-1.0f), s)), both(1.0f)));
                    R::write(raw + 3 * R::kBytes, t, ec, mul2f(mul2f(o, fma2f(skip, u, y)), slope));
                }
            }
        }
        dskip = add2f(dskip, tskip);
        dbias = add2f(dbias, tbias);
        __syncwarp();
        {
            const int64_t tl = t0 + R::token(lane);
            S *odu = static_cast<S *>(a.p.du) + at.b * a.p.du_batch, *odd = static_cast<S *>(a.p.ddelta) + at.b * a.p.ddelta_batch;
            S *odz = static_cast<S *>(a.p.dz) + at.b * a.p.dz_batch;
            if (ALN) {
                R::put16(raw, odd + tl * a.p.ddelta_token + cs, a.p.ddelta_token, left, in, lane);
                R::put16(raw + R::kBytes, odu + tl * a.p.du_token + cs, a.p.du_token, left, in, lane);
                if (gated)
                    R::put16(raw + 3 * R::kBytes, odz + tl * a.p.dz_token + cs, a.p.dz_token, left, in, lane);
            } else {
                R::put_each(raw, odd + cb, a.p.ddelta_token, t0, left, channels, lane);
                R::put_each(raw + R::kBytes, odu + cb, a.p.du_token, t0, left, channels, lane);
                if (gated)
                    R::put_each(raw + 3 * R::kBytes, odz + cb, a.p.dz_token, t0, left, channels, lane);
            }
        }
        __syncthreads();  // the rows may be written again; the next tile's B and C are there
    }
    for (int64_t t = begin > end ? begin : end; t < stop; ++t)  // past the sequence's end
        for (int c = lane; c < channels; c += 32) {
            Codec<S>::store1(static_cast<S *>(a.p.du) + at.b * a.p.du_batch + t * a.p.du_token + cb + c, 0.0f);
            Codec<S>::store1(static_cast<S *>(a.p.ddelta) + at.b * a.p.ddelta_batch + t * a.p.ddelta_token + cb + c, 0.0f);
            if (gated)
                Codec<S>::store1(static_cast<S *>(a.p.dz) + at.b * a.p.dz_batch + t * a.p.dz_token + cb + c, 0.0f);
        }
    if (at.s == 0 && a.p.dinit != nullptr)
        r.store(a.p.dinit + (at.b * a.p.dim + at.ch) * N, N, at.n0, at.cl, ALN || a.nvec);
    const int64_t part = at.b * SEG + at.s;
    dA.store(a.dA_part + (part * a.p.dim + at.ch) * N, N, at.n0, at.cl, ALN || a.nvec);
    float v[4];
    unpack2f(dskip, v[0], v[1]);
    unpack2f(dbias, v[2], v[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int d = kPairs; d < 32; d <<= 1)
            v[e] += __shfl_xor_sync(kFull, v[e], d);
        if (lane < kPairs && (e & 1) < el)
            (e < 2 ? a.dD_part : a.dbias_part)[part * a.p.dim + cb + ec + (e & 1)] = v[e];
    }
}

// rows values `stride` apart, in eight sums that are then added in pairs: the
// loads are in flight together, and rounding grows with the logarithm of what is added.
__device__ __forceinline__ float sum_rows(const float *p, int64_t stride, int64_t rows) {
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    int64_t k = 0;
    for (; k + 16 <= rows; k += 16) {
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            x[e] = p[(k + e) * stride];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            v[e % 8] += x[e];
    }
    if (k + 8 <= rows) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += p[(k + e) * stride];
        k += 8;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (k + e < rows)
            v[e] += p[(k + e) * stride];
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
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
            const float v = t < ssm_len(a, b) ? sum_rows(a.shared + ((g * a.plan.ctiles * B + b) * L + t) * (2 * np) + which * np + s,
                                                         B * L * (2 * np), a.plan.ctiles)
                                              : 0.0f;
            S *to = which ? static_cast<S *>(a.p.dC) + b * a.p.dC_batch + t * a.p.dC_token
                          : static_cast<S *>(a.p.dB) + b * a.p.dB_batch + t * a.p.dB_token;
            Codec<S>::store1(to + g * N + s, v);
        } else if (i < shared + params) {
            const int64_t j = i - shared;
            a.p.dA[j] = sum_rows(a.dA_part + j, params, parts);
        } else {
            const int64_t j = i - shared - params;
            const float v = sum_rows(a.dD_part + j, D, parts), w = sum_rows(a.dbias_part + j, D, parts);
            if (a.p.dD != nullptr)
                a.p.dD[j] = v;
            if (a.p.ddelta_bias != nullptr)
                a.p.ddelta_bias[j] = w;
        }
    }
}

// ---- launches ------------------------------------------------------------------------------
template <class S, int P, bool ALN> static cudaError_t grad_go(const SsmArgs &a, const Launch &L) {
    const int64_t grid = a.p.batch * a.p.groups * a.plan.ctiles * a.plan.segments;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    if (grid > 0) {
        const size_t smem = GradSmem<S, P>::kBytes;
        cudaError_t e = ssm_smem(k_ssm_grad<S, P, ALN>, smem);
        if (e != cudaSuccess)
            return e;
        note_launch();
        if ((e = launch_pdl(k_ssm_grad<S, P, ALN>, (unsigned)grid, kSsmThreads, smem, L.stream, a)) != cudaSuccess)
            return e;
    }
    const int64_t items = a.p.batch * a.p.len * a.p.groups * 2 * a.p.nstate + a.p.dim * a.p.nstate + a.p.dim;
    int64_t jgrid = (items + 255) / 256;
    if (jgrid > 16 * (int64_t)L.sm_count)
        jgrid = 16 * (int64_t)L.sm_count;
    note_launch();
    return launch_pdl(k_ssm_grad_join<S>, (unsigned)jgrid, 256, 0, L.stream, a, 4 * P);
}
template <class S> static cudaError_t grad_states(const SsmArgs &a, const Launch &L) {
#define MT_LANES(P) \
    case P: return a.aligned ? grad_go<S, P, true>(a, L) : grad_go<S, P, false>(a, L)
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
