// mt_ssm_prompt.cuh -- the selective state space scan of whole prompts: the
// carries of the segments, and the forward kernel.
//
// Work split. A lane owns two neighbouring channels with up to 16 of their
// states in registers (K of them; P lanes share a channel pair when there are
// more), so at up to 16 states the sum over states never leaves the lane and a
// channel's step size, gate and output are made where they are used. B and C
// are the same for all channels of a group: a warp widens 8 tokens of them into
// shared memory and reads them back as broadcasts, half a clock per value
// and 64 channels. (A lane of 4 channels x 4 states, the gradient's shape, reads B and C with 4
// addresses a warp, at twice the cost, and needs 12 operations a token for the sum over lanes; it
// measured 347 us for one prompt of 16384 tokens x 2048 channels with 16 states, bf16, where
// this takes 227: carries, chain and forward pass. 16 states of one channel a lane: 291.)
//
// Latency: u, delta, z, B and C of the next 8 tokens are copied into shared memory (cp.async, in
// storage form, so that no register holds them) while 8 are worked on; and the
// exponentials of later tokens do not wait for the recurrence.
#pragma once

#include "mt_ssm.cuh"

namespace mt {

constexpr int kStep = kSsmTile;  // tokens per stage, and per checkpoint
constexpr int kAhead = 4;         // tokens whose step sizes are made together
constexpr int kPromptCtas = 3;    // CTAs an SM: 16 warps at 128 registers measured 294 us against 261 at 12 of 168 (same code)

// ROWS rows of up to `values` <= MOST values each, by 32-bit words: the words that a row's
// live values touch, to dst + row * pitch (16-bit values that start in the middle of a word stay
// there, half a word in). f32 rows are whole words, with zeros where there is nothing.
template <class S, int ROWS, int MOST>
__device__ __forceinline__ void copy_words(uint32_t dst, int pitch, const S *base, int64_t stride, int64_t t0, int left, int values,
                                           int lane) {
    constexpr int kWords = sizeof(S) == 4 ? MOST : MOST / 2 + 1, kEach = 32 / ROWS;  // lanes of a row
    const int t = lane / kEach, w0 = lane % kEach;
    const uintptr_t at = (uintptr_t)(base + (t0 + t) * stride), from = (at & ~(uintptr_t)3) + 4 * w0;
    const uint32_t to = dst + t * pitch + 4 * w0;
    // words of the row from this lane's first on
    const int words = t < left && values > 0 ? (int)((at + values * sizeof(S) + 3 - from) >> 2) : 0;
#pragma unroll
    for (int w = 0; w < kWords; w += kEach) {
        if constexpr (sizeof(S) == 4) {
            if (MOST % kEach == 0 || w + w0 < MOST)
                cp_async_zfill<4>(to + 4 * w, w < words ? (const void *)(from + 4 * w) : (const void *)base, w < words);
        } else {
            if (w < words)
                cp_async_zfill<4>(to + 4 * w, (const void *)(from + 4 * w), true);
        }
    }
}
// How far into its first word row t of a tensor starts, in bytes.
template <class S> __device__ __forceinline__ uint32_t row_skip(const S *base, int64_t stride, int64_t t) {
    if (sizeof(S) == 4)
        return 0u;
    return ((uint32_t)(uintptr_t)base + (uint32_t)t * (uint32_t)stride * (uint32_t)sizeof(S)) & 3u;
}

// A warp's CW channels of kStep tokens in shared memory, in storage form and
// aligned, zeros where there is nothing. Rows whose channels start on a 16-byte
// boundary are copied in 16-byte pieces. Any other row (odd sizes and offsets) is copied as
// the 32-bit words that its live channels touch (a word that holds a live value is inside the
// tensor's memory page) and settle() moves the channels to their places: the
// loop that works on them has one aligned read and no branch either way.
template <class S, int CW> struct Rows8 {
    static constexpr int kPitch = CW * (int)sizeof(S) + 16;
    static constexpr int kBytes = kStep * kPitch;
    static constexpr int kPiece = CW * (int)sizeof(S) < 16 ? CW * (int)sizeof(S) : 16;  // bytes moved as one
    static constexpr int kEach = kPiece / (int)sizeof(S);  // channels of a piece
    static constexpr int kChunks = CW / kEach;             // pieces of a token
    static constexpr int kTokens = 32 / kChunks < kStep ? 32 / kChunks : kStep;  // that a warp moves together
    // the lane's first channel and token of a stage
    static __device__ __forceinline__ int chunk(int lane) { return lane % kChunks * kEach; }
    static __device__ __forceinline__ int token(int lane) { return lane / kChunks; }
    // `at` is where the lane's piece of the stage's first tokens lies; `left` tokens exist
    static __device__ __forceinline__ void fetch16(uint32_t dst, const S *at, int64_t stride, int left, bool in, int lane) {
        const uint32_t to = dst + token(lane) * kPitch + chunk(lane) * (int)sizeof(S);
#pragma unroll
        for (int i = 0; i < kStep / kTokens; ++i) {
            if (kTokens * kChunks == 32 || lane < kTokens * kChunks)
                cp_async_zfill<kPiece>(to + i * kTokens * kPitch, at + i * kTokens * stride, in && token(lane) + i * kTokens < left);
        }
    }
    static __device__ __forceinline__ void fetch_words(uint32_t dst, const S *base, int64_t stride, int64_t t0, int left, int channels,
                                                       int lane) {
        copy_words<S, kStep, CW>(dst, kPitch, base, stride, t0, left, channels, lane);
    }
    // rows that fetch_words copied; the caller syncs the warp before and after
    static __device__ __forceinline__ void settle(char *rows, const S *base, int64_t stride, int64_t t0, int left, int channels,
                                                  int lane) {
        if constexpr (sizeof(S) == 4)
            return;  // whole words, and zeros where there is nothing
        constexpr int kLanes = CW / 2 < 32 ? CW / 2 : 32, kTok = 32 / kLanes;  // a lane a channel pair, kTok tokens together
        constexpr int kEach = (kStep + kTok - 1) / kTok;
        const int c = lane % kLanes * 2;
        S v[kEach][2];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int t = lane / kLanes + i * kTok;
            const S *p = reinterpret_cast<const S *>(rows + (t < kStep ? t : 0) * kPitch + row_skip(base, stride, t0 + t)) + c;
            v[i][0] = t < left && c < channels ? p[0] : S(0.0f);
            v[i][1] = t < left && c + 1 < channels ? p[1] : S(0.0f);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int t = lane / kLanes + i * kTok;
            if (t < kStep) {
                S *to = reinterpret_cast<S *>(rows + t * kPitch) + c;
                to[0] = v[i][0];
                to[1] = v[i][1];
            }
        }
    }
    // channels c, c + 1 (c even) of token t of the stage
    static __device__ __forceinline__ f32x2 read(const char *rows, int t, int c) {
        const char *row = rows + t * kPitch + c * (int)sizeof(S);
        if constexpr (sizeof(S) == 4) {
            return *reinterpret_cast<const f32x2 *>(row);
        } else {
            float a, b;
            Codec<S>::two(*reinterpret_cast<const uint32_t *>(row), a, b);
            return pack2f(a, b);
        }
    }
    static __device__ __forceinline__ void write(char *rows, int t, int c, f32x2 x) {
        char *row = rows + t * kPitch + c * (int)sizeof(S);
        if constexpr (sizeof(S) == 4) {
            *reinterpret_cast<f32x2 *>(row) = x;
        } else {
            float a, b;
            unpack2f(x, a, b);
            *reinterpret_cast<uint32_t *>(row) = Codec<S>::pack2(a, b);
        }
    }
    // tokens left .. kStep - 1 of a stage of delta: -inf, of which softplus (after any bias) makes the step 0 that they
    // take. So they go through softplus where the live tokens have none, too: a 0 here would come out as the bias
    static __device__ __forceinline__ void no_steps(char *rows, int left, int lane) {
        for (int t = left; t < kStep; ++t)
            for (int c = lane; c < CW; c += 32)
                Codec<S>::store1(reinterpret_cast<S *>(rows + t * kPitch) + c, __int_as_float((int)0xff800000u));
    }
    // the rows of the `left` tokens to global memory
    static __device__ __forceinline__ void put16(const char *rows, S *at, int64_t stride, int left, bool in, int lane) {
        const char *from = rows + token(lane) * kPitch + chunk(lane) * (int)sizeof(S);
#pragma unroll
        for (int i = 0; i < kStep / kTokens; ++i)
            if (in && token(lane) + i * kTokens < left && (kTokens * kChunks == 32 || lane < kTokens * kChunks)) {
                using W = typename std::conditional<kPiece == 16, uint4, uint2>::type;
                *reinterpret_cast<W *>(at + i * kTokens * stride) = *reinterpret_cast<const W *>(from + i * kTokens * kPitch);
            }
    }
    static __device__ __forceinline__ void put_each(const char *rows, S *base, int64_t stride, int64_t t0, int left, int channels,
                                                    int lane) {
        constexpr int kRow = CW < 32 ? CW : 32, kTok = 32 / kRow;  // lanes of a token, tokens together
        const int c0 = lane % kRow;
        S *to = base + (t0 + lane / kRow) * stride + c0;
#pragma unroll
        for (int t = lane / kRow; t < kStep; t += kTok) {
#pragma unroll
            for (int c = 0; c < CW; c += kRow)
                if (t < left && c0 + c < channels)
                    to[c] = reinterpret_cast<const S *>(rows + t * kPitch)[c0 + c];
            to += kTok * stride;
        }
    }
};

// K states of a lane's two channels, two neighbouring states a register pair.
template <int K> struct Rows {
    f32x2 v[2][K / 2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int k = 0; k < K / 2; ++k)
                v[c][k] = 0ull;
    }
    __device__ __forceinline__ void load(const float *rows, int64_t nstate, int n0, int cl, bool vec, float scale = 1.0f) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int k = 0; k < K; k += 4) {
                float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (c < cl) {
                    const float *r = rows + c * nstate + n0 + k;
                    if (vec) {
                        if (n0 + k < nstate) {
                            const float4 w = *reinterpret_cast<const float4 *>(r);
                            x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n0 + k + e < nstate)
                                x[e] = r[e];
                    }
                }
                v[c][k / 2] = pack2f(x[0] * scale, x[1] * scale);
                v[c][k / 2 + 1] = pack2f(x[2] * scale, x[3] * scale);
            }
        }
    }
    __device__ __forceinline__ void store(float *rows, int64_t nstate, int n0, int cl, bool vec) const {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (c < cl) {
#pragma unroll
                for (int k = 0; k < K; k += 4) {
                    float x[4];
                    unpack2f(v[c][k / 2], x[0], x[1]);
                    unpack2f(v[c][k / 2 + 1], x[2], x[3]);
                    float *r = rows + c * nstate + n0 + k;
                    if (vec) {
                        if (n0 + k < nstate)
                            *reinterpret_cast<float4 *>(r) = make_float4(x[0], x[1], x[2], x[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n0 + k + e < nstate)
                                r[e] = x[e];
                    }
                }
            }
        }
    }
};

// Where a warp's work lies.
template <int K, int P> struct PromptPlace {
    static constexpr int CW = 32 * 2 / P, NP = K * P;
    int64_t b, s, g, ch, cw;  // sequence, segment, group; first channel of the lane and of the warp
    int n0, cl, channels;     // first state of the lane, its live channels and the warp's
    __device__ __forceinline__ void set(const SsmArgs &a, int64_t w, int64_t segments, int64_t first, int lane) {
        const int64_t ct = w % a.plan.ctiles;
        w /= a.plan.ctiles;
        g = w % a.p.groups;
        w /= a.p.groups;
        s = w % segments + first;
        b = w / segments;
        const int64_t c = ct * CW + (lane / P) * 2, left = a.gdim - c, all = a.gdim - ct * CW;
        n0 = (lane % P) * K;
        cl = left <= 0 ? 0 : left >= 2 ? 2 : (int)left;
        channels = all < CW ? (int)all : CW;
        ch = g * a.gdim + c;
        cw = g * a.gdim + ct * CW;
    }
};

// B or C of kStep tokens: copied in storage form (in vectors of four states,
// which each lane widens itself, or by words), then widened to f32.
template <class S, int NP> struct States8 {
    static constexpr int kVecs = kStep * NP / 4, kPer = (kVecs + 31) / 32;
    static constexpr int kPitch = NP * (int)sizeof(S) + 8;  // of a token copied by words
    static constexpr int kBytes = (kStep * kPitch + 15) / 16 * 16;
    static __device__ __forceinline__ int live(int left, int t, int s, int nstate) {
        const int n = t < left ? nstate - s : 0;
        return n <= 0 ? 0 : n > 4 ? 4 : n;
    }
    static __device__ __forceinline__ void fetch(uint32_t dst, const S *base, int64_t stride, int64_t t0, int left, int nstate,
                                                 int lane, bool vec) {
        if (!vec) {
            copy_words<S, kStep, NP>(dst, kPitch, base, stride, t0, left, nstate, lane);
            return;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = 32 * i + lane, t = v / (NP / 4), s = v % (NP / 4) * 4;
            const bool in = live(left, t, s, nstate) == 4;
            if (v < kVecs)
                cp_async_zfill<4 * sizeof(S)>(dst + v * 4 * (int)sizeof(S), in ? base + (t0 + t) * stride + s : base, in);
        }
    }
    // after the copies have arrived: a warp's, and its lanes are in step, unless vec
    static __device__ __forceinline__ void widen(float *to, const char *raw, const S *base, int64_t stride, int64_t t0, int left,
                                                 int nstate, int lane, bool vec) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = 32 * i + lane, t = v / (NP / 4), s = v % (NP / 4) * 4;
            if (v < kVecs) {
                Raw4<S> w;
                if (vec) {
                    w.load(reinterpret_cast<const S *>(raw) + 4 * v, true, 4);
                } else {
                    const char *row = raw + t * kPitch + row_skip(base, stride, t0 + t);
                    w.load(reinterpret_cast<const S *>(row) + s, false, live(left, t, s, nstate));
                }
                float x[4];
                w.widen(x);
                *reinterpret_cast<float4 *>(to + 4 * v) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
    }
};

// Bytes of shared memory per warp: two stages of 3 activations and `shared` of
// B and C in storage form, and those widened.
template <class S, int K, int P, int SHARED> struct PromptSmem {
    using R = Rows8<S, 32 * 2 / P>;
    using B = States8<S, K * P>;
    static constexpr int kStage = 3 * R::kBytes + SHARED * B::kBytes;
    static constexpr int kWide = SHARED * kStep * K * P * 4;
    static constexpr int kBytes = 2 * kStage + kWide;
};

// Two channels' values of a parameter; 0 where there is none.
__device__ __forceinline__ f32x2 pair_of(const float *p, int64_t ch, int cl) {
    return pack2f(p != nullptr && cl > 0 ? p[ch] : 0.0f, p != nullptr && cl > 1 ? p[ch + 1] : 0.0f);
}

// ---- carries of the segments ---------------------------------------------------------
// Forward: the state that a segment leaves from zero (segment 0: from the
// first state). REV: the same of the adjoint, r = a (r + C g) from the last token
// down. One exponential and three multiply-adds a pair; no output.
template <class S, int K, int P, bool REV, bool ALN>
__global__ void __launch_bounds__(kSsmThreads, kPromptCtas) k_ssm_carry(const __grid_constant__ SsmArgs a, int64_t warps) {
    using Q = PromptPlace<K, P>;
    using M = PromptSmem<S, K, P, 1>;
    using R = typename M::R;
    using St = typename M::B;
    constexpr int NP = Q::NP;
    extern __shared__ float4 smem4[];
    const int lane = threadIdx.x & 31;
    char *stage = reinterpret_cast<char *>(smem4) + (threadIdx.x >> 5) * M::kBytes;
    float *sb = reinterpret_cast<float *>(stage + 2 * M::kStage);
    pdl_prologue();
    const int64_t w = (int64_t)blockIdx.x * kSsmWarps + (threadIdx.x >> 5);
    if (w >= warps)
        return;
    Q at;
    at.set(a, w, a.plan.segments - 1, REV ? 1 : 0, lane);  // the last (REV: first) segment's carry goes nowhere
    const int64_t N = a.p.nstate, n = ssm_len(a, at.b);
    const int64_t begin = at.s * a.plan.seg_len;
    const int64_t end = begin + a.plan.seg_len < n ? begin + a.plan.seg_len : n;
    Rows<K> A, h;
    A.load(a.p.A + at.ch * N, N, at.n0, at.cl, ALN || a.nvec, kLog2e);
    h.zero();
    if (!REV && at.s == 0) {
        const int64_t slot = ssm_slot(a, at.b);
        if (a.p.carry_in && a.p.state != nullptr && slot >= 0)
            h.load(a.p.state + (slot * a.p.dim + at.ch) * N, N, at.n0, at.cl, ALN || a.nvec);
        // the state is written by the next launch's last segment while its first
        // one starts: that one reads this copy, in the place of the last carry
        const int64_t spare = (at.b * a.plan.segments + a.plan.segments - 1) * a.p.dim + at.ch;
        h.store(a.carry + spare * N, N, at.n0, at.cl, ALN || a.nvec);
    }
    f32x2 sum = 0ull;
    const f32x2 bias = pair_of(a.p.delta_bias, at.ch, at.cl);
    const S *dp = static_cast<const S *>(a.p.delta) + at.b * a.p.delta_batch + at.cw;
    const S *xp = static_cast<const S *>(REV ? a.p.dout : a.p.u) + at.b * (REV ? a.p.dout_batch : a.p.u_batch) + at.cw;
    const S *zp = static_cast<const S *>(a.p.z) + at.b * a.p.z_batch + at.cw;
    const S *bp = static_cast<const S *>(REV ? a.p.C : a.p.B) + at.b * (REV ? a.p.C_batch : a.p.B_batch) + at.g * N;
    const int64_t dt_ = a.p.delta_token, zt = a.p.z_token, xt = REV ? a.p.dout_token : a.p.u_token, bt = REV ? a.p.C_token : a.p.B_token;
    const bool gated = REV && a.p.z != nullptr, softplus = a.p.softplus;
    const int steps = end > begin ? (int)((end - begin + kStep - 1) / kStep) : 0;
    const int64_t from = begin + (REV && steps > 0 ? (int64_t)(steps - 1) * kStep : 0);  // the first stage's first token
    const bool in = R::chunk(lane) < at.channels;
    const int64_t lane0 = in ? R::chunk(lane) : 0, lane_t = from + R::token(lane);
    const S *d16 = dp + lane_t * dt_ + lane0, *x16 = xp + lane_t * xt + lane0, *z16 = zp + lane_t * zt + lane0;
    const auto fetch = [&](int k, int64_t t0) {
        const int left = end - t0 < kStep ? (int)(end - t0) : kStep;
        const uint32_t to = smem_addr(stage) + (k & 1) * M::kStage;
        if (ALN) {
            R::fetch16(to, d16, dt_, left, in, lane);
            R::fetch16(to + R::kBytes, x16, xt, left, in, lane);
            if (gated)
                R::fetch16(to + 2 * R::kBytes, z16, zt, left, in, lane);
            constexpr int kBy = REV ? -kStep : kStep;
            d16 += kBy * dt_;
            x16 += kBy * xt;
            z16 += kBy * zt;
        } else {
            R::fetch_words(to, dp, dt_, t0, left, at.channels, lane);
            R::fetch_words(to + R::kBytes, xp, xt, t0, left, at.channels, lane);
            if (gated)
                R::fetch_words(to + 2 * R::kBytes, zp, zt, t0, left, at.channels, lane);
        }
        St::fetch(to + 3 * R::kBytes, bp, bt, t0, left, (int)N, lane, ALN || a.bvec);
        cp_async_commit();
    };
    if (steps > 0)
        fetch(0, from);
    const int cq = (lane / P) * 2;
    int64_t t0 = from;
    for (int k = 0; k < steps; ++k, t0 += REV ? -kStep : kStep) {
        char *raw = stage + (k & 1) * M::kStage;
        cp_async_wait_all();
        __syncwarp();  // everyone's copies are here, and nobody reads the other stage any more
        if (k + 1 < steps)
            fetch(k + 1, REV ? t0 - kStep : t0 + kStep);
        const int left = end - t0 < kStep ? (int)(end - t0) : kStep;
        if (!ALN) {
            R::settle(raw, dp, dt_, t0, left, at.channels, lane);
            R::settle(raw + R::kBytes, xp, xt, t0, left, at.channels, lane);
            if (gated)
                R::settle(raw + 2 * R::kBytes, zp, zt, t0, left, at.channels, lane);
            __syncwarp();
        }
        if (left < kStep)
            R::no_steps(raw, left, lane);
        St::widen(sb, raw + 3 * R::kBytes, bp, bt, t0, left, (int)N, lane, ALN || a.bvec);
        __syncwarp();
#pragma unroll
        for (int ii = 0; ii < kStep; ii += kAhead) {
            const int i = REV ? kStep - kAhead - ii : ii;
            f32x2 d[kAhead], x[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                d[j] = add2f(R::read(raw, i + j, cq), bias);
                x[j] = R::read(raw + R::kBytes, i + j, cq);
            }
            // chosen, not branched on: a branch would keep one group's work from the next one's
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                d[j] = choose_2f(softplus || i + j >= left, softplus_2f(d[j]), d[j]);
            if (REV) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const f32x2 z = R::read(raw + 2 * R::kBytes, i + j, cq);
                    x[j] = choose_2f(gated, mul2f(x[j], mul2f(z, sigmoid_2f(z))), x[j]);
                }
            }
            const float *row = sb + i * NP + at.n0;
#pragma unroll
            for (int jj = 0; jj < kAhead; ++jj) {
                const int j = REV ? kAhead - 1 - jj : jj;
                sum = add2f(sum, d[j]);
                float dc[2], xc[2];
                unpack2f(d[j], dc[0], dc[1]);
                unpack2f(REV ? x[j] : mul2f(d[j], x[j]), xc[0], xc[1]);
                const f32x2 d2[2] = {both(dc[0]), both(dc[1])}, x2[2] = {both(xc[0]), both(xc[1])};
#pragma unroll
                for (int q = 0; q < K / 4; ++q) {
                    f32x2 b[2];
                    lds_pairs(row + j * NP + 4 * q, b[0], b[1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            f32x2 &hv = h.v[c][2 * q + e];
                            const f32x2 dec = ex2_2f(exponent2f(d2[c], A.v[c][2 * q + e]));
                            hv = REV ? mul2f(dec, fma2f(x2[c], b[e], hv)) : fma2f(dec, hv, mul2f(x2[c], b[e]));
                        }
                    }
                }
            }
        }
    }
    const int64_t row = (at.b * a.plan.segments + at.s) * a.p.dim + at.ch;
    h.store(a.carry + row * N, N, at.n0, at.cl, ALN || a.nvec);
    float s[2];
    unpack2f(sum, s[0], s[1]);
    if (lane % P == 0)
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (c < at.cl)
                a.decay[row + c] = s[c];
}

// Carries to first states: each carry is replaced by the state (REV: the adjoint)
// that its segment starts from. A lane holds V states of a channel over kChain segments, whose
// loads are all in flight at once, and up to 16 warps of a CTA hold the segments after one another: each
// combines its own, and goes over the sums of those before it, so the loads of 128
// segments are waited for once. 9 us (caches empty) for 8 sequences of 7 segments of 65536 states; a lane that
// walked down all segments of one state took 30, more in the addresses than in the sums.
constexpr int kChain = 8, kChainMost = 16;
struct ChainPlan {
    int chunks, lanes;  // of a CTA: groups of kChain segments, and lanes of a group
};
static inline ChainPlan chain_plan(int64_t segments) {
    int c = 1;
    while (c < kChainMost && (int64_t)c * kChain < segments)
        c *= 2;
    return {c, c < 8 ? 256 / c : 32};
}
template <int V> __device__ __forceinline__ void get_states(const float *p, float (&x)[V]) {
    if constexpr (V == 4)
        lds4(p, x);
    else
        x[0] = *p;
}
template <int V> __device__ __forceinline__ void put_states(float *p, const float (&x)[V]) {
    if constexpr (V == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else
        *p = x[0];
}
template <bool REV, int V>
__global__ void __launch_bounds__(32 * kChainMost) k_ssm_chain(const __grid_constant__ SsmArgs a, int lanes, int chunks) {
    __shared__ float s_h[32 * kChainMost * V], s_sum[32 * kChainMost];
    pdl_prologue();
    const int chunk = threadIdx.x / lanes, x = threadIdx.x - chunk * lanes;
    const int64_t per = a.p.dim * a.p.nstate, S = a.plan.segments, mine = ((int64_t)blockIdx.x * lanes + x) * V;
    const bool in = mine < per;
    const int64_t e = in ? mine : 0, ch = per <= 0xffffffffll ? (uint32_t)e / (uint32_t)a.p.nstate : e / a.p.nstate;
    const int64_t by = REV ? -per : per, sum_by = REV ? -a.p.dim : a.p.dim;
    float A[V];
    get_states<V>(a.p.A + e, A);
#pragma unroll
    for (int v = 0; v < V; ++v)
        A[v] *= kLog2e;
    for (int64_t b = blockIdx.y; b < a.p.batch; b += gridDim.y) {
        float *c = a.carry + (b * S + (REV ? S - 1 : 0)) * per + e;
        const float *sum = a.decay + (b * S + (REV ? S - 1 : 0)) * a.p.dim + ch;
        // forward: segment 0 starts from the copy in the last place, and its carry already holds it
        float h[V] = {};
        if (!REV)
            get_states<V>(c + (S - 1) * per, h);
        else if (a.p.dfinal != nullptr)
            get_states<V>(a.p.dfinal + b * per + e, h);
        for (int64_t first = 0; first < S; first += (int64_t)chunks * kChain) {
            const int64_t j0 = first + chunk * kChain;
            const int live = S - 1 - j0 < kChain ? (int)(S - 1 - j0) : kChain;  // the last one's carry goes nowhere
            float next[kChain][V], dec[kChain];
#pragma unroll
            for (int k = 0; k < kChain; ++k) {
                dec[k] = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    next[k][v] = 0.0f;
                if (k < live) {
                    get_states<V>(c + (j0 + k) * by, next[k]);
                    dec[k] = sum[(j0 + k) * sum_by];
                }
            }
            const auto advance = [&](int k) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    h[v] = !REV && k == 0 && j0 == 0 ? next[k][v] : fmaf(ex2f(A[v] * dec[k]), h[v], next[k][v]);
            };
            float past[V];  // the state after all of the CTA's chunks
            if (chunks > 1) {
                float all = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    past[v] = h[v];
                    h[v] = chunk == 0 ? h[v] : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < kChain; ++k) {
                    advance(k);
                    all += dec[k];
                }
#pragma unroll
                for (int v = 0; v < V; ++v)
                    s_h[v * lanes * chunks + threadIdx.x] = h[v];
                s_sum[threadIdx.x] = all;
                __syncthreads();
                for (int i = 0; i < chunks; ++i) {
                    const float d = s_sum[i * lanes + x];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (i == chunk)
                            h[v] = past[v];
                        const float y = s_h[v * lanes * chunks + i * lanes + x];
                        past[v] = i == 0 ? y : fmaf(ex2f(A[v] * d), past[v], y);
                    }
                }
                __syncthreads();  // the sums are read, and every lane has the copy in the last place
            }
#pragma unroll
            for (int k = 0; k < kChain; ++k) {
                if (in && k <= live)
                    put_states<V>(c + (j0 + k) * by, h);
                advance(k);
            }
            if (chunks > 1) {  // one chunk alone takes all segments in one turn
#pragma unroll
                for (int v = 0; v < V; ++v)
                    h[v] = past[v];
            }
        }
    }
}

// ---- forward -----------------------------------------------------------------------------
template <class S, int K, int P, bool ALN>
__global__ void __launch_bounds__(kSsmThreads, kPromptCtas) k_ssm(const __grid_constant__ SsmArgs a, int64_t warps) {
    using Q = PromptPlace<K, P>;
    constexpr int NP = Q::NP;
    using M = PromptSmem<S, K, P, 2>;
    using R = typename M::R;
    using St = typename M::B;
    extern __shared__ float4 smem4[];
    const int lane = threadIdx.x & 31;
    char *stage = reinterpret_cast<char *>(smem4) + (threadIdx.x >> 5) * M::kBytes;
    float *sb = reinterpret_cast<float *>(stage + 2 * M::kStage), *sc = sb + kStep * NP;
    pdl_prologue();
    const int64_t w = (int64_t)blockIdx.x * kSsmWarps + (threadIdx.x >> 5);
    if (w >= warps)
        return;
    Q at;
    at.set(a, w, a.plan.segments, 0, lane);
    const int64_t N = a.p.nstate;
    const int64_t slot = ssm_slot(a, at.b);
    const bool active = slot >= 0 || a.p.state == nullptr;
    const int64_t begin = at.s * a.plan.seg_len;
    const int64_t stop = begin + a.plan.seg_len < a.p.len ? begin + a.plan.seg_len : a.p.len;
    const int64_t n = active ? ssm_len(a, at.b) : 0;
    const int64_t end = n < stop ? n : stop;
    float *state = a.p.state != nullptr && active ? a.p.state + (slot * a.p.dim + at.ch) * N : nullptr;
    Rows<K> A, h;
    A.load(a.p.A + at.ch * N, N, at.n0, at.cl, ALN || a.nvec, kLog2e);
    h.zero();
    if (a.plan.segments > 1)
        h.load(a.carry + ((at.b * a.plan.segments + at.s) * a.p.dim + at.ch) * N, N, at.n0, at.cl, ALN || a.nvec);
    else if (a.p.carry_in && state != nullptr)
        h.load(state, N, at.n0, at.cl, ALN || a.nvec);
    const f32x2 bias = pair_of(a.p.delta_bias, at.ch, at.cl), skip = pair_of(a.p.D, at.ch, at.cl);
    const S *dp = static_cast<const S *>(a.p.delta) + at.b * a.p.delta_batch + at.cw;
    const S *up = static_cast<const S *>(a.p.u) + at.b * a.p.u_batch + at.cw;
    const S *zp = static_cast<const S *>(a.p.z) + at.b * a.p.z_batch + at.cw;
    const S *bp = static_cast<const S *>(a.p.B) + at.b * a.p.B_batch + at.g * N;
    const S *cp = static_cast<const S *>(a.p.C) + at.b * a.p.C_batch + at.g * N;
    S *op = static_cast<S *>(a.p.out) + at.b * a.p.out_batch + at.cw;
    const bool gated = a.p.z != nullptr, softplus = a.p.softplus;
    const bool writer = lane % P == 0;  // one of the lanes of a channel pair keeps its output
    const int steps = end > begin ? (int)((end - begin + kStep - 1) / kStep) : 0;
    const bool in = R::chunk(lane) < at.channels;
    const int64_t lane0 = in ? R::chunk(lane) : 0, lane_t = begin + R::token(lane);
    const S *d16 = dp + lane_t * a.p.delta_token + lane0, *u16 = up + lane_t * a.p.u_token + lane0;
    const S *z16 = zp + lane_t * a.p.z_token + lane0;
    S *o16 = op + lane_t * a.p.out_token + lane0;
    const auto fetch = [&](int k, int64_t t0) {
        const int left = end - t0 < kStep ? (int)(end - t0) : kStep;
        const uint32_t to = smem_addr(stage) + (k & 1) * M::kStage;
        if (ALN) {
            R::fetch16(to, d16, a.p.delta_token, left, in, lane);
            R::fetch16(to + R::kBytes, u16, a.p.u_token, left, in, lane);
            if (gated)
                R::fetch16(to + 2 * R::kBytes, z16, a.p.z_token, left, in, lane);
            d16 += kStep * a.p.delta_token;
            u16 += kStep * a.p.u_token;
            z16 += kStep * a.p.z_token;
        } else {
            R::fetch_words(to, dp, a.p.delta_token, t0, left, at.channels, lane);
            R::fetch_words(to + R::kBytes, up, a.p.u_token, t0, left, at.channels, lane);
            if (gated)
                R::fetch_words(to + 2 * R::kBytes, zp, a.p.z_token, t0, left, at.channels, lane);
        }
        St::fetch(to + 3 * R::kBytes, bp, a.p.B_token, t0, left, (int)N, lane, ALN || a.bvec);
        St::fetch(to + 3 * R::kBytes + St::kBytes, cp, a.p.C_token, t0, left, (int)N, lane, ALN || a.bvec);
        cp_async_commit();
    };
    if (steps > 0)
        fetch(0, begin);
    const int cq = (lane / P) * 2;
    int64_t t0 = begin;
    for (int k = 0; k < steps; ++k, t0 += kStep) {
        char *raw = stage + (k & 1) * M::kStage;
        if (a.p.checkpoints != nullptr)
            h.store(a.p.checkpoints + ((at.b * a.ntiles + t0 / kStep) * a.p.dim + at.ch) * N, N, at.n0, at.cl, ALN || a.nvec);
        cp_async_wait_all();
        __syncwarp();  // everyone's copies are here, and nobody reads the other stage any more
        if (k + 1 < steps)
            fetch(k + 1, t0 + kStep);
        const int left = end - t0 < kStep ? (int)(end - t0) : kStep;
        if (!ALN) {
            R::settle(raw, dp, a.p.delta_token, t0, left, at.channels, lane);
            R::settle(raw + R::kBytes, up, a.p.u_token, t0, left, at.channels, lane);
            if (gated)
                R::settle(raw + 2 * R::kBytes, zp, a.p.z_token, t0, left, at.channels, lane);
            __syncwarp();
        }
        if (left < kStep)
            R::no_steps(raw, left, lane);
        St::widen(sb, raw + 3 * R::kBytes, bp, a.p.B_token, t0, left, (int)N, lane, ALN || a.bvec);
        St::widen(sc, raw + 3 * R::kBytes + St::kBytes, cp, a.p.C_token, t0, left, (int)N, lane, ALN || a.bvec);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kStep; i += kAhead) {
            f32x2 d[kAhead], u[kAhead], y[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                d[j] = add2f(R::read(raw, i + j, cq), bias);
                u[j] = R::read(raw + R::kBytes, i + j, cq);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                d[j] = choose_2f(softplus || i + j >= left, softplus_2f(d[j]), d[j]);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                f32x2 acc[2] = {0ull, 0ull};
                const float *rowb = sb + (i + j) * NP + at.n0, *rowc = sc + (i + j) * NP + at.n0;
                float dc[2], xc[2];
                unpack2f(d[j], dc[0], dc[1]);
                unpack2f(mul2f(d[j], u[j]), xc[0], xc[1]);
                const f32x2 d2[2] = {both(dc[0]), both(dc[1])}, x2[2] = {both(xc[0]), both(xc[1])};
#pragma unroll
                for (int q = 0; q < K / 4; ++q) {
                    f32x2 bb[2], cc[2];
                    lds_pairs(rowb + 4 * q, bb[0], bb[1]);
                    lds_pairs(rowc + 4 * q, cc[0], cc[1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            f32x2 &hv = h.v[c][2 * q + e];
                            hv = fma2f(ex2_2f(exponent2f(d2[c], A.v[c][2 * q + e])), hv, mul2f(x2[c], bb[e]));
                            acc[c] = fma2f(cc[e], hv, acc[c]);
                        }
                    }
                }
                float s[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float lo, hi;
                    unpack2f(acc[c], lo, hi);
                    s[c] = lo + hi;
#pragma unroll
                    for (int m = 1; m < P; m <<= 1)
                        s[c] += __shfl_xor_sync(kFull, s[c], m);
                }
                y[j] = fma2f(skip, u[j], pack2f(s[0], s[1]));
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const f32x2 z = R::read(raw + 2 * R::kBytes, i + j, cq);
                y[j] = choose_2f(gated, mul2f(y[j], mul2f(z, sigmoid_2f(z))), y[j]);
            }
            // into the place of delta, which every lane of the pair has used
            if (P == 1 || writer) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    R::write(raw, i + j, cq, y[j]);
            }
        }
        __syncwarp();
        if (ALN) {
            R::put16(raw, o16, a.p.out_token, left, in, lane);
            o16 += kStep * a.p.out_token;
        } else {
            R::put_each(raw, op, a.p.out_token, t0, left, at.channels, lane);
        }
    }
    for (int64_t t = begin > end ? begin : end; t < stop; ++t)  // past the sequence's end
        for (int c = lane; c < at.channels; c += 32)
            Codec<S>::store1(op + t * a.p.out_token + c, 0.0f);
    if (state != nullptr && at.s == a.plan.segments - 1)
        h.store(state, N, at.n0, at.cl, ALN || a.nvec);
}

// ---- launches ------------------------------------------------------------------------------
template <class K> static cudaError_t ssm_smem(K kernel, size_t bytes) {
    return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) : cudaSuccess;
}

template <class S, int K, int P, bool REV, bool ALN> static cudaError_t carry_go(const SsmArgs &a, const Launch &L) {
    SsmArgs c = a;
    c.plan.ctiles = (a.gdim + 64 / P - 1) / (64 / P);
    const int64_t warps = a.p.batch * a.p.groups * c.plan.ctiles * (a.plan.segments - 1);
    const ChainPlan at = chain_plan(a.plan.segments);
    const int64_t each = a.nvec ? 4 : 1;
    const int64_t grid = (warps + kSsmWarps - 1) / kSsmWarps, chain = (a.p.dim * a.p.nstate + at.lanes * each - 1) / (at.lanes * each);
    if (grid > INT32_MAX || chain > INT32_MAX)
        return cudaErrorInvalidValue;
    const size_t smem = kSsmWarps * PromptSmem<S, K, P, 1>::kBytes;
    cudaError_t e = ssm_smem(k_ssm_carry<S, K, P, REV, ALN>, smem);
    if (e != cudaSuccess)
        return e;
    note_launch();
    e = launch_pdl(k_ssm_carry<S, K, P, REV, ALN>, (unsigned)grid, kSsmThreads, smem, L.stream, c, warps);
    if (e != cudaSuccess)
        return e;
    note_launch();
    return launch_pdl_2d(a.nvec ? k_ssm_chain<REV, 4> : k_ssm_chain<REV, 1>, dim3((unsigned)chain, (unsigned)(a.p.batch < 65535 ? a.p.batch : 65535)),
                         (unsigned)(at.lanes * at.chunks), L.stream, a, at.lanes, at.chunks);
}
template <class S, int K, int P, bool ALN> static cudaError_t prompt_go(const SsmArgs &a, const Launch &L) {
    cudaError_t e;
    if (a.plan.segments > 1 && (e = carry_go<S, K, P, false, ALN>(a, L)) != cudaSuccess)
        return e;
    const int64_t warps = a.p.batch * a.p.groups * a.plan.ctiles * a.plan.segments;
    const int64_t grid = (warps + kSsmWarps - 1) / kSsmWarps;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    const size_t smem = kSsmWarps * PromptSmem<S, K, P, 2>::kBytes;
    if ((e = ssm_smem(k_ssm<S, K, P, ALN>, smem)) != cudaSuccess)
        return e;
    note_launch();
    return launch_pdl(k_ssm<S, K, P, ALN>, (unsigned)grid, kSsmThreads, smem, L.stream, a, warps);
}

// by the number of states, rounded up to what a lane (and P lanes) hold
#define MT_BY_STATES(n, f)              \
    if ((n) <= 4) return f(4, 1);       \
    if ((n) <= 8) return f(8, 1);       \
    if ((n) <= 16) return f(16, 1);     \
    if ((n) <= 32) return f(16, 2);     \
    if ((n) <= 64) return f(16, 4);     \
    return f(16, 8)
template <class S> static cudaError_t prompt_states(const SsmArgs &a, const Launch &L) {
#define MT_GO(K, P) (a.aligned ? prompt_go<S, K, P, true>(a, L) : prompt_go<S, K, P, false>(a, L))
    MT_BY_STATES(a.p.nstate, MT_GO);
#undef MT_GO
}
template <class S> static cudaError_t adjoint_carries(const SsmArgs &a, const Launch &L) {
#define MT_GO(K, P) (a.aligned ? carry_go<S, K, P, true, true>(a, L) : carry_go<S, K, P, true, false>(a, L))
    MT_BY_STATES(a.p.nstate, MT_GO);
#undef MT_GO
}
#undef MT_BY_STATES

}  // namespace mt
