// mt_conv.cu -- the short causal convolution of each channel over the tokens,
// with bias and SiLU, its gradient, and its single-token form.
//
//   p_t = bias + sum_{k < W} w_k x_{t-W+1+k},  out_t = p_t or p_t * sigmoid(p_t)
//
// where the W-1 inputs before token 0 come from a state (or are 0) and the
// last W-1 inputs are left in it. 2W + 5 operations per value of 2 or 4 bytes
// read and written: bound by bytes. A lane owns four channels (neighbours,
// moved as one, or 32 apart where the rows fit no vector) and walks down a span of
// tokens with the W-1 inputs before the present one in registers, so an input is
// read once, plus W-1 per span; products are made for two channels at a time.
#include <type_traits>

#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

constexpr int kConvThreads = 128;

// Four values of one lane in storage form: neighbouring channels moved as one
// (ALN), or channels 32 apart (rows that no vector fits), of which `live` exist.
template <class S, bool ALN> struct Quad {
    Raw4<S> w;
    __device__ __forceinline__ void load(const S *p, int live) {
        if constexpr (ALN) {
            w.load(p, true, 4);
        } else {
            S v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = e < live ? p[32 * e] : S(0.0f);
            w.w = *reinterpret_cast<typename VecOf<S, 4>::T *>(v);
        }
    }
    __device__ __forceinline__ void zero() {
        if constexpr (sizeof(S) == 4)
            w.w = make_uint4(0u, 0u, 0u, 0u);
        else
            w.w = make_uint2(0u, 0u);
    }
    __device__ __forceinline__ void store(S *p, int live) const {
        if constexpr (ALN) {
            *reinterpret_cast<typename VecOf<S, 4>::T *>(p) = w.w;
        } else {
            const S *v = reinterpret_cast<const S *>(&w.w);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < live)
                    p[32 * e] = v[e];
        }
    }
    __device__ __forceinline__ void widen(f32x2 (&x)[2]) const {
        float v[4];
        w.widen(v);
        x[0] = pack2f(v[0], v[1]);
        x[1] = pack2f(v[2], v[3]);
    }
    __device__ __forceinline__ void narrow(const f32x2 (&x)[2]) {
        float v[4];
        unpack2f(x[0], v[0], v[1]);
        unpack2f(x[1], v[2], v[3]);
        w.w = narrow4<S>(v);
    }
};
// Tokens on their way to a lane: GROUPS groups of EACH quads, asked for in
// order and taken in order. Quads that are vectors are copied into the lane's
// own places in shared memory, so no register waits for them and the whole ring is in flight;
// the others are loaded one group ahead.
template <class S, bool ALN, int GROUPS, int EACH> struct Ring {
    static constexpr int kBytes = ALN ? GROUPS * EACH * 4 * (int)sizeof(S) : 0;  // of a lane
    char *mine;  // the lane's place in the first quad; quads lie 32 lanes apart
    Quad<S, ALN> next[ALN ? 1 : EACH];
    __device__ __forceinline__ void set(char *warp, int lane) { mine = warp + lane * 4 * (int)sizeof(S); }
    // ALL: all EACH tokens exist
    template <bool ALL> __device__ __forceinline__ void ask(int group, const S *from, int64_t stride, int left, int live) {
        if constexpr (ALN) {
            const uint32_t to = smem_addr(mine) + group % GROUPS * (EACH * 32 * 4 * (int)sizeof(S));
#pragma unroll
            for (int j = 0; j < EACH; ++j) {
                const bool in = ALL || j < left;
                cp_async_zfill<4 * sizeof(S)>(to + j * 32 * 4 * (int)sizeof(S), in ? from + j * stride : from, in);
            }
            cp_async_commit();
        } else {
#pragma unroll
            for (int j = 0; j < EACH; ++j) {
                next[j].zero();
                if (ALL || j < left)
                    next[j].load(from + j * stride, live);
            }
        }
    }
    __device__ __forceinline__ void take(int group, Quad<S, ALN> (&v)[EACH]) {
        if constexpr (ALN) {
#pragma unroll
            for (int j = 0; j < EACH; ++j)
                v[j].w.w = *reinterpret_cast<const typename VecOf<S, 4>::T *>(mine + (group % GROUPS * EACH + j) * 32 * 4 * (int)sizeof(S));
        } else {
#pragma unroll
            for (int j = 0; j < EACH; ++j)
                v[j] = next[j];
        }
    }
};

// A lane's first channel, how many it has, and the distance between them.
template <bool ALN> struct ConvLane {
    int64_t c;
    int live;
    __device__ __forceinline__ void set(int64_t group, int lane, int64_t dim) {  // 128 channels a warp
        c = group * 128 + (ALN ? 4 * lane : lane);
        if (ALN)
            live = c < dim ? 4 : 0;  // dim is a multiple of four
        else
            live = c >= dim ? 0 : (dim - c + 31) / 32 < 4 ? (int)((dim - c + 31) / 32) : 4;
    }
    static __device__ __forceinline__ int step(int e) { return ALN ? e : 32 * e; }
};

// Weights and bias are f32 or the activations' type.
template <class S> __device__ __forceinline__ float param(const void *p, int64_t i, bool f32) {
    return f32 ? static_cast<const float *>(p)[i] : Codec<S>::load1(static_cast<const S *>(p) + i);
}

struct ConvDims {
    int64_t batch, len, dim, width, nslots;
    int64_t xb, xt, ob, ot, gb, gt, db, dt;  // strides: x, out, dout, dx
    int silu, carry_in, wf32;
    const int32_t *slots, *lens;
    const void *weight, *bias;
};

static ConvDims conv_dims(const mt_conv_args &a) {
    ConvDims d;
    d.batch = a.batch; d.len = a.len; d.dim = a.dim; d.width = a.width; d.nslots = a.nslots;
    d.xb = a.x_batch; d.xt = a.x_token; d.ob = a.out_batch; d.ot = a.out_token;
    d.gb = a.dout_batch; d.gt = a.dout_token; d.db = a.dx_batch; d.dt = a.dx_token;
    d.silu = a.silu != 0; d.carry_in = a.carry_in != 0; d.wf32 = a.wdtype == MT_F32;
    d.slots = a.slots; d.lens = a.lens; d.weight = a.weight; d.bias = a.bias;
    return d;
}

// The state's row of sequence b; -1 where it has none.
__device__ __forceinline__ int64_t slot_of(const int32_t *slots, int64_t nslots, int64_t b) {
    const int64_t s = slots != nullptr ? (int64_t)slots[b] : b;
    return s >= 0 && s < nslots ? s : -1;
}
__device__ __forceinline__ int64_t live_len(const int32_t *lens, int64_t len, int64_t b) {
    const int64_t n = lens != nullptr ? (int64_t)lens[b] : len;
    return n < 0 ? 0 : n > len ? len : n;
}

// x at token t of a sequence (t >= -(W-1)): the state's before token 0, zeros
// from the sequence's end on (what is stored there is not read).
template <class S, bool ALN>
__device__ __forceinline__ void input_at(Quad<S, ALN> &v, const S *x, const S *state, const ConvDims &d, int64_t t, int64_t n,
                                         int live) {
    if (t < 0) {
        if (state != nullptr)
            v.load(state + (t + d.width - 1) * d.dim, live);
        else
            v.zero();
    } else if (t < n) {
        v.load(x + t * d.xt, live);
    } else {
        v.zero();
    }
}
// weights and bias of a lane's channels, two channels a register pair
template <class S, bool ALN, int W>
__device__ __forceinline__ void conv_params(const ConvDims &d, const ConvLane<ALN> &at, f32x2 (&w)[W][2], f32x2 (&bias)[2]) {
    float b[4], k4[W][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t c = at.c + at.step(e);
        const bool in = e < at.live;
        b[e] = in && d.bias != nullptr ? param<S>(d.bias, c, d.wf32) : 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k)
            k4[k][e] = in ? param<S>(d.weight, c * W + k, d.wf32) : 0.0f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        bias[h] = pack2f(b[2 * h], b[2 * h + 1]);
#pragma unroll
        for (int k = 0; k < W; ++k)
            w[k][h] = pack2f(k4[k][2 * h], k4[k][2 * h + 1]);
    }
}

// ---- forward ------------------------------------------------------------------------
// Tokens per lane: at 64 the W-1 inputs read twice are a twentieth of the
// bytes and come from L2. 32 tokens a lane measured 54 us where 64 and 128 take 47 (4 x 4096 tokens x 4096
// channels, bf16, W = 4: 268 MB, 85 % of the copy's rate). Rows that fit no vector (4095 channels) are loaded value by value, one group
// ahead: 68 us (58 %), in f32 90 against 84 (87 and 94 %).
constexpr int kConvSpan = 64;
constexpr int kConvAhead = 4, kConvGroups = 4;  // tokens of a group, groups on their way

template <class S, bool ALN, int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads, 5) k_conv(const S *x, S *out, S *state, ConvDims d, int64_t groups,
                                                       int64_t spans) {
    pdl_prologue();
    using Rng = Ring<S, ALN, kConvGroups, kConvAhead>;
    __shared__ __align__(16) char s_ring[ALN ? kConvThreads * Rng::kBytes : 16];
    Rng ring;
    const int64_t i = (int64_t)blockIdx.x * (kConvThreads / 32) + (threadIdx.x >> 5);
    const int64_t cgroup = i % groups, bs = i / groups;
    const int64_t span = bs % spans, b = bs / spans;
    if (b >= d.batch)
        return;
    ConvLane<ALN> at;
    at.set(cgroup, threadIdx.x & 31, d.dim);
    if (at.live == 0)
        return;
    const int64_t n = live_len(d.lens, d.len, b);
    const int64_t t0 = span * kConvSpan, t1 = t0 + kConvSpan < d.len ? t0 + kConvSpan : d.len;
    bool active = true;
    S *st = nullptr;
    if (d.slots != nullptr || state != nullptr) {
        const int64_t slot = slot_of(d.slots, d.nslots, b);
        active = slot >= 0;
        if (active && state != nullptr)
            st = state + slot * (W - 1) * d.dim + at.c;
    }
    const S *xs = x + b * d.xb + at.c;
    S *os = out + b * d.ob + t0 * d.ot + at.c;
    f32x2 w[W][2], bias[2];
    conv_params<S, ALN, W>(d, at, w, bias);
    f32x2 h[W][2];  // h[0..W-2]: the inputs before the present one
    const S *from = d.carry_in ? st : nullptr;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        Quad<S, ALN> v;
        input_at<S, ALN>(v, xs, from, d, t0 - (W - 1) + k, n, at.live);
        v.widen(h[k]);
    }
    const int tokens = (int)(t1 - t0), here = !active || n <= t0 ? 0 : n < t1 ? (int)(n - t0) : tokens;  // that exist
    const S *xt = xs + t0 * d.xt;
    constexpr int kDeep = ALN ? kConvGroups : 1;
    ring.set(s_ring + (threadIdx.x >> 5) * 32 * Rng::kBytes, threadIdx.x & 31);
#pragma unroll
    for (int g = 0; g < kDeep; ++g)
        ring.template ask<false>(g, xt + g * kConvAhead * d.xt, d.xt, here - g * kConvAhead, at.live);
    xt += kDeep * kConvAhead * d.xt;
    int group = 0;
    // FULL: the batch's tokens, and those asked for, all exist
    const auto batch = [&](int tt, auto full) {
        constexpr bool FULL = decltype(full)::value;
        Quad<S, ALN> v[kConvAhead];
        if (ALN)
            cp_async_wait<kDeep - 1>();
        ring.take(group, v);
        ring.template ask<FULL>(group, xt, d.xt, here - tt - kDeep * kConvAhead, at.live);  // in the place of what was taken
        xt += kConvAhead * d.xt;
#pragma unroll
        for (int j = 0; j < kConvAhead; ++j) {
            v[j].widen(h[W - 1]);
            f32x2 o[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f32x2 p = bias[e];
#pragma unroll
                for (int k = 0; k < W; ++k)
                    p = fma2f(w[k][e], h[k][e], p);
                if (SILU)
                    p = mul2f(p, sigmoid_2f(p));
                o[e] = FULL || tt + j < here ? p : 0ull;
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    h[k][e] = h[k + 1][e];
            }
            v[j].narrow(o);
            if (FULL || tt + j < tokens)
                v[j].store(os, at.live);
            os += d.ot;
        }
    };
    for (int tt = 0; tt < tokens; tt += kConvAhead, ++group) {
        if (tt + (kDeep + 1) * kConvAhead <= here)
            batch(tt, std::true_type());
        else
            batch(tt, std::false_type());
    }
    // The lane of the first span is the only one that reads the state, so it
    // is also the one that writes it: the last W-1 inputs of the sequence.
    if (span == 0 && st != nullptr) {
        Quad<S, ALN> last[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            input_at<S, ALN>(last[k], xs, from, d, n - (W - 1) + k, n, at.live);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            last[k].store(st + k * d.dim, at.live);
    }
}

// ---- one token of each sequence --------------------------------------------------------
template <class S, bool ALN, int W>
__global__ void __launch_bounds__(kConvThreads) k_conv_step(const S *x, S *out, S *state, ConvDims d, int64_t groups) {
    pdl_prologue();
    const int64_t i = (int64_t)blockIdx.x * (kConvThreads / 32) + (threadIdx.x >> 5);
    const int64_t group = i % groups, b = i / groups;
    if (b >= d.batch)
        return;
    ConvLane<ALN> at;
    at.set(group, threadIdx.x & 31, d.dim);
    if (at.live == 0)
        return;
    const int64_t slot = d.slots != nullptr || state != nullptr ? slot_of(d.slots, d.nslots, b) : b;
    Quad<S, ALN> o;
    o.zero();
    if (slot >= 0) {
        S *st = state + slot * (W - 1) * d.dim + at.c;
        Quad<S, ALN> v[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            v[k].load(st + k * d.dim, at.live);
        v[W - 1].load(x + b * d.xb + at.c, at.live);
        f32x2 w[W][2], p[2], h[2];
        conv_params<S, ALN, W>(d, at, w, p);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            v[k].widen(h);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                p[e] = fma2f(w[k][e], h[e], p[e]);
        }
        if (d.silu) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                p[e] = mul2f(p[e], sigmoid_2f(p[e]));
        }
        o.narrow(p);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            v[k + 1].store(st + k * d.dim, at.live);
    }
    o.store(out + b * d.ob + at.c, at.live);
}

// ---- gradient ----------------------------------------------------------------------------
// With g_t = dout_t * act'(p_t): dx_t = sum_k w_k g_{t+W-1-k}, dw_k = sum_t g_t x_{t-W+1+k},
// dbias = sum_t g_t. A lane walks up a span of tokens; at token t it makes p_t and g_t from W inputs
// in registers, adds to its W+1 sums, and finishes dx of token t-W+1, whose last
// g this is. Tokens past the span's end, whose g its last W-1 dx need, are walked
// too, without the sums. The sums of a span are 4(W+1) bytes against its
// 6 * kGradSpan bytes of activations; they are added over a CTA's spans in
// shared memory, written once per CTA and added by a second kernel in order.
// 30 us for 2 x 4099 tokens x 2048 channels, f16, W = 4 (101 MB, 15 us of the copy's rate; 3.3 TB/s). Its 98 instructions a lane
// and token are 11 us of the SMs' issue slots (47 % busy), so neither those nor the bytes bound it, but the cut: 288 CTAs of 512 tokens x
// 128 channels, of which 32 hold three tokens and the others lie two or one on 152 SMs, 13 warps an SM (128 registers), each a chain of 67 tokens.
// 8 x 4096 tokens x 4096 channels (2048 CTAs) reach 4.6 TB/s, one sequence of 2048 tokens x 1024 channels (32 CTAs) takes 18.7 us.
// Spans of 16, 32 and 128 tokens measured 45, 38 and 62 us where 64 took 36: shorter ones walk the W-1 tokens past the end more often,
// longer ones leave warps out. Rows that fit no vector: 47 us with 2047 channels (f32 73 against 40). With W = 4 that form keeps more than 128
// registers a thread, and spills 100 bytes (f32 316).
constexpr int kFew = 4, kGradGroups = 2;  // tokens of a group, groups on their way
constexpr int kGradSpan = 64;
constexpr int kGradSpans = 8;  // a CTA: 128 channels x 8 spans, a warp a span
constexpr int kGradThreads = 32 * kGradSpans;

// out_t's derivative by p_t
__device__ __forceinline__ f32x2 act_grad(f32x2 p) {
    const f32x2 s = sigmoid_2f(p);
    return mul2f(s, fma2f(p, add2f(both(1.0f), mul2f(both(-1.0f), s)), both(1.0f)));
}

template <class S, bool ALN, int W, bool SILU>
__global__ void __launch_bounds__(kGradThreads, 2) k_conv_grad(const S *x, const S *dout, S *dx, const S *state, S *dstate,
                                                            float *partial, ConvDims d, int64_t groups, int64_t span_blocks) {
    using Rng = Ring<S, ALN, kGradGroups, kFew>;
    // the rings, and after them the sums
    constexpr int kRings = ALN ? 2 * kGradThreads * Rng::kBytes : 16, kSums = (W + 1) * kGradSpans * 128 * 4;
    __shared__ __align__(16) char s_ring[kRings > kSums ? kRings : kSums];
    float(*s_sum)[kGradSpans][128] = reinterpret_cast<float(*)[kGradSpans][128]>(s_ring);
    pdl_prologue();
    const int lane = threadIdx.x & 31, sp = threadIdx.x >> 5;
    const int64_t cgroup = blockIdx.x % groups, rest = blockIdx.x / groups;
    const int64_t sb = rest % span_blocks, b = rest / span_blocks;
    ConvLane<ALN> at;
    at.set(cgroup, lane, d.dim);
    f32x2 sums[W + 1][2];  // dw, then dbias
#pragma unroll
    for (int k = 0; k <= W; ++k)
        sums[k][0] = sums[k][1] = 0ull;
    const int64_t t0 = (sb * kGradSpans + sp) * kGradSpan;
    if (at.live > 0 && (t0 < d.len || (t0 == 0 && dstate != nullptr))) {
        const int64_t n = live_len(d.lens, d.len, b);
        const int64_t t1 = t0 + kGradSpan < d.len ? t0 + kGradSpan : d.len;
        const S *xs = x + b * d.xb + at.c;
        const S *st = d.carry_in && state != nullptr ? state + b * (W - 1) * d.dim + at.c : nullptr;
        S *dst = t0 == 0 && dstate != nullptr ? dstate + b * (W - 1) * d.dim + at.c : nullptr;
        f32x2 w[W][2], bias[2];
        conv_params<S, ALN, W>(d, at, w, bias);
        f32x2 h[W][2], q[W][2];  // q[j]: the sum so far of dx of token t-W+1+j (the newest begins at j = W-1)
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            Quad<S, ALN> v;
            input_at<S, ALN>(v, xs, st, d, t0 - (W - 1) + k, n, at.live);
            v.widen(h[k]);
        }
#pragma unroll
        for (int k = 0; k < W; ++k)
            q[k][0] = q[k][1] = 0ull;
        const int tokens = (int)(t1 - t0), walk = tokens + W - 1;  // the last W-1 only finish this span's dx
        const int here = n <= t0 ? 0 : n - t0 < walk ? (int)(n - t0) : walk;  // that exist
        const S *xp = xs + t0 * d.xt, *gp = dout + b * d.gb + t0 * d.gt + at.c;
        S *dp = dx + b * d.db + t0 * d.dt + at.c;
        constexpr int kDeep = ALN ? kGradGroups : 1;
        Rng rx, rg;
        rx.set(s_ring + sp * 64 * Rng::kBytes, lane);
        rg.set(s_ring + (sp * 64 + 32) * Rng::kBytes, lane);
#pragma unroll
        for (int g = 0; g < kDeep; ++g) {
            rx.template ask<false>(g, xp + g * kFew * d.xt, d.xt, here - g * kFew, at.live);
            rg.template ask<false>(g, gp + g * kFew * d.gt, d.gt, here - g * kFew, at.live);
        }
        xp += kDeep * kFew * d.xt;
        gp += kDeep * kFew * d.gt;
        dp -= (W - 1) * d.dt;
        int group = 0;
        // FULL: the batch's tokens are this span's, their dx too, and those asked for exist
        const auto batch = [&](int tt, auto full) {
            constexpr bool FULL = decltype(full)::value;
            Quad<S, ALN> vx[kFew], vg[kFew];
            if (ALN)
                cp_async_wait<2 * kDeep - 2>();
            rx.take(group, vx);
            rg.take(group, vg);
            rx.template ask<FULL>(group, xp, d.xt, here - tt - kDeep * kFew, at.live);  // in the place of what was taken
            rg.template ask<FULL>(group, gp, d.gt, here - tt - kDeep * kFew, at.live);
            xp += kFew * d.xt;
            gp += kFew * d.gt;
#pragma unroll
            for (int j = 0; j < kFew; ++j) {
                f32x2 g[2], o[2];
                vx[j].widen(h[W - 1]);
                vg[j].widen(g);
                const bool own = FULL || tt + j < tokens;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f32x2 p = bias[e];
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        p = fma2f(w[k][e], h[k][e], p);
                    if (SILU)
                        g[e] = mul2f(g[e], act_grad(p));
                    const f32x2 gs = own ? g[e] : 0ull;
                    sums[W][e] = add2f(sums[W][e], gs);
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        sums[k][e] = fma2f(gs, h[k][e], sums[k][e]);
                        q[k][e] = fma2f(w[k][e], g[e], q[k][e]);  // g_t reaches dx of tokens t-W+1+k with w_k
                    }
                    o[e] = q[0][e];
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) {
                        q[k][e] = q[k + 1][e];
                        h[k][e] = h[k + 1][e];
                    }
                    q[W - 1][e] = 0ull;
                }
                const int to = tt + j - (W - 1);  // the token whose dx is done
                if (!FULL && to >= here)
                    o[0] = o[1] = 0ull;
                vg[j].narrow(o);
                if (FULL || (to >= 0 && to < tokens))
                    vg[j].store(dp, at.live);
                else if (to < 0 && dst != nullptr)
                    vg[j].store(dst + (to + W - 1) * d.dim, at.live);
                dp += d.dt;
            }
        };
        for (int tt = 0; tt < walk; tt += kFew, ++group) {
            if (tt >= W - 1 && tt + kFew <= tokens && tt + (kDeep + 1) * kFew <= here)
                batch(tt, std::true_type());
            else
                batch(tt, std::false_type());
        }
    }
    cp_async_wait_all();
    __syncthreads();  // the rings are done with
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        float v[4];
        unpack2f(sums[k][0], v[0], v[1]);
        unpack2f(sums[k][1], v[2], v[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s_sum[k][sp][(ALN ? 4 * lane : lane) + at.step(e)] = v[e];
    }
    __syncthreads();
    float *row = partial + (b * span_blocks + sb) * (W + 1) * d.dim;
    for (int i = threadIdx.x; i < (W + 1) * 128; i += kGradThreads) {
        const int k = i / 128, c = i % 128;
        const int64_t ch = cgroup * 128 + c;
        if (ch < d.dim) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < kGradSpans; ++j)
                s += s_sum[k][j][c];
            row[k * d.dim + ch] = s;
        }
    }
}

__global__ void __launch_bounds__(256) k_conv_grad_join(const float *partial, float *dweight, float *dbias, int64_t dim,
                                                        int64_t width, int64_t rows) {
    pdl_prologue();
    // a warp per (channel, quantity) would read strided: a lane per channel, one quantity per grid row
    const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const int64_t k = blockIdx.y;
    __shared__ float s_part[8][33];
    float s = 0.0f;
    if (c < dim)
        for (int64_t r = threadIdx.x >> 5; r < rows; r += 8)
            s += partial[(r * (width + 1) + k) * dim + c];
    s_part[threadIdx.x >> 5][threadIdx.x & 31] = s;
    __syncthreads();
    if (threadIdx.x < 32 && c < dim) {
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v += s_part[j][threadIdx.x];
        if (k < width)
            dweight[c * width + k] = v;
        else if (dbias != nullptr)
            dbias[c] = v;
    }
}

static int64_t conv_span_blocks(int64_t len) {
    const int64_t b = (len + kGradSpan * kGradSpans - 1) / (kGradSpan * kGradSpans);
    return b > 0 ? b : 1;
}

int64_t conv_grad_scratch_slots(int64_t batch, int64_t len, int64_t dim, int64_t width) {
    return (batch * conv_span_blocks(len) * (width + 1) * dim + 1) / 2;
}

static bool fits(const void *p, int64_t a, int64_t b, int64_t bytes) {  // of four values
    return (uintptr_t)p % bytes == 0 && a % 4 == 0 && b % 4 == 0;
}

template <class S, bool ALN, int W> static cudaError_t conv_go(const mt_conv_args &a, int what, const Launch &L) {
    const ConvDims d = conv_dims(a);
    const int64_t groups = (a.dim + 127) / 128;  // of channels: a warp's
    const S *x = static_cast<const S *>(a.x);
    S *state = static_cast<S *>(a.state);
    if (what == 0) {
        const int64_t spans = a.len > 0 ? (a.len + kConvSpan - 1) / kConvSpan : 1;
        const int64_t grid = (a.batch * spans * groups + kConvThreads / 32 - 1) / (kConvThreads / 32);
        if (grid > INT32_MAX)
            return cudaErrorInvalidValue;
        note_launch();
        return launch_pdl(d.silu ? k_conv<S, ALN, W, true> : k_conv<S, ALN, W, false>, (unsigned)grid, kConvThreads, 0, L.stream, x, static_cast<S *>(a.out), state, d, groups, spans);
    }
    if (what == 1) {
        const int64_t grid = (a.batch * groups + kConvThreads / 32 - 1) / (kConvThreads / 32);
        if (grid > INT32_MAX)
            return cudaErrorInvalidValue;
        note_launch();
        return launch_pdl(k_conv_step<S, ALN, W>, (unsigned)grid, kConvThreads, 0, L.stream, x, static_cast<S *>(a.out), state, d, groups);
    }
    const int64_t span_blocks = conv_span_blocks(a.len);
    const int64_t grid = a.batch * groups * span_blocks;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    float *partial = static_cast<float *>(a.scratch);
    if (grid > 0) {
        note_launch();
        const cudaError_t e = launch_pdl(d.silu ? k_conv_grad<S, ALN, W, true> : k_conv_grad<S, ALN, W, false>, (unsigned)grid, kGradThreads, 0, L.stream, x,
                                         static_cast<const S *>(a.dout), static_cast<S *>(a.dx), static_cast<const S *>(state),
                                         static_cast<S *>(a.dstate), partial, d, groups, span_blocks);
        if (e != cudaSuccess)
            return e;
    }
    note_launch();
    return launch_pdl_2d(k_conv_grad_join, dim3((unsigned)((a.dim + 31) / 32), (unsigned)(W + 1)), 256, L.stream, (const float *)partial, a.dweight, a.dbias, (int64_t)a.dim, (int64_t)W,
                              a.batch * span_blocks);
}

template <class S, bool ALN> static cudaError_t conv_width(const mt_conv_args &a, int what, const Launch &L) {
    switch (a.width) {
    case 1: return conv_go<S, ALN, 1>(a, what, L);
    case 2: return conv_go<S, ALN, 2>(a, what, L);
    case 3: return conv_go<S, ALN, 3>(a, what, L);
    case 4: return conv_go<S, ALN, 4>(a, what, L);
    default: return cudaErrorInvalidValue;
    }
}

template <class S> static cudaError_t conv_type(const mt_conv_args &a, int what, const Launch &L) {
    constexpr int64_t v = 4 * sizeof(S);
    bool aligned = a.dim % 4 == 0 && fits(a.x, a.x_batch, a.x_token, v) && fits(a.state, 0, 0, v);
    if (what == 2)
        aligned = aligned && fits(a.dout, a.dout_batch, a.dout_token, v) && fits(a.dx, a.dx_batch, a.dx_token, v) && fits(a.dstate, 0, 0, v);
    else
        aligned = aligned && fits(a.out, a.out_batch, a.out_token, v);
    return aligned ? conv_width<S, true>(a, what, L) : conv_width<S, false>(a, what, L);
}

static cudaError_t conv_any(const mt_conv_args &a, int what, const Launch &L) {
    switch (a.dtype) {
    case MT_F32: return conv_type<float>(a, what, L);
    case MT_BF16: return conv_type<__nv_bfloat16>(a, what, L);
    case MT_F16: return conv_type<__half>(a, what, L);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t conv_launch(const mt_conv_args &a, const Launch &L) { return conv_any(a, 0, L); }
cudaError_t conv_step_launch(const mt_conv_args &a, const Launch &L) { return conv_any(a, 1, L); }
cudaError_t conv_grad_launch(const mt_conv_args &a, const Launch &L) { return conv_any(a, 2, L); }

}  // namespace mt
