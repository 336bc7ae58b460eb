// mt_conv.cu -- the short causal convolution of each channel over the tokens,
// with bias and SiLU, its gradient, and its single-token form.
//
//   p_t = bias + sum_{k < W} w_k x_{t-W+1+k},  out_t = p_t or p_t * sigmoid(p_t)
//
// where the W-1 inputs before token 0 come from a state (or are 0) and the
// last W-1 inputs are left in it. 2W + 5 operations per value of 2 or 4 bytes
// read and written: bound by bytes. A lane owns V neighbouring channels (16
// bytes, or one value where the rows fit no vector) and walks down a span of
// tokens with the W-1 inputs before the present one in registers, so an input is
// read once, plus W-1 per span; a warp's lanes are neighbouring channels.
#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

constexpr int kConvThreads = 128;

// V values of one lane.
template <class S, int V> struct Lane {
    float x[V];
    __device__ __forceinline__ void load(const S *p) {
        if constexpr (V == 1)
            x[0] = Codec<S>::load1(p);
        else
            Codec<S>::unpack(*reinterpret_cast<const uint4 *>(p), x);
    }
    __device__ __forceinline__ void store(S *p) const {
        if constexpr (V == 1)
            Codec<S>::store1(p, x[0]);
        else
            *reinterpret_cast<uint4 *>(p) = Codec<S>::pack(x);
    }
    __device__ __forceinline__ void fill(float v) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = v;
    }
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
template <class S, int V>
__device__ __forceinline__ void input_at(Lane<S, V> &v, const S *x, const S *state, const ConvDims &d, int64_t t,
                                         int64_t n) {
    if (t < 0) {
        if (state != nullptr)
            v.load(state + (t + d.width - 1) * d.dim);
        else
            v.fill(0.0f);
    } else if (t < n) {
        v.load(x + t * d.xt);
    } else {
        v.fill(0.0f);
    }
}

// ---- forward ------------------------------------------------------------------------
// Tokens per lane: at 32 the W-1 inputs read twice are a tenth of the
// bytes and come from L2.
constexpr int kConvSpan = 32;
constexpr int kConvAhead = 8;  // tokens loaded together

template <class S, int V, int W>
__global__ void __launch_bounds__(kConvThreads) k_conv(const S *x, S *out, S *state, ConvDims d, int64_t lanes,
                                                       int64_t spans) {
    pdl_prologue();
    const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    const int64_t lane = i % lanes, bs = i / lanes;
    const int64_t span = bs % spans, b = bs / spans;
    if (b >= d.batch)
        return;
    const int64_t c = lane * V;
    const int64_t n = live_len(d.lens, d.len, b);
    const int64_t t0 = span * kConvSpan, t1 = t0 + kConvSpan < d.len ? t0 + kConvSpan : d.len;
    bool active = true;
    S *st = nullptr;
    if (d.slots != nullptr || state != nullptr) {
        const int64_t slot = slot_of(d.slots, d.nslots, b);
        active = slot >= 0;
        if (active && state != nullptr)
            st = state + slot * (W - 1) * d.dim + c;
    }
    const S *xs = x + b * d.xb + c;
    S *os = out + b * d.ob + c;
    float w[W][V], bias[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        bias[e] = d.bias != nullptr ? param<S>(d.bias, c + e, d.wf32) : 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k)
            w[k][e] = param<S>(d.weight, (c + e) * W + k, d.wf32);
    }
    Lane<S, V> h[W];  // h[0..W-2]: the inputs before the present one
    const S *from = d.carry_in ? st : nullptr;
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        input_at<S, V>(h[k], xs, from, d, t0 - (W - 1) + k, n);
    for (int64_t tt = t0; tt < t1; tt += kConvAhead) {
        Lane<S, V> v[kConvAhead];
#pragma unroll
        for (int j = 0; j < kConvAhead; ++j) {
            if (tt + j < n && tt + j < t1)
                v[j].load(xs + (tt + j) * d.xt);
            else
                v[j].fill(0.0f);
        }
#pragma unroll
        for (int j = 0; j < kConvAhead; ++j) {
            if (tt + j < t1) {
                h[W - 1] = v[j];
                Lane<S, V> o;
                const bool live = active && tt + j < n;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float p = bias[e];
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        p = fmaf(w[k][e], h[k].x[e], p);
                    if (d.silu)
                        p *= sigmoidf(p);
                    o.x[e] = live ? p : 0.0f;
                }
                o.store(os + (tt + j) * d.ot);
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    h[k] = h[k + 1];
            }
        }
    }
    // The lane of the first span is the only one that reads the state, so it
    // is also the one that writes it: the last W-1 inputs of the sequence.
    if (span == 0 && st != nullptr) {
        Lane<S, V> last[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            input_at<S, V>(last[k], xs, from, d, n - (W - 1) + k, n);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            last[k].store(st + k * d.dim);
    }
}

// ---- one token of each sequence --------------------------------------------------------
template <class S, int V, int W>
__global__ void __launch_bounds__(kConvThreads) k_conv_step(const S *x, S *out, S *state, ConvDims d, int64_t lanes) {
    pdl_prologue();
    const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    const int64_t lane = i % lanes, b = i / lanes;
    if (b >= d.batch)
        return;
    const int64_t c = lane * V;
    const int64_t slot = d.slots != nullptr || state != nullptr ? slot_of(d.slots, d.nslots, b) : b;
    Lane<S, V> o;
    o.fill(0.0f);
    if (slot >= 0) {
        S *st = state + slot * (W - 1) * d.dim + c;
        Lane<S, V> h[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            h[k].load(st + k * d.dim);
        h[W - 1].load(x + b * d.xb + c);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float p = d.bias != nullptr ? param<S>(d.bias, c + e, d.wf32) : 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k)
                p = fmaf(param<S>(d.weight, (c + e) * W + k, d.wf32), h[k].x[e], p);
            o.x[e] = d.silu ? p * sigmoidf(p) : p;
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            h[k + 1].store(st + k * d.dim);
    }
    o.store(out + b * d.ob + c);
}

// ---- gradient ----------------------------------------------------------------------------
// With g_t = dout_t * act'(p_t): dx_t = sum_k w_k g_{t+W-1-k}, dw_k = sum_t g_t x_{t-W+1+k},
// dbias = sum_t g_t. A lane walks up a span of tokens; at token t it makes p_t and g_t from W inputs
// in registers, adds to its W+1 sums, and finishes dx of token t-W+1, whose last
// g this is. Tokens past the span's end, whose g its last W-1 dx need, are walked
// too, without the sums. The sums of a span are 4(W+1) bytes against its
// 6 * kGradSpan bytes of activations; they are added over a CTA's spans in
// shared memory, written once per CTA and added by a second kernel in order.
constexpr int kGradSpan = 64;
constexpr int kGradLanes = 32, kGradSpans = 8;  // a CTA: 32 lanes of channels x 8 spans
constexpr int kGradThreads = kGradLanes * kGradSpans;

// out_t's derivative by p_t
__device__ __forceinline__ float act_grad(float p, bool silu) {
    if (!silu)
        return 1.0f;
    const float s = sigmoidf(p);
    return s * fmaf(p, 1.0f - s, 1.0f);
}

template <class S, int V, int W>
__global__ void __launch_bounds__(kGradThreads) k_conv_grad(const S *x, const S *dout, S *dx, const S *state, S *dstate,
                                                            float *partial, ConvDims d, int64_t lane_blocks,
                                                            int64_t span_blocks) {
    __shared__ float s_sum[kGradSpans][kGradLanes * V + 1];
    pdl_prologue();
    const int lane = threadIdx.x % kGradLanes, sp = threadIdx.x / kGradLanes;
    const int64_t lb = blockIdx.x % lane_blocks, rest = blockIdx.x / lane_blocks;
    const int64_t sb = rest % span_blocks, b = rest / span_blocks;
    const int64_t c = (lb * kGradLanes + lane) * V;
    const bool on = c < d.dim;
    float dw[W][V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        db[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k)
            dw[k][e] = 0.0f;
    }
    const int64_t t0 = (sb * kGradSpans + sp) * kGradSpan;
    if (on && (t0 < d.len || (t0 == 0 && dstate != nullptr))) {
        const int64_t n = live_len(d.lens, d.len, b);
        const int64_t t1 = t0 + kGradSpan < d.len ? t0 + kGradSpan : d.len;
        const S *xs = x + b * d.xb + c, *gs = dout + b * d.gb + c;
        S *ds = dx + b * d.db + c;
        const S *st = d.carry_in && state != nullptr ? state + b * (W - 1) * d.dim + c : nullptr;
        float w[W][V], bias[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            bias[e] = d.bias != nullptr ? param<S>(d.bias, c + e, d.wf32) : 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k)
                w[k][e] = param<S>(d.weight, (c + e) * W + k, d.wf32);
        }
        Lane<S, V> h[W];
        float q[W][V];  // q[j]: the sum so far of dx of token t-W+1+j (the newest begins at j = W-1)
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            input_at<S, V>(h[k], xs, st, d, t0 - (W - 1) + k, n);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e)
                q[k][e] = 0.0f;
        // tokens t1 .. t1+W-2 only finish this span's dx
        for (int64_t tt = t0; tt < t1 + W - 1; tt += 4) {
            Lane<S, V> vx[4], vg[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t t = tt + j;
                if (t < n && t < t1 + W - 1) {
                    vx[j].load(xs + t * d.xt);
                    vg[j].load(gs + t * d.gt);
                } else {
                    vx[j].fill(0.0f);
                    vg[j].fill(0.0f);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t t = tt + j;
                if (t < t1 + W - 1) {
                    h[W - 1] = vx[j];
                    Lane<S, V> o;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float p = bias[e];
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            p = fmaf(w[k][e], h[k].x[e], p);
                        const float g = vg[j].x[e] * act_grad(p, d.silu);
                        if (t < t1) {
                            db[e] += g;
#pragma unroll
                            for (int k = 0; k < W; ++k)
                                dw[k][e] = fmaf(g, h[k].x[e], dw[k][e]);
                        }
                        // g_t reaches dx of tokens t-W+1+k with w_k
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            q[k][e] = fmaf(w[k][e], g, q[k][e]);
                        o.x[e] = q[0][e];
#pragma unroll
                        for (int k = 0; k < W - 1; ++k)
                            q[k][e] = q[k + 1][e];
                        q[W - 1][e] = 0.0f;
                    }
                    const int64_t to = t - (W - 1);
                    if (to >= t0) {
                        if (to >= n)
                            o.fill(0.0f);
                        o.store(ds + to * d.dt);
                    } else if (t0 == 0 && dstate != nullptr) {
                        o.store(dstate + b * (W - 1) * d.dim + (to + W - 1) * d.dim + c);
                    }
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        h[k] = h[k + 1];
                }
            }
        }
    }
    // the CTA's sums, one quantity after the other
    float *row = partial + (b * span_blocks + sb) * (W + 1) * d.dim;
#pragma unroll
    for (int k = 0; k <= W; ++k) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            s_sum[sp][lane * V + e] = k < W ? dw[k < W ? k : 0][e] : db[e];
        __syncthreads();
        for (int i = threadIdx.x; i < kGradLanes * V; i += kGradThreads) {
            const int64_t ch = lb * kGradLanes * V + i;
            if (ch < d.dim) {
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < kGradSpans; ++j)
                    s += s_sum[j][i];
                row[k * d.dim + ch] = s;
            }
        }
        __syncthreads();
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

static bool fits(const void *p, int64_t a, int64_t b, int64_t e) {
    return (uintptr_t)p % 16 == 0 && a % e == 0 && b % e == 0;
}

template <class S, int V, int W> static cudaError_t conv_go(const mt_conv_args &a, int what, const Launch &L) {
    const ConvDims d = conv_dims(a);
    const int64_t lanes = a.dim / V;
    const S *x = static_cast<const S *>(a.x);
    S *state = static_cast<S *>(a.state);
    if (what == 0) {
        const int64_t spans = a.len > 0 ? (a.len + kConvSpan - 1) / kConvSpan : 1;
        const int64_t grid = (a.batch * spans * lanes + kConvThreads - 1) / kConvThreads;
        if (grid > INT32_MAX)
            return cudaErrorInvalidValue;
        note_launch();
        return launch_pdl(k_conv<S, V, W>, (unsigned)grid, kConvThreads, 0, L.stream, x, static_cast<S *>(a.out), state, d, lanes, spans);
    }
    if (what == 1) {
        const int64_t grid = (a.batch * lanes + kConvThreads - 1) / kConvThreads;
        if (grid > INT32_MAX)
            return cudaErrorInvalidValue;
        note_launch();
        return launch_pdl(k_conv_step<S, V, W>, (unsigned)grid, kConvThreads, 0, L.stream, x, static_cast<S *>(a.out), state, d, lanes);
    }
    const int64_t lane_blocks = (lanes + kGradLanes - 1) / kGradLanes, span_blocks = conv_span_blocks(a.len);
    const int64_t grid = a.batch * lane_blocks * span_blocks;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    float *partial = static_cast<float *>(a.scratch);
    if (grid > 0) {
        note_launch();
        const cudaError_t e = launch_pdl(k_conv_grad<S, V, W>, (unsigned)grid, kGradThreads, 0, L.stream, x,
                                         static_cast<const S *>(a.dout), static_cast<S *>(a.dx), static_cast<const S *>(state),
                                         static_cast<S *>(a.dstate), partial, d, lane_blocks, span_blocks);
        if (e != cudaSuccess)
            return e;
    }
    note_launch();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.dim + 31) / 32), (unsigned)(W + 1));
    cfg.blockDim = dim3(256);
    cfg.stream = L.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_conv_grad_join, (const float *)partial, a.dweight, a.dbias, (int64_t)a.dim, (int64_t)W,
                              a.batch * span_blocks);
}

template <class S, int V> static cudaError_t conv_width(const mt_conv_args &a, int what, const Launch &L) {
    switch (a.width) {
    case 1: return conv_go<S, V, 1>(a, what, L);
    case 2: return conv_go<S, V, 2>(a, what, L);
    case 3: return conv_go<S, V, 3>(a, what, L);
    case 4: return conv_go<S, V, 4>(a, what, L);
    default: return cudaErrorInvalidValue;
    }
}

template <class S> static cudaError_t conv_type(const mt_conv_args &a, int what, const Launch &L) {
    constexpr int E = Codec<S>::E;
    bool vec = a.dim % E == 0 && fits(a.x, a.x_batch, a.x_token, E) && fits(a.state, 0, 0, E);
    if (what == 2)
        vec = vec && fits(a.dout, a.dout_batch, a.dout_token, E) && fits(a.dx, a.dx_batch, a.dx_token, E) && fits(a.dstate, 0, 0, E);
    else
        vec = vec && fits(a.out, a.out_batch, a.out_token, E);
    return vec ? conv_width<S, E>(a, what, L) : conv_width<S, 1>(a, what, L);
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
