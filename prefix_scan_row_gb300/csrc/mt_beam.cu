// mt_beam.cu -- a beam search's selection over beams and vocabulary.
//
// Two kernels. In the first every warp reads a span of one beam's logits, a group of 1024 (f32: 512) after the other, and leaves the
// sum of their exponentials and each group's largest value: one pass at the speed of memory, with no word between warps.
// The second has a CTA a sequence: it joins the sums, and keeps the beams_out best groups, by the score of their largest logit and,
// where those are equal, by their place. That loses nothing: a logit that is among the beams_out first cannot be in a group that
// as many groups are before, since each of those holds a logit before it. So only beams_out groups are read
// again, and the few logits in them that reach the last one's score are ranked. Where there are many such logits (equal ones, or
// high ones beside each other), the same step over the groups' vectors, and then over theirs, leaves few.
//
// Bound: the first kernel by bytes, f32, and by its instructions, 16-bit (an exponential a logit; issue 63 %, XU 38 %); the second
// by its chain of loads, barriers and comparisons, 8 to 10 us. Both together, us in a CUDA graph (share of the measured copy rate, 6798 GB/s):
// 64 x 16 x 131072 logits f32 91 (87 %), bf16 55 (71 %); 64 x 8 x 32768 bf16 16.8 (29 %); 1 x 4 x 32768 f32 7.8. Rows that are not
// aligned take two loads for a vector: 64 x 16 x 131071 bf16 84 (47 %). All logits equal, 64 x 16 x 131072 bf16: 106.
#include <initializer_list>

#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

namespace {

constexpr int kBeamThreads = 256;  // of the first kernel
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32;
constexpr int kBatch = 4;        // vectors of a lane in a group
constexpr int kMostBatches = 8;  // groups of a warp
constexpr int kGroupVectors = 32 * kBatch;

// Values as unsigned numbers in their order, -0 below 0; not for NaN, whose sign is anything.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
constexpr uint32_t kOrderLow = 0x007fffffu;  // of -inf
// A score is a pair of f32, the value rounded and what that leaves: 48 bits, by f32 additions (f64 ones take a
// warp 16 clocks of the SM each here, and a few thousand scores are made). As a number in their order; 0 is below all of them.
__device__ __forceinline__ uint64_t order_of(float high, float low) { return (uint64_t)order_of(high + 0.0f) << 32 | order_of(low + 0.0f); }
__device__ __forceinline__ float score_of(uint64_t k) { return value_of((uint32_t)(k >> 32)); }
// a + b and its rounding error (Knuth's sum)
__device__ __forceinline__ float two_sum(float a, float b, float &error) {
    const float s = a + b, t = s - a;
    error = (a - (s - t)) + (b - t);
    return s;
}
// (x - top) + (high + low)
__device__ __forceinline__ uint64_t score_order(float x, float top, float high, float low) {
    float e0, e1;
    const float d = two_sum(x, -top, e0), s = two_sum(d, high, e1), rest = e1 + (e0 + low), sum = s + rest;
    return fabsf(s) < Lim<float>::hi() ? order_of(sum, rest - (sum - s)) : order_of(s, 0.0f);
}
// NaN as -inf, +inf as the largest finite value.
__device__ __forceinline__ float tidy(float x, float most) { return x == x ? fminf(x, most) : Lim<float>::lo(); }

// The power of two that a span's sum is relative to: below 2^23 from 0 where its largest value is below 2^22; others' sums
// are relative to exp of that value; and a span with no sum.
constexpr float kFarTop = 4194304.0f;
constexpr int kNoPower = 1 << 30, kLeastPower = -(1 << 30);

// A 16-byte vector of logits.
template <class S> struct Logits;
template <> struct Logits<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ float most() { return 3.402823466e38f; }
    static __device__ __forceinline__ uint4 none() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    static __device__ __forceinline__ float larger(float m, float x) {
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(x));
        return m;
    }
    using Most = float;
    static __device__ __forceinline__ Most low() { return Lim<float>::lo(); }
    static __device__ __forceinline__ Most max_of(Most m, const uint4 &w) {
        return larger(larger(larger(larger(m, __uint_as_float(w.x)), __uint_as_float(w.y)), __uint_as_float(w.z)), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ float widen(Most m) { return m; }
};
template <class S, uint32_t LOW, uint32_t HIGH> struct LogitsOf16 {
    static constexpr int E = 8;
    static __device__ __forceinline__ float most() {
        float a, b;
        Codec<S>::two(HIGH, a, b);
        return a;
    }
    static __device__ __forceinline__ uint4 none() { return make_uint4(LOW, LOW, LOW, LOW); }
    using Most = uint32_t;  // two maxima
    static __device__ __forceinline__ Most low() { return LOW; }
    static __device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t x);
    static __device__ __forceinline__ Most max_of(Most m, const uint4 &w) { return larger(larger(m, larger(w.x, w.y)), larger(w.z, w.w)); }
    static __device__ __forceinline__ float widen(Most m) {
        float a, b;
        Codec<S>::two(m, a, b);
        return Logits<float>::larger(a, b);
    }
};
template <> __device__ __forceinline__ uint32_t LogitsOf16<__nv_bfloat16, 0xff80ff80u, 0x7f7f7f7fu>::larger(uint32_t m, uint32_t x) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
    return m;
}
template <> __device__ __forceinline__ uint32_t LogitsOf16<__half, 0xfc00fc00u, 0x7bff7bffu>::larger(uint32_t m, uint32_t x) {
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
    return m;
}
template <> struct Logits<__nv_bfloat16> : LogitsOf16<__nv_bfloat16, 0xff80ff80u, 0x7f7f7f7fu> {};
template <> struct Logits<__half> : LogitsOf16<__half, 0xfc00fc00u, 0x7bff7bffu> {};

// In the scratch: a span's sum (in units of 2^-40), its largest value and power; then the groups' largest values, as numbers in order.
struct BeamPlan {
    int batches;    // groups of a span
    int64_t spans;  // of a beam's logits
};
// Spans as long as leave enough warps, us by the warps asked for, 152 x 8, 152 x 64 and 152 x 256: 64 x 8 x 32768 bf16 19.1, 16.8, 16.6;
// 64 x 16 x 131071 bf16 83.9, 83.7, 90.7; 5 x 7 x 100003 f16 13.8, 13.3, 13.2.
constexpr int64_t kEnoughSpans = 152 * 32 * 2;
BeamPlan beam_plan(int64_t rows, int64_t vocab, int64_t size) {
    BeamPlan p;
    for (p.batches = kMostBatches;; p.batches /= 2) {
        const int64_t bytes = (int64_t)p.batches * kGroupVectors * 16;
        p.spans = (vocab * size + bytes - 1) / bytes;
        if (p.batches == 1 || rows * p.spans >= kEnoughSpans)
            return p;
    }
}

// The vector of logits from token `at` on, -inf behind the row. WORDS < 0: rows are made of aligned vectors. Otherwise the row begins
// WORDS words (and, `half` 16, another 16 bits) behind an aligned vector, and the values come from the two aligned ones that they lie
// in, each of which holds a logit of the row at least. Which thread has which token does not depend on a row's address,
// so that equal rows have equal sums.
template <class S, int WORDS> __device__ __forceinline__ uint4 load_logits(const S *x, int64_t at, int64_t vocab, int half) {
    constexpr int E = Logits<S>::E;
    uint4 w = Logits<S>::none();
    if (at >= vocab)
        return w;
    if constexpr (WORDS < 0) {
        return ld_stream(reinterpret_cast<const uint4 *>(x + at));
    } else {
        const uintptr_t from = (uintptr_t)(x + at) & ~(uintptr_t)15;
        const uint4 p = *reinterpret_cast<const uint4 *>(from);
        const uint4 q = from + 16 < (uintptr_t)(x + vocab) ? *reinterpret_cast<const uint4 *>(from + 16) : w;
        const uint32_t o[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
        w = make_uint4(__funnelshift_r(o[WORDS], o[WORDS + 1], half), __funnelshift_r(o[WORDS + 1], o[WORDS + 2], half),
                       __funnelshift_r(o[WORDS + 2], o[WORDS + 3], half), __funnelshift_r(o[WORDS + 3], o[WORDS + 4], half));
        if (at + E > vocab) {
            uint4 none = Logits<S>::none();
            S *s = reinterpret_cast<S *>(&w);
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (at + k >= vocab)
                    s[k] = reinterpret_cast<S *>(&none)[k];
        }
        return w;
    }
}
// A lane's part of a span: its largest value, and the sum, in f32, of up to 64 terms in each of four places (which is what a beam's sum is
// good to, some 1e-7; from there on nothing is lost above 2^-30 of a span), of 2^(log2(e) x - k) with k the whole number next to log2(e) times
// the largest (kept between -+kMostPower). One multiply-add, rounded once, makes an exponent, and a larger k scales the sum by
// a power of two. (A sum relative to exp of the largest would take a subtraction for each logit.)
constexpr float kMostPower = 8388608.0f;
__device__ __forceinline__ float power_of(float top) { return fminf(fmaxf(rintf(kLog2e * top), -kMostPower), kMostPower); }
template <class S> struct Part {
    using L = Logits<S>;
    float top, power;
    f32x2 s0, s1;
    __device__ __forceinline__ void begin() {
        top = Lim<float>::lo();
        power = -kMostPower;
        s0 = s1 = 0ull;
    }
    __device__ __forceinline__ float largest(const uint4 (&w)[kBatch]) const {
        typename L::Most most = L::low();
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            most = L::max_of(most, w[j]);
        return L::widen(most);
    }
    // returns the batch's largest value
    __device__ __forceinline__ float add(uint4 (&w)[kBatch]) {
        float m = largest(w);
        if (!(m < Lim<float>::hi())) {  // an infinity or NaN among them: made finite
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                float f[L::E];
                Codec<S>::unpack(w[j], f);
#pragma unroll
                for (int q = 0; q < L::E; ++q)
                    f[q] = tidy(f[q], L::most());
                w[j] = Codec<S>::pack(f);
            }
            m = largest(w);
        }
        top = fmaxf(top, m);
        const float p = power_of(top);
        const f32x2 scale = both(ex2f(power - p)), less = both(-p);
        power = p;
        s0 = mul2f(s0, scale);
        s1 = mul2f(s1, scale);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            float f[L::E];
            Codec<S>::unpack(w[j], f);
#pragma unroll
            for (int q = 0; q < L::E; q += 4) {
                s0 = add2f(s0, ex2_2f(fma2f(pack2f(f[q], f[q + 1]), both(kLog2e), less)));
                s1 = add2f(s1, ex2_2f(fma2f(pack2f(f[q + 2], f[q + 3]), both(kLog2e), less)));
            }
        }
        return m;
    }
    __device__ __forceinline__ float sum() const {
        float a, b;
        unpack2f(add2f(s0, s1), a, b);
        return a + b;
    }
};
// The span from token `begin` on, `lane_at` the lane's place in a row of vectors; the next batch is on its way while one is worked
// on. Lane t gets group t's largest value.
template <class S, int WORDS>
__device__ __forceinline__ uint32_t read_span(Part<S> &part, const S *x, int64_t begin, int64_t vocab, int batches, int lane, int half) {
    constexpr int E = Logits<S>::E;
    const int64_t first = begin + lane * E;
    uint32_t mine = kOrderLow;
    if constexpr (WORDS >= 0) {  // a vector comes from two, which would have to be there before they are one: no batch ahead, more warps
#pragma unroll 1
        for (int t = 0; t < batches; ++t) {
            uint4 w[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                w[j] = load_logits<S, WORDS>(x, first + (t * kBatch + j) * (32 * E), vocab, half);
            const uint32_t m = __reduce_max_sync(kFull, order_of(part.add(w) + 0.0f));
            mine = lane == t ? m : mine;
        }
    } else {
        uint4 w[2][kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            w[0][j] = load_logits<S, WORDS>(x, first + j * (32 * E), vocab, half);
#pragma unroll 1
        for (int t = 0; t < batches; t += 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (t + u < batches) {
                    if (t + u + 1 < batches) {
#pragma unroll
                        for (int j = 0; j < kBatch; ++j)
                            w[1 - u][j] = load_logits<S, WORDS>(x, first + ((t + u + 1) * kBatch + j) * (32 * E), vocab, half);
                    }
                    const uint32_t m = __reduce_max_sync(kFull, order_of(part.add(w[u]) + 0.0f));
                    mine = lane == t + u ? m : mine;
                }
            }
        }
    }
    return mine;
}

// VEC: rows are made of aligned vectors. Five CTAs an SM (48 registers): 64 x 16 x 131071 bf16 84 us, with four 98.
template <class S, bool VEC> __global__ void __launch_bounds__(kBeamThreads, 5) k_beam_read(const __grid_constant__ mt_beam_args a, BeamPlan plan) {
    constexpr int E = Logits<S>::E;
    pdl_prologue();
    const int lane = threadIdx.x % 32;
    const int64_t id = (int64_t)blockIdx.x * (kBeamThreads / 32) + threadIdx.x / 32, rows = a.batch * a.beams;
    const int64_t row = id / plan.spans, span = id - row * plan.spans, b = row / a.beams, beam = row - b * a.beams;
    if (row >= rows || (a.finished != nullptr && a.finished[row] != 0))
        return;
    const S *x = static_cast<const S *>(a.logits) + b * a.logits_batch + beam * a.logits_beam;
    const int64_t begin = span * plan.batches * (kGroupVectors * E);
    Part<S> part;
    part.begin();
    uint32_t mine;
    if constexpr (VEC) {
        mine = read_span<S, -1>(part, x, begin, a.vocab, plan.batches, lane, 0);
    } else {
        const int half = (int)((uintptr_t)x & 2) * 8;
        switch ((uintptr_t)x % 16 / 4) {
        case 0: mine = read_span<S, 0>(part, x, begin, a.vocab, plan.batches, lane, half); break;
        case 1: mine = read_span<S, 1>(part, x, begin, a.vocab, plan.batches, lane, half); break;
        case 2: mine = read_span<S, 2>(part, x, begin, a.vocab, plan.batches, lane, half); break;
        default: mine = read_span<S, 3>(part, x, begin, a.vocab, plan.batches, lane, half);
        }
    }
    const float top = value_of(__reduce_max_sync(kFull, mine)), power = power_of(top);
    const bool by_power = fabsf(top) < kFarTop;
    float s = part.sum() * ex2f(part.power - power);
    if (!by_power && top != Lim<float>::lo()) {  // far out, where log2(e) x is no longer exact enough: relative to exp(top)
        s = 0.0f;
#pragma unroll 1
        for (int i = 0; i < plan.batches * kBatch; ++i) {
            const int64_t at = begin + (i * 32 + lane) * E;
            float t = 0.0f;
#pragma unroll
            for (int q = 0; q < E; ++q)
                if (at + q < a.vocab)
                    t += ex2f(kLog2e * (tidy(Codec<S>::load1(x + at + q), Logits<S>::most()) - top));
            s += t;
        }
    }
    // the lanes' sums as whole numbers, whose sum has no order
    const uint32_t high = (uint32_t)(s * 0x1p18f), low = (uint32_t)((s * 0x1p18f - (float)high) * 0x1p22f);
    const uint32_t low_all = __reduce_add_sync(kFull, low), high_all = __reduce_add_sync(kFull, high);
    uint64_t *stat = static_cast<uint64_t *>(a.scratch) + 2 * id;
    uint32_t *groups = reinterpret_cast<uint32_t *>(static_cast<uint64_t *>(a.scratch) + 2 * rows * plan.spans) + id * plan.batches;
    if (lane == 0) {
        stat[0] = top == Lim<float>::lo() ? 0 : (uint64_t)low_all + ((uint64_t)high_all << 22);
        stat[1] = __float_as_uint(top) | (uint64_t)(uint32_t)(top == Lim<float>::lo() ? kLeastPower : by_power ? (int)power : kNoPower) << 32;
    }
    if (lane < plan.batches)
        groups[lane] = mine;
}

// log(2) as a pair, and as one whose first part has 9 bits, so that a small whole number times it is exact
constexpr double kLn2Double = 0.693147180559945309417;
constexpr float kLn2Low = (float)(kLn2Double - (double)kLn2), kLn2Few = 355.0f / 512.0f, kLn2FewLow = (float)(kLn2Double - (double)kLn2Few);

// Logarithms of c = 1 - j / 128, j below 64, as f32 pairs: the series of 2 atanh((c - 1) / (c + 1)), summed by the compiler.
struct LogTable {
    float high[64], low[64];
    constexpr LogTable() : high(), low() {
        for (int j = 0; j < 64; ++j) {
            const double c = 1.0 - j / 128.0, r = (c - 1.0) / (c + 1.0);
            double sum = 0.0, power = r;
            for (int k = 1; k < 60; k += 2) {
                sum += power / k;
                power *= r * r;
            }
            high[j] = (float)(2.0 * sum);
            low[j] = (float)(2.0 * sum - (double)(float)(2.0 * sum));
        }
    }
};
__constant__ LogTable kLogTable = LogTable();

// The score of a beam's largest logit, as a pair: prior - log(sum of exp(x - top)), with `sum` in units of 2^-30 relative to 2^power
// (the terms' exponents are x log2(e) with log2(e) as f32, so top's is taken the same), or (kNoPower) a double.
// In f32 pairs, good to 2e-9 (64-bit arithmetic's latency made 1.7 of the join's 7.7 us): with c of 7 bits next to 1 / m,
// log(2^e m) = e log(2) - log(c) + log(c m), whose last argument is within 1/128 of 1.
__device__ __forceinline__ void best_score(float prior, uint64_t sum, int power, float top, float &high, float &low) {
    if (power == kNoPower) {
        const double s = (double)prior - log(__longlong_as_double((long long)sum));
        high = (float)s;
        low = (float)(s - (double)high);
        return;
    }
    const int e = 63 - __clzll((long long)sum);
    const uint64_t bits = sum << (63 - e);  // m = bits / 2^63
    const float m_high = (float)(uint32_t)(bits >> 40) * 0x1p-23f, m_low = (float)(uint32_t)(bits >> 16 & 0xffffffu) * 0x1p-47f;
    const int j = 128 - (int)rintf(128.0f * rcpf(m_high));  // 0 to 64
    const int at = j < 63 ? j : 63;
    const float c = 1.0f - (float)at * 0.0078125f, p = m_high * c, z = (p - 1.0f) + fmaf(m_high, c, -p) + m_low * c;
    float log1 = fmaf(z, 1.0f / 7.0f, -1.0f / 6.0f);  // log(1 + z) - z
    log1 = fmaf(log1, z, 0.2f);
    log1 = fmaf(log1, z, -0.25f);
    log1 = fmaf(log1, z, 1.0f / 3.0f);
    log1 = fmaf(log1, z, -0.5f) * z * z;
    // (power - log2(e) top) log(2), exactly but for its last rounding; and e log(2), whose first part has few bits
    const float t = kLog2e * top, d = (float)power - t, d_low = -fmaf(kLog2e, top, -t);
    const float w = d * kLn2, w_low = fmaf(d, kLn2, -w) + (d * kLn2Low + d_low * kLn2);
    const float f = (float)(e - 30), e_high = f * kLn2Few, e_low = f * kLn2FewLow;
    float r0, r1, r2, r3, s = two_sum(prior, -e_high, r0);
    s = two_sum(s, kLogTable.high[at], r1);
    s = two_sum(s, -z, r2);
    s = two_sum(s, -w, r3);
    const float rest = (r0 + r1) + (r2 + r3) + ((kLogTable.low[at] - e_low) - (log1 + w_low));
    high = s + rest;
    low = rest - (high - s);
    if (!(fabsf(s) < Lim<float>::hi()))
        low = 0.0f;
}

// A block of logits, or one, as it is chosen: by its score's number, then by the lower place. Score 0 is none.
struct Choice {
    uint64_t score, place;
    __device__ __forceinline__ bool before(const Choice &o) const { return score > o.score || (score == o.score && place < o.place); }
};
constexpr int kChosen = 1024;  // that may reach the threshold
constexpr int kAhead = 4;                 // vectors of a thread on their way
constexpr int kPart = kJoinThreads / 32;  // threads that share a first choice, and that rank one
struct ChooseShared {
    Choice best[32], kept[kChosen], list[kBeamsMost];
    Choice threshold;
    int count;
};
__device__ __forceinline__ Choice first_of(Choice c, int lanes) {
    for (int d = 1; d < lanes; d *= 2) {
        const Choice o = {__shfl_xor_sync(kFull, c.score, d), __shfl_xor_sync(kFull, c.place, d)};
        c = o.before(c) ? o : c;
    }
    return c;
}
// How many of n choices are before c, counted by the kPart threads that hold the same c.
__device__ __forceinline__ int rank_of(const Choice &c, const Choice *of, int n) {
    int before = 0;
    for (int q = threadIdx.x % kPart; q < n; q += kPart)
        before += of[q].before(c);
#pragma unroll
    for (int d = 1; d < kPart; d *= 2)
        before += __shfl_xor_sync(kFull, before, d);
    return before;
}
__device__ __forceinline__ void keep(ChooseShared &s, const Choice &c) {
    const int at = atomicAdd(&s.count, 1);
    if (at < kChosen)
        s.kept[at] = c;
}
// The K first of the kept ones to s.list. A barrier before and one after.
__device__ __forceinline__ void rank_kept(ChooseShared &s, int count, int K) {
    for (int t0 = 0; t0 < count; t0 += 32) {
        const int t = t0 + threadIdx.x / kPart;
        const Choice c = t < count ? s.kept[t] : Choice{0, ~0ull};
        const int before = rank_of(c, s.kept, count);
        if (t < count && before < K && threadIdx.x % kPart == 0)
            s.list[before] = c;
    }
}
// The K first of get(0) .. get(n - 1), in order, in s.list; returns how many there are (K at most). A threshold that K of them
// reach at least is the K-th of the first ones of 32 parts of the CTA; few others reach it, and where that is not so (in one
// part, more than there is place for) they are taken one after the other. A barrier before it, behind the last read of s.count;
// ends with one.
template <class F> __device__ __forceinline__ int choose(int64_t n, int K, ChooseShared &s, F get) {
    const int tid = threadIdx.x, lane = tid % 32;
    Choice mine = {0, ~0ull};
#pragma unroll 4
    for (int64_t i = tid; i < n; i += kJoinThreads) {
        const Choice c = get(i);
        if (c.before(mine))
            mine = c;
    }
    if (mine.score == 0)
        mine.place = ~(uint64_t)tid;  // no two are equal
    const Choice top = first_of(mine, kPart);
    if (tid % kPart == 0)
        s.best[tid / kPart] = top;
    if (tid == 0)
        s.count = 0;
    __syncthreads();
    if (rank_of(top, s.best, 32) == K - 1 && tid % kPart == 0)
        s.threshold = top;
    __syncthreads();
    const Choice least = s.threshold;
    if (n <= kJoinThreads) {  // a thread had one
        if (mine.score != 0 && !least.before(mine))
            keep(s, mine);
    } else if (mine.score != 0 && !least.before(mine)) {
        for (int64_t i = tid; i < n; i += kJoinThreads) {
            const Choice c = get(i);
            if (c.score != 0 && !least.before(c))
                keep(s, c);
        }
    }
    __syncthreads();
    const int count = s.count;
    if (count <= kChosen) {
        rank_kept(s, count, K);
    } else {
        Choice last = {~0ull, 0};
        for (int t = 0; t < K; ++t) {
            mine = {0, ~0ull};
            for (int64_t i = tid; i < n; i += kJoinThreads) {
                const Choice c = get(i);
                if (last.before(c) && c.before(mine))
                    mine = c;
            }
            mine = first_of(mine, 32);
            if (lane == 0)
                s.best[tid / 32] = mine;
            __syncthreads();
            last = first_of(s.best[lane % kJoinWarps], kJoinWarps);
            if (tid == 0)
                s.list[t] = last;
            __syncthreads();
        }
    }
    __syncthreads();
    return count < K ? count : K;
}

template <class S, bool VEC> __global__ void __launch_bounds__(kJoinThreads) k_beam_join(const __grid_constant__ mt_beam_args a, BeamPlan plan) {
    constexpr int E = Logits<S>::E;
    __shared__ ChooseShared s;
    __shared__ uint64_t sums[kBeamsMost];
    __shared__ int powers[kBeamsMost];
    __shared__ float priors[kBeamsMost], tops[kBeamsMost];
    __shared__ float highs[kBeamsMost], lows[kBeamsMost];  // the scores of the beams' largest logits
    __shared__ float cuts[kBeamsMost];
    __shared__ uint64_t blocks[kBeamsMost];
    __shared__ int32_t spare[kBeamsMost];
    __shared__ uint32_t finished, ended;  // finished beams, and those of them that go on
    pdl_prologue();
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, beams = (int)a.beams, K = (int)a.beams_out;
    const int spans = (int)plan.spans;
    const uint64_t *stats = static_cast<const uint64_t *>(a.scratch) + 2 * b * beams * plan.spans;
    const uint32_t *groups =
        reinterpret_cast<const uint32_t *>(static_cast<const uint64_t *>(a.scratch) + 2 * a.batch * beams * plan.spans) + b * beams * plan.spans * plan.batches;
    if (tid == 0)
        finished = ended = 0;
    const int group = beams > K ? beams : K;
    const int32_t slot = a.slots != nullptr && tid < group ? a.slots[b * group + tid] : 0;
    __syncthreads();
    for (int k = warp; k < beams; k += kJoinWarps) {
        const ulonglong2 *mine = reinterpret_cast<const ulonglong2 *>(stats) + (int64_t)k * spans;
        const ulonglong2 none = make_ulonglong2(0, (uint64_t)(uint32_t)kLeastPower << 32 | 0xff800000u);
        ulonglong2 own[kAhead];  // those of the first spans, on their way before it is known whether they count
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            own[u] = lane + 32 * u < spans ? mine[lane + 32 * u] : none;
        const float prior = a.prior != nullptr ? tidy(a.prior[b * beams + k], 3.402823466e38f) : 0.0f;
        const bool done = a.finished != nullptr && a.finished[b * beams + k] != 0;
        const bool reads = !done && prior != Lim<float>::lo();
        float top = Lim<float>::lo();
        int power = kLeastPower;
        uint64_t sum = 0;
        if (reads) {
            auto top_of = [](const ulonglong2 &o) { return __uint_as_float((uint32_t)o.y); };
            auto power_in = [](const ulonglong2 &o) { return (int)(uint32_t)(o.y >> 32); };
            auto each = [&](auto f) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    f(own[u]);
                for (int c = lane + 32 * kAhead; c < spans; c += 32)
                    f(mine[c]);
            };
            each([&](const ulonglong2 &o) {
                top = fmaxf(top, top_of(o));
                power = max(power, power_in(o));
            });
            top = value_of(__reduce_max_sync(kFull, order_of(top)));
            power = __reduce_max_sync(kFull, power);
            if (power == kNoPower) {  // far out: sums in 64 bits, relative to the largest value
                double all = 0.0;
                each([&](const ulonglong2 &o) {
                    const double m = (double)top_of(o);
                    const int p = power_in(o);
                    if (p != kLeastPower)
                        all += (double)o.x * 0x1p-40 * exp(m - (double)top + (p == kNoPower ? 0.0 : ((double)p - m * (double)kLog2e) * kLn2Double));
                });
                for (int o = 16; o > 0; o /= 2)
                    all += __shfl_xor_sync(kFull, all, o);
                sum = (uint64_t)__double_as_longlong(all);
            } else {
                each([&](const ulonglong2 &o) { sum += o.x >> 10 >> min(power - power_in(o), 53); });
                for (int o = 16; o > 0; o /= 2)
                    sum += __shfl_xor_sync(kFull, sum, o);
            }
        }
        if (lane == 0) {
            sums[k] = sum;
            powers[k] = power;
            tops[k] = top;
            priors[k] = prior;
            if (done)
                atomicOr(&finished, 1u << k);
            if (done && prior != Lim<float>::lo())
                atomicOr(&ended, 1u << k);
        }
    }
    __syncthreads();
    // a lane makes each beam's logarithm
    if (warp == 0 && lane < beams && powers[lane] != kLeastPower)
        best_score(priors[lane], sums[lane], powers[lane], tops[lane], highs[lane], lows[lane]);
    __syncthreads();
    auto score = [&](int k, float x) { return score_order(x, tops[k], highs[k], lows[k]); };
    // places: the beam, and the group, vector or token in its row
    const int per_beam = spans * plan.batches;
    int n = choose((int64_t)beams * per_beam, K, s, [&](int64_t i) {
        const int k = (int)i / per_beam, g = (int)i - k * per_beam;
        const uint32_t o = groups[i];  // of a beam that was not read it is not looked at
        return Choice{powers[k] != kLeastPower && o > kOrderLow ? score(k, value_of(o)) : 0, (uint64_t)k << 32 | (uint32_t)g};
    });
    if (tid < n)
        blocks[tid] = s.list[tid].place;
    // What a logit has to reach for the last group's score, a little less for the roundings: the others' scores are not made.
    if (tid < beams) {
        const float last = score_of(s.list[K - 1].score), at = last - highs[tid];
        cuts[tid] = n < K ? Lim<float>::lo() : tops[tid] + at - 1e-6f * (fabsf(at) + fabsf(last) + fabsf(highs[tid]) + fabsf(tops[tid]));
    }
    auto row_of = [&](int k) { return static_cast<const S *>(a.logits) + b * a.logits_batch + k * a.logits_beam; };
    auto logit = [&](const S *x, int64_t at) { return tidy(Codec<S>::load1(x + at), Logits<S>::most()); };
    auto choice = [&](int k, float x, uint32_t at) {
        return Choice{x == Lim<float>::lo() || x < cuts[k] ? 0 : score(k, x + 0.0f), (uint64_t)k << 32 | at};
    };
    if (tid == 0)
        s.count = 0;
    __syncthreads();
    // The logits of these groups that reach it, with the ends of beams that are finished: hardly more than beams_out.
    for (int i0 = tid; i0 < n * kGroupVectors; i0 += kJoinThreads * kAhead) {
        float f[kAhead][E];
        int64_t at[kAhead];
        int k[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kJoinThreads;
            const uint64_t block = i < n * kGroupVectors ? blocks[i / kGroupVectors] : 0;
            k[u] = (int)(block >> 32);
            at[u] = i < n * kGroupVectors ? ((int64_t)(uint32_t)block * kGroupVectors + i % kGroupVectors) * E : a.vocab;
            const S *x = row_of(k[u]) + at[u];
            if (VEC && at[u] < a.vocab) {
                Codec<S>::unpack(*reinterpret_cast<const uint4 *>(x), f[u]);
            } else {
#pragma unroll
                for (int q = 0; q < E; ++q)
                    f[u][q] = at[u] + q < a.vocab ? Codec<S>::load1(x + q) : Lim<float>::lo();
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float cut = cuts[k[u]];
            uint32_t reach = 0;
#pragma unroll
            for (int q = 0; q < E; ++q)
                reach |= !(f[u][q] < cut) && f[u][q] != Lim<float>::lo() ? 1u << q : 0u;
            for (; reach != 0; reach &= reach - 1) {
                const int q = __ffs(reach) - 1;
                float x = f[u][0];
#pragma unroll
                for (int o = 1; o < E; ++o)
                    x = q == o ? f[u][o] : x;
                const Choice c = choice(k[u], tidy(x, Logits<S>::most()), (uint32_t)(at[u] + q));
                if (c.score != 0)
                    keep(s, c);
            }
        }
    }
    if (tid < beams && (ended >> tid & 1u))
        keep(s, {order_of(priors[tid], 0.0f), (uint64_t)tid << 32 | (uint32_t)a.eos});
    __syncthreads();
    const int count = s.count;
    if (count <= kChosen) {
        rank_kept(s, count, K);
        n = count < K ? count : K;
        __syncthreads();
    } else {
        // Or there are many: of the groups' vectors the first ones, and of their logits.
        __syncthreads();  // every warp has read the count, which choose() begins anew
        n = choose((int64_t)n * kGroupVectors, K, s, [&](int64_t i) {
            const uint64_t block = blocks[i / kGroupVectors];
            const int k = (int)(block >> 32);
            const uint32_t v = (uint32_t)block * kGroupVectors + (uint32_t)(i % kGroupVectors);
            const int64_t at = (int64_t)v * E;
            const S *x = row_of(k);
            float m = Lim<float>::lo();
#pragma unroll
            for (int q = 0; q < E; ++q)
                if (at + q < a.vocab)
                    m = fmaxf(m, logit(x, at + q));
            return choice(k, m, v);
        });
        if (tid < n)
            blocks[tid] = s.list[tid].place;
        __syncthreads();
        const int logits = n * E;
        n = choose((int64_t)logits + beams, K, s, [&](int64_t i) {
            if (i >= logits) {
                const int k = (int)i - logits;
                return Choice{ended >> k & 1u ? order_of(priors[k], 0.0f) : 0, (uint64_t)k << 32 | (uint32_t)a.eos};
            }
            const uint64_t block = blocks[i / E];
            const int k = (int)(block >> 32);
            const int64_t at = (int64_t)(uint32_t)block * E + i % E;
            return choice(k, at < a.vocab ? logit(row_of(k), at) : Lim<float>::lo(), (uint32_t)at);
        });
    }
    if (warp != 0)
        return;
    const Choice chosen = lane < n ? s.list[lane] : Choice{order_of(Lim<float>::lo(), 0.0f), 0};
    int parent = (int)(chosen.place >> 32), tok = (int)(uint32_t)chosen.place;
    if (n < K) {  // behind all that may come next what may not, in order
        int64_t next = 0;
        for (int j = n; j < K; ++j, ++next) {
            while (__any_sync(kFull, lane < n && parent * a.vocab + tok == next))
                ++next;
            if (lane == j) {
                parent = (int)(next / a.vocab);
                tok = (int)(next % a.vocab);
            }
        }
    }
    const bool out = lane < K;
    const int64_t to = b * K + lane;
    if (out) {
        a.tokens[to] = tok;
        a.parents[to] = parent;
        a.scores[to] = score_of(chosen.score);
        if (a.finished_out != nullptr)
            a.finished_out[to] = (finished >> parent & 1u) != 0 || tok == a.eos;
    }
    if (a.slots == nullptr)
        return;
    const uint32_t sames = __match_any_sync(kFull, out ? parent : 32 + lane);
    const bool stays = out && __ffs(sames) - 1 == lane;
    const uint32_t members = group == 32 ? kFull : (1u << group) - 1;
    const uint32_t free = members & ~__reduce_or_sync(kFull, stays ? 1u << parent : 0u);
    const uint32_t moving = __ballot_sync(kFull, lane < group && !stays);
    const int32_t old = __shfl_sync(kFull, slot, parent);
    // the lanes that move, and those behind the beams, take the free slots in order
    if (free >> lane & 1u)
        spare[__popc(free & ((1u << lane) - 1))] = slot;
    __syncwarp();
    const int32_t fresh = spare[__popc(moving & ((1u << lane) - 1)) & 31];
    if (lane < group)
        a.slots[b * group + lane] = stays ? old : fresh;
    if (out) {
        a.src[to] = stays ? -1 : old;
        a.dst[to] = stays ? -1 : fresh;
    }
}

template <class S> cudaError_t launch(const mt_beam_args &a, const Launch &L) {
    const BeamPlan plan = beam_plan(a.batch * a.beams, a.vocab, sizeof(S));
    const int64_t vector = Logits<S>::E, warps = kBeamThreads / 32, blocks = (a.batch * a.beams * plan.spans + warps - 1) / warps;
    if (blocks > INT32_MAX || a.batch > INT32_MAX)
        return cudaErrorInvalidValue;
    const bool vec = (uintptr_t)a.logits % 16 == 0 && a.vocab % vector == 0 && a.logits_batch % vector == 0 && a.logits_beam % vector == 0;
    note_launch();
    const cudaError_t e = vec ? launch_pdl(k_beam_read<S, true>, (unsigned)blocks, kBeamThreads, 0, L.stream, a, plan)
                              : launch_pdl(k_beam_read<S, false>, (unsigned)blocks, kBeamThreads, 0, L.stream, a, plan);
    if (e != cudaSuccess)
        return e;
    note_launch();
    return vec ? launch_pdl(k_beam_join<S, true>, (unsigned)a.batch, kJoinThreads, 0, L.stream, a, plan)
               : launch_pdl(k_beam_join<S, false>, (unsigned)a.batch, kJoinThreads, 0, L.stream, a, plan);
}

}  // namespace

// No smaller than what any smaller call takes, although a smaller call may cut its rows into more and shorter spans: spans of
// fewer groups than the most are chosen only where spans of twice as many are fewer than kEnoughSpans, so there are less than twice
// that many of them, and no more than these rows have.
int64_t beam_scratch_slots(int64_t batch, int64_t beams, int64_t, int64_t vocab) {
    int64_t most = 0;
    for (const int64_t size : {2, 4})  // of the types
        for (int batches = kMostBatches; batches >= 1; batches /= 2) {
            const int64_t bytes = (int64_t)batches * kGroupVectors * 16;
            int64_t spans = batch * beams * ((vocab * size + bytes - 1) / bytes);
            if (batches < kMostBatches && spans > 2 * kEnoughSpans)
                spans = 2 * kEnoughSpans;
            const int64_t slots = 2 * spans + (spans * batches + 1) / 2;
            most = slots > most ? slots : most;
        }
    return most;
}

cudaError_t beam_launch(const mt_beam_args &a, const Launch &L) {
    switch (a.dtype) {
    case MT_F32: return launch<float>(a, L);
    case MT_BF16: return launch<__nv_bfloat16>(a, L);
    case MT_F16: return launch<__half>(a, L);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace mt
