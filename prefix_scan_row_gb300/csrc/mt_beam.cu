// mt_beam.cu -- a beam search's selection over beams and vocabulary.
//
// Two kernels. The first gives every CTA a chunk of one beam's logits: its largest value, the sum of
// exp(x - largest), and its beams_out first tokens in order. The second has a CTA a sequence: it joins the
// chunks of each beam, then the beams, and gives out the slots.
//
// Within a beam the order of the scores is the order of the logits, so only joining beams needs scores; they are
// made and compared in 64 bits there, a few hundred of them. What bounds the whole is reading the logits once.
#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamKept = 1024;  // logits of a chunk that may reach the threshold

// Values as unsigned numbers in their order, -0 below 0; not for NaN, whose sign is anything.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
constexpr uint32_t kOrderLow = 0x007fffffu;   // of -inf
constexpr uint32_t kOrderHigh = 0xff800000u;  // of +inf
// The power of two that a chunk's sum is relative to: below 2^23 from 0 where its largest value is below 2^22; others' sums
// are relative to exp of that value; and a chunk with no sum.
constexpr float kFarTop = 4194304.0f;
constexpr int kNoPower = 1 << 30, kLeastPower = -(1 << 30);
// NaN as -inf, +inf as the largest finite value.
__device__ __forceinline__ float tidy(float x, float most) { return x == x ? fminf(x, most) : Lim<float>::lo(); }
// Larger values first, of equal ones the lower token; 0 and -0 are equal.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) { return (uint64_t)order_of(x + 0.0f) << 32 | (uint32_t)~token; }

__device__ __forceinline__ uint32_t redux_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
// The largest of a warp's keys.
__device__ __forceinline__ uint64_t warp_max(uint64_t key) {
    const uint32_t hi = redux_max((uint32_t)(key >> 32));
    const uint32_t lo = redux_max((uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
    return (uint64_t)hi << 32 | lo;
}

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

// A chunk's place in the scratch: sum (in units of 2^-40), largest value and power, then beams_out keys, 0 for none.
struct BeamPlan {
    int per_thread;  // logits of a thread: 64 or 16
    int64_t chunks;  // of a beam's logits
    int64_t slots;   // of a chunk
};
// A CTA's chunk: large, so that what follows the reading costs little beside it, where there are many CTAs all the same.
BeamPlan beam_plan(int64_t rows, int64_t beams_out, int64_t vocab) {
    BeamPlan p;
    auto chunks = [&](int per_thread) { return (vocab + per_thread * kBeamThreads - 1) / (per_thread * kBeamThreads); };
    p.per_thread = rows * chunks(64) >= 2 * 152 ? 64 : 16;
    p.chunks = chunks(p.per_thread);
    p.slots = beams_out + 2;
    return p;
}

// Rows that are not made of aligned vectors: the thread's vectors, tokens begin + j * 2048 (or 1024) on, from the aligned
// ones that they touch (each holds a logit of the row at least). Which thread has which token does not depend on a row's address,
// so that equal rows have equal sums.
template <class S, int V, int WORDS> __device__ __forceinline__ void stage_shifted(uint4 *own, const S *x, int64_t begin, int64_t vocab) {
    constexpr int E = Logits<S>::E;
    const uintptr_t end = (uintptr_t)(x + vocab);
    const int half = (int)((uintptr_t)x & 2) * 8;
#pragma unroll 4
    for (int j = 0; j < V; ++j) {
        const int64_t at = begin + j * (kBeamThreads * E);
        uint4 w = Logits<S>::none();
        if (at < vocab) {
            const uintptr_t from = (uintptr_t)(x + at) & ~(uintptr_t)15;
            const uint4 p = *reinterpret_cast<const uint4 *>(from);
            const uint4 q = from + 16 < end ? *reinterpret_cast<const uint4 *>(from + 16) : w;
            const uint32_t o[9] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w, 0};
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
        }
        own[j * kBeamThreads] = w;
    }
}

// A value that beams_out logits of the CTA reach at least: of the maxima of every LANES threads the beams_out-th largest.
// And the largest. LANES threads count together what is before their group's maximum. Few logits reach it: of 16384
// independent ones about 22 for 16 of 32 groups, and 44 for 32 of 64 (130 for 32 of 32).
template <int LANES>
__device__ __forceinline__ void find_threshold(uint32_t mine, int K, uint32_t *group_max, uint32_t &threshold, uint32_t &top_order) {
    constexpr int kGroups = kBeamThreads / LANES, kPart = kGroups / LANES;
    const int lane = threadIdx.x % 32, g = threadIdx.x / LANES, part = lane % LANES * kPart;
    uint32_t m = mine;
#pragma unroll
    for (int d = 1; d < LANES; d *= 2)
        m = max(m, __shfl_xor_sync(kFull, m, d));
    if (lane % LANES == 0)
        group_max[g] = m;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int q = 0; q < kPart; q += 4) {
        const uint4 o = *reinterpret_cast<const uint4 *>(&group_max[part + q]);
        before += o.x > m || (o.x == m && part + q < g);
        before += o.y > m || (o.y == m && part + q + 1 < g);
        before += o.z > m || (o.z == m && part + q + 2 < g);
        before += o.w > m || (o.w == m && part + q + 3 < g);
    }
#pragma unroll
    for (int d = 1; d < LANES; d *= 2)
        before += __shfl_xor_sync(kFull, before, d);
    if (lane % LANES == 0 && before == K - 1)
        threshold = m;
    if (lane % LANES == 0 && before == 0)
        top_order = m;
    __syncthreads();
}

// Thread t's logits from `least` on, as keys; their number goes on beyond the places that there are.
template <class S, int PER>
__device__ __forceinline__ void keep_reached(const uint4 *staged, int t, int lane, uint32_t begin, uint32_t least, uint64_t *kept, uint32_t &count) {
    constexpr int E = Logits<S>::E, kWords = PER / E * 4;  // 32-bit words of a thread
#pragma unroll
    for (int i = 0; i < kWords; i += 32) {
        const int word = i + lane;
        if (word < kWords) {
            const int j = word / 4, q = word % 4 * (E / 4);
            const uint32_t w = reinterpret_cast<const uint32_t *>(staged + j * kBeamThreads + t)[word % 4];
            float f[2];
            if constexpr (E == 8)
                Codec<S>::two(w, f[0], f[1]);
            else
                f[0] = __uint_as_float(w);
            const uint32_t token = begin + (uint32_t)(j * (kBeamThreads * E) + t * E + q);
#pragma unroll
            for (int k = 0; k < E / 4; ++k) {
                const uint64_t key = key_of(f[k], token + k);
                if ((uint32_t)(key >> 32) >= least) {
                    const uint32_t n = atomicAdd(&count, 1u);
                    if (n < kBeamKept)
                        kept[n] = key;
                }
            }
        }
    }
}

// A thread's logits stay in its own places of shared memory, where they are copied to and read from three times: for
// their maxima, for the sum, and (of few threads) for those that reach the threshold. VEC: rows are made of aligned vectors.
template <class S, int PER, bool VEC> __global__ void __launch_bounds__(kBeamThreads) k_beam_chunk(const __grid_constant__ mt_beam_args a, BeamPlan plan) {
    using L = Logits<S>;
    constexpr int E = L::E, V = PER / E;  // values of a vector, vectors of a thread
    __shared__ __align__(16) uint32_t group_max[kBeamThreads / 4];
    __shared__ uint32_t threshold, top_order, count;
    __shared__ uint32_t sum_low[kBeamWarps], sum_high[kBeamWarps];
    __shared__ uint64_t kept[kBeamKept];
    extern __shared__ __align__(16) uint4 staged[];
    pdl_prologue();
    const uint32_t chunks = (uint32_t)plan.chunks, beams = (uint32_t)a.beams;
    const int64_t row = blockIdx.x / chunks, chunk = blockIdx.x % chunks, b = (uint32_t)row / beams, beam = (uint32_t)row % beams;
    if (a.finished != nullptr && a.finished[row] != 0)
        return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, K = (int)a.beams_out;
    const S *x = static_cast<const S *>(a.logits) + b * a.logits_batch + beam * a.logits_beam;
    // vector j of the thread: tokens first + j * 2048 (or 1024) and on
    const int64_t first = chunk * (kBeamThreads * PER) + threadIdx.x * E;
    uint4 *own = staged + threadIdx.x;  // vector j: own[j * kBeamThreads]
    if constexpr (VEC) {
        const uint32_t own_at = (uint32_t)__cvta_generic_to_shared(own);
        const S *from = x + first;
        if ((chunk + 1) * (kBeamThreads * PER) <= a.vocab) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                cp_async_zfill<16>(own_at + j * (kBeamThreads * 16), from + j * (kBeamThreads * E), true);
        } else {
            const int left = (int)(a.vocab - first < INT32_MAX ? a.vocab - first : INT32_MAX);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (j * (kBeamThreads * E) < left)
                    cp_async_zfill<16>(own_at + j * (kBeamThreads * 16), from + j * (kBeamThreads * E), true);
                else
                    own[j * kBeamThreads] = L::none();
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
    } else {
        switch ((uintptr_t)x % 16 / 4) {
        case 0: stage_shifted<S, V, 0>(own, x, first, a.vocab); break;
        case 1: stage_shifted<S, V, 1>(own, x, first, a.vocab); break;
        case 2: stage_shifted<S, V, 2>(own, x, first, a.vocab); break;
        default: stage_shifted<S, V, 3>(own, x, first, a.vocab);
        }
    }
    __syncwarp();
    uint32_t mine;  // the thread's largest value
    for (bool again = false;; again = true) {
        typename L::Most most = L::low();
#pragma unroll
        for (int j = 0; j < V; ++j)
            most = L::max_of(most, own[j * kBeamThreads]);
        const float widest = L::widen(most);
        mine = widest == widest ? order_of(widest + 0.0f) : ~0u;
        if (threadIdx.x == 0)
            count = 0;
        if (K <= 16)
            find_threshold<8>(mine, K, group_max, threshold, top_order);
        else
            find_threshold<4>(mine, K, group_max, threshold, top_order);
        if (again || top_order < kOrderHigh)
            break;
        // an infinity or NaN among them: made finite, and once more
#pragma unroll 1
        for (int j = 0; j < V; ++j) {
            float f[E];
            Codec<S>::unpack(own[j * kBeamThreads], f);
#pragma unroll
            for (int q = 0; q < E; ++q)
                f[q] = tidy(f[q], L::most());
            own[j * kBeamThreads] = Codec<S>::pack(f);
        }
    }
    uint64_t *out = static_cast<uint64_t *>(a.scratch) + (row * plan.chunks + chunk) * plan.slots;
    const uint32_t top = top_order;
    if (top <= kOrderLow) {  // nothing here may come next
        if (threadIdx.x < plan.slots)
            out[threadIdx.x] = threadIdx.x == 1 ? __float_as_uint(Lim<float>::lo()) | (uint64_t)(uint32_t)kLeastPower << 32 : 0;
        return;
    }
    // the logits that reach the threshold: few lanes have one, and the warp goes through each of theirs together
    const uint32_t least = threshold > kOrderLow ? threshold : kOrderLow + 1;
    for (uint32_t lanes = __ballot_sync(kFull, mine >= least); lanes != 0; lanes &= lanes - 1)
        keep_reached<S, PER>(staged, warp * 32 + __ffs(lanes) - 1, lane, (uint32_t)(chunk * (kBeamThreads * PER)), least, kept, count);
    // Sum of exp(x - top): f32 in the thread, then whole numbers, whose sum has no order. Where top is not too far out, of
    // 2^(log2(e) x - k) with the whole number k next to log2(e) top: one multiply-add, rounded once, makes the
    // exponent, and sums of chunks differ by powers of two.
    const bool by_power = fabsf(value_of(top)) < kFarTop;
    const float power = rintf(kLog2e * value_of(top));
    {
        f32x2 s0 = 0ull, s1 = 0ull;
        auto add = [&](auto term) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float f[E];
                Codec<S>::unpack(own[j * kBeamThreads], f);
#pragma unroll
                for (int q = 0; q < E; q += 4) {
                    s0 = add2f(s0, ex2_2f(term(pack2f(f[q], f[q + 1]))));
                    s1 = add2f(s1, ex2_2f(term(pack2f(f[q + 2], f[q + 3]))));
                }
            }
        };
        const f32x2 scale = both(kLog2e), less = both(by_power ? -power : -value_of(top));
        if (by_power)
            add([&](f32x2 v) { return fma2f(v, scale, less); });
        else
            add([&](f32x2 v) { return mul2f(add2f(v, less), scale); });
        float p, r;
        unpack2f(add2f(s0, s1), p, r);
        const float s = p + r;
        const uint32_t high = (uint32_t)(s * 0x1p20f), low = (uint32_t)((s * 0x1p20f - (float)high) * 0x1p20f);
        const uint32_t low_all = __reduce_add_sync(kFull, low), high_all = __reduce_add_sync(kFull, high);
        if (lane == 0) {
            sum_low[warp] = low_all;
            sum_high[warp] = high_all;
        }
    }
    __syncthreads();
    int n = (int)count;
    if (n > kBeamKept) {
        // More equal values than there is place for (a mask of a finite value, for instance): those above the threshold,
        // and of those at it the first beams_out, vector after vector.
        __syncthreads();
        if (threadIdx.x == 0)
            count = 0;
        __syncthreads();
        for (uint32_t lanes = __ballot_sync(kFull, mine > least); lanes != 0; lanes &= lanes - 1)
            keep_reached<S, PER>(staged, warp * 32 + __ffs(lanes) - 1, lane, (uint32_t)(chunk * (kBeamThreads * PER)), least + 1, kept, count);
        __syncthreads();
        n = (int)count;  // places behind those take the equal ones
        int had = 0;
#pragma unroll 1
        for (int j = 0; j < V && had < K && n + K <= kBeamKept; ++j) {
            float f[E];
            Codec<S>::unpack(own[j * kBeamThreads], f);
            uint32_t equal = 0;
#pragma unroll
            for (int q = 0; q < E; ++q)
                equal |= order_of(f[q] + 0.0f) == least ? 1u << q : 0u;
            int before = __popc(equal), all = before;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(kFull, before, d);
                before += lane >= d ? o : 0;
            }
            if (lane == 31)
                group_max[j % 2 * kBeamWarps + warp] = (uint32_t)before;
            before += had - all;
            __syncthreads();
#pragma unroll
            for (int q = 0; q < kBeamWarps; ++q) {
                const int o = (int)group_max[j % 2 * kBeamWarps + q];
                before += q < warp ? o : 0;
                had += o;
            }
            for (; equal != 0 && before < K; equal &= equal - 1, ++before) {
                const int q = __ffs(equal) - 1;
                kept[n + before] = (uint64_t)least << 32 | (uint32_t)~(uint32_t)(first + j * (kBeamThreads * E) + q);
            }
        }
        n = n + K <= kBeamKept ? n + (had < K ? had : K) : kBeamKept + 1;
        __syncthreads();
    }
    if (n <= kBeamKept) {
        for (int t = threadIdx.x; t < n; t += kBeamThreads) {
            const uint64_t key = kept[t];
            int before = 0;
            for (int q = 0; q < n; ++q)
                before += kept[q] > key;
            if (before < K)
                out[2 + before] = key;
        }
        for (int t = n + threadIdx.x; t < K; t += kBeamThreads)
            out[2 + t] = 0;
    } else {
        // too many in too few places: the largest key below the last one, beams_out times
        uint64_t last = ~0ull;
        for (int t = 0; t < K; ++t) {
            uint64_t m = 0;
#pragma unroll 1
            for (int j = 0; j < V; ++j) {
                float f[E];
                Codec<S>::unpack(own[j * kBeamThreads], f);
#pragma unroll
                for (int q = 0; q < E; ++q) {
                    const uint64_t key = key_of(f[q], (uint32_t)(first + j * (kBeamThreads * E) + q));
                    if ((uint32_t)(key >> 32) >= least && key < last && key > m)
                        m = key;
                }
            }
            m = warp_max(m);
            __syncthreads();
            if (lane == 0)
                kept[warp] = m;
            __syncthreads();
            last = kept[0];
#pragma unroll
            for (int q = 1; q < kBeamWarps; ++q)
                last = kept[q] > last ? kept[q] : last;
            if (threadIdx.x == 0)
                out[2 + t] = last;
        }
    }
    if (threadIdx.x == 0) {
        uint64_t sum = 0;
#pragma unroll
        for (int q = 0; q < kBeamWarps; ++q)
            sum += (uint64_t)sum_low[q] + ((uint64_t)sum_high[q] << 20);
        out[0] = sum;
        out[1] = __float_as_uint(value_of(top)) | (uint64_t)(uint32_t)(by_power ? (int)power : kNoPower) << 32;
    }
}

// 64-bit scores as unsigned numbers in the order of their values.
__device__ __forceinline__ uint64_t order_of(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double score_of(uint64_t k) { return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k)); }

// The 32 largest of two lists that a warp holds in falling order, a key a lane.
__device__ __forceinline__ uint64_t join_lists(uint64_t p, uint64_t q, int lane) {
    const uint64_t o = __shfl_sync(kFull, q, 31 - lane);
    p = o > p ? o : p;  // rising, then falling: sorted by halves
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
        const uint64_t r = __shfl_xor_sync(kFull, p, d);
        p = ((lane & d) == 0) == (r > p) ? r : p;
    }
    return p;
}

// The logarithm of a beam's sum relative to its largest value: `sum` in units of 2^-30 relative to 2^power, or (kNoPower)
// a double relative to exp(top). The terms' exponents are x log2(e) with log2(e) as f32, so top's is taken the same.
__device__ __forceinline__ double log_of_sum(uint64_t sum, int power, float top) {
    if (power == kNoPower)
        return log(__longlong_as_double((long long)sum));
    return log((double)sum * 0x1p-30) + ((double)power - (double)top * (double)kLog2e) * 0.693147180559945309417;
}

// A warp a beam, and one more for the logarithms of all (64-bit arithmetic is slow here: a warp's instruction takes 16 clocks of
// the SM, so a lane makes each beam's, not a warp).
constexpr int kJoinAhead = 8;  // lists on their way
__global__ void __launch_bounds__(32 * kBeamsMost) k_beam_join(const __grid_constant__ mt_beam_args a, BeamPlan plan) {
    __shared__ uint64_t score[kBeamsMost][kBeamsMost];  // of each beam's first continuations, in order
    __shared__ int32_t token[kBeamsMost][kBeamsMost];
    __shared__ uint64_t sums[kBeamsMost];
    __shared__ int powers[kBeamsMost];
    __shared__ float tops[kBeamsMost];
    __shared__ double less[kBeamsMost];  // the logarithms
    pdl_prologue();
    const int64_t b = blockIdx.x;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, k = warp, chunks = (int)plan.chunks, beams = (int)a.beams;
    const int K = (int)a.beams_out, n = (int)(a.vocab < K ? a.vocab : K);  // continuations of a beam that can matter
    const int64_t row = b * a.beams + (k < beams ? k : 0);
    const uint64_t *mine = static_cast<const uint64_t *>(a.scratch) + row * plan.chunks * plan.slots;
    const float prior = a.prior != nullptr ? tidy(a.prior[row], 3.402823466e38f) : 0.0f;
    const bool done = a.finished != nullptr && a.finished[row] != 0;
    const bool reads = k < beams && !done && prior != Lim<float>::lo();
    uint64_t list[kJoinAhead];
    if (reads) {
#pragma unroll
        for (int q = 0; q < kJoinAhead; ++q)
            list[q] = q < chunks && lane < K ? mine[q * plan.slots + 2 + lane] : 0;
        float top = Lim<float>::lo();
        int power = kLeastPower;
        uint64_t sum = 0;
        if (chunks <= 32) {
            if (lane < chunks) {
                sum = mine[lane * plan.slots];
                const uint64_t o = mine[lane * plan.slots + 1];
                top = __uint_as_float((uint32_t)o);
                power = (int)(uint32_t)(o >> 32);
            }
        } else {
            for (int c = lane; c < chunks; c += 32) {
                const uint64_t o = mine[c * plan.slots + 1];
                top = fmaxf(top, __uint_as_float((uint32_t)o));
                power = max(power, (int)(uint32_t)(o >> 32));
            }
        }
        const int own_power = power;
        top = value_of(redux_max(order_of(top)));
        power = __reduce_max_sync(kFull, power);
        if (power == kNoPower) {  // far out: sums in 64 bits, relative to the largest value
            double all = 0.0;
            for (int c = lane; c < chunks; c += 32) {
                const uint64_t o = mine[c * plan.slots + 1];
                const double m = (double)__uint_as_float((uint32_t)o), s = (double)mine[c * plan.slots] * 0x1p-40;
                const int p = (int)(uint32_t)(o >> 32);
                if (p != kLeastPower)
                    all += s * exp(m - (double)top + (p == kNoPower ? 0.0 : ((double)p - m * (double)kLog2e) * 0.693147180559945309417));
            }
            for (int o = 16; o > 0; o /= 2)
                all += __shfl_xor_sync(kFull, all, o);
            sum = (uint64_t)__double_as_longlong(all);
        } else {
            if (chunks <= 32) {
                sum = sum >> 10 >> min(power - own_power, 53);
            } else {
                for (int c = lane; c < chunks; c += 32)
                    sum += mine[c * plan.slots] >> 10 >> min(power - (int)(uint32_t)(mine[c * plan.slots + 1] >> 32), 53);
            }
            for (int o = 16; o > 0; o /= 2)
                sum += __shfl_xor_sync(kFull, sum, o);
        }
        if (lane == 0) {
            sums[k] = sum;
            powers[k] = power;
            tops[k] = top;
        }
    } else if (k < beams && lane == 0) {
        powers[k] = kLeastPower;
    }
    __syncthreads();
    const int logs = blockDim.x / 32 - 1;  // the warp of the logarithms, a beam's own too where there are 32
    if (warp == logs && lane < beams)
        less[lane] = powers[lane] == kLeastPower ? 0.0 : log_of_sum(sums[lane], powers[lane], tops[lane]);
    uint64_t key = 0;
    if (reads && powers[k] != kLeastPower) {
        for (int c0 = 0; c0 < chunks; c0 += kJoinAhead) {
#pragma unroll
            for (int q = 0; q < kJoinAhead; ++q)
                if (c0 + q < chunks) {
                    key = c0 + q == 0 ? list[q] : join_lists(key, list[q], lane);
                    const int c = c0 + q + kJoinAhead;
                    list[q] = c < chunks && lane < K ? mine[c * plan.slots + 2 + lane] : 0;
                }
        }
    }
    __syncthreads();
    if (k < beams) {
        const int has = __popc(__ballot_sync(kFull, key != 0));  // logits that may come next, as far as they matter
        int32_t tok = (int32_t)~(uint32_t)key;
        double s = Lim<double>::lo();
        if (key != 0)
            s = (double)prior + (((double)value_of((uint32_t)(key >> 32)) - (double)tops[k]) - less[k]);
        if (done && prior != Lim<float>::lo()) {  // the end with the beam's score, then the other tokens in order
            tok = lane == 0 ? (int)a.eos : lane - 1 < a.eos ? lane - 1 : lane;
            if (lane == 0)
                s = (double)prior;
        } else if (has < n) {
            // all that may come next is in the list: behind it the tokens that may not, in order
            int next = 0;
            for (int j = has; j < n; ++j, ++next) {
                while (__any_sync(kFull, lane < has && tok == next))
                    ++next;
                if (lane == j)
                    tok = next;
            }
        }
        if (lane < n) {
            token[k][lane] = tok;
            score[k][lane] = order_of(s);
        }
    }
    __syncthreads();
    if (warp != 0)
        return;
    // beams side by side, each with its best continuation that is left; of equal scores the lowest beam's
    int at = 0, parent = 0, place = 0;
    uint64_t best = 0;
    for (int j = 0; j < K; ++j) {
        const bool has = lane < a.beams && at < n;
        const uint64_t s = has ? score[lane][at] : 0ull;  // 0 is below every score's number
        const uint64_t m = warp_max(s);
        const int from = __ffs(__ballot_sync(kFull, has && s == m)) - 1;
        const int its = __shfl_sync(kFull, at, from);
        if (lane == j) {
            best = m;
            parent = from;
            place = its;
        }
        at += lane == from;
    }
    const int tok = token[parent][place];
    const bool out = lane < K;
    const int64_t to = b * K + lane;
    const bool ended = a.finished != nullptr && out && a.finished[b * a.beams + parent] != 0;
    const int group = (int)(a.beams > K ? a.beams : K);
    const int32_t slot = a.slots != nullptr && lane < group ? a.slots[b * group + lane] : 0;
    __syncwarp();
    if (out) {
        a.tokens[to] = tok;
        a.parents[to] = parent;
        a.scores[to] = (float)score_of(best);
        if (a.finished_out != nullptr)
            a.finished_out[to] = ended || tok == a.eos;
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
        token[0][__popc(free & ((1u << lane) - 1))] = slot;
    __syncwarp();
    const int32_t fresh = token[0][__popc(moving & ((1u << lane) - 1)) & 31];
    if (lane < group)
        a.slots[b * group + lane] = stays ? old : fresh;
    if (out) {
        a.src[to] = stays ? -1 : old;
        a.dst[to] = stays ? -1 : fresh;
    }
}

template <class S, int PER, bool VEC> cudaError_t launch_chunks(const mt_beam_args &a, const BeamPlan &plan, unsigned blocks, const Launch &L) {
    static PerDevice ready;
    constexpr int smem = kBeamThreads * PER * (int)sizeof(S);
    const cudaError_t e = allow_shared(k_beam_chunk<S, PER, VEC>, smem, ready);
    if (e != cudaSuccess)
        return e;
    note_launch();
    return launch_pdl(k_beam_chunk<S, PER, VEC>, blocks, kBeamThreads, smem, L.stream, a, plan);
}
template <class S> cudaError_t launch(const mt_beam_args &a, const Launch &L) {
    const BeamPlan plan = beam_plan(a.batch * a.beams, a.beams_out, a.vocab);
    const int64_t blocks = a.batch * a.beams * plan.chunks, vector = Logits<S>::E;
    if (blocks > INT32_MAX)
        return cudaErrorInvalidValue;
    const bool vec = (uintptr_t)a.logits % 16 == 0 && a.vocab % vector == 0 && a.logits_batch % vector == 0 && a.logits_beam % vector == 0;
    const unsigned n = (unsigned)blocks;
    const cudaError_t e = plan.per_thread == 64 ? (vec ? launch_chunks<S, 64, true>(a, plan, n, L) : launch_chunks<S, 64, false>(a, plan, n, L))
                                                : (vec ? launch_chunks<S, 16, true>(a, plan, n, L) : launch_chunks<S, 16, false>(a, plan, n, L));
    if (e != cudaSuccess)
        return e;
    note_launch();
    return launch_pdl(k_beam_join, (unsigned)a.batch, (unsigned)(32 * (a.beams < kBeamsMost ? a.beams + 1 : kBeamsMost)), 0, L.stream, a, plan);
}

}  // namespace

int64_t beam_scratch_slots(int64_t batch, int64_t beams, int64_t beams_out, int64_t vocab) {
    const BeamPlan plan = beam_plan(batch * beams, beams_out, vocab);
    return batch * beams * plan.chunks * plan.slots;
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
