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
constexpr int64_t kBeamChunk = 8192;  // logits of a CTA

// Logits as unsigned numbers in the order of their values; NaN as -inf, +inf as the largest finite value, -0 as 0.
__device__ __forceinline__ float tidy(float x) {
    x = x == x ? x : Lim<float>::lo();
    return fminf(x, 3.402823466e38f) + 0.0f;
}
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
// Larger values first, of equal ones the lower token.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) { return (uint64_t)order_of(x) << 32 | (uint32_t)~token; }

__device__ __forceinline__ uint32_t redux_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
// The largest of a warp's keys.
__device__ __forceinline__ uint64_t warp_max(uint64_t key) {
    const uint32_t hi = redux_max((uint32_t)(key >> 32));
    const uint32_t lo = redux_max((uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
    return (uint64_t)hi << 32 | lo;
}

// A chunk's place in the scratch: sum and largest value, then beams_out keys.
struct BeamPlan {
    int64_t chunks;  // of a beam's logits
    int64_t slots;   // of a chunk
};
BeamPlan beam_plan(int64_t beams_out, int64_t vocab) { return {(vocab + kBeamChunk - 1) / kBeamChunk, beams_out + 2}; }

template <class S> __global__ void __launch_bounds__(kBeamThreads) k_beam_chunk(mt_beam_args a, BeamPlan plan) {
    __shared__ uint64_t best[kBeamThreads / 32];
    __shared__ double part[kBeamThreads / 32];
    pdl_prologue();
    const int64_t row = blockIdx.x / plan.chunks, chunk = blockIdx.x - row * plan.chunks, b = row / a.beams, k = row - b * a.beams;
    if (a.finished != nullptr && a.finished[row] != 0)
        return;
    const int64_t first = chunk * kBeamChunk;
    const int n = (int)(a.vocab - first < kBeamChunk ? a.vocab - first : kBeamChunk);
    const S *x = static_cast<const S *>(a.logits) + b * a.logits_batch + k * a.logits_beam + first;
    uint64_t *mine = static_cast<uint64_t *>(a.scratch) + (row * plan.chunks + chunk) * plan.slots;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint64_t last = ~0ull;
    float top = 0.0f;
    for (int j = 0; j < a.beams_out && j < n; ++j) {
        uint64_t m = 0;
        for (int t = threadIdx.x; t < n; t += kBeamThreads) {
            const uint64_t key = key_of(tidy(Codec<S>::load1(x + t)), (uint32_t)(first + t));
            if (key < last && key > m)
                m = key;
        }
        m = warp_max(m);
        if (lane == 0)
            best[warp] = m;
        __syncthreads();
        last = best[0];
        for (int w = 1; w < kBeamThreads / 32; ++w)
            last = best[w] > last ? best[w] : last;
        __syncthreads();
        if (j == 0)
            top = value_of((uint32_t)(last >> 32));
        if (threadIdx.x == 0)
            mine[2 + j] = last;
    }
    for (int j = n + threadIdx.x; j < a.beams_out; j += kBeamThreads)
        mine[2 + j] = 0;
    double sum = 0.0;
    if (top != Lim<float>::lo())
        for (int t = threadIdx.x; t < n; t += kBeamThreads)
            sum += (double)ex2f(kLog2e * (tidy(Codec<S>::load1(x + t)) - top));
    for (int o = 16; o > 0; o /= 2)
        sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0)
        part[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kBeamThreads / 32; ++w)
            sum += part[w];
        mine[0] = (uint64_t)__double_as_longlong(sum);
        mine[1] = __float_as_uint(top);
    }
}

// 64-bit scores as unsigned numbers in the order of their values.
__device__ __forceinline__ uint64_t order_of(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double score_of(uint64_t k) { return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k)); }

__global__ void __launch_bounds__(kBeamThreads) k_beam_join(mt_beam_args a, BeamPlan plan) {
    __shared__ uint64_t score[kBeamsMost][kBeamsMost];  // of each beam's first continuations, in order
    __shared__ int32_t token[kBeamsMost][kBeamsMost];
    pdl_prologue();
    const int64_t b = blockIdx.x;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int K = (int)a.beams_out, n = (int)(a.vocab < K ? a.vocab : K);  // continuations of a beam that can matter
    for (int k = warp; k < a.beams; k += kBeamThreads / 32) {
        const int64_t row = b * a.beams + k;
        float prior = a.prior != nullptr ? a.prior[row] : 0.0f;
        prior = tidy(prior);
        const bool done = a.finished != nullptr && a.finished[row] != 0;
        const uint64_t *mine = static_cast<const uint64_t *>(a.scratch) + row * plan.chunks * plan.slots;
        float top = Lim<float>::lo();
        double sum = 0.0;
        if (!done) {
            for (int64_t c = lane; c < plan.chunks; c += 32)
                top = fmaxf(top, __uint_as_float((uint32_t)mine[c * plan.slots + 1]));
            top = value_of(redux_max(order_of(top)));
            for (int64_t c = lane; c < plan.chunks; c += 32) {
                const float m = __uint_as_float((uint32_t)mine[c * plan.slots + 1]);
                if (m != Lim<float>::lo())
                    sum += __longlong_as_double((long long)mine[c * plan.slots]) * exp((double)m - (double)top);
            }
            for (int o = 16; o > 0; o /= 2)
                sum += __shfl_xor_sync(kFull, sum, o);
        }
        if (done || prior == Lim<float>::lo() || top == Lim<float>::lo()) {
            // no logits count: the end with the prior's score (done), and tokens in order that may not come next
            if (lane < n) {
                const bool end = done && lane == 0;
                token[k][lane] = !done ? lane : end ? (int)a.eos : lane - 1 < a.eos ? lane - 1 : lane;
                score[k][lane] = order_of(end ? (double)prior : (double)Lim<float>::lo());
            }
        } else {
            const double less = log(sum);
            uint64_t last = ~0ull;
            for (int j = 0; j < n; ++j) {
                uint64_t m = 0;
                for (int64_t c = lane; c < plan.chunks; c += 32)
                    for (int q = 0; q < K; ++q) {
                        const uint64_t key = mine[c * plan.slots + 2 + q];
                        if (key < last) {
                            m = key > m ? key : m;
                            break;
                        }
                    }
                last = warp_max(m);
                if (lane == 0) {
                    const double x = (double)value_of((uint32_t)(last >> 32)) - (double)top;
                    token[k][j] = (int32_t)~(uint32_t)last;
                    score[k][j] = order_of((double)prior + (x - less));
                }
            }
        }
    }
    __syncthreads();
    if (warp != 0)
        return;
    // beams side by side, each with its best continuation that is left; of equal scores the lowest beam's
    int at = 0, parent = 0, tok = 0;
    float best = 0.0f;
    for (int j = 0; j < K; ++j) {
        const bool has = lane < a.beams && at < n;
        const uint64_t s = has ? score[lane][at] : 0ull;  // 0 is below every score's number
        const uint64_t m = warp_max(s);
        const int from = __ffs(__ballot_sync(kFull, has && s == m)) - 1;
        if (lane == j) {
            best = (float)score_of(m);
            parent = from;
        }
        const int t = token[from][__shfl_sync(kFull, at, from)];
        if (lane == j)
            tok = t;
        at += lane == from;
    }
    const bool out = lane < K;
    const int64_t to = b * K + lane;
    const bool done = a.finished != nullptr && out && a.finished[b * a.beams + parent] != 0;
    const int group = (int)(a.beams > K ? a.beams : K);
    const int32_t slot = a.slots != nullptr && lane < group ? a.slots[b * group + lane] : 0;
    __syncwarp();
    if (out) {
        a.tokens[to] = tok;
        a.parents[to] = parent;
        a.scores[to] = best;
        if (a.finished_out != nullptr)
            a.finished_out[to] = done || tok == a.eos;
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
    const int rank = __popc(moving & ((1u << lane) - 1));
    const int32_t fresh = __shfl_sync(kFull, slot, __fns(free, 0, rank + 1) & 31);
    if (lane < group)
        a.slots[b * group + lane] = stays ? old : fresh;
    if (out) {
        a.src[to] = stays ? -1 : old;
        a.dst[to] = stays ? -1 : fresh;
    }
}

template <class S> cudaError_t launch(const mt_beam_args &a, const Launch &L) {
    const BeamPlan plan = beam_plan(a.beams_out, a.vocab);
    const int64_t blocks = a.batch * a.beams * plan.chunks;
    if (blocks > INT32_MAX)
        return cudaErrorInvalidValue;
    note_launch();
    const cudaError_t e = launch_pdl(k_beam_chunk<S>, (unsigned)blocks, kBeamThreads, 0, L.stream, a, plan);
    if (e != cudaSuccess)
        return e;
    note_launch();
    return launch_pdl(k_beam_join, (unsigned)a.batch, kBeamThreads, 0, L.stream, a, plan);
}

}  // namespace

int64_t beam_scratch_slots(int64_t batch, int64_t beams, int64_t beams_out, int64_t vocab) {
    const BeamPlan plan = beam_plan(beams_out, vocab);
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
