// mt_embed.cu -- embedding lookup with scaling, and the gradient of its table
// by sorted tokens.
//
// Lookup: out[i, :] = scale * table[tok_i, :]. Nothing but bytes: one row read
// and one written per token, 16 bytes a lane and four of them in flight.
//
// Gradient: dtable[v, :] = scale * sum over the tokens i with tok_i = v of
// dout[i, :], which is reduce-by-key with rows for values. Summing by atomics
// would make the result depend on the order the hardware takes them in, so
// the tokens are sorted first, stably, and each run is summed in the order of
// its positions:
//   k_embed_sort  every CTA owns a range of table rows, reads all tokens and
//                 places those of its range, with no word between CTAs: the
//                 number of tokens below its range, which it counts on the way,
//                 is where its part of the order begins;
//   k_embed_sum   a piece of the sorted order per CTA: runs inside the piece are
//                 finished, the first and last run may go on in the neighbours
//                 and leave a partial sum; further CTAs clear the rows that no
//                 token names;
//   k_embed_join  adds the partial sums of a run over its pieces, in order.
#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

// ---- lookup ---------------------------------------------------------------------
constexpr int kEmbThreads = 256;
constexpr int kEmbUnroll = 4;

// E values of a row by one lane: neighbouring (VEC, one 16-byte access) or a
// warp's width apart (rows that no 16-byte access fits).
template <class S, bool VEC> struct RowPart {
    static constexpr int E = Codec<S>::E;
    static constexpr int kSpan = 32 * E;  // columns of a warp
    float x[E];
    __device__ __forceinline__ void load(const S *row, int64_t col0, int64_t dim, int lane) {
        if (VEC) {
            const int64_t c = col0 + lane * E;
            if (c < dim)
                Codec<S>::unpack(ld_stream(reinterpret_cast<const uint4 *>(row + c)), x);
            else
                zero();
        } else {
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const int64_t c = col0 + lane + 32 * k;
                x[k] = c < dim ? Codec<S>::load1(row + c) : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < E; ++k)
            x[k] = 0.0f;
    }
};

template <class S, class Tok, bool VEC>
__global__ void __launch_bounds__(kEmbThreads) k_embed(const Tok *tokens, int64_t ntokens, const S *table, int64_t vocab,
                                                       int64_t dim, float scale, S *out, int64_t chunks) {
    pdl_prologue();
    using R = RowPart<S, VEC>;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kEmbThreads / 32);
    for (int64_t w = (int64_t)blockIdx.x * (kEmbThreads / 32) + (threadIdx.x >> 5); w < ntokens * chunks; w += warps) {
        const int64_t i = w / chunks, col0 = (w - i * chunks) * (R::kSpan * kEmbUnroll);
        const int64_t tok = (int64_t)tokens[i];
        const bool has = tok >= 0 && tok < vocab;  // any other token names no row: zeros
        const S *row = table + (has ? tok : 0) * dim;
        S *to = out + i * dim;
        R r[kEmbUnroll];
#pragma unroll
        for (int k = 0; k < kEmbUnroll; ++k) {
            if (has)
                r[k].load(row, col0 + k * R::kSpan, dim, lane);
            else
                r[k].zero();
        }
#pragma unroll
        for (int k = 0; k < kEmbUnroll; ++k) {
            const int64_t c0 = col0 + k * R::kSpan;
#pragma unroll
            for (int e = 0; e < R::E; ++e)
                r[k].x[e] *= scale;
            if (VEC) {
                const int64_t c = c0 + lane * R::E;
                if (c < dim)
                    st_v4(reinterpret_cast<uint4 *>(to + c), Codec<S>::pack(r[k].x));
            } else {
#pragma unroll
                for (int e = 0; e < R::E; ++e) {
                    const int64_t c = c0 + lane + 32 * e;
                    if (c < dim)
                        Codec<S>::store1(to + c, r[k].x[e]);
                }
            }
        }
    }
}

template <class S, class Tok>
static cudaError_t embed_go(const void *tokens, int64_t n, const void *table, int64_t vocab, int64_t dim, float scale,
                            void *out, const Launch &L) {
    const bool vec = dim % Codec<S>::E == 0 && (uintptr_t)table % 16 == 0 && (uintptr_t)out % 16 == 0;
    const int64_t span = 32 * Codec<S>::E * kEmbUnroll;
    const int64_t chunks = (dim + span - 1) / span;
    const int64_t want = (n * chunks + kEmbThreads / 32 - 1) / (kEmbThreads / 32);
    const unsigned grid = (unsigned)(want < (1 << 30) ? want : (1 << 30));
    note_launch();
    const Tok *t = static_cast<const Tok *>(tokens);
    const S *tab = static_cast<const S *>(table);
    S *o = static_cast<S *>(out);
    return vec ? launch_pdl(k_embed<S, Tok, true>, grid, kEmbThreads, 0, L.stream, t, n, tab, vocab, dim, scale, o, chunks)
               : launch_pdl(k_embed<S, Tok, false>, grid, kEmbThreads, 0, L.stream, t, n, tab, vocab, dim, scale, o, chunks);
}

cudaError_t embed_launch(const void *tokens, bool wide, int64_t n, const void *table, int64_t vocab, int64_t dim,
                         int dtype, float scale, void *out, const Launch &L) {
#define MT_EMBED(S)                                                                              \
    return wide ? embed_go<S, int64_t>(tokens, n, table, vocab, dim, scale, out, L)              \
                : embed_go<S, int32_t>(tokens, n, table, vocab, dim, scale, out, L)
    switch (dtype) {
    case MT_F32: MT_EMBED(float);
    case MT_BF16: MT_EMBED(__nv_bfloat16);
    case MT_F16: MT_EMBED(__half);
    default: return cudaErrorInvalidValue;
    }
#undef MT_EMBED
}

// ---- the sort ---------------------------------------------------------------------
// Work: every CTA reads all T tokens twice (from L2), T/32 a warp, counting
// its range's tokens by warp and row, and then places them. A warp's tokens are
// a contiguous part of the array and are taken in order, so equal tokens keep
// their order: within 32 by their lane, between warps by the counts. Reading
// T tokens in every CTA costs ctas * 4T bytes of L2 traffic (10 MB at T = 16384),
// less than the launches that passing digit counts between CTAs would take.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRows = 1024;  // most table rows per CTA: 32 warps x 1024 counts are 128 KB
constexpr int kSortAhead = 8;

template <class Tok>
__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const Tok *tokens, int64_t ntokens, int64_t vocab,
                                                             int rows, int32_t *start, int32_t *order) {
    extern __shared__ int32_t cnt[];  // [warps][rows]
    __shared__ int32_t s_warp[kSortWarps], s_less;
    pdl_prologue();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t lo = (int64_t)blockIdx.x * rows;
    const int64_t hi = lo + rows < vocab ? lo + rows : vocab;
    const int live = (int)(hi - lo);
    for (int i = tid; i < kSortWarps * rows; i += kSortThreads)
        cnt[i] = 0;
    if (tid == 0)
        s_less = 0;
    __syncthreads();
    const int64_t per = ((ntokens + kSortThreads - 1) / kSortThreads) * 32;  // tokens per warp, whole groups of 32
    const int64_t begin = per * warp < ntokens ? per * warp : ntokens;
    const int64_t end = begin + per < ntokens ? begin + per : ntokens;
    int32_t *mine = cnt + warp * rows;
    int less = 0;
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kSortAhead) {
        int64_t t[kSortAhead];
#pragma unroll
        for (int k = 0; k < kSortAhead; ++k) {
            const int64_t i = i0 + 32 * k + lane;
            t[k] = i < end ? (int64_t)tokens[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < kSortAhead; ++k) {
            less += t[k] >= 0 && t[k] < lo;
            if (t[k] >= lo && t[k] < hi)
                atomicAdd(&mine[t[k] - lo], 1);
        }
    }
    less = __reduce_add_sync(kFull, less);
    if (lane == 0)
        atomicAdd(&s_less, less);
    __syncthreads();
    // one table row a thread (rows <= threads): its tokens before each warp's, and in all
    int total = 0;
    if (tid < live)
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = cnt[w * rows + tid];
            cnt[w * rows + tid] = total;
            total += c;
        }
    int incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, d);
        if (lane >= d)
            incl += v;
    }
    if (lane == 31)
        s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = s_warp[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(kFull, v, d);
            if (lane >= d)
                v += u;
        }
        s_warp[lane] = v;
    }
    __syncthreads();
    const int first = s_less + (warp > 0 ? s_warp[warp - 1] : 0) + incl - total;
    if (tid < live) {
        start[lo + tid] = first;
        if (lo + tid + 1 == vocab)
            start[vocab] = first + total;
        for (int w = 0; w < kSortWarps; ++w)
            cnt[w * rows + tid] += first;
    }
    __syncthreads();
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kSortAhead) {
        int64_t t[kSortAhead];
#pragma unroll
        for (int k = 0; k < kSortAhead; ++k) {
            const int64_t i = i0 + 32 * k + lane;
            t[k] = i < end ? (int64_t)tokens[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < kSortAhead; ++k) {
            const bool in = t[k] >= lo && t[k] < hi;
            const unsigned any = __ballot_sync(kFull, in);
            if (any == 0)
                continue;
            if (in) {
                const int r = (int)(t[k] - lo);
                const unsigned same = __match_any_sync(any, r);
                const int rank = __popc(same & ((1u << lane) - 1u));
                const int at = mine[r];
                __syncwarp(any);
                if (rank == 0)
                    mine[r] = at + __popc(same);
                order[at + rank] = (int32_t)(i0 + 32 * k + lane);
            }
            __syncwarp();
        }
    }
}

// ---- the sums -----------------------------------------------------------------------
template <class G, int E, bool VEC>
__device__ __forceinline__ void put_row(G *row, int64_t col0, int64_t dim, int lane, const float (&x)[E], float scale,
                                        bool accumulate) {
    float v[E];
    if (VEC) {  // E neighbouring columns, whole vectors
        const int64_t c = col0 + lane * E;
        if (c >= dim)
            return;
        constexpr int EG = Codec<G>::E;
        constexpr int kStep = EG < E ? EG : E;
#pragma unroll
        for (int b = 0; b < E; b += kStep) {
            if constexpr (EG <= E) {
                float y[EG];
                if (accumulate) {
                    Codec<G>::unpack(*reinterpret_cast<const uint4 *>(row + c + b), y);
                } else {
#pragma unroll
                    for (int k = 0; k < EG; ++k)
                        y[k] = 0.0f;
                }
#pragma unroll
                for (int k = 0; k < EG; ++k)
                    y[k] = fmaf(scale, x[b + k], y[k]);
                st_v4(reinterpret_cast<uint4 *>(row + c + b), Codec<G>::pack(y));
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int64_t c = col0 + lane + 32 * k;
            if (c < dim) {
                v[k] = accumulate ? Codec<G>::load1(row + c) : 0.0f;
                Codec<G>::store1(row + c, fmaf(scale, x[k], v[k]));
            }
        }
    }
}

struct EmbSumArgs {
    const int32_t *start, *order;
    float *partial;  // [pieces][2][dim]: of the run that came in, of the run that goes on
    int64_t vocab, dim, pieces;
    int piece;
    float scale;
    int accumulate;
    int64_t clear_ctas;
};

constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kSumAhead = 4;  // rows of dout in flight per warp
constexpr int kPieceMost = 1024;

// One CTA sums one piece of the sorted order, each warp its columns: it walks
// the piece's rows with four of them in flight, and where the token changes
// the run's sum leaves the registers. The dout rows are read once, so this
// is bound by bytes: T*H of dout and V*H of the table's gradient, the larger part.
template <class S, class G, class Tok, bool VEC>
__global__ void __launch_bounds__(kSumThreads) k_embed_sum(const Tok *tokens, const S *dout, G *dtable, EmbSumArgs a) {
    __shared__ int32_t s_pos[kPieceMost], s_tok[kPieceMost];
    pdl_prologue();
    using R = RowPart<S, VEC>;
    constexpr int E = R::E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if ((int64_t)blockIdx.x >= a.pieces) {  // rows that no token names
        if (a.accumulate)
            return;
        float z[E];
#pragma unroll
        for (int k = 0; k < E; ++k)
            z[k] = 0.0f;
        const int64_t w0 = ((int64_t)blockIdx.x - a.pieces) * kSumWarps + warp;
        for (int64_t v = w0; v < a.vocab; v += a.clear_ctas * kSumWarps)
            if (a.start[v] == a.start[v + 1])
                for (int64_t c0 = 0; c0 < a.dim; c0 += R::kSpan)
                    put_row<G, E, VEC>(dtable + v * a.dim, c0, a.dim, lane, z, 0.0f, false);
        return;
    }
    const int64_t total = a.start[a.vocab];
    const int64_t p0 = (int64_t)blockIdx.x * a.piece;
    if (p0 >= total)
        return;
    const int n = (int)(total - p0 < a.piece ? total - p0 : a.piece);
    for (int i = tid; i < n; i += kSumThreads) {
        const int32_t at = a.order[p0 + i];
        s_pos[i] = at;
        s_tok[i] = (int32_t)tokens[at];
    }
    __syncthreads();
    const bool comes_in = a.start[s_tok[0]] < p0;           // the first run began before this piece
    const bool goes_on = a.start[s_tok[n - 1] + 1] > p0 + n;  // the last run ends after it
    float *head = a.partial + (int64_t)blockIdx.x * 2 * a.dim, *tail = head + a.dim;
    for (int64_t c0 = (int64_t)warp * R::kSpan; c0 < a.dim; c0 += (int64_t)kSumWarps * R::kSpan) {
        R buf[kSumAhead];
#pragma unroll
        for (int k = 0; k < kSumAhead; ++k)
            if (k < n)
                buf[k].load(dout + (int64_t)s_pos[k] * a.dim, c0, a.dim, lane);
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.0f;
        bool first = true;
        for (int i0 = 0; i0 < n; i0 += kSumAhead) {
#pragma unroll
            for (int k = 0; k < kSumAhead; ++k) {
                const int i = i0 + k;
                if (i < n) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        acc[e] += buf[k].x[e];
                    if (i + kSumAhead < n)
                        buf[k].load(dout + (int64_t)s_pos[i + kSumAhead] * a.dim, c0, a.dim, lane);
                    const int32_t tok = s_tok[i];
                    const bool last = i + 1 == n;
                    if (last || s_tok[i + 1] != tok) {
                        if (first && comes_in)
                            put_row<float, E, VEC>(head, c0, a.dim, lane, acc, 1.0f, false);
                        else if (last && goes_on)
                            put_row<float, E, VEC>(tail, c0, a.dim, lane, acc, 1.0f, false);
                        else
                            put_row<G, E, VEC>(dtable + (int64_t)tok * a.dim, c0, a.dim, lane, acc, a.scale, a.accumulate);
                        first = false;
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            acc[e] = 0.0f;
                    }
                }
            }
        }
    }
}

// The run that begins in piece p and goes on: its sum over the pieces, in order.
template <class G, class Tok>
__global__ void __launch_bounds__(kSumThreads) k_embed_join(const Tok *tokens, G *dtable, EmbSumArgs a) {
    pdl_prologue();
    const int64_t p = blockIdx.x;
    const int64_t total = a.start[a.vocab];
    const int64_t end = (p + 1) * a.piece;
    if (end >= total)
        return;
    const int32_t tok = (int32_t)tokens[a.order[end - 1]];
    const int64_t from = a.start[tok], to = a.start[tok + 1];
    if (to <= end || from < p * a.piece)
        return;
    const int64_t q = (to - 1) / a.piece;  // its last piece
    for (int64_t c = (int64_t)blockIdx.y * kSumThreads + threadIdx.x; c < a.dim; c += (int64_t)gridDim.y * kSumThreads) {
        float s = a.partial[(p * 2 + 1) * a.dim + c];
#pragma unroll 4
        for (int64_t k = p + 1; k <= q; ++k)
            s += a.partial[k * 2 * a.dim + c];
        G *at = dtable + (int64_t)tok * a.dim + c;
        Codec<G>::store1(at, fmaf(a.scale, s, a.accumulate ? Codec<G>::load1(at) : 0.0f));
    }
}

EmbedGradPlan embed_grad_plan(int64_t tokens, int64_t vocab, int64_t dim) {
    EmbedGradPlan p;
    // a CTA of the sort for every SM, with at least 32 rows each and at most kSortRows
    int64_t rows = (vocab + 151) / 152;
    rows = rows < 32 ? 32 : rows > kSortRows ? kSortRows : rows;
    p.rows_per_cta = rows;
    p.ctas = (vocab + rows - 1) / rows;
    // short pieces spread a long run over the GPU; their partial sums stay few
    p.piece = 32;
    while (p.piece < kPieceMost && tokens / p.piece > 4096)
        p.piece *= 2;
    p.pieces = (tokens + p.piece - 1) / p.piece;
    p.start_slots = (vocab + 1 + 3) / 4 * 2;  // int32, 16-byte rounded
    p.order_slots = (tokens + 3) / 4 * 2;
    p.partial_slots = p.pieces * dim;  // two rows of f32 a piece
    return p;
}

template <class S, class G, class Tok>
static cudaError_t embed_grad_go(const void *tokens, int64_t n, const void *dout, int64_t vocab, int64_t dim, float scale,
                                 void *dtable, bool accumulate, uint64_t *scratch, const Launch &L) {
    const EmbedGradPlan p = embed_grad_plan(n, vocab, dim);
    EmbSumArgs a;
    int32_t *start = reinterpret_cast<int32_t *>(scratch);
    int32_t *order = reinterpret_cast<int32_t *>(scratch + p.start_slots);
    a.start = start;
    a.order = order;
    a.partial = reinterpret_cast<float *>(scratch + p.start_slots + p.order_slots);
    a.vocab = vocab;
    a.dim = dim;
    a.pieces = p.pieces;
    a.piece = (int)p.piece;
    a.scale = scale;
    a.accumulate = accumulate;
    a.clear_ctas = accumulate ? 0 : 2 * (int64_t)L.sm_count;
    const Tok *t = static_cast<const Tok *>(tokens);
    const S *d = static_cast<const S *>(dout);
    G *g = static_cast<G *>(dtable);
    const size_t smem = (size_t)p.rows_per_cta * kSortWarps * 4;
    cudaError_t e = cudaFuncSetAttribute(k_embed_sort<Tok>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortRows * kSortWarps * 4);
    if (e != cudaSuccess)
        return e;
    note_launch();
    e = launch_pdl(k_embed_sort<Tok>, (unsigned)p.ctas, kSortThreads, smem, L.stream, t, n, vocab, (int)p.rows_per_cta, start, order);
    if (e != cudaSuccess)
        return e;
    const bool vec = dim % Codec<S>::E == 0 && dim % Codec<G>::E == 0 && (uintptr_t)dout % 16 == 0 &&
                     (uintptr_t)dtable % 16 == 0 && sizeof(G) >= sizeof(S);
    const unsigned grid = (unsigned)(p.pieces + a.clear_ctas);
    if (grid > 0) {
        note_launch();
        e = vec ? launch_pdl(k_embed_sum<S, G, Tok, true>, grid, kSumThreads, 0, L.stream, t, d, g, a)
                : launch_pdl(k_embed_sum<S, G, Tok, false>, grid, kSumThreads, 0, L.stream, t, d, g, a);
        if (e != cudaSuccess)
            return e;
    }
    if (p.pieces > 1) {
        note_launch();
        e = launch_pdl(k_embed_join<G, Tok>, (unsigned)(p.pieces - 1), kSumThreads, 0, L.stream, t, g, a);
    }
    return e;
}

cudaError_t embed_grad_launch(const void *tokens, bool wide, int64_t n, const void *dout, int dtype, int64_t vocab,
                              int64_t dim, float scale, void *dtable, int grad_dtype, bool accumulate, uint64_t *scratch,
                              const Launch &L) {
#define MT_EMBED_GRAD(S, G)                                                                                       \
    return wide ? embed_grad_go<S, G, int64_t>(tokens, n, dout, vocab, dim, scale, dtable, accumulate, scratch, L) \
                : embed_grad_go<S, G, int32_t>(tokens, n, dout, vocab, dim, scale, dtable, accumulate, scratch, L)
    if (grad_dtype == MT_F32) {
        switch (dtype) {
        case MT_F32: MT_EMBED_GRAD(float, float);
        case MT_BF16: MT_EMBED_GRAD(__nv_bfloat16, float);
        case MT_F16: MT_EMBED_GRAD(__half, float);
        default: return cudaErrorInvalidValue;
        }
    }
    if (grad_dtype != dtype)
        return cudaErrorInvalidValue;
    if (dtype == MT_BF16)
        MT_EMBED_GRAD(__nv_bfloat16, __nv_bfloat16);
    MT_EMBED_GRAD(__half, __half);
#undef MT_EMBED_GRAD
}

}  // namespace mt
