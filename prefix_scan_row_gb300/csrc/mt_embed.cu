// mt_embed.cu -- embedding lookup with scaling, and the gradient of its table
// by sorted tokens.
//
// Lookup: out[i, :] = scale * table[tok_i, :]. Nothing but bytes: one row read
// and one written per token, 16 bytes a lane and four of them in flight. 20.3 us for 8192
// rows of 4096 bf16 (134 MB), 97 % of the copy's rate.
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
constexpr int kSortAhead = 16;

template <class Tok>
__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const Tok *tokens, int64_t ntokens, int64_t vocab,
                                                             int rows, int32_t *start, int32_t *order, int32_t *sorted) {
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
    // tokens as 32-bit numbers; any that names no row as -1, which is in no range and below none
    const int lo32 = (int)lo;
    const auto token = [&](int64_t i) {
        if (i >= end)
            return -1;
        const Tok t = tokens[i];
        return t >= 0 && t < (Tok)vocab ? (int)t : -1;
    };
    int less = 0;
    int t[kSortAhead];  // up to 32 * kSortAhead tokens a warp are read once for both passes
    const bool once = per <= 32 * kSortAhead;
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kSortAhead) {
#pragma unroll
        for (int k = 0; k < kSortAhead; ++k)
            t[k] = token(i0 + 32 * k + lane);
#pragma unroll
        for (int k = 0; k < kSortAhead; ++k) {
            less += (unsigned)t[k] < (unsigned)lo32;
            if ((unsigned)(t[k] - lo32) < (unsigned)live && t[k] >= 0)
                atomicAdd(&mine[t[k] - lo32], 1);
        }
    }
    less = __reduce_add_sync(kFull, less);
    if (lane == 0)
        atomicAdd(&s_less, less);
    __syncthreads();
    // one table row a thread (rows <= threads): its tokens before each warp's, and in all
    int total = 0;
    if (tid < live)
#pragma unroll
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
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w)
            cnt[w * rows + tid] += first;
    }
    __syncthreads();
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kSortAhead) {
        if (!once) {
#pragma unroll
            for (int k = 0; k < kSortAhead; ++k)
                t[k] = token(i0 + 32 * k + lane);
        }
#pragma unroll
        for (int k = 0; k < kSortAhead; ++k) {
            const bool in = (unsigned)(t[k] - lo32) < (unsigned)live && t[k] >= 0;
            const unsigned any = __ballot_sync(kFull, in);
            if (any == 0)
                continue;
            if (in) {
                const int r = t[k] - lo32;
                const unsigned same = __match_any_sync(any, r);
                const int rank = __popc(same & ((1u << lane) - 1u));
                const int at = mine[r];
                __syncwarp(any);
                if (rank == 0)
                    mine[r] = at + __popc(same);
                order[at + rank] = (int32_t)(i0 + 32 * k + lane);
                sorted[at + rank] = t[k];
            }
            __syncwarp();
        }
    }
}

// ---- the sums -----------------------------------------------------------------------
// Columns of a row by one lane: two quads 128 apart (VEC: each a vector, of 8 or
// 16 bytes, so that stores of f32 are whole sectors too), or eight a warp's width apart.
template <bool VEC> struct Part {
    static constexpr int kSpan = 256;  // columns of a warp
    float x[8];
    static __device__ __forceinline__ int64_t col(int64_t c0, int k, int lane) {
        return VEC ? c0 + 128 * (k / 4) + 4 * lane + k % 4 : c0 + lane + 32 * k;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = 0.0f;
    }
    // the same of a row in storage form
    template <class S> struct Raw {
        typename VecOf<S, 4>::T w[2];
        __device__ __forceinline__ void load(const S *row, int64_t c0, int64_t dim, int lane) {
            if (VEC) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t c = col(c0, 4 * k, lane);
                    w[k] = *reinterpret_cast<const typename VecOf<S, 4>::T *>(row + (c < dim ? c : 0));  // past the end: not stored
                }
            } else {
                S v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int64_t c = col(c0, k, lane);
                    v[k] = row[c < dim ? c : 0];
                }
                w[0] = *reinterpret_cast<typename VecOf<S, 4>::T *>(v);
                w[1] = *reinterpret_cast<typename VecOf<S, 4>::T *>(v + 4);
            }
        }
        __device__ __forceinline__ void add(Part &to) const {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float v[4];
                widen4<S>(w[k], v);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    to.x[4 * k + e] += v[e];
            }
        }
    };
    template <class S> __device__ __forceinline__ void load(const S *row, int64_t c0, int64_t dim, int lane) {
        if (VEC) {
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
                const int64_t c = col(c0, k, lane);
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (c < dim)
                    widen4<S>(*reinterpret_cast<const typename VecOf<S, 4>::T *>(row + c), v);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[k + e] = v[e];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int64_t c = col(c0, k, lane);
                x[k] = c < dim ? Codec<S>::load1(row + c) : 0.0f;
            }
        }
    }
    template <class G>
    __device__ __forceinline__ void store(G *row, int64_t c0, int64_t dim, int lane, float scale, bool accumulate) const {
        Part old;
        if (accumulate)
            old.load(row, c0, dim, lane);
        else
            old.zero();
        if (VEC) {
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
                const int64_t c = col(c0, k, lane);
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = fmaf(scale, x[k + e], old.x[k + e]);
                if (c < dim)
                    *reinterpret_cast<typename VecOf<G, 4>::T *>(row + c) = narrow4<G>(v);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int64_t c = col(c0, k, lane);
                if (c < dim)
                    Codec<G>::store1(row + c, fmaf(scale, x[k], old.x[k]));
            }
        }
    }
};

struct EmbSumArgs {
    const int32_t *start, *order, *sorted;
    float *partial;  // [pieces][2][dim]: of the run that came in, of the run that goes on
    int32_t *last;   // [pieces]: the last piece of the run that begins here and goes on, or 0
    int64_t vocab, dim, pieces, ntokens;
    int piece;
    float scale;
    int accumulate;
    int64_t clear_ctas;
};

constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kSumAhead = 8;  // rows of dout in flight per warp
constexpr int kPieceMost = 1024;
constexpr int kClearRows = 16;  // looked at together by a clearing warp

// One CTA sums one piece of the sorted order, each warp its columns: it takes
// the piece's rows a few at a time, all loaded before the first is added, and where the token
// changes the run's sum leaves the registers. Where each sum goes is worked
// out once for the piece, so a row costs its loads, its additions and one test. The dout rows are read once: bound
// by bytes, T*H of dout and V*H of the table's gradient, the larger part: of the 80 us of 16384 tokens
// of 2048 bf16 into 32768 rows of f32, 59 are here, 336 MB at 5.7 TB/s (stores alone reach 5.2).
constexpr int kNowhere = -1, kHead = -2, kTail = -3;  // where a row's sum goes, but for a row of the table

template <class S, class G, bool VEC>
__global__ void __launch_bounds__(kSumThreads, 2) k_embed_sum(const S *dout, G *dtable, EmbSumArgs a) {
    __shared__ int32_t s_pos[kPieceMost], s_to[kPieceMost], s_tok[kPieceMost];
    pdl_prologue();
    using R = Part<VEC>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // pieces and clearing CTAs take turns, so that reading and writing overlap
    const int64_t pair = blockIdx.x / 2, both = a.pieces < a.clear_ctas ? a.pieces : a.clear_ctas;
    const bool clears = pair < both ? (blockIdx.x & 1) != 0 : a.clear_ctas > a.pieces;
    const int64_t index = pair < both ? pair : (int64_t)blockIdx.x - both;
    if (clears) {  // rows that no token names
        R z;
        z.zero();
        for (int64_t v0 = (index * kSumWarps + warp) * kClearRows; v0 < a.vocab; v0 += a.clear_ctas * kSumWarps * kClearRows) {
            const int64_t v = v0 + lane;
            unsigned none = __ballot_sync(kFull, lane < kClearRows && v < a.vocab && a.start[v < a.vocab ? v : 0] == a.start[v < a.vocab ? v + 1 : 0]);
            for (; none != 0; none &= none - 1) {
                const int64_t row = v0 + __ffs(none) - 1;
                for (int64_t c0 = 0; c0 < a.dim; c0 += R::kSpan)
                    z.store(dtable + row * a.dim, c0, a.dim, lane, 0.0f, false);
            }
        }
        return;
    }
    const int64_t total = a.start[a.vocab];
    const int64_t p0 = index * a.piece;
    for (int i = tid; i < a.piece && p0 + i < a.ntokens; i += kSumThreads) {  // past the total: not used
        s_pos[i] = a.order[p0 + i];
        s_tok[i] = a.sorted[p0 + i];
    }
    if (p0 >= total) {
        if (tid == 0)
            a.last[index] = 0;
        return;
    }
    const int n = (int)(total - p0 < a.piece ? total - p0 : a.piece);
    __syncthreads();
    for (int i = tid; i < n; i += kSumThreads) {
        const int32_t tok = s_tok[i];
        int32_t to = kNowhere;
        if (i + 1 == n || s_tok[i + 1] != tok) {
            const int64_t from = a.start[tok], end = a.start[tok + 1];
            to = from < p0 ? kHead : end > p0 + n ? kTail : tok;
            if (i + 1 == n)  // a run that begins here and goes on is this piece's to join
                a.last[index] = to == kTail ? (int32_t)((end - 1) / a.piece) : 0;
        }
        s_to[i] = to;
    }
    __syncthreads();
    float *head = a.partial + index * 2 * a.dim, *tail = head + a.dim;
    for (int64_t c0 = (int64_t)warp * R::kSpan; c0 < a.dim; c0 += (int64_t)kSumWarps * R::kSpan) {
        R acc;
        acc.zero();
        for (int i0 = 0; i0 < n; i0 += kSumAhead) {
            typename R::template Raw<S> buf[kSumAhead];
#pragma unroll
            for (int k = 0; k < kSumAhead; ++k)
                buf[k].load(dout + (int64_t)s_pos[i0 + k < n ? i0 + k : n - 1] * a.dim, c0, a.dim, lane);
#pragma unroll
            for (int k = 0; k < kSumAhead; ++k) {
                if (i0 + k < n) {
                    buf[k].add(acc);
                    const int32_t to = s_to[i0 + k];
                    if (to != kNowhere) {
                        if (to >= 0)
                            acc.store(dtable + (int64_t)to * a.dim, c0, a.dim, lane, a.scale, a.accumulate);
                        else
                            acc.store(to == kHead ? head : tail, c0, a.dim, lane, 1.0f, false);
                        acc.zero();
                    }
                }
            }
        }
    }
}

// Runs that go on: their sums over the pieces. A warp takes one of the CTA's eight
// pieces, and 128 columns of the run that begins there; a run over more than
// kFewPieces is left to all eight warps, of which each adds every eighth
// piece, and the eight sums are added in order: a token that fills
// hundreds of pieces is not one chain of loads.
constexpr int kFewPieces = 12;

template <class G>
__global__ void __launch_bounds__(kSumThreads) k_embed_join(G *dtable, EmbSumArgs a) {
    __shared__ float s_sum[kSumWarps][128];
    pdl_prologue();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t p0 = (int64_t)blockIdx.x * kSumWarps, c0 = (int64_t)blockIdx.y * 128 + lane;  // columns c0 + 32 k
    const int32_t mine = lane < kSumWarps && p0 + lane < a.pieces ? a.last[p0 + lane] : 0;
    const auto add = [&](int64_t from, int64_t to, int64_t first, int64_t by, float (&s)[4]) {
#pragma unroll 4
        for (int64_t k = from; k <= to; k += by) {
            const float *row = a.partial + (k == first ? k * 2 + 1 : k * 2) * a.dim;  // where it begins: the run that goes on
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[e] += c0 + 32 * e < a.dim ? row[c0 + 32 * e] : 0.0f;
        }
    };
    const auto put = [&](int64_t p, const float (&s)[4]) {
        G *row = dtable + (int64_t)a.sorted[(p + 1) * a.piece - 1] * a.dim;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c0 + 32 * e < a.dim)
                Codec<G>::store1(row + c0 + 32 * e, fmaf(a.scale, s[e], a.accumulate ? Codec<G>::load1(row + c0 + 32 * e) : 0.0f));
    };
    const int64_t q = __shfl_sync(kFull, mine, warp), p = p0 + warp;
    if (q != 0 && q - p < kFewPieces) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        add(p, q, p, 1, s);
        put(p, s);
    }
    unsigned many = __ballot_sync(kFull, mine != 0 && mine - (p0 + lane) >= kFewPieces);
    for (; many != 0; many &= many - 1) {  // the same for all warps
        const int i = __ffs(many) - 1;
        const int64_t first = p0 + i, end = __shfl_sync(kFull, mine, i);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        add(first + warp, end, first, kSumWarps, s);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s_sum[warp][lane + 32 * e] = s[e];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int w = 1; w < kSumWarps; ++w)
                    s[e] += s_sum[w][lane + 32 * e];
            }
            put(first, s);
        }
        __syncthreads();
    }
}

EmbedGradPlan embed_grad_plan(int64_t tokens, int64_t vocab, int64_t dim) {
    EmbedGradPlan p;
    // a CTA of the sort for every SM, with at least 32 rows each and at most kSortRows
    int64_t rows = (vocab + 151) / 152;
    rows = rows < 32 ? 32 : rows > kSortRows ? kSortRows : rows;
    p.rows_per_cta = rows;
    p.ctas = (vocab + rows - 1) / rows;
    // short pieces spread the rows, and a long run, over the GPU; their partial sums stay few
    p.piece = 8;
    while (p.piece < kPieceMost && tokens / p.piece > 1024)
        p.piece *= 2;
    p.pieces = (tokens + p.piece - 1) / p.piece;
    p.start_slots = (vocab + 1 + 3) / 4 * 2;  // int32, 16-byte rounded
    p.order_slots = (tokens + 3) / 4 * 2;
    p.partial_slots = p.pieces * dim;  // two rows of f32 a piece
    p.last_slots = (p.pieces + 3) / 4 * 2;
    return p;
}

template <class S, class G, class Tok>
static cudaError_t embed_grad_go(const void *tokens, int64_t n, const void *dout, int64_t vocab, int64_t dim, float scale,
                                 void *dtable, bool accumulate, uint64_t *scratch, const Launch &L) {
    const EmbedGradPlan p = embed_grad_plan(n, vocab, dim);
    EmbSumArgs a;
    int32_t *start = reinterpret_cast<int32_t *>(scratch);
    int32_t *order = reinterpret_cast<int32_t *>(scratch + p.start_slots);
    int32_t *sorted = reinterpret_cast<int32_t *>(scratch + p.start_slots + p.order_slots);
    a.start = start;
    a.order = order;
    a.sorted = sorted;
    a.last = reinterpret_cast<int32_t *>(scratch + p.start_slots + 2 * p.order_slots);
    a.partial = reinterpret_cast<float *>(scratch + p.start_slots + 2 * p.order_slots + p.last_slots);
    a.vocab = vocab;
    a.dim = dim;
    a.pieces = p.pieces;
    a.ntokens = n;
    a.piece = (int)p.piece;
    a.scale = scale;
    a.accumulate = accumulate;
    a.clear_ctas = accumulate ? 0 : (vocab + kClearRows * kSumWarps - 1) / (kClearRows * kSumWarps);
    if (a.clear_ctas > 4 * (int64_t)L.sm_count)
        a.clear_ctas = 4 * (int64_t)L.sm_count;
    const Tok *t = static_cast<const Tok *>(tokens);
    const S *d = static_cast<const S *>(dout);
    G *g = static_cast<G *>(dtable);
    const size_t smem = (size_t)p.rows_per_cta * kSortWarps * 4;
    cudaError_t e = cudaFuncSetAttribute(k_embed_sort<Tok>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortRows * kSortWarps * 4);
    if (e != cudaSuccess)
        return e;
    note_launch();
    e = launch_pdl(k_embed_sort<Tok>, (unsigned)p.ctas, kSortThreads, smem, L.stream, t, n, vocab, (int)p.rows_per_cta, start, order, sorted);
    if (e != cudaSuccess)
        return e;
    const bool vec = dim % 4 == 0 && (uintptr_t)dout % (4 * sizeof(S)) == 0 && (uintptr_t)dtable % (4 * sizeof(G)) == 0;
    const unsigned grid = (unsigned)(p.pieces + a.clear_ctas);
    if (grid > 0) {
        note_launch();
        e = vec ? launch_pdl(k_embed_sum<S, G, true>, grid, kSumThreads, 0, L.stream, d, g, a)
                : launch_pdl(k_embed_sum<S, G, false>, grid, kSumThreads, 0, L.stream, d, g, a);
        if (e != cudaSuccess)
            return e;
    }
    if (p.pieces > 1) {
        note_launch();
        e = launch_pdl_2d(k_embed_join<G>, dim3((unsigned)((p.pieces + kSumWarps - 1) / kSumWarps), (unsigned)((dim + 127) / 128)), kSumThreads, L.stream, g, a);
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
