// mt_copy.cu -- copies between slots of state pools.
//
// Rows of a pool of layers lie far apart, so a CTA takes one chunk of a row and plane, 16 KB, with the widest accesses that the
// pool's addresses and sizes allow. Where there are many pairs it takes that chunk of up to 32 of them, since most pairs of
// a beam search copy nothing and a CTA for each costs more than the rest of its work. Only bytes count: each is read
// once and written once. 64 sequences of 8 beams, 192 copies of 287 KB in each of 4 layers: 66 us in a CUDA graph, 98 % of the measured
// copy rate (6798 GB/s); one sequence of 4 beams, one layer: 2.0.
#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyInFlight = 4;                                       // loads of a thread before its stores
constexpr int64_t kCopyChunk = 16 * kCopyThreads * kCopyInFlight;      // bytes of a CTA
// More CTAs than these take more pairs each. us, by one pair a CTA, this rule, and one wave of CTAs (152 x 8): 64 x 8 beams x 4 layers, 3 of
// 8 beams copied 83.9, 66.0, 69.6; 7 of 8 106, 91, 98; one layer 22.7, 17.9, 15.1; 8 x 4 beams x 4 layers 6.4, 6.4, 5.9.
constexpr int64_t kEnoughCtas = 152 * 8 * 4;

struct CopyPool {
    char *base;
    int64_t nslots, row_bytes, row_stride, plane_stride;
    int64_t first;   // of the grid's first axis: the pools before it
    int64_t chunks;  // of a row
    int bytes;       // of an access: 16, 8, 4, 2 or 1
};
struct CopyArgs {
    const int32_t *src, *dst;
    int64_t pairs;
    int npools, per_cta;  // pairs of a CTA
    CopyPool pool[MT_MOST_POOLS];
};

template <class T> __device__ __forceinline__ void copy_span(const char *from, char *to, int64_t bytes) {
    const T *f = reinterpret_cast<const T *>(from);
    T *t = reinterpret_cast<T *>(to);
    const int n = (int)(bytes / (int64_t)sizeof(T));
    for (int k0 = threadIdx.x; k0 < n; k0 += kCopyThreads * kCopyInFlight) {
        T v[kCopyInFlight];
#pragma unroll
        for (int k = 0; k < kCopyInFlight; ++k)
            if (k0 + k * kCopyThreads < n)
                v[k] = f[k0 + k * kCopyThreads];
#pragma unroll
        for (int k = 0; k < kCopyInFlight; ++k)
            if (k0 + k * kCopyThreads < n)
                t[k0 + k * kCopyThreads] = v[k];
    }
}

__global__ void __launch_bounds__(kCopyThreads) k_state_copy(const __grid_constant__ CopyArgs a) {
    pdl_prologue();
    int which = 0;
    while (which + 1 < a.npools && (int64_t)blockIdx.x >= a.pool[which + 1].first)
        ++which;
    const CopyPool &p = a.pool[which];
    const int64_t at = (int64_t)blockIdx.x - p.first, plane = at / p.chunks, chunk = at - plane * p.chunks;
    const int64_t begin = chunk * kCopyChunk;
    const int64_t bytes = p.row_bytes - begin < kCopyChunk ? p.row_bytes - begin : kCopyChunk;
    char *rows = p.base + plane * p.plane_stride + begin;
    const int lane = threadIdx.x % 32;
    for (int64_t i0 = (int64_t)blockIdx.y * a.per_cta; i0 < a.pairs; i0 += (int64_t)gridDim.y * a.per_cta) {
        int32_t s = -1, d = -1;
        if (lane < a.per_cta && i0 + lane < a.pairs) {
            s = a.src[i0 + lane];
            d = a.dst[i0 + lane];
        }
        for (uint32_t left = __ballot_sync(kFull, s >= 0 && s < p.nslots && d >= 0 && d < p.nslots && s != d); left != 0; left &= left - 1) {
            const int q = __ffs(left) - 1;
            const char *from = rows + (int64_t)__shfl_sync(kFull, s, q) * p.row_stride;
            char *to = rows + (int64_t)__shfl_sync(kFull, d, q) * p.row_stride;
            switch (p.bytes) {
            case 16: copy_span<uint4>(from, to, bytes); break;
            case 8: copy_span<uint2>(from, to, bytes); break;
            case 4: copy_span<uint32_t>(from, to, bytes); break;
            case 2: copy_span<uint16_t>(from, to, bytes); break;
            default: copy_span<uint8_t>(from, to, bytes);
            }
        }
    }
}

}  // namespace

cudaError_t copy_launch(const int32_t *src, const int32_t *dst, int64_t pairs, const mt_pool *pools, int64_t npools,
                        const Launch &L) {
    CopyArgs a;
    a.src = src;
    a.dst = dst;
    a.pairs = pairs;
    a.npools = 0;
    int64_t blocks = 0;
    for (int64_t k = 0; k < npools; ++k) {
        const mt_pool &p = pools[k];
        if (p.nslots == 0 || p.planes == 0 || p.row_bytes == 0)
            continue;
        CopyPool &q = a.pool[a.npools++];
        q.base = static_cast<char *>(p.base);
        q.nslots = p.nslots;
        q.row_bytes = p.row_bytes;
        q.row_stride = p.row_stride;
        q.plane_stride = p.planes > 1 ? p.plane_stride : 0;
        q.first = blocks;
        q.chunks = (p.row_bytes + kCopyChunk - 1) / kCopyChunk;
        q.bytes = 16;
        const uint64_t all = (uint64_t)(uintptr_t)p.base | (uint64_t)q.row_bytes | (uint64_t)q.row_stride | (uint64_t)q.plane_stride;
        while (all % q.bytes != 0)
            q.bytes /= 2;
        blocks += q.chunks * p.planes;
        if (blocks > INT32_MAX)
            return cudaErrorInvalidValue;
    }
    if (blocks == 0)
        return cudaSuccess;
    a.per_cta = 1;
    while (a.per_cta < 32 && blocks * ((pairs + a.per_cta - 1) / a.per_cta) > kEnoughCtas)
        a.per_cta *= 2;
    const int64_t rows = (pairs + a.per_cta - 1) / a.per_cta;
    note_launch();
    const dim3 grid((unsigned)blocks, (unsigned)(rows < 65535 ? rows : 65535));
    return launch_pdl_2d(k_state_copy, grid, kCopyThreads, L.stream, a);
}

}  // namespace mt
