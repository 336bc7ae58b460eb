// mt_gated.cu -- plans and launches of the gated scan, and the join of its parameter's sums.
#include "mt_gated.cuh"

namespace mt {

// CTAs that share a sequence's tokens: one where sequences and channels give every SM work, and otherwise as many as find
// place at once, two an SM. A cluster's CTAs wait for one another at every tile, so it pays only then. bf16, all gates, prompt, us, in
// clusters of 1, 2, 4 and 8 CTAs: 4 x 2048 tokens x 4096 channels (256 CTAs without clusters) 73, 89, 86, 101; 16384 tokens x
// 2048 (32) 339, 224, 117, 98 (eight warps of 8 tokens a CTA). Of the sizes with the same number of tiles the smallest.
// The scratch is sized on the host, so the plan counts GB300's 152 SMs, and by the cluster's size the CTAs that were found to run
// at once: clusters lie within a group of SMs, so not all places can be taken (a prompt of 2048 tokens
// and its gradient in 264 CTAs, 44 clusters of 6, 23 and 32 us; in 288, 48 clusters, 33 and 51).
constexpr int kPlaces[] = {0, 304, 304, 276, 276, 264, 264, 252, 264}, kMostCtas = 8;
static int gated_ctas(int64_t batch, int64_t len, int64_t dim, int64_t cta_tokens) {
    const int64_t units = batch * ((dim + kGatedSlab - 1) / kGatedSlab), tiles = (len + cta_tokens - 1) / cta_tokens;
    int64_t n = kMostCtas;
    while (n > 1 && (units * n > kPlaces[n] || n > tiles))
        --n;
    const int64_t rounds = (tiles + n - 1) / n;
    return rounds > 0 ? (int)((tiles + rounds - 1) / rounds) : 1;
}

// A sum of every CTA and channel, no fewer than any smaller call has, although one may take larger clusters: these have as many CTAs as there are
// tiles at most, and only where all CTAs, of 64 channels each, are no more than the places for clusters of two.
int64_t gated_scratch_slots(int64_t batch, int64_t len, int64_t dim) {
    const int64_t tiles = (len + kBwdWarps * kBwdT - 1) / (kBwdWarps * kBwdT), shared = kPlaces[2] * kGatedSlab;
    const int64_t sums = batch * dim, more = sums * (tiles < 1 ? 1 : tiles < kMostCtas ? tiles : kMostCtas);
    const int64_t most = more < shared ? more : shared;
    return ((sums > most ? sums : most) + 1) / 2;
}

// Sums of parts [rows, dim] over the rows, in order: a warp's lanes share 32 channels, its CTA's warps the rows.
static __global__ void __launch_bounds__(256) k_gated_rate_join(const float *part, float *drate, int64_t rows, int64_t dim) {
    __shared__ float sums[8][32];
    pdl_prologue();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t d = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (d < dim)
        for (int64_t k = warp; k < rows; k += 8)
            s += part[k * dim + d];
    sums[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || d >= dim)
        return;
#pragma unroll
    for (int w = 1; w < 8; ++w)
        s += sums[w][lane];
    drate[d] = s;
}

// b is a token's stride, which the kernels for whole vectors take in 32 bits (in bytes)
static bool fits(const void *p, int64_t a, int64_t b, int64_t bytes, int64_t values) {
    return (uintptr_t)p % bytes == 0 && a % values == 0 && b % values == 0 && b > -(1 << 29) && b < 1 << 29;
}
// whether `bytes` of every tensor's channels can be moved as one
static bool all_fit(const mt_gated_args &p, int64_t bytes, bool step, bool grad) {
    const int64_t v = bytes / (p.dtype == MT_F32 ? 4 : 2), t = step ? 0 : 1;
    bool fit = p.dim % v == 0 && fits(p.x, p.x_batch, p.x_token * t, bytes, v) && fits(p.r, p.r_batch, p.r_token * t, bytes, v) &&
               (p.i == nullptr || fits(p.i, p.i_batch, p.i_token * t, bytes, v)) &&
               (p.z == nullptr || fits(p.z, p.z_batch, p.z_token * t, bytes, v));
    if (!grad)
        return fit && fits(p.out, p.out_batch, p.out_token * t, bytes, v);
    return fit && fits(p.dout, p.dout_batch, p.dout_token, bytes, v) && fits(p.dx, p.dx_batch, p.dx_token, bytes, v) &&
           fits(p.dr, p.dr_batch, p.dr_token, bytes, v) && (p.i == nullptr || fits(p.di, p.di_batch, p.di_token, bytes, v)) &&
           (p.z == nullptr || fits(p.dz, p.dz_batch, p.dz_token, bytes, v));
}

static GatedArgs gated_args(const mt_gated_args &p, int64_t cta_tokens, const Launch &L) {
    GatedArgs g;
    g.p = p;
    g.slabs = (int)((p.dim + kGatedSlab - 1) / kGatedSlab);
    g.ctas = gated_ctas(p.batch, p.len, p.dim, cta_tokens);
    g.ntiles = (p.len + kGatedTile - 1) / kGatedTile;
    g.limit = L.spin_limit != kDefaultSpin ? L.spin_limit : kCopyWaitLimit;  // the test hook's, where it is set
    g.silent = L.skip_tile;
    return g;
}

#define MT_BY_TYPE(f, ...)                              \
    switch (p.dtype) {                                  \
    case MT_F32: return f##_f32(__VA_ARGS__);           \
    case MT_BF16: return f##_bf16(__VA_ARGS__);         \
    case MT_F16: return f##_f16(__VA_ARGS__);           \
    default: return cudaErrorInvalidValue;              \
    }
cudaError_t gated_launch(const mt_gated_args &p, const Launch &L) {
    const GatedArgs g = gated_args(p, kGatedWarps * gated_cluster_tokens(p.dtype == MT_F32 ? 4 : 2), L);
    const bool vec = all_fit(p, 16, false, false);
    if (p.batch * g.slabs * g.ctas > INT32_MAX)
        return cudaErrorInvalidValue;
    MT_BY_TYPE(gated_forward, g, vec, L)
}
cudaError_t gated_step_launch(const mt_gated_args &a, const Launch &L) {
    mt_gated_args p = a;
    p.len = 1;
    const GatedArgs g = gated_args(p, kFwdT, L);
    const bool vec = all_fit(p, p.dtype == MT_F32 ? 8 : 4, true, false);
    if (p.batch * ((p.dim + 1) / 2) / 128 >= INT32_MAX)
        return cudaErrorInvalidValue;
    MT_BY_TYPE(gated_single, g, vec, L)
}
static cudaError_t backward(const GatedArgs &g, float *part, const Launch &L) {
    const mt_gated_args &p = g.p;
    const bool vec = all_fit(p, 16, false, true);
    MT_BY_TYPE(gated_backward, g, part, vec, L)
}
cudaError_t gated_grad_launch(const mt_gated_args &p, const Launch &L) {
    const GatedArgs g = gated_args(p, kBwdWarps * kBwdT, L);
    float *part = p.drate != nullptr ? static_cast<float *>(p.scratch) : nullptr;
    if (p.batch * g.slabs * g.ctas > INT32_MAX)
        return cudaErrorInvalidValue;
    if (p.batch > 0) {
        const cudaError_t e = backward(g, part, L);
        if (e != cudaSuccess)
            return e;
    }
    if (p.drate == nullptr)
        return cudaSuccess;
    note_launch();
    return launch_pdl(k_gated_rate_join, (unsigned)((p.dim + 31) / 32), 256, 0, L.stream, part, p.drate, p.batch * g.ctas, p.dim);
}
#undef MT_BY_TYPE

}  // namespace mt
