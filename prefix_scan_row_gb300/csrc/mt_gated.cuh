// mt_gated.cuh -- the gated scan's mathematics, and its kernels, instantiated per activation type (mt_gated_*.cu).
//
//   s = sigma(r);  a = exp(-rate s), w = sqrt(1 - a^2)  or, without rate,  a = 1 - s, w = s
//   h_t = a_t h_{t-1} + w_t v_t,  v = sigma(i) x or x,  out = h or h z sigma(z)
//
// Gradient, with g_t the gradient by h_t (from out_t, and from h_{t+1} through a_{t+1}):
//   dh = dout z sigma(z),  g_t = dh_t + a_{t+1} g_{t+1},  dz = dout h sigma(z) (1 + z (1 - sigma(z)))
//   dx = g w sigma(i),  di = dx x (1 - sigma(i))
//   rate: with u = rate s, da/du = -a and dw/du = a^2 / w, so e = g (v a^2 / w - h_{t-1} a) s,
//         dr = e rate (1 - s), drate = sum of e;  no rate: dr = g (v - h_{t-1}) s (1 - s)
//
// Both recurrences are scans with the operator (a, b) o (a', b') = (a a', a' b + b'). The floor is bytes: a
// token's channel is 6 to 8 of them at 16-bit storage (gradient 10 to 18), and its 5 to 8 exponentials,
// reciprocals and roots, at 30.5 a clock and SM, take less.
//
// So every input is read once: the token axis is cut over the warps of a CTA, and where sequences and channels alone
// do not fill the GPU over the CTAs of a cluster too. A warp has kT tokens of 64 channels, a lane a pair of channels in
// a register pair; it makes the decays and inputs of its tokens, and their product and sum as one element of the
// scan. The elements meet in shared memory, those of a cluster's CTAs in each other's, and each warp then
// knows its first state and finishes its tokens, whose decays and inputs are still in registers. Nothing is
// computed or read twice. A cluster's CTAs are resident together, so their waits for one another end.
//
// Measured, all gates, us (share of the measured copy rate, 6798 GB/s): 16 x 1024 tokens x 4096 channels bf16, prompt 111
// (89 %), gradient 221 (81 %); 4 x 2048 x 4096 bf16 68 (73 %) and 121 (73 %): 256 CTAs leave some SMs two and others one, and
// the schedulers, the exponentials' unit and the multiply-adds' are each 25 to 55 % busy (78 instructions for a pair's token in
// the prompt, 136 in the gradient); 16384 x 2048 bf16 86 (58 %) and 147 (60 %): the same, and clusters' waits; 8 x 2048 x 4096
// f32 211 (94 %) and 410 (87 %).
#pragma once

#include <initializer_list>
#include <type_traits>

#include "mt_seq.cuh"
#include "mt_seq.h"

namespace mt {

constexpr int kGatedSlab = 64;   // channels of a warp
// A prompt's CTA: its warps and their tokens. us, all gates but where said, 4096 channels, by sequences x tokens (CTAs).
// 16-bit, four warps of 16 tokens, two CTAs an SM, up to three CTAs an SM in all, and beyond that of 8 tokens, four CTAs an SM, whose ends
// leave less idle; against eight warps of 8: 4 x 2048 (256) 69, 73; without output gate 4 x 4096 (256) 107, 117; 7 x 2048 (448) 108, 110;
// 8 x 2048 (512) 128, of 16 tokens 134, eight warps 140; 16 x 1024 (1024) 112, 123, 125. 4 tokens, eight warps, three CTAs an SM, 4 x 2048: 115.
// f32, eight warps of 8 tokens, one CTA an SM: 8 x 2048 (512) 211, four warps 246.
// Clusters, two of whose CTAs have to be on an SM: four warps, of 16 and f32 of 8 tokens; against eight of 8, as measured together: bf16 16384 x 2048
// channels 91, 107 (one warp joining for all: 99), 86 now; 2 x 2048 44, 49; f32 16384 x 2048 channels 127, 221, 115 now; 4096 64, 76.
constexpr int kGatedWarps = 4, kGatedWholeWarps = 8;
constexpr int kFwdT = 8, kFwdMoreT = 16;
constexpr int gated_cluster_tokens(int bytes) { return bytes == 4 ? kFwdT : kFwdMoreT; }
constexpr int kGatedStages = 2;  // tiles of a warp on their way or in use

struct GatedArgs {
    mt_gated_args p;
    int slabs;       // of 64 channels
    int ctas;        // of a cluster
    int64_t ntiles;  // checkpoints of a sequence
    uint32_t limit;  // polls of a wait for a cluster's CTAs
    int64_t silent;  // test hook: the CTA that tells the others nothing (-1: none)
};

__device__ __forceinline__ int64_t gated_len(const mt_gated_args &p, int64_t b) {
    const int64_t n = p.lens != nullptr ? (int64_t)p.lens[b] : p.len;
    return n < 0 ? 0 : n > p.len ? p.len : n;
}
__device__ __forceinline__ int64_t gated_slot(const mt_gated_args &p, int64_t b) {
    const int64_t s = p.slots != nullptr ? (int64_t)p.slots[b] : b;
    return s >= 0 && s < p.nslots ? s : -1;
}

struct alignas(16) Element {  // of the scan
    f32x2 a, h;
};

// ---- clusters -----------------------------------------------------------------------------------
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Two pairs to the same place in another CTA's shared memory, counted by the barrier at the same place there: data and
// signal go one way together, where stores and a barrier of the cluster go there, back, and there again.
__device__ __forceinline__ void cluster_send(uint32_t here, uint32_t bar_here, unsigned rank, f32x2 a, f32x2 b) {
    uint32_t there, bar;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(bar_here), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];"
                 :: "r"(there), "l"(a), "l"(b), "r"(bar) : "memory");
}
// One poll for phase `parity`. What another CTA sent is acquired at the cluster's scope: a poll's scope is its own CTA unless it says so.
__device__ __forceinline__ bool cluster_try_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// What the CTAs of a cluster tell one another: the scan's elements of two tiles, and how far a CTA came that stopped early.
// Waits are bounded. One that gives up is reported as the look-back's are, its CTA stops before the next tile, and the others, which
// wait for that tile's elements, follow: no call waits longer than the limit twice. A CTA that ends while elements are on their way to it would
// leave them a place that is no longer its own; so whoever stops says how many tiles' elements it has sent, and each waits for the rest.
constexpr int kAllSent = INT32_MAX;
struct ClusterShared {
    Element element[2][8][32];       // by the tile's side, of each CTA
    alignas(8) uint64_t arrived[2];  // a side's elements are all here
    int late[2];                     // a wait of this side gave up
    int stopped;                     // a CTA of the cluster stopped early
    int sent[8];                     // and then the tiles whose elements it has sent
};
constexpr uint32_t kElementBytes = 32 * sizeof(Element);
// Before the cluster's first barrier. `silent`: the test hook's CTA, which stops before its first tile.
__device__ __forceinline__ void cluster_begin(ClusterShared &s, bool silent) {
    if (threadIdx.x == 0) {
        mbar_init(&s.arrived[0], 1);
        mbar_init(&s.arrived[1], 1);
        fence_mbar_init();
        s.late[0] = s.stopped = 0;
        s.late[1] = silent;  // as if of the tile before the first
        for (int q = 0; q < 8; ++q)
            s.sent[q] = kAllSent;
    }
}
// Until all CTAs' elements of a tile are here.
__device__ __forceinline__ void cluster_await(ClusterShared &s, int side, uint32_t parity, uint32_t limit) {
    for (uint32_t i = 0; i < limit; ++i)
        if (cluster_try_wait(&s.arrived[side], parity))
            return;
    atomicCAS(&g_mt_err, 0, kErrTimeout);
    s.late[side] = 1;
}
// Behind the loop, of all threads. This CTA has sent its elements of `done` of `tiles` tiles.
__device__ __forceinline__ void cluster_end(ClusterShared &s, unsigned rank, int ctas, int done, int tiles) {
    if (done < tiles && threadIdx.x < ctas) {
        uint32_t sent, stopped;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(sent) : "r"(smem_addr(&s.sent[rank])), "r"(threadIdx.x));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(stopped) : "r"(smem_addr(&s.stopped)), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.s32 [%0], %1;" :: "r"(sent), "r"(done) : "memory");
        asm volatile("st.shared::cluster.s32 [%0], %1;" :: "r"(stopped), "r"(1) : "memory");
    }
    cluster_arrive();  // no CTA ends that another might still send to
    cluster_wait();
    if (threadIdx.x != 0 || (s.late[0] | s.late[1] | s.stopped) == 0)
        return;
    // The tile before has a wait of this CTA, which may have given up, for everyone's elements: those never sent are counted as here. The next one
    // has none yet, and those that came further have sent theirs; nobody comes further than that without this CTA's.
    for (int t = done > 0 ? done - 1 : 0; t <= done && t < tiles; ++t) {
        uint32_t missing = 0;
        for (int q = 0; q < ctas; ++q)
            missing += s.sent[q] <= t ? kElementBytes : 0;
        if (t == done)
            mbar_arrive_expect_tx(&s.arrived[t & 1], (uint32_t)ctas * kElementBytes);
        if (missing != 0)
            asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" :: "r"(smem_addr(&s.arrived[t & 1])), "r"(missing) : "memory");
        for (uint32_t i = 0; i < kCopyWaitLimit; ++i)  // all have been sent
            if (cluster_try_wait(&s.arrived[t & 1], (uint32_t)(t >> 1 & 1)))
                break;
    }
}

// ---- a pair of channels ---------------------------------------------------------------------------
__device__ __forceinline__ f32x2 less2f(float a, f32x2 b) { return fma2f(b, both(-1.0f), both(a)); }  // a - b
__device__ __forceinline__ f32x2 max2f(f32x2 a, f32x2 b) {
    float x, y, v, w;
    unpack2f(a, x, y);
    unpack2f(b, v, w);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(v));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(y) : "f"(w));
    return pack2f(x, y);
}
__device__ __forceinline__ f32x2 rsqrt_2f(f32x2 v) {
    float a, b;
    unpack2f(v, a, b);
    asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(b));
    return pack2f(a, b);
}

// sigma(x) and 1 - sigma(x), each to f32's relative precision: 1 / (1 + e) and e / (1 + e) with e = exp(-x), which is
// kept below 2^126 (x above -87.3) so that neither is 0 * inf; the minimum passes NaN on. Less 2^-126, which is lost in any sigma above
// 2^-102, the former is 0 there: a gate at its type's lowest value is shut for any finite value beside it. (A choice between e s and
// 1 - s instead: gradients 2 to 3 % slower.)
__device__ __forceinline__ f32x2 least_2f(f32x2 v, float most) {
    float a, b;
    unpack2f(v, a, b);
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(most));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(most));
    return pack2f(a, b);
}
__device__ __forceinline__ void sigmoid_both_2f(f32x2 x, f32x2 &s, f32x2 &c) {
    const f32x2 e = least_2f(ex2_2f(mul2f(both(-kLog2e), x)), 0x1p126f), least = rcp_2f(add2f(both(1.0f), e));
    s = add2f(least, both(-0x1p-126f));
    c = mul2f(e, least);
}

// 1 - exp(-u) = u (1 - u/2! + u^2/3! - ...), Taylor's series of the exponential, for u below 1/4: the first
// term left out is below 4.9e-8 of the sum. The decay next to 1 is 1 minus this, so that a long memory's
// decays keep f32's precision and w = sqrt(1 - a^2) its relative one, which 1 - a * a does not.
constexpr float kNear = 0.25f;
__device__ __forceinline__ f32x2 one_minus_exp_small_2f(f32x2 u) {
    f32x2 p = both(-1.0f / 720.0f);
    p = fma2f(p, u, both(1.0f / 120.0f));
    p = fma2f(p, u, both(-1.0f / 24.0f));
    p = fma2f(p, u, both(1.0f / 6.0f));
    p = fma2f(p, u, both(-0.5f));
    p = fma2f(p, u, both(1.0f));
    return mul2f(u, p);
}

// With rate: the decay and q = 1 - a^2, 0 where 1 - a is below f32's normal numbers (there w = sqrt(q) and its derivative count as 0:
// 1 / w would be up to 2^75 in a sum over tokens, of which q has few bits or none).
__device__ __forceinline__ f32x2 mul_normal_2f(f32x2 a, f32x2 b) {  // numbers that are not normal count as 0
    f32x2 r;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void decay_2f(f32x2 u, f32x2 &a, f32x2 &q) {
    const f32x2 small = one_minus_exp_small_2f(u), big = ex2_2f(mul2f(both(-kLog2e), u));
    const f32x2 far = less2f(1.0f, big), near = less2f(1.0f, small);
    float u0, u1, s0, s1, b0, b1, f0, f1, n0, n1;
    unpack2f(u, u0, u1);
    unpack2f(small, s0, s1);
    unpack2f(big, b0, b1);
    unpack2f(far, f0, f1);
    unpack2f(near, n0, n1);
    a = pack2f(u0 < kNear ? n0 : b0, u1 < kNear ? n1 : b1);
    const f32x2 d = pack2f(u0 < kNear ? s0 : f0, u1 < kNear ? s1 : f1);  // 1 - a
    q = mul_normal_2f(d, less2f(2.0f, d));                             // (1 - a) (1 + a)
}
// 1 / sqrt(q), or 0 where q is 0
__device__ __forceinline__ f32x2 rsqrt_or_0_2f(f32x2 q) {
    float q0, q1, r0, r1;
    unpack2f(q, q0, q1);
    unpack2f(rsqrt_2f(q), r0, r1);
    return pack2f(q0 == 0.0f ? 0.0f : r0, q1 == 0.0f ? 0.0f : r1);
}
// sqrt(q) = q / sqrt(q), with the least normal number at least in the root, so that 0 stays 0
constexpr float kLeast = 0x1p-126f;
__device__ __forceinline__ f32x2 root_2f(f32x2 q) { return mul2f(q, rsqrt_2f(max2f(q, both(kLeast)))); }
// sqrt(q) sigma(i) = q / sqrt(q (1 + e)^2) with e = exp(-i): one root for both. (1 + e)^2 is out of range for i below -44, where this may be 0:
// off by less than 2^-63. Prompts of 4 x 2048 tokens x 4096 channels bf16, us: this 68, a root and a reciprocal 75, this and those
// for tiles with gates so low 71, but 126 for 112 with 16 x 1024 tokens.
__device__ __forceinline__ f32x2 root_sigmoid_2f(f32x2 q, f32x2 i) {
    const f32x2 n = add2f(both(1.0f), ex2_2f(mul2f(both(-kLog2e), i)));
    return mul2f(q, rsqrt_2f(mul2f(mul2f(max2f(q, both(kLeast)), n), n)));
}

// ---- rows of activations --------------------------------------------------------------------------
template <class S> struct Pair;  // two neighbouring values
template <> struct Pair<float> {
    using T = uint2;
    __device__ __forceinline__ static f32x2 widen(const uint2 &w) { return pack2f(__uint_as_float(w.x), __uint_as_float(w.y)); }
    __device__ __forceinline__ static uint2 narrow(float a, float b) { return make_uint2(__float_as_uint(a), __float_as_uint(b)); }
};
template <> struct Pair<__nv_bfloat16> {
    using T = uint32_t;
    __device__ __forceinline__ static f32x2 widen(uint32_t w) {
        float a, b;
        Codec<__nv_bfloat16>::two(w, a, b);
        return pack2f(a, b);
    }
    __device__ __forceinline__ static uint32_t narrow(float a, float b) { return Codec<__nv_bfloat16>::pack2(a, b); }
};
template <> struct Pair<__half> {
    using T = uint32_t;
    __device__ __forceinline__ static f32x2 widen(uint32_t w) {
        float a, b;
        Codec<__half>::two(w, a, b);
        return pack2f(a, b);
    }
    __device__ __forceinline__ static uint32_t narrow(float a, float b) { return Codec<__half>::pack2(a, b); }
};

// A tensor's rows for one sequence and slab. Where VEC, a token's stride in bytes is below 2^31, and a row's
// address one multiply-add.
template <class S, bool VEC> struct Rows {
    S *at;  // token 0, the slab's first channel
    int64_t token;
    __device__ __forceinline__ Rows(const void *p, int64_t batch, int64_t token_, int64_t b, int64_t c0)
        : at(p == nullptr ? nullptr : const_cast<S *>(static_cast<const S *>(p)) + b * batch + c0), token(token_) {}
    // of a tile: where its first row begins in a 16-byte vector, and what a token adds to that
    int low = 0, token_low = 0;
    __device__ __forceinline__ void begin_tile(int t0) {
        if constexpr (!VEC) {
            low = (int)((uintptr_t)row(t0) & 15);
            token_low = (int)(token * (int64_t)sizeof(S) & 15);
        }
    }
    __device__ __forceinline__ S *row(int t) const {
        if constexpr (VEC)
            return reinterpret_cast<S *>(reinterpret_cast<char *>(at) + (int64_t)t * (int)((int)token * (int)sizeof(S)));
        else
            return at + t * token;
    }
};

// A lane's two channels: neighbours where rows are vectors, and otherwise half a slab apart, so that a warp's single values are
// together: 4 x 2048 tokens x 4095 channels, all gates, gradient, us: bf16 212 for 286 as neighbours, f32 271 for 321.
template <bool VEC> constexpr int kFar = VEC ? 1 : kGatedSlab / 2;

// T tokens of a tensor in a warp's part of shared memory, 64 channels each. VEC: the rows are 16-byte aligned and
// whole vectors. Otherwise rows are copied as the aligned vectors that they touch (each holds a channel of the row) and read from
// where they begin in the first; or, WORDS, f32 value by value.
// 4 x 2048 tokens x 4095 channels, all gates, us: bf16 prompt 106 and gradient 206 (4096 channels 68 and 121); f32 gradient by words 390, by
// vectors 260; f32 prompt 182 and 164, but 8 x 1027 x 1001 without input gate 43.0 and 44.7, 3 x 515 x 1001 without output gate 12.4 and 13.4.
template <class S, int T, bool VEC, bool WORDS = false> struct Tile {
    static constexpr int kPitch = kGatedSlab * (int)sizeof(S) + (VEC ? 0 : 16);
    static constexpr int kBytes = T * kPitch;
    static constexpr int kRow = kGatedSlab * (int)sizeof(S) / 16, kPer = 16 / (int)sizeof(S);  // vectors of a row, values of one
    // The first n tokens (T at most) from token t0 on, `live` of the slab's channels; `r` from the lane's own vector on where VEC (lane_rows).
    static __device__ __forceinline__ void copy(uint32_t to, const Rows<S, VEC> &r, int t0, int n, int live, int lane) {
        if constexpr (VEC) {
            if (lane % kRow * kPer >= live)
                return;
#pragma unroll
            for (int k = 0; k < T * kRow / 32; ++k) {
                const int row = k * (32 / kRow) + lane / kRow;
                if (n >= T || row < n)
                    cp_async_zfill<16>(to + k * 512 + lane * 16, r.row(t0 + row), true);
            }
        } else if constexpr (WORDS) {
#pragma unroll
            for (int k = 0; k < 2 * T; ++k)
                if (k / 2 < n && k % 2 * 32 + lane < live)
                    cp_async_zfill<4>(to + k / 2 * kPitch + (k % 2 * 32 + lane) * 4, r.row(t0 + k / 2) + k % 2 * 32 + lane, true);
        } else {
            constexpr int kVectors = kPitch / 16;  // that a row can touch
#pragma unroll
            for (int k = 0; k < (T * kVectors + 31) / 32; ++k) {
                const int q = k * 32 + lane, row = q / kVectors, col = q % kVectors;
                const uintptr_t from = (uintptr_t)r.row(t0 + row);
                if (row < n && row < T && col * 16 < (int)(from & 15) + live * (int)sizeof(S))
                    cp_async_zfill<16>(to + row * kPitch + col * 16, (const void *)((from & ~(uintptr_t)15) + col * 16), true);
            }
        }
    }
    // The rows as copy takes them.
    static __device__ __forceinline__ Rows<S, VEC> lane_rows(Rows<S, VEC> r, int lane) {
        if constexpr (VEC)
            if (r.at != nullptr)
                r.at += lane % kRow * kPer;
        return r;
    }
    // The lane's channels of the tile's row.
    static __device__ __forceinline__ f32x2 read(const char *at, const Rows<S, VEC> &r, int row, int lane) {
        using P = typename Pair<S>::T;
        if constexpr (VEC)
            return Pair<S>::widen(*reinterpret_cast<const P *>(at + row * kPitch + lane * (int)sizeof(P)));
        const S *from = reinterpret_cast<const S *>(at + row * kPitch + (WORDS ? 0 : (r.low + row * r.token_low) & 15)) + lane;
        return pack2f(Codec<S>::load1(from), Codec<S>::load1(from + kFar<VEC>));
    }
    // Rows from n on hold `v` in every channel.
    static __device__ __forceinline__ void fill(char *at, int n, S v, int lane) {
        for (int row = n; row < T; ++row)
            for (int k = lane; k < kPitch / (int)sizeof(S); k += 32)
                reinterpret_cast<S *>(at + row * kPitch)[k] = v;
    }
};

// A lane's pair: channels FAR apart, of which those at 0 to `live` - 1 exist (VEC: none or both).
template <class S, bool VEC, int FAR> __device__ __forceinline__ void put_pair(S *to, int live, f32x2 v) {
    float a, b;
    unpack2f(v, a, b);
    if constexpr (VEC) {
        if (live > 0)
            *reinterpret_cast<typename Pair<S>::T *>(to) = Pair<S>::narrow(a, b);
    } else {
        if (live > 0)
            Codec<S>::store1(to, a);
        if (live > FAR)
            Codec<S>::store1(to + FAR, b);
    }
}
// f32 rows of states and parameters, from the lane's first channel on
template <int FAR> __device__ __forceinline__ f32x2 get_state(const float *p, int live) {
    return pack2f(live > 0 ? p[0] : 0.0f, live > FAR ? p[FAR] : 0.0f);
}
// Rates, of which those below 0 count as 0. The maximum also has the load waited for before the tiles: where a product within
// their loop is the first to use it, the gradient of 4 x 2048 tokens x 4096 channels bf16 takes 146 us for 121.
template <int FAR> __device__ __forceinline__ f32x2 get_rate(const float *p, int live) { return max2f(get_state<FAR>(p, live), both(0.0f)); }
template <int FAR> __device__ __forceinline__ void put_state(float *p, int live, f32x2 v) {
    float a, b;
    unpack2f(v, a, b);
    if (live > 0)
        p[0] = a;
    if (live > FAR)
        p[FAR] = b;
}

// ---- prompts ----------------------------------------------------------------------------------------
template <class S, bool VEC, int T> using FwdTile = Tile<S, T, VEC, sizeof(S) == 4>;

// With room for all four tensors, used or not: with less a cluster's f32 CTAs go three an SM, and unevenly (2 x 2048 x 4096, no
// output gate, 72 us for 57).
template <class S, bool VEC, int T> struct FwdShared {
    static constexpr int kTile = FwdTile<S, VEC, T>::kBytes;
    static constexpr int kIn = 2 * kTile, kZ = 3 * kTile;  // behind x and r
    static constexpr int kStage = 4 * kTile;
    static constexpr int kWarp = kGatedStages * kStage;
};

// IN and Z: the call has an input gate, an output gate; CLUSTER: CTAs share the tokens.
// W: warps of the CTA; fewer where these have all tokens.
template <class S, bool RATE, bool VEC, bool IN, bool Z, bool CLUSTER, int W, int T>
__global__ void __launch_bounds__(32 * W, 128 / W / T) k_gated(const __grid_constant__ GatedArgs g) {
    using In = FwdTile<S, VEC, T>;
    using Shared = FwdShared<S, VEC, T>;
    constexpr int kCtaTokens = W * T;
    constexpr int FAR = kFar<VEC>;
    extern __shared__ __align__(16) char staged[];
    __shared__ Element of_warps[2][W][32];
    __shared__ ClusterShared others;
    const int ctas = CLUSTER ? g.ctas : 1;
    if (ctas > 1) {
        cluster_begin(others, blockIdx.x == g.silent);
        cluster_arrive();  // waited for below: no CTA sends to one that has not begun
    }
    pdl_prologue();
    const mt_gated_args &p = g.p;
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = ctas > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / ctas, b = unit / g.slabs, c0 = (unit - b * g.slabs) * kGatedSlab;
    const int live = (int)(p.dim - c0 < kGatedSlab ? p.dim - c0 : kGatedSlab), at0 = VEC ? 2 * lane : lane, mine = live - at0;
    const int64_t slot = gated_slot(p, b);
    const bool active = slot >= 0 || p.state == nullptr;
    const int len = active ? (int)gated_len(p, b) : 0, total = (int)p.len;
    Rows<S, VEC> x = In::lane_rows({p.x, p.x_batch, p.x_token, b, c0}, lane), r = In::lane_rows({p.r, p.r_batch, p.r_token, b, c0}, lane),
                       in = In::lane_rows({p.i, p.i_batch, p.i_token, b, c0}, lane), z = In::lane_rows({p.z, p.z_batch, p.z_token, b, c0}, lane);
    const Rows<S, VEC> out(p.out, p.out_batch, p.out_token, b, c0 + at0);
    constexpr bool has_in = IN, has_z = Z;
    const int64_t c = c0 + at0;
    const f32x2 rate = RATE ? get_rate<FAR>(p.rate + c, mine) : 0ull;
    f32x2 carry = 0ull;
    if (active && p.state != nullptr && p.carry_in)
        carry = get_state<FAR>(p.state + slot * p.dim + c, mine);
    char *own = staged + warp * Shared::kWarp;
    const uint32_t own_at = (uint32_t)__cvta_generic_to_shared(own);
    const int step = ctas * kCtaTokens, first = rank * kCtaTokens + warp * T;

    auto ask = [&](int t0, int stage) {
        const int n = len - t0;
        if (n > 0) {
            const uint32_t to = own_at + (uint32_t)(stage * Shared::kStage);
            In::copy(to, x, t0, n, live, lane);
            In::copy(to + Shared::kTile, r, t0, n, live, lane);
            if (has_in)
                In::copy(to + Shared::kIn, in, t0, n, live, lane);
            if (has_z)
                In::copy(to + Shared::kZ, z, t0, n, live, lane);
        }
        cp_async_commit();
    };
    for (int w = warps; w < W; ++w)  // of warps that are not there; all that are write the same
        of_warps[0][w][lane] = {both(1.0f), 0ull};
    ask(first, 0);
    ask(first + step, 1);
    if (ctas > 1)
        cluster_wait();

    int side = 0;
    uint32_t parity = 0;  // of the barriers' phases, each of which serves every other tile
    int base = 0;
    const int tiles = (len + step - 1) / step;
    for (; base < len; base += step, side ^= 1) {
        const int t0 = base + first, n = len - t0;
        char *at = own + side * Shared::kStage;
        cp_async_wait<kGatedStages - 1>();
        __syncwarp();
        if (n < T) {  // tokens behind the end: a shut gate, which leaves the state
            const int has = n < 0 ? 0 : n;
            In::fill(at, has, S(0.0f), lane);
            In::fill(at + Shared::kTile, has, S(Lim<float>::lo()), lane);
            if (has_in)
                In::fill(at + Shared::kIn, has, S(0.0f), lane);
            if (has_z)
                In::fill(at + Shared::kZ, has, S(0.0f), lane);
            __syncwarp();
        }
        for (Rows<S, VEC> *rows : {&x, &r, &in, &z})
            rows->begin_tile(t0);
        f32x2 a[T], v[T], gate[T];
        Element e = {both(1.0f), 0ull};
#pragma unroll
        for (int k = 0; k < T; ++k) {
            const f32x2 rr = In::read(at + Shared::kTile, r, k, lane);
            f32x2 w;
            if constexpr (RATE) {
                f32x2 q;
                decay_2f(mul2f(rate, sigmoid_2f(rr)), a[k], q);
                w = has_in ? root_sigmoid_2f(q, In::read(at + Shared::kIn, in, k, lane)) : root_2f(q);
            } else {
                sigmoid_both_2f(rr, w, a[k]);
                if (has_in)
                    w = mul2f(w, sigmoid_2f(In::read(at + Shared::kIn, in, k, lane)));
            }
            v[k] = mul2f(w, In::read(at, x, k, lane));
            if (has_z) {
                const f32x2 zz = In::read(at + Shared::kZ, z, k, lane);
                gate[k] = mul2f(zz, sigmoid_2f(zz));
            }
            e.h = fma2f(a[k], e.h, v[k]);
            e.a = mul2f(e.a, a[k]);
        }
        __syncwarp();
        ask(t0 + kGatedStages * step, side);
        of_warps[side][warp][lane] = e;
        __syncthreads();
        if (ctas > 1 && others.late[side ^ 1])  // a side's mark is not written again before all have passed the next barrier
            break;
        f32x2 h = carry;  // before the CTA's first token
        if (ctas == 1) {
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w == warp)
                    h = carry;
                const Element o = of_warps[side][w][lane];
                carry = fma2f(o.a, carry, o.h);
            }
        } else {
            // every warp joins the CTA's elements, and tells its share of the cluster's CTAs
            Element all = {both(1.0f), 0ull}, before = all;  // of the warps before this one
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w == warp)
                    before = all;
                const Element o = of_warps[side][w][lane];
                all.h = fma2f(o.a, all.h, o.h);
                all.a = mul2f(all.a, o.a);
            }
            if (threadIdx.x == 0)
                mbar_arrive_expect_tx(&others.arrived[side], (uint32_t)ctas * kElementBytes);
            for (int q = warp; q < ctas; q += W)
                cluster_send(smem_addr(&others.element[side][rank][lane]), smem_addr(&others.arrived[side]), (unsigned)q, all.a, all.h);
            cluster_await(others, side, parity, g.limit);
            parity ^= (uint32_t)side;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (q == rank)
                    h = carry;
                if (q < ctas) {
                    const Element o = others.element[side][q][lane];
                    carry = fma2f(o.a, carry, o.h);
                }
            }
            h = fma2f(before.a, h, before.h);
        }
        if (p.checkpoints != nullptr && warp * T % kGatedTile == 0 && n > 0)
            put_state<FAR>(p.checkpoints + (b * g.ntiles + t0 / kGatedTile) * p.dim + c, mine, h);
        auto finish = [&](bool whole) {
#pragma unroll
            for (int k = 0; k < T; ++k) {
                h = fma2f(a[k], h, v[k]);
                f32x2 y = h;
                if (has_z)
                    y = mul2f(h, gate[k]);
                if (whole || k < n)
                    put_pair<S, VEC, FAR>(out.row(t0 + k), mine, y);
            }
        };
        if (n >= T)
            finish(true);
        else
            finish(false);
    }
    cp_async_wait<0>();
    if (ctas > 1)
        cluster_end(others, (unsigned)rank, ctas, base / step, tiles);
    for (int t = len + rank * warps + warp; t < total; t += ctas * warps)
        put_pair<S, VEC, FAR>(out.row(t), mine, 0ull);
    if (active && p.state != nullptr && rank == 0 && warp == 0)
        put_state<FAR>(p.state + slot * p.dim + c, mine, carry);
}

// ---- gradients ----------------------------------------------------------------------------------------
// From the last tokens to the first. A warp's tokens give two elements, the recurrence's from the checkpoint before
// them and its adjoint's from behind; with both carries known the states and the gradients by them
// follow, and what a token's gradients take besides is in registers: eight tokens' worth of it, in all that a thread can
// have. So an SM holds eight such warps, in two CTAs. Twice the warps of four tokens, which take the carries' work twice as
// often, against these, us, all gates, 4096 channels, bf16: 4 x 2048 tokens 140 and 121, 8 x 2048 253 and 237; no output gate 4 x 4096 254 and 198.
constexpr int kBwdT = 8;
constexpr int kBwdWarps = 4;

template <class S, bool VEC> struct BwdShared {
    static constexpr int kTile = Tile<S, kBwdT, VEC>::kBytes;
    static constexpr int kIn = 3 * kTile, kZ = 4 * kTile;  // behind x, r and dout
    static constexpr int kStage = 5 * kTile;
    static constexpr int kWarp = kGatedStages * kStage;
};

template <class S, bool RATE, bool VEC, bool IN, bool Z, bool CLUSTER>
__global__ void __launch_bounds__(32 * kBwdWarps, 2) k_gated_grad(const __grid_constant__ GatedArgs g, float *rate_part) {
    using In = Tile<S, kBwdT, VEC>;
    using Shared = BwdShared<S, VEC>;
    constexpr int W = kBwdWarps;
    constexpr int kCtaTokens = W * kBwdT;
    constexpr int kMarkWarps = kGatedTile / kBwdT;  // that share a checkpoint
    static_assert(kCtaTokens % kGatedTile == 0 && kGatedTile % kBwdT == 0, "a CTA's tokens begin at a checkpoint");
    constexpr int FAR = kFar<VEC>;
    extern __shared__ __align__(16) char staged[];
    __shared__ Element of_warps[2][W][32];
    __shared__ Element back_of_warps[2][W][32];  // the adjoint's
    __shared__ ClusterShared others;
    const int ctas = CLUSTER ? g.ctas : 1;
    if (ctas > 1) {
        cluster_begin(others, blockIdx.x == g.silent);
        cluster_arrive();  // waited for below: no CTA sends to one that has not begun
    }
    pdl_prologue();
    const mt_gated_args &p = g.p;
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = ctas > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / ctas, b = unit / g.slabs, c0 = (unit - b * g.slabs) * kGatedSlab;
    const int live = (int)(p.dim - c0 < kGatedSlab ? p.dim - c0 : kGatedSlab), at0 = VEC ? 2 * lane : lane, mine = live - at0;
    const int len = (int)gated_len(p, b), total = (int)p.len;
    Rows<S, VEC> x = In::lane_rows({p.x, p.x_batch, p.x_token, b, c0}, lane), r = In::lane_rows({p.r, p.r_batch, p.r_token, b, c0}, lane),
                       in = In::lane_rows({p.i, p.i_batch, p.i_token, b, c0}, lane), z = In::lane_rows({p.z, p.z_batch, p.z_token, b, c0}, lane),
                       dout = In::lane_rows({p.dout, p.dout_batch, p.dout_token, b, c0}, lane);
    const int64_t c = c0 + at0;
    const Rows<S, VEC> dx(p.dx, p.dx_batch, p.dx_token, b, c), dr(p.dr, p.dr_batch, p.dr_token, b, c), di(p.di, p.di_batch, p.di_token, b, c),
        dz(p.dz, p.dz_batch, p.dz_token, b, c);
    constexpr bool has_in = IN, has_z = Z;
    const f32x2 rate = RATE ? get_rate<FAR>(p.rate + c, mine) : 0ull;
    f32x2 carry = p.dfinal != nullptr ? get_state<FAR>(p.dfinal + b * p.dim + c, mine) : 0ull;
    f32x2 rate_sum = 0ull;
    char *own = staged + warp * Shared::kWarp;
    const uint32_t own_at = (uint32_t)__cvta_generic_to_shared(own);
    const int step = ctas * kCtaTokens, first = rank * kCtaTokens + warp * kBwdT;

    auto ask = [&](int base, int stage) {
        const int t0 = base + first, n = len - t0;
        if (base >= 0 && n > 0) {
            const uint32_t to = own_at + (uint32_t)(stage * Shared::kStage);
            In::copy(to, x, t0, n, live, lane);
            In::copy(to + Shared::kTile, r, t0, n, live, lane);
            if (has_in)
                In::copy(to + Shared::kIn, in, t0, n, live, lane);
            if (has_z)
                In::copy(to + Shared::kZ, z, t0, n, live, lane);
            In::copy(to + 2 * Shared::kTile, dout, t0, n, live, lane);
        }
        cp_async_commit();
    };
    const int last = len > 0 ? (len - 1) / step * step : -1;  // where the last CTAs' tokens begin
    for (int w = warps; w < W; ++w)  // of warps that are not there; all that are write the same
        of_warps[0][w][lane] = back_of_warps[0][w][lane] = {both(1.0f), 0ull};
    ask(last, 0);
    ask(last - step, 1);
    if (ctas > 1)
        cluster_wait();

    int side = 0;
    uint32_t parity = 0;  // of the barriers' phases, each of which serves every other tile
    int base = last;
    const int tiles = len > 0 ? last / step + 1 : 0;
    for (; base >= 0; base -= step, side ^= 1) {
        const int t0 = base + first, n = len - t0;
        char *at = own + side * Shared::kStage;
        f32x2 h = 0ull;  // before the first token of the checkpoint's warps
        if (t0 / kGatedTile * kGatedTile < len)
            h = get_state<FAR>(p.checkpoints + (b * g.ntiles + t0 / kGatedTile) * p.dim + c, mine);
        cp_async_wait<kGatedStages - 1>();
        __syncwarp();
        if (n < kBwdT) {  // tokens behind the end: a shut gate, which passes states and gradients by them
            const int has = n < 0 ? 0 : n;
            In::fill(at, has, S(0.0f), lane);
            In::fill(at + Shared::kTile, has, S(Lim<float>::lo()), lane);
            In::fill(at + 2 * Shared::kTile, has, S(0.0f), lane);
            if (has_in)
                In::fill(at + Shared::kIn, has, S(0.0f), lane);
            if (has_z)
                In::fill(at + Shared::kZ, has, S(0.0f), lane);
            __syncwarp();
        }
        for (Rows<S, VEC> *rows : {&x, &r, &in, &z, &dout})
            rows->begin_tile(t0);
        // per token: decay, w v (later the state before it), dh; w sigma(i), x (1 - sigma(i)), dz / h; and of
        // e = g as (m - h_{t-1}), with as = a s and m = v a / w (without rate 1 and v), those and dr / e
        f32x2 a[kBwdT], v[kBwdT], dh[kBwdT], to_x[kBwdT], to_i[kBwdT], to_z[kBwdT], as[kBwdT], m[kBwdT], to_r[kBwdT];
        Element e = {both(1.0f), 0ull};
#pragma unroll
        for (int k = 0; k < kBwdT; ++k) {
            f32x2 s, cs, w, rw = 0ull;
            sigmoid_both_2f(In::read(at + Shared::kTile, r, k, lane), s, cs);
            if constexpr (RATE) {
                f32x2 q;
                decay_2f(mul2f(rate, s), a[k], q);
                rw = rsqrt_or_0_2f(q);
                w = mul2f(q, rw);
            } else {
                a[k] = cs;
                w = s;
            }
            const f32x2 xx = In::read(at, x, k, lane), dy = In::read(at + 2 * Shared::kTile, dout, k, lane);
            f32x2 vv = xx;
            to_x[k] = w;
            to_i[k] = 0ull;
            if (has_in) {
                f32x2 si, ci;
                sigmoid_both_2f(In::read(at + Shared::kIn, in, k, lane), si, ci);
                vv = mul2f(xx, si);
                to_x[k] = mul2f(w, si);
                to_i[k] = mul2f(xx, ci);
            }
            dh[k] = dy;
            to_z[k] = 0ull;
            if (has_z) {
                f32x2 sz, cz;
                const f32x2 zz = In::read(at + Shared::kZ, z, k, lane);
                sigmoid_both_2f(zz, sz, cz);
                dh[k] = mul2f(dy, mul2f(zz, sz));
                to_z[k] = mul2f(dy, mul2f(sz, fma2f(zz, cz, both(1.0f))));
            }
            v[k] = mul2f(w, vv);
            if constexpr (RATE) {
                as[k] = mul2f(a[k], s);
                m[k] = mul2f(vv, mul2f(a[k], rw));
                to_r[k] = mul2f(rate, cs);
            } else {
                m[k] = vv;
                to_r[k] = mul2f(s, cs);
            }
            e.h = fma2f(a[k], e.h, v[k]);
            e.a = mul2f(e.a, a[k]);
        }
        f32x2 back = 0ull;
#pragma unroll
        for (int k = kBwdT - 1; k >= 0; --k)
            back = mul2f(a[k], add2f(dh[k], back));
        __syncwarp();
        ask(base - kGatedStages * step, side);
        of_warps[side][warp][lane] = e;
        back_of_warps[side][warp][lane] = {e.a, back};
        __syncthreads();
        if (ctas > 1 && others.late[side ^ 1])  // a side's mark is not written again before all have passed the next barrier
            break;
        // the state before this warp's tokens
        for (int w = warp / kMarkWarps * kMarkWarps; w < warp; ++w) {
            const Element o = of_warps[side][w][lane];
            h = fma2f(o.a, h, o.h);
        }
        f32x2 gh = carry;  // by the state after the CTA's last token
        if (ctas == 1) {
#pragma unroll
            for (int w = W - 1; w >= 0; --w) {
                if (w == warp)
                    gh = carry;
                const Element o = back_of_warps[side][w][lane];
                carry = fma2f(o.a, carry, o.h);
            }
        } else {
            // every warp joins the CTA's elements of the adjoint, and tells its share of the cluster's CTAs
            Element all = {both(1.0f), 0ull}, behind = all;  // of the warps behind this one
#pragma unroll
            for (int w = W - 1; w >= 0; --w) {
                if (w == warp)
                    behind = all;
                const Element o = back_of_warps[side][w][lane];
                all.h = fma2f(o.a, all.h, o.h);
                all.a = mul2f(all.a, o.a);
            }
            if (threadIdx.x == 0)
                mbar_arrive_expect_tx(&others.arrived[side], (uint32_t)ctas * kElementBytes);
            for (int q = warp; q < ctas; q += W)
                cluster_send(smem_addr(&others.element[side][rank][lane]), smem_addr(&others.arrived[side]), (unsigned)q, all.a, all.h);
            cluster_await(others, side, parity, g.limit);
            parity ^= (uint32_t)side;
#pragma unroll
            for (int q = 7; q >= 0; --q) {
                if (q == rank)
                    gh = carry;
                if (q < ctas) {
                    const Element o = others.element[side][q][lane];
                    carry = fma2f(o.a, carry, o.h);
                }
            }
            gh = fma2f(behind.a, gh, behind.h);
        }
#pragma unroll
        for (int k = 0; k < kBwdT; ++k) {
            const f32x2 now = fma2f(a[k], h, v[k]);
            v[k] = h;
            to_z[k] = mul2f(to_z[k], now);
            h = now;
        }
        auto finish = [&](bool whole) {
#pragma unroll
            for (int k = kBwdT - 1; k >= 0; --k) {
                const f32x2 gt = add2f(dh[k], gh);
                gh = mul2f(gt, a[k]);
                f32x2 to = fma2f(v[k], both(-1.0f), m[k]), gr;
                if (RATE) {
                    to = mul2f(mul2f(gt, to), as[k]);
                    gr = mul2f(to, to_r[k]);
                } else {  // a shut gate's 0 before the product of what may both be large
                    gr = mul2f(gt, mul2f(to, to_r[k]));
                }
                const f32x2 gx = mul2f(gt, to_x[k]);
                if (whole || k < n) {
                    if (RATE)
                        rate_sum = add2f(rate_sum, to);
                    put_pair<S, VEC, FAR>(dx.row(t0 + k), mine, gx);
                    put_pair<S, VEC, FAR>(dr.row(t0 + k), mine, gr);
                    if (has_in)
                        put_pair<S, VEC, FAR>(di.row(t0 + k), mine, mul2f(gx, to_i[k]));
                    if (has_z)
                        put_pair<S, VEC, FAR>(dz.row(t0 + k), mine, to_z[k]);
                }
            }
        };
        if (n >= kBwdT)
            finish(true);
        else
            finish(false);
    }
    cp_async_wait<0>();
    if (ctas > 1)
        cluster_end(others, (unsigned)rank, ctas, (last - base) / step, tiles);
    for (int t = len + rank * warps + warp; t < total; t += ctas * warps) {
        put_pair<S, VEC, FAR>(dx.row(t), mine, 0ull);
        put_pair<S, VEC, FAR>(dr.row(t), mine, 0ull);
        if (has_in)
            put_pair<S, VEC, FAR>(di.row(t), mine, 0ull);
        if (has_z)
            put_pair<S, VEC, FAR>(dz.row(t), mine, 0ull);
    }
    if (p.dinit != nullptr && rank == 0 && warp == 0)
        put_state<FAR>(p.dinit + b * p.dim + c, mine, carry);
    if (RATE && rate_part != nullptr) {
        __syncthreads();  // the loop's last reads of back_of_warps
        back_of_warps[0][warp][lane].h = rate_sum;
        __syncthreads();
        if (warp == 0) {
            f32x2 s = 0ull;
#pragma unroll
            for (int w = 0; w < W; ++w)
                s = add2f(s, back_of_warps[0][w][lane].h);
            put_state<FAR>(rate_part + (b * ctas + rank) * p.dim + c, mine, s);
        }
    }
}

// ---- single tokens ----------------------------------------------------------------------------------
// A thread a pair of channels of one sequence.
template <class S, bool RATE, bool VEC> __global__ void __launch_bounds__(128) k_gated_step(const __grid_constant__ GatedArgs g) {
    pdl_prologue();
    const mt_gated_args &p = g.p;
    const int64_t pairs = (p.dim + 1) / 2, at = (int64_t)blockIdx.x * 128 + threadIdx.x, b = at / pairs;
    if (b >= p.batch)
        return;
    const int64_t c = (at - b * pairs) * 2;
    const int live = (int)(p.dim - c < 2 ? p.dim - c : 2);
    const int64_t slot = gated_slot(p, b);
    S *out = static_cast<S *>(p.out) + b * p.out_batch + c;
    if (slot < 0) {
        put_pair<S, VEC, 1>(out, live, 0ull);
        return;
    }
    auto get = [&](const void *q, int64_t batch) {
        const S *s = static_cast<const S *>(q) + b * batch + c;
        if constexpr (VEC)
            return Pair<S>::widen(*reinterpret_cast<const typename Pair<S>::T *>(s));
        else
            return pack2f(Codec<S>::load1(s), live > 1 ? Codec<S>::load1(s + 1) : 0.0f);
    };
    float *state = p.state + slot * p.dim + c;
    const f32x2 r = get(p.r, p.r_batch), x = get(p.x, p.x_batch), i = p.i != nullptr ? get(p.i, p.i_batch) : 0ull,
                z = p.z != nullptr ? get(p.z, p.z_batch) : 0ull, h = get_state<1>(state, live);
    f32x2 a, w;
    if constexpr (RATE) {
        f32x2 q;
        decay_2f(mul2f(get_rate<1>(p.rate + c, live), sigmoid_2f(r)), a, q);
        w = root_2f(q);
    } else {
        sigmoid_both_2f(r, w, a);
    }
    if (p.i != nullptr)
        w = mul2f(w, sigmoid_2f(i));
    const f32x2 now = fma2f(a, h, mul2f(w, x));
    put_state<1>(state, live, now);
    put_pair<S, VEC, 1>(out, live, p.z != nullptr ? mul2f(now, mul2f(z, sigmoid_2f(z))) : now);
}

// ---- launches ---------------------------------------------------------------------------------------
// Whether this translation unit has launched a cluster: no other of its kernels waits, and its error word is not read for them.
static std::atomic<bool> g_clusters{false};
static cudaError_t clusters_take_error(int *code) {
    *code = 0;
    if (!g_clusters.load(std::memory_order_relaxed))
        return cudaSuccess;
    const int zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(code, g_mt_err, sizeof(int));
    return e != cudaSuccess || *code == 0 ? e : cudaMemcpyToSymbol(g_mt_err, &zero, sizeof(int));
}
template <class... KArgs, class... Args>
static cudaError_t launch_cluster(void (*kernel)(KArgs...), int64_t grid, unsigned block, int smem, int cluster, cudaStream_t stream,
                                  Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cluster > 1)
        g_clusters.store(true, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Warps of a CTA of W: no more than have tokens, so that more short sequences are on an SM. 64 x 16 tokens x 4096 channels, bf16, all
// gates, us: prompt 11, gradient 25; with all warps 27 and 62.
static int gated_warps(const GatedArgs &g, int most, int tokens) {
    const int64_t n = (g.p.len + tokens - 1) / tokens;
    return g.ctas > 1 || n > most ? most : n < 1 ? 1 : (int)n;
}
// Shared memory that three CTAs of an SM cannot have: with calls that leave registers for three some SMs would get three and
// others one (4 x 4096 x 4096, bf16: prompt without output gate 147 us for 107, gradient without any but r 157 for 138).
constexpr int kThird = 80 * 1024;
template <class S, bool RATE, bool VEC, bool IN, bool Z, bool CLUSTER, int W, int T>
static cudaError_t gated_forward_of(const GatedArgs &g, const Launch &L) {
    static PerDevice ready;
    constexpr int smem = FwdShared<S, VEC, T>::kWarp, all = T == kFwdMoreT && W * smem < kThird ? kThird : W * smem;
    const cudaError_t e = allow_shared(k_gated<S, RATE, VEC, IN, Z, CLUSTER, W, T>, all, ready);
    if (e != cudaSuccess)
        return e;
    const int warps = gated_warps(g, W, T);
    note_launch();
    return launch_cluster(k_gated<S, RATE, VEC, IN, Z, CLUSTER, W, T>, g.p.batch * g.slabs * g.ctas, 32 * warps,
                          warps == W ? all : warps * smem, g.ctas, L.stream, g);
}
template <class S, bool RATE, bool VEC, bool IN, bool Z, bool CLUSTER>
static cudaError_t gated_backward_of(const GatedArgs &g, float *part, const Launch &L) {
    static PerDevice ready;
    constexpr int smem = BwdShared<S, VEC>::kWarp, all = kBwdWarps * smem < kThird ? kThird : kBwdWarps * smem;
    const cudaError_t e = allow_shared(k_gated_grad<S, RATE, VEC, IN, Z, CLUSTER>, all, ready);
    if (e != cudaSuccess)
        return e;
    const int warps = gated_warps(g, kBwdWarps, kBwdT);
    note_launch();
    return launch_cluster(k_gated_grad<S, RATE, VEC, IN, Z, CLUSTER>, g.p.batch * g.slabs * g.ctas, 32 * warps,
                          warps == kBwdWarps ? all : warps * smem, g.ctas, L.stream, g, part);
}
// The kernel of a call's gates: f(std::bool_constant of the input gate, of the output gate).
template <class F> static cudaError_t by_gates(const mt_gated_args &p, F f) {
    if (p.i != nullptr)
        return p.z != nullptr ? f(std::true_type(), std::true_type()) : f(std::true_type(), std::false_type());
    return p.z != nullptr ? f(std::false_type(), std::true_type()) : f(std::false_type(), std::false_type());
}
template <class S, bool RATE, bool VEC> static cudaError_t gated_forward(const GatedArgs &g, const Launch &L) {
    return by_gates(g.p, [&](auto in, auto z) {
        if (g.ctas > 1)
            return gated_forward_of<S, RATE, VEC, in(), z(), true, kGatedWarps, gated_cluster_tokens(sizeof(S))>(g, L);
        if constexpr (sizeof(S) == 4)
            return gated_forward_of<S, RATE, VEC, in(), z(), false, kGatedWholeWarps, kFwdT>(g, L);
        else if (g.p.batch * g.slabs > 3 * 152)
            return gated_forward_of<S, RATE, VEC, in(), z(), false, kGatedWarps, kFwdT>(g, L);
        else
            return gated_forward_of<S, RATE, VEC, in(), z(), false, kGatedWarps, kFwdMoreT>(g, L);
    });
}
template <class S, bool RATE, bool VEC> static cudaError_t gated_backward(const GatedArgs &g, float *part, const Launch &L) {
    return by_gates(g.p, [&](auto in, auto z) {
        if (g.ctas > 1)
            return gated_backward_of<S, RATE, VEC, in(), z(), true>(g, part, L);
        return gated_backward_of<S, RATE, VEC, in(), z(), false>(g, part, L);
    });
}
template <class S, bool RATE, bool VEC> static cudaError_t gated_single(const GatedArgs &g, const Launch &L) {
    const int64_t threads = g.p.batch * ((g.p.dim + 1) / 2);
    note_launch();
    return launch_cluster(k_gated_step<S, RATE, VEC>, (threads + 127) / 128, 128, 0, 1, L.stream, g);
}

#define MT_GATED_BY(f, ...)                                                                              \
    (g.p.rate != nullptr ? (vec ? f<S, true, true>(__VA_ARGS__) : f<S, true, false>(__VA_ARGS__))        \
                         : (vec ? f<S, false, true>(__VA_ARGS__) : f<S, false, false>(__VA_ARGS__)))
#define MT_GATED_TYPE(name, T)                                                                                                      \
    using S = T;                                                                                                                    \
    cudaError_t gated_forward_##name(const GatedArgs &g, bool vec, const Launch &L) { return MT_GATED_BY(gated_forward, g, L); }    \
    cudaError_t gated_single_##name(const GatedArgs &g, bool vec, const Launch &L) { return MT_GATED_BY(gated_single, g, L); }      \
    cudaError_t gated_##name##_take_error(int *code) { return clusters_take_error(code); }
#define MT_GATED_GRAD_TYPE(name, T)                                                                                                 \
    using S = T;                                                                                                                    \
    cudaError_t gated_backward_##name(const GatedArgs &g, float *part, bool vec, const Launch &L) {                                 \
        return MT_GATED_BY(gated_backward, g, part, L);                                                                             \
    }                                                                                                                               \
    cudaError_t gated_grad_##name##_take_error(int *code) { return clusters_take_error(code); }

#define MT_GATED_DECL(name)                                                                  \
    cudaError_t gated_forward_##name(const GatedArgs &g, bool vec, const Launch &L);         \
    cudaError_t gated_backward_##name(const GatedArgs &g, float *part, bool vec, const Launch &L); \
    cudaError_t gated_single_##name(const GatedArgs &g, bool vec, const Launch &L);
MT_GATED_DECL(f32)
MT_GATED_DECL(bf16)
MT_GATED_DECL(f16)
#undef MT_GATED_DECL

}  // namespace mt
