// mt_seq.cuh -- what the sequence-model kernels (embedding lookup, short
// causal convolution, selective state space scan) share: widening loads and
// rounding stores of a few neighbouring channels, and the scalar functions.
//
// Activations are f32, bf16 or f16 and are widened to f32 at the load; every
// product, sum and state is f32; a result is rounded once, to nearest even,
// at its store.
#pragma once

#include "mt_tile.cuh"

namespace mt {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// launch_pdl for grids of two dimensions.
template <class... KArgs, class... Args>
static cudaError_t launch_pdl_2d(void (*kernel)(KArgs...), dim3 grid, unsigned block, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// The dynamic shared memory of a kernel is allowed once per device.
template <class F> static cudaError_t allow_shared(F kernel, int bytes, PerDevice &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev >= kMaxDevices || done.get(dev) != 0)
        return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done.set(dev, 1);
    return e;
}

// ---- four neighbouring values -------------------------------------------------
// as one vector access when `vec` (then p is aligned to four values) and all four
// are `live`, otherwise value by value; those that do not exist load as 0.
template <class S, int V> struct VecOf;
template <> struct VecOf<float, 4> { using T = uint4; };
template <> struct VecOf<__nv_bfloat16, 4> { using T = uint2; };
template <> struct VecOf<__half, 4> { using T = uint2; };

template <class S> __device__ __forceinline__ void widen4(const typename VecOf<S, 4>::T &w, float (&x)[4]);
template <> __device__ __forceinline__ void widen4<float>(const uint4 &w, float (&x)[4]) { Codec<float>::unpack(w, x); }
template <> __device__ __forceinline__ void widen4<__nv_bfloat16>(const uint2 &w, float (&x)[4]) {
    Codec<__nv_bfloat16>::two(w.x, x[0], x[1]);
    Codec<__nv_bfloat16>::two(w.y, x[2], x[3]);
}
template <> __device__ __forceinline__ void widen4<__half>(const uint2 &w, float (&x)[4]) {
    Codec<__half>::two(w.x, x[0], x[1]);
    Codec<__half>::two(w.y, x[2], x[3]);
}
template <class S> __device__ __forceinline__ typename VecOf<S, 4>::T narrow4(const float (&x)[4]);
template <> __device__ __forceinline__ uint4 narrow4<float>(const float (&x)[4]) { return Codec<float>::pack(x); }
template <> __device__ __forceinline__ uint2 narrow4<__nv_bfloat16>(const float (&x)[4]) {
    return make_uint2(Codec<__nv_bfloat16>::pack2(x[0], x[1]), Codec<__nv_bfloat16>::pack2(x[2], x[3]));
}
template <> __device__ __forceinline__ uint2 narrow4<__half>(const float (&x)[4]) {
    return make_uint2(Codec<__half>::pack2(x[0], x[1]), Codec<__half>::pack2(x[2], x[3]));
}

// Four values kept in their storage form, so that a load can be in flight
// while earlier ones are worked on.
template <class S> struct Raw4 {
    typename VecOf<S, 4>::T w;
    __device__ __forceinline__ void load(const S *p, bool vec, int live) {
        if (vec && live == 4) {
            w = *reinterpret_cast<const typename VecOf<S, 4>::T *>(p);
        } else {
            S v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = k < live ? p[k] : S(0.0f);
            w = *reinterpret_cast<typename VecOf<S, 4>::T *>(v);
        }
    }
    __device__ __forceinline__ void widen(float (&x)[4]) const { widen4<S>(w, x); }
};

// ---- asynchronous copies to shared memory ------------------------------------------
// Zeros where `in` is false (the source is then not read).
template <int BYTES> __device__ __forceinline__ void cp_async_zfill(uint32_t dst, const void *src, bool in) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" :: "r"(dst), "l"(src), "r"(in ? BYTES : 0), "n"(BYTES) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most LEFT of the thread's groups are on their way
template <int LEFT> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(LEFT) : "memory"); }

// ---- scalar functions ---------------------------------------------------------
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcpf(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoidf(float x) { return rcpf(1.0f + ex2f(-kLog2e * x)); }

// log(1 + exp(x)) = max(x, 0) + log(1 + e), e = exp(-|x|) in (0, 1], and
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3, by the odd series of atanh
// (the classical series for a logarithm): the first term left out is below
// 1.5e-8 of the sum. No cancellation, so the small steps that a scan lives on
// (exp(x) far below 1) keep f32's relative precision, which log(1 + exp(x))
// evaluated as written does not.
__device__ __forceinline__ float softplusf(float x) {
    const float e = ex2f(-kLog2e * fabsf(x));
    const float s = e * rcpf(2.0f + e);
    const float q = s * s;
    float p = 1.0f / 13.0f;
    p = fmaf(p, q, 1.0f / 11.0f);
    p = fmaf(p, q, 1.0f / 9.0f);
    p = fmaf(p, q, 1.0f / 7.0f);
    p = fmaf(p, q, 1.0f / 5.0f);
    p = fmaf(p, q, 1.0f / 3.0f);
    p = fmaf(p, q, 1.0f);
    return fmaf(2.0f * s, p, fmaxf(x, 0.0f));
}

// ---- two f32 lanes in a register pair -------------------------------------------
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2f(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2f(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2f(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2f(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2f(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 both(float x) { return pack2f(x, x); }
__device__ __forceinline__ f32x2 ex2_2f(f32x2 v) {
    float a, b;
    unpack2f(v, a, b);
    return pack2f(ex2f(a), ex2f(b));
}

__device__ __forceinline__ f32x2 rcp_2f(f32x2 v) {
    float a, b;
    unpack2f(v, a, b);
    return pack2f(rcpf(a), rcpf(b));
}
// Exponent of a decay, d * A in powers of two. The unit's exponential is low by about 2e-8 of its
// value on average, and a state that remembers n tokens sees that n times. The constant takes it back in a multiply-add where
// the product alone would be as dear. Mean error by decay, without it and with it (a million arguments a range):
//   0.5 to 0.7    -2.5e-8 (the constant is lost in the argument's rounding)     0.97 to 0.996      -2.6e-8, -0.8e-8
//   0.7 to 0.97   -1.7e-8, +0.1e-8                                              0.9973 and above   -0.7e-8, +1.1e-8
// So decays above 0.9973 are worse off, where the lean is smallest. Errors of scans stay at the level of f32: relative
// to 64 bits, dA over 2048 tokens x 2048 channels x 16 states 7e-7 (without the constant 1.4e-6, torch operations 8e-6), and with
// A of 0.01 to 0.02, whose states remember thousands of 8192 tokens, dA 8e-7 (9e-7, 3.7e-5) and states 6e-7 (8e-7, 3.9e-5).
// Half the constant is a little better there, and worse by up to two thirds at the common decays.
// Up to 8e-8 the unit's answer is 1 exactly, so a token with d = 0 still leaves the state alone, bit for bit.
constexpr float kExponentLow = 2.6e-8f;
__device__ __forceinline__ f32x2 exponent2f(f32x2 d, f32x2 A) { return fma2f(d, A, both(kExponentLow)); }

// softplusf and sigmoidf of two values: half the multiply-add instructions.
__device__ __forceinline__ f32x2 softplus_2f(f32x2 x) {
    float a, b;
    unpack2f(x, a, b);
    const f32x2 e = pack2f(ex2f(-kLog2e * fabsf(a)), ex2f(-kLog2e * fabsf(b)));
    const f32x2 s = mul2f(e, rcp_2f(add2f(both(2.0f), e)));
    const f32x2 q = mul2f(s, s);
    f32x2 p = both(1.0f / 13.0f);
    p = fma2f(p, q, both(1.0f / 11.0f));
    p = fma2f(p, q, both(1.0f / 9.0f));
    p = fma2f(p, q, both(1.0f / 7.0f));
    p = fma2f(p, q, both(1.0f / 5.0f));
    p = fma2f(p, q, both(1.0f / 3.0f));
    p = fma2f(p, q, both(1.0f));
    return fma2f(add2f(s, s), p, pack2f(fmaxf(a, 0.0f), fmaxf(b, 0.0f)));
}
__device__ __forceinline__ f32x2 sigmoid_2f(f32x2 x) { return rcp_2f(add2f(both(1.0f), ex2_2f(mul2f(both(-kLog2e), x)))); }

// a where yes, else b
__device__ __forceinline__ f32x2 choose_2f(bool yes, f32x2 a, f32x2 b) {
    float a0, a1, b0, b1;
    unpack2f(a, a0, a1);
    unpack2f(b, b0, b1);
    return pack2f(yes ? a0 : b0, yes ? a1 : b1);
}

}  // namespace mt
