// norm_kernels.cuh -- shared device code of the group-norm operators: typed vector access, the
// activations and their derivatives, and the parameters every kernel gets.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mh3a_internal.cuh"
#include "tc_ptx.cuh"

namespace mh3a {
namespace norm {

// What a launch works on.  Strides in elements; y, dx and dy as documented in mh3a.h.
struct NormArgs {
    const void* x;
    const void* dy;
    void* out;  // y (forward) or dx (backward)
    long long xb, xr, gb, gr;
    const float *weight, *bias, *alpha, *beta;
    const int* lengths;
    float* mean;
    float* rstd;
    float *dweight, *dbias, *dalpha, *dbeta;
    float* ws;
    int B, T, C, G, D;
    float eps;
    int chunks, rows;  // row chunks per item and rows per chunk
    int ctiles, tx;    // channel tiles per row, threads along the channels
};

__device__ __forceinline__ int valid_rows(const NormArgs& a, int b) {
    if (!a.lengths) return a.T;
    const int n = __ldg(a.lengths + b);
    return n < 0 ? 0 : (n > a.T ? a.T : n);
}

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V elements as they lie in memory.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}

// Pairs of neighbouring elements, for the packed fp32x2 instructions.
__device__ __forceinline__ float2 pair_of(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ float2 pair_of(const __half* v) { return __half22float2(*reinterpret_cast<const __half2*>(v)); }
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* v) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(v);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
template <typename T, int V>
__device__ __forceinline__ void unpack_pairs(const Pack<T, V>& p, float2 (&f)[V / 2]) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[i] = pair_of(p.v + 2 * i);
}

__device__ __forceinline__ void put_pair(float* v, float2 f) { *reinterpret_cast<float2*>(v) = f; }
__device__ __forceinline__ void put_pair(__half* v, float2 f) {
    *reinterpret_cast<__half2*>(v) = __floats2half2_rn(f.x, f.y);
}
__device__ __forceinline__ void put_pair(__nv_bfloat16* v, float2 f) {
    *reinterpret_cast<__nv_bfloat162*>(v) = __floats2bfloat162_rn(f.x, f.y);
}

template <typename T, int V>
__device__ __forceinline__ void store_pairs(T* p, const float2 (&f)[V / 2]) {
    Pack<T, V> o;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) put_pair(o.v + 2 * i, f[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = o;
}

// V per-channel parameters by 16-byte loads, `other` for a null array: c is a multiple of V, C too, p 16-byte
// aligned.
template <int V>
__device__ __forceinline__ void load_param_vec(const float* p, int c, float other, float2 (&f)[V / 2]) {
    if (p) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p + c) + i);
            f[2 * i] = make_float2(v.x, v.y);
            f[2 * i + 1] = make_float2(v.z, v.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) f[i] = make_float2(other, other);
    }
}

// n / d by a multiplication: mul = ceil(2^32 / d) gives the exact quotient for n d < 2^32, which
// holds for thread indices and for channels of one slab.
struct FastDiv {
    unsigned d, mul;
};
__device__ __forceinline__ unsigned operator/(unsigned n, FastDiv f) { return f.d == 1 ? n : __umulhi(n, f.mul); }

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }

// v within [-c, c]; NaN stays NaN.
__device__ __forceinline__ float clamp_nan(float v, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(-c));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(r) : "f"(c));
    return r;
}

// sin(theta) and cos(theta) up to a common sign, theta = alpha u: what sin^2 and sin cos need, both
// of period pi; two values at a time in packed fp32x2 operations.
//
// fp32 tensors (PRECISE): the phase is reduced to [-pi/2, pi/2] by the Cody-Waite method (pi as
// fp32(pi) plus the fp32 remainder, the product's rounding error carried along from one fma), then the
// Taylor series (truncated terms below 7e-10).  k = rint(theta / pi) comes from adding and taking away
// 1.5 2^23, right for |theta| below 2^22 pi; farther out fp32 leaves theta no fraction of a period, and
// the clamp keeps the result a sine.
//
// 16-bit tensors: the hardware sine, whose 2^-21 absolute error is far below the rounding of y and dx; its
// argument loses |theta| 2^-24 as the product itself does, so a reduction first would gain nothing.  In the
// parameters' gradients, fp32 sums, it does show: off by 2.3 to 5.5 x 10^-7 of their size where the series
// gives 1.1 to 2.4 x 10^-7 (1 to 160000 rows), of inputs that are rounded to 2^-9 or 2^-12 themselves.
template <bool PRECISE, bool COS>
__device__ __forceinline__ void sin_cos_mod_pi(float2 alpha, float2 u, float2* sn, float2* cs) {
    const float2 v = __fmul2_rn(alpha, u);
    if (!PRECISE) {
        *sn = make_float2(__sinf(v.x), __sinf(v.y));
        if (COS) *cs = make_float2(__cosf(v.x), __cosf(v.y));
        return;
    }
    const float2 e = __ffma2_rn(alpha, u, neg2(v));
    const float2 k = __fadd2_rn(__ffma2_rn(v, both(0.318309886183790671538f), both(12582912.f)), both(-12582912.f));
    float2 r = __ffma2_rn(k, both(-3.14159274101257324219f), v);
    r = __fadd2_rn(__ffma2_rn(k, both(8.74227800037248297e-08f), r), e);
    r = make_float2(clamp_nan(r.x, 1.6f), clamp_nan(r.y, 1.6f));
    const float2 r2 = __fmul2_rn(r, r);
    float2 p = both(1.0f / 6227020800.0f);
    p = __ffma2_rn(p, r2, both(-1.0f / 39916800.0f));
    p = __ffma2_rn(p, r2, both(1.0f / 362880.0f));
    p = __ffma2_rn(p, r2, both(-1.0f / 5040.0f));
    p = __ffma2_rn(p, r2, both(1.0f / 120.0f));
    p = __ffma2_rn(p, r2, both(-1.0f / 6.0f));
    *sn = __ffma2_rn(__fmul2_rn(r, r2), p, r);
    if (COS) {
        float2 q = both(-1.0f / 87178291200.0f);
        q = __ffma2_rn(q, r2, both(1.0f / 479001600.0f));
        q = __ffma2_rn(q, r2, both(-1.0f / 3628800.0f));
        q = __ffma2_rn(q, r2, both(1.0f / 40320.0f));
        q = __ffma2_rn(q, r2, both(-1.0f / 720.0f));
        q = __ffma2_rn(q, r2, both(1.0f / 24.0f));
        q = __ffma2_rn(q, r2, both(-0.5f));
        *cs = __ffma2_rn(q, r2, both(1.0f));
    }
}

__device__ __forceinline__ float ex2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (Also 1 / (beta + 1e-9), for all types: within one unit in the last place, where a division is within half.)
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x for x in [1, 2^126]: a first guess by taking x's bits (exponent and fraction, so a piecewise linear
// logarithm) from a constant, then a step of Newton's iteration and one of third order for what is left.
// The constant minimises the guess's largest relative error, 0.051 (by search); then 2.6e-3, then 1.7e-8,
// below the roundings (8e-8 in all).  From 2^125.9 on the guess is no normal number any more, which leaves
// 1.2e-6 at 2^126; beyond 1.9 2^126 the subtraction gives no number at all.
__device__ __forceinline__ float rcp_newton(float x) {
    float y = __uint_as_float(0x7ef31000u - __float_as_uint(x));
    y = fmaf(y, fmaf(-x, y, 1.f), y);
    const float r = fmaf(-x, y, 1.f);
    return fmaf(y, fmaf(r, r, r), y);
}

// 1 / (1 + e^-u).  16-bit tensors take the hardware's exponential and reciprocal (each a few ulp;
// results below 2^-126 become 0), without the scaling that keeps subnormal numbers, but for one of
// the two reciprocals: the unit that computes these takes eight cycles for a warp, and three of them beside
// five multiplications take less time than four (7 items of [3001, 200] 9.36 us with both by the unit, 9.11
// with one).  The two channels of a pair so differ by a few units of 2^-24 for equal u, and nowhere else.
template <bool PRECISE>
__device__ __forceinline__ float2 sigmoid(float2 u) {
    if (PRECISE) return make_float2(1.0f / (1.0f + expf(-u.x)), 1.0f / (1.0f + expf(-u.y)));
    const float2 t = __fmul2_rn(u, both(-1.44269504088896341f));
    const float2 e = __fadd2_rn(make_float2(ex2_ftz(t.x), ex2_ftz(t.y)), both(1.f));
    return make_float2(rcp_ftz(e.x), e.y > 0x1p126f ? 0.f : rcp_newton(e.y));  // 0 where rcp_ftz gives 0; NaN stays
}

// y = act(u) of two neighbouring channels; ib = 1 / (beta + 1e-9)
template <int ACT, bool PRECISE>
__device__ __forceinline__ float2 act_fwd(float2 u, float2 al, float2 ib) {
    if (ACT == MH3A_ACT_SILU) return __fmul2_rn(u, sigmoid<PRECISE>(u));
    if (ACT == MH3A_ACT_SNAKE_BETA) {
        float2 sn, cs;
        sin_cos_mod_pi<PRECISE, false>(al, u, &sn, &cs);
        return __ffma2_rn(__fmul2_rn(sn, sn), ib, u);
    }
    return u;
}

// act'(u), and for SnakeBeta the factors of dalpha and dbeta: dalpha = sum dy *pa,
// dbeta = -sum dy *pb (1/beta^2 follows once, after the sum).
template <int ACT, bool PRECISE>
__device__ __forceinline__ float2 act_slope(float2 u, float2 al, float2 ib, float2* pa, float2* pb) {
    if (ACT == MH3A_ACT_SILU) {
        const float2 s = sigmoid<PRECISE>(u);
        return __fmul2_rn(s, __ffma2_rn(u, __ffma2_rn(s, both(-1.f), both(1.f)), both(1.f)));
    }
    if (ACT == MH3A_ACT_SNAKE_BETA) {
        float2 sn, cs;
        sin_cos_mod_pi<PRECISE, true>(al, u, &sn, &cs);
        const float2 s2 = __fmul2_rn(__fmul2_rn(__fadd2_rn(sn, sn), cs), ib);  // sin(2 alpha u) / beta
        *pa = __fmul2_rn(u, s2);
        *pb = __fmul2_rn(sn, sn);
        return __ffma2_rn(al, s2, both(1.f));
    }
    return both(1.f);
}

// Sums of one channel in the backward pass: 0 du, 1 du xh, 2 dy * (factor of dalpha), 3 dy * (factor
// of dbeta).
template <int ACT>
constexpr int kSums = ACT == MH3A_ACT_SNAKE_BETA ? 4 : 2;

}  // namespace norm
}  // namespace mh3a
