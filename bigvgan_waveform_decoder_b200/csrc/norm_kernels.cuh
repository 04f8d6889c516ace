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

template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& p, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f<T>(p.v[i]);
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

template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const float (&f)[V]) {
    Pack<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.v[i] = from_f<T>(f[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = o;
}

// Loads V per-channel parameters; channels beyond C and a null array give `other`.
template <int V>
__device__ __forceinline__ void load_param(const float* p, int c, int C, float other, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (p && c + i < C) ? __ldg(p + c + i) : other;
}

// sin(theta) and cos(theta) up to a common sign, theta = alpha u: what sin^2 and sin cos need, both
// of period pi.  The phase is reduced to [-pi/2, pi/2] by the Cody-Waite method (pi as fp32(pi)
// plus the fp32 remainder, the product's rounding error carried along from one fma).  fp32 tensors
// take the Taylor series there (truncated terms below 7e-10); 16-bit tensors take the hardware
// sine, whose 2^-21 absolute error is far below their rounding.
template <bool PRECISE>
__device__ __forceinline__ void sin_cos_mod_pi(float alpha, float u, float* sn, float* cs) {
    const float v = alpha * u;
    const float e = fmaf(alpha, u, -v);
    const float k = rintf(v * 0.318309886183790671538f);
    float r = fmaf(-k, 3.14159274101257324219f, v);
    r = fmaf(-k, -8.74227800037248297e-08f, r) + e;
    if (PRECISE) {
        const float r2 = r * r;
        float p = 1.0f / 6227020800.0f;
        p = fmaf(p, r2, -1.0f / 39916800.0f);
        p = fmaf(p, r2, 1.0f / 362880.0f);
        p = fmaf(p, r2, -1.0f / 5040.0f);
        p = fmaf(p, r2, 1.0f / 120.0f);
        p = fmaf(p, r2, -1.0f / 6.0f);
        *sn = fmaf(r * r2, p, r);
        float q = -1.0f / 87178291200.0f;
        q = fmaf(q, r2, 1.0f / 479001600.0f);
        q = fmaf(q, r2, -1.0f / 3628800.0f);
        q = fmaf(q, r2, 1.0f / 40320.0f);
        q = fmaf(q, r2, -1.0f / 720.0f);
        q = fmaf(q, r2, 1.0f / 24.0f);
        q = fmaf(q, r2, -0.5f);
        *cs = fmaf(q, r2, 1.0f);
    } else {
        *sn = __sinf(r);
        *cs = __cosf(r);
    }
}

template <bool PRECISE>
__device__ __forceinline__ float sigmoid(float u) {
    if (PRECISE) return 1.0f / (1.0f + expf(-u));
    return __fdividef(1.0f, 1.0f + __expf(-u));
}

// y = act(u); ib = 1 / (beta + 1e-9)
template <int ACT, bool PRECISE>
__device__ __forceinline__ float act_fwd(float u, float al, float ib) {
    if (ACT == MH3A_ACT_SILU) return u * sigmoid<PRECISE>(u);
    if (ACT == MH3A_ACT_SNAKE_BETA) {
        float sn, cs;
        sin_cos_mod_pi<PRECISE>(al, u, &sn, &cs);
        return fmaf(sn * sn, ib, u);
    }
    return u;
}

// act'(u), and for SnakeBeta the factors of dalpha and dbeta: dalpha = sum dy *pa,
// dbeta = -sum dy *pb (1/beta^2 follows once, after the sum).
template <int ACT, bool PRECISE>
__device__ __forceinline__ float act_slope(float u, float al, float ib, float* pa, float* pb) {
    if (ACT == MH3A_ACT_SILU) {
        const float s = sigmoid<PRECISE>(u);
        return s * fmaf(u, 1.0f - s, 1.0f);
    }
    if (ACT == MH3A_ACT_SNAKE_BETA) {
        float sn, cs;
        sin_cos_mod_pi<PRECISE>(al, u, &sn, &cs);
        const float s2 = 2.0f * sn * cs * ib;  // sin(2 alpha u) / beta
        *pa = u * s2;
        *pb = sn * sn;
        return fmaf(al, s2, 1.0f);
    }
    return 1.0f;
}

}  // namespace norm
}  // namespace mh3a
