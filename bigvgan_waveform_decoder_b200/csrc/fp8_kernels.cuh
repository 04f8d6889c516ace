// fp8_kernels.cuh -- launchers and device helpers of the fp8 operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "mh3a_internal.cuh"
#include "ops_common.cuh"
#include "tc_ptx.cuh"

namespace mh3a {
namespace fp8 {

constexpr int kBlock = 128;       // values under one scale along the inner axis
constexpr float kMax = 448.0f;    // largest e4m3 value
constexpr float kTiny = 0x1p-100f;  // blocks whose largest magnitude is below this are scaled as if it were this

// Larger of two values; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A wait by a whole warp, the same answer in all lanes: what follows has to be done by all or by none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns = 1000000000ull) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, limit_ns));
}

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Two 16-bit values, the first in the low half.
template <typename T>
__device__ __forceinline__ float2 pair(uint32_t w) {
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Four consecutive elements; `vec`: they all exist and are aligned to their size, else the `n` that
// exist are read one by one and the others are 0.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p, bool vec, int n) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (vec) {
        if constexpr (sizeof(T) == 4) {
            v = *reinterpret_cast<const float4*>(p);
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            const float2 lo = pair<T>(q.x), hi = pair<T>(q.y);
            v = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
    } else {
        if (n > 0) v.x = as_float<T>(p[0]);
        if (n > 1) v.y = as_float<T>(p[1]);
        if (n > 2) v.z = as_float<T>(p[2]);
        if (n > 3) v.w = as_float<T>(p[3]);
    }
    return v;
}

__device__ __forceinline__ float amax4(float4 v) {
    return max_nan(max_nan(fabsf(v.x), fabsf(v.y)), max_nan(fabsf(v.z), fabsf(v.w)));
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

struct QuantArgs {
    const void* x;
    long long xs;  // elements between rows of x
    unsigned char* q;
    long long qs;  // bytes between rows of q
    float* scale;
    int rows, cols;
    int vec;       // four adjacent elements of x can be read at once
    int vec16;     // rows of 16-bit x start on 16-byte boundaries, rows of q on 8-byte ones
};

// Launchers: number of kernels, or -1.
int launch_quantize(const QuantArgs& a, int dtype, int block_rows, int transpose, cudaStream_t s);

struct MatmulArgs {
    const void* a;
    long long as;
    const float* sa;
    const void* b;
    long long bs;
    const float* sb;
    int b_block_rows;
    int M, N, K;
    const float* bias;
    void* out;
    long long os;
    int out_dtype;
};
int launch_matmul(const MatmulArgs& m, cudaStream_t s);

struct FewRowsArgs {
    const void* x;
    long long xs;
    const unsigned char* w;
    long long ws;
    const float* sw;
    int w_block_rows;
    int M, N, K;
    const float* bias;
    void* y;
    long long ys;
};
int launch_few_rows(const FewRowsArgs& a, int dtype, cudaStream_t s);

}  // namespace fp8
}  // namespace mh3a
