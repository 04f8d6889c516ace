// fp8_quantize.cu -- fp8 (e4m3) with one scale for each block of 128 values.
//
// Bound by memory: one read of x, one byte written an element.  Two kernels: one for blocks within a
// row, a half-warp a block, and one for blocks that span 128 rows, which reads a 128 x 128 tile into
// registers (64 values a thread, all loads in flight at once) and, where the transpose is stored,
// turns it around in shared memory so that both sides move whole lines.
#include "fp8_kernels.cuh"

namespace mh3a {
namespace fp8 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void block_scale(float amax, float* scale, float* factor) {
    const float a = max_nan(amax, kTiny);
    *scale = __fdiv_rn(a, kMax);
    *factor = __fdiv_rn(kMax, a);
}

// Blocks of 128 within a row.  A warp takes 128 columns of 4 consecutive rows: lane l holds columns
// 4 l .. 4 l + 3 of each, so four loads are in flight; a block's 32 rows of scales are one line.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_quant_rows(const QuantArgs a, int blocks) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    constexpr int R = 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rg = blockIdx.x / blocks, kb = blockIdx.x % blocks;
    const int r0 = (rg * (kThreads / 32) + warp) * R;
    const int c = kb * kBlock + lane * 4;
    const int left = a.cols - c;
    const T* x = static_cast<const T*>(a.x) + (long long)r0 * a.xs + c;
    float4 v[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        v[i] = r0 + i < a.rows && left > 0 ? load4<T>(x + i * a.xs, a.vec && left >= 4, left) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float m = amax4(v[i]);
#pragma unroll
        for (int off = 16; off; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        float s, f;
        block_scale(m, &s, &f);
        if (r0 + i >= a.rows) break;
        const uint32_t q = pack4(__fmul_rn(v[i].x, f), __fmul_rn(v[i].y, f), __fmul_rn(v[i].z, f), __fmul_rn(v[i].w, f));
        unsigned char* to = a.q + (long long)(r0 + i) * a.qs + c;
        if (left >= 4) {
            *reinterpret_cast<uint32_t*>(to) = q;
        } else {
            for (int k = 0; k < left; ++k) to[k] = (unsigned char)(q >> (8 * k));
        }
        if (lane == 0) a.scale[(long long)kb * a.rows + r0 + i] = s;
    }
}

// A 128 x 128 tile: warp w holds rows 16 w .. 16 w + 15, lane l columns 4 l .. 4 l + 3.
// COLUMNS: every column of the tile is a block (of the transpose's row), else the tile is one block.
// TRANSPOSE: the transpose is stored.
template <typename T, bool COLUMNS, bool TRANSPOSE>
__global__ void __launch_bounds__(kThreads) k_quant_tile(const QuantArgs a, int col_tiles) {
    constexpr int R = 16, kPitch = kBlock + 16;
    __shared__ __align__(16) float red[kThreads / 32][kBlock];
    __shared__ __align__(16) unsigned char turned[TRANSPOSE ? kBlock * kPitch : 16];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rt = blockIdx.x / col_tiles, ct = blockIdx.x % col_tiles;
    const int r0 = rt * kBlock + warp * R, c = ct * kBlock + lane * 4;
    const int left = a.cols - c;
    const T* x = static_cast<const T*>(a.x) + (long long)r0 * a.xs + c;
    float4 v[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        v[i] = r0 + i < a.rows && left > 0 ? load4<T>(x + i * a.xs, a.vec && left >= 4, left) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        m.x = max_nan(m.x, fabsf(v[i].x));
        m.y = max_nan(m.y, fabsf(v[i].y));
        m.z = max_nan(m.z, fabsf(v[i].z));
        m.w = max_nan(m.w, fabsf(v[i].w));
    }
    float4 f;
    const int outer = COLUMNS ? a.cols : 0;
    if (COLUMNS) {
        *reinterpret_cast<float4*>(&red[warp][lane * 4]) = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const float4 o = *reinterpret_cast<const float4*>(&red[w][lane * 4]);
            m.x = max_nan(m.x, o.x);
            m.y = max_nan(m.y, o.y);
            m.z = max_nan(m.z, o.z);
            m.w = max_nan(m.w, o.w);
        }
        float4 s;
        block_scale(m.x, &s.x, &f.x);
        block_scale(m.y, &s.y, &f.y);
        block_scale(m.z, &s.z, &f.z);
        block_scale(m.w, &s.w, &f.w);
        if (warp == 0) {
            float* to = a.scale + (long long)rt * outer + c;
            if (left > 0) to[0] = s.x;
            if (left > 1) to[1] = s.y;
            if (left > 2) to[2] = s.z;
            if (left > 3) to[3] = s.w;
        }
    } else {
        float t = max_nan(max_nan(m.x, m.y), max_nan(m.z, m.w));
#pragma unroll
        for (int off = 16; off; off >>= 1) t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, off));
        if (lane == 0) red[0][warp] = t;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) t = max_nan(t, red[0][w]);
        float s;
        block_scale(t, &s, &f.x);
        f.y = f.z = f.w = f.x;
        if (threadIdx.x == 0) {
            const int row_tiles = (a.rows + kBlock - 1) / kBlock;
            a.scale[TRANSPOSE ? (long long)rt * col_tiles + ct : (long long)ct * row_tiles + rt] = s;
        }
    }
    if (TRANSPOSE) {
        // 16 consecutive rows of x are 16 bytes of a row of the transpose
        const float* fv = &f.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q[i] = pack4(__fmul_rn((&v[4 * i].x)[j], fv[j]), __fmul_rn((&v[4 * i + 1].x)[j], fv[j]),
                             __fmul_rn((&v[4 * i + 2].x)[j], fv[j]), __fmul_rn((&v[4 * i + 3].x)[j], fv[j]));
            *reinterpret_cast<uint4*>(turned + (lane * 4 + j) * kPitch + warp * R) = make_uint4(q[0], q[1], q[2], q[3]);
        }
        __syncthreads();
        const int width = min(kBlock, a.rows - rt * kBlock);  // bytes of each stored row
        for (int k = threadIdx.x; k < kBlock * (kBlock / 16); k += kThreads) {
            const int row = k >> 3, at = (k & 7) * 16;
            if (ct * kBlock + row >= a.cols || at >= width) continue;
            unsigned char* to = a.q + (long long)(ct * kBlock + row) * a.qs + (long long)rt * kBlock + at;
            const unsigned char* from = turned + row * kPitch + at;
            if (at + 16 <= width) {
                *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
            } else {
                for (int i = 0; i < width - at; ++i) to[i] = from[i];
            }
        }
    } else {
        unsigned char* to = a.q + (long long)r0 * a.qs + c;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (r0 + i >= a.rows) break;
            const uint32_t q = pack4(__fmul_rn(v[i].x, f.x), __fmul_rn(v[i].y, f.y), __fmul_rn(v[i].z, f.z), __fmul_rn(v[i].w, f.w));
            if (left >= 4) {
                *reinterpret_cast<uint32_t*>(to + i * a.qs) = q;
            } else {
                for (int k = 0; k < left; ++k) (to + i * a.qs)[k] = (unsigned char)(q >> (8 * k));
            }
        }
    }
}

template <typename T>
int launch(const QuantArgs& a, int block_rows, int transpose, cudaStream_t s) {
    const long long kb = (a.cols + kBlock - 1) / kBlock, rb = (a.rows + kBlock - 1) / kBlock;
    cudaError_t e;
    if (block_rows == 1 && !transpose) {
        const int groups = (int)((a.rows + 31LL) / 32);
        e = launch_dependent(k_quant_rows<T>, dim3((unsigned)(kb * groups)), dim3(kThreads), 0, s, a, (int)kb);
    } else if (block_rows == 1) {
        e = launch_dependent(k_quant_tile<T, true, true>, dim3((unsigned)(kb * rb)), dim3(kThreads), 0, s, a, (int)kb);
    } else if (transpose) {
        e = launch_dependent(k_quant_tile<T, false, true>, dim3((unsigned)(kb * rb)), dim3(kThreads), 0, s, a, (int)kb);
    } else {
        e = launch_dependent(k_quant_tile<T, false, false>, dim3((unsigned)(kb * rb)), dim3(kThreads), 0, s, a, (int)kb);
    }
    return e == cudaSuccess ? 1 : -1;
}

}  // namespace

int launch_quantize(const QuantArgs& a, int dtype, int block_rows, int transpose, cudaStream_t s) {
    switch (dtype) {
        case MH3A_DTYPE_F32: return launch<float>(a, block_rows, transpose, s);
        case MH3A_DTYPE_F16: return launch<__half>(a, block_rows, transpose, s);
        default: return launch<__nv_bfloat16>(a, block_rows, transpose, s);
    }
}

}  // namespace fp8
}  // namespace mh3a
