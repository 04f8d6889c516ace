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

// The same for 16-bit x, 16 bytes a lane: a half-warp a block, a warp 256 columns of 4 rows.  The largest
// magnitude is found on packed pairs, and the two quotients of a block are formed once, by lane 0 .. 3
// of its half-warp for rows 0 .. 3, and handed around.  (Four elements a lane and every quotient in
// every lane: 25 us against 11.5 at [12800, 2048] bf16.)
template <typename T>
__global__ void __launch_bounds__(kThreads) k_quant_rows16(const QuantArgs a, int pairs) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    constexpr int R = 4;
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rg = blockIdx.x / pairs, kp = blockIdx.x % pairs;
    const int r0 = (rg * (kThreads / 32) + warp) * R;
    const int c = kp * 2 * kBlock + lane * 8;
    if (r0 >= a.rows) return;
    const int left = a.cols - c;
    const T* x = static_cast<const T*>(a.x) + (long long)r0 * a.xs + c;
    union Vec {
        uint4 q;
        T2 h[4];
        uint32_t w[4];
        T e[8];
    } v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        v[i].q = make_uint4(0, 0, 0, 0);
        if (r0 + i < a.rows) {
            if (left >= 8) {
                v[i].q = *reinterpret_cast<const uint4*>(x + i * a.xs);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < left) v[i].e[k] = x[i * a.xs + k];
            }
        }
    }
    float mine = 0.f;  // the largest magnitude of the block whose quotients this lane forms
#pragma unroll
    for (int i = 0; i < R; ++i) {
        T2 m = __hmax2_nan(__hmax2_nan(__habs2(v[i].h[0]), __habs2(v[i].h[1])), __hmax2_nan(__habs2(v[i].h[2]), __habs2(v[i].h[3])));
#pragma unroll
        for (int off = 8; off; off >>= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&m), off);
            m = __hmax2_nan(m, *reinterpret_cast<const T2*>(&o));
        }
        const float2 f = pair<T>(*reinterpret_cast<const uint32_t*>(&m));
        const float t = max_nan(f.x, f.y);
        mine = (lane & 3) == i ? t : mine;
    }
    float s, f;
    block_scale(mine, &s, &f);
    const int kb = kp * 2 + (lane >> 4);
    if ((lane & 15) < R && r0 + (lane & 15) < a.rows && kb * kBlock < a.cols) a.scale[(long long)kb * a.rows + r0 + (lane & 15)] = s;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, (lane & 16) + i);
        if (r0 + i >= a.rows || left <= 0) continue;
        float2 p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = __fmul2_rn(pair<T>(v[i].w[k]), make_float2(fi, fi));
        const uint2 q = make_uint2(pack4(p[0].x, p[0].y, p[1].x, p[1].y), pack4(p[2].x, p[2].y, p[3].x, p[3].y));
        unsigned char* to = a.q + (long long)(r0 + i) * a.qs + c;
        if (left >= 8) {
            *reinterpret_cast<uint2*>(to) = q;
        } else {
            for (int k = 0; k < left; ++k) to[k] = (unsigned char)((k < 4 ? q.x : q.y) >> (8 * (k & 3)));
        }
    }
}

// Four adjacent elements as they are stored.
template <typename T>
struct Four {
    using Raw = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
    Raw raw;
    __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ void load_some(const T* p, int n) {
        raw = Raw{};
        T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) e[k] = p[k];
    }
    __device__ __forceinline__ float4 get() const {
        if constexpr (sizeof(T) == 4) {
            return raw;
        } else {
            const float2 a = pair<T>(raw.x), b = pair<T>(raw.y);
            return make_float4(a.x, a.y, b.x, b.y);
        }
    }
};

// A 128 x 128 tile: warp w holds rows 16 w .. 16 w + 15, lane l columns 4 l .. 4 l + 3.
// COLUMNS: every column of the tile is a block (of the transpose's row), else the tile is one block.
// TRANSPOSE: the transpose is stored.
template <typename T, bool COLUMNS, bool TRANSPOSE>
__global__ void __launch_bounds__(kThreads) k_quant_tile(const QuantArgs a, int col_tiles) {
    constexpr int R = 16;
    __shared__ __align__(16) float red[kThreads / 32][kBlock];
    __shared__ __align__(16) unsigned char turned[TRANSPOSE ? kBlock * kBlock : 16];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rt = blockIdx.x / col_tiles, ct = blockIdx.x % col_tiles;
    const int r0 = rt * kBlock + warp * R, c = ct * kBlock + lane * 4;
    const int left = a.cols - c;
    const T* x = static_cast<const T*>(a.x) + (long long)r0 * a.xs + c;
    Four<T> v[R];
    if (a.vec && (ct + 1) * kBlock <= a.cols && (rt + 1) * kBlock <= a.rows) {  // all loads at once
#pragma unroll
        for (int i = 0; i < R; ++i) v[i].load(x + i * a.xs);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) v[i].load_some(x + i * a.xs, r0 + i < a.rows ? left : 0);
    }
    float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float4 t = v[i].get();
        m.x = max_nan(m.x, fabsf(t.x));
        m.y = max_nan(m.y, fabsf(t.y));
        m.z = max_nan(m.z, fabsf(t.z));
        m.w = max_nan(m.w, fabsf(t.w));
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
        // (piece w of column c stands at w ^ (c / 4 mod 8): 8 lanes then meet no bank twice, here and below)
        uint32_t q[4][4];  // [column][word]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = v[4 * i + k].get();
            q[0][i] = pack4(__fmul_rn(t[0].x, f.x), __fmul_rn(t[1].x, f.x), __fmul_rn(t[2].x, f.x), __fmul_rn(t[3].x, f.x));
            q[1][i] = pack4(__fmul_rn(t[0].y, f.y), __fmul_rn(t[1].y, f.y), __fmul_rn(t[2].y, f.y), __fmul_rn(t[3].y, f.y));
            q[2][i] = pack4(__fmul_rn(t[0].z, f.z), __fmul_rn(t[1].z, f.z), __fmul_rn(t[2].z, f.z), __fmul_rn(t[3].z, f.z));
            q[3][i] = pack4(__fmul_rn(t[0].w, f.w), __fmul_rn(t[1].w, f.w), __fmul_rn(t[2].w, f.w), __fmul_rn(t[3].w, f.w));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(turned + (lane * 4 + j) * kBlock + (warp ^ (lane & 7)) * 16) = make_uint4(q[j][0], q[j][1], q[j][2], q[j][3]);
        __syncthreads();
        const int width = min(kBlock, a.rows - rt * kBlock);  // bytes of each stored row
        for (int k = threadIdx.x; k < kBlock * (kBlock / 16); k += kThreads) {
            const int row = k >> 3, at = (k & 7) * 16;
            if (ct * kBlock + row >= a.cols || at >= width) continue;
            unsigned char* to = a.q + (long long)(ct * kBlock + row) * a.qs + (long long)rt * kBlock + at;
            const unsigned char* from = turned + row * kBlock + ((k & 7) ^ ((row >> 2) & 7)) * 16;
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
            const float4 t = v[i].get();
            const uint32_t q = pack4(__fmul_rn(t.x, f.x), __fmul_rn(t.y, f.y), __fmul_rn(t.z, f.z), __fmul_rn(t.w, f.w));
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
    if (block_rows == 1 && !transpose && a.vec16) {
        if constexpr (sizeof(T) == 2) {
            const int pairs = (int)((kb + 1) / 2);
            e = launch_dependent(k_quant_rows16<T>, dim3((unsigned)(pairs * ((a.rows + 31LL) / 32))), dim3(kThreads), 0, s, a, pairs);
        } else {
            return -1;
        }
    } else if (block_rows == 1 && !transpose) {
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
