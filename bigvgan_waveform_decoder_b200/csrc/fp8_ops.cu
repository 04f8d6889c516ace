// fp8_ops.cu -- entry points of the fp8 operators, and the linear layer of a few rows.
//
// Few rows (a decode frame by frame): the product is bound by reading the weights once, 1 byte each,
// so it runs on the CUDA cores: a warp takes two weight rows, a lane 16 bytes of each at a time, the next
// 2048 columns on their way while the present ones are multiplied; the
// rows of x are quantised by every block for itself (from L2) instead of by a launch of its own.
#include "fp8_kernels.cuh"

namespace mh3a {
namespace fp8 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSlab = 2048;  // K values of x held at a time
constexpr int kLane = 16;    // K values of a lane and step
constexpr int kSteps = kSlab / (32 * kLane);

// 16 e4m3 values -> floats
__device__ __forceinline__ void unpack16(uint4 q, float (&f)[16]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * h)), __NV_E4M3);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r));
            f[4 * i + 2 * h] = v.x;
            f[4 * i + 2 * h + 1] = v.y;
        }
    }
}

// MR rows of x, two rows of w for each warp.  xs: the slab's quantised values, [row][step][quarter][lane] of
// float4, so that a warp reads 512 consecutive bytes; ss: the scales of their blocks of 128 (8 lanes).  A lane's 16
// products stand for themselves times two scales, the smaller of which is multiplied first: so nothing in between
// leaves the range of fp32 that the result does not leave (x of 1e36 with weights of 1, say).
template <typename T, typename O, int MR>
__global__ void __launch_bounds__(kThreads) k_fp8_few_rows(const FewRowsArgs a, int x_vec) {
    constexpr int RW = 2;
    __shared__ float4 xs[MR][kSteps][4][32];
    __shared__ float ss[MR][kSteps][4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = (blockIdx.x * kWarps + warp) * RW;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    float acc[RW][MR];
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int m = 0; m < MR; ++m) acc[r][m] = 0.f;
    const int NB = (a.N + a.w_block_rows - 1) / a.w_block_rows;
    // a lane's 16 bytes of each row and step, from slab k0
    auto fetch = [&](uint4(&w)[RW][kSteps], int k0) {
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int t = 0; t < kSteps; ++t) {
                const int k = k0 + (t * 32 + lane) * kLane, n = n0 + r;
                w[r][t] = make_uint4(0, 0, 0, 0);
                if (n < a.N && k < a.K) {
                    const unsigned char* from = a.w + (long long)n * a.ws + k;
                    if (k + kLane <= a.K) {
                        w[r][t] = __ldcs(reinterpret_cast<const uint4*>(from));
                    } else {
                        uint32_t q[4] = {0, 0, 0, 0};
                        for (int i = 0; i < a.K - k; ++i) q[i >> 2] |= (uint32_t)from[i] << (8 * (i & 3));
                        w[r][t] = make_uint4(q[0], q[1], q[2], q[3]);
                    }
                }
            }
    };
    uint4 next[RW][kSteps];
    fetch(next, 0);
    for (int k0 = 0; k0 < a.K; k0 += kSlab) {
        uint4 w[RW][kSteps];
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int t = 0; t < kSteps; ++t) w[r][t] = next[r][t];
        if (k0) __syncthreads();
        // 16 values a lane, 8 lanes a block of 128
        for (int j = warp; j < MR * kSteps; j += kWarps) {
            const int m = j / kSteps, t = j % kSteps, k = k0 + (t * 32 + lane) * kLane;
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int left = m < a.M ? a.K - (k + 4 * i) : 0;
                v[i] = left > 0 ? load4<T>(static_cast<const T*>(a.x) + m * a.xs + k + 4 * i, x_vec && left >= 4, left)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float top = max_nan(max_nan(amax4(v[0]), amax4(v[1])), max_nan(amax4(v[2]), amax4(v[3])));
#pragma unroll
            for (int off = 4; off; off >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float b = max_nan(top, kTiny), s = __fdiv_rn(b, kMax), f = __fdiv_rn(kMax, b);
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = pack4(__fmul_rn(v[i].x, f), __fmul_rn(v[i].y, f), __fmul_rn(v[i].z, f), __fmul_rn(v[i].w, f));
            float u[16];
            unpack16(make_uint4(q[0], q[1], q[2], q[3]), u);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                xs[m][t][i][lane] = make_float4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
            if (lane % 8 == 0) ss[m][t][lane / 8] = s;
        }
        __syncthreads();
        if (k0 + kSlab < a.K) fetch(next, k0 + kSlab);  // on their way while this slab is added up
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            const int k = k0 + (t * 32 + lane) * kLane;
            if (k >= a.K) break;
            float s[RW], f[RW][16];
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                s[r] = __ldg(a.sw + (long long)(k / kBlock) * NB + min(n0 + r, a.N - 1) / a.w_block_rows);
                unpack16(w[r][t], f[r]);
            }
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                float d[RW];
#pragma unroll
                for (int r = 0; r < RW; ++r) d[r] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 v = xs[m][t][i][lane];
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        d[r] = fmaf(v.x, f[r][4 * i], d[r]);
                        d[r] = fmaf(v.y, f[r][4 * i + 1], d[r]);
                        d[r] = fmaf(v.z, f[r][4 * i + 2], d[r]);
                        d[r] = fmaf(v.w, f[r][4 * i + 3], d[r]);
                    }
                }
                const float sx = ss[m][t][lane / 8];
#pragma unroll
                for (int r = 0; r < RW; ++r) acc[r][m] = fmaf(d[r] * fminf(sx, s[r]), max_nan(sx, s[r]), acc[r][m]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int m = 0; m < MR; ++m) {
#pragma unroll
            for (int off = 16; off; off >>= 1) acc[r][m] += __shfl_xor_sync(0xffffffffu, acc[r][m], off);
        }
    if (lane < RW && n0 + lane < a.N) {
        const float b = a.bias ? __ldg(a.bias + n0 + lane) : 0.f;
#pragma unroll
        for (int m = 0; m < MR; ++m)
            if (m < a.M) static_cast<O*>(a.y)[m * a.ys + n0 + lane] = (O)((lane ? acc[1][m] : acc[0][m]) + b);
    }
}

template <typename T, int MR>
int few(const FewRowsArgs& a, cudaStream_t s) {
    const int x_vec = aligned(a.x, 4 * sizeof(T)) && a.xs % 4 == 0;
    const unsigned grid = (unsigned)((a.N + 2LL * kWarps - 1) / (2 * kWarps));
    return launch_dependent(k_fp8_few_rows<T, T, MR>, dim3(grid), dim3(kThreads), 0, s, a, x_vec) == cudaSuccess ? 1 : -1;
}

template <typename T>
int few(const FewRowsArgs& a, cudaStream_t s) {
    return a.M == 1 ? few<T, 1>(a, s) : a.M == 2 ? few<T, 2>(a, s) : few<T, 4>(a, s);
}

constexpr int kMostSize = 1 << 30;

bool size_ok(int n) { return n >= 1 && n <= kMostSize; }
bool dtype_ok(int d) { return d >= MH3A_DTYPE_F32 && d <= MH3A_DTYPE_BF16; }
size_t elem(int d) { return d == MH3A_DTYPE_F32 ? 4 : 2; }
bool stored_ok(const void* q, long long stride, int cols) {
    return q && aligned(q, 16) && stride >= cols && stride % 16 == 0 && stride < (1LL << 40);
}
long long blocks(int n) { return (n + (long long)kBlock - 1) / kBlock; }

// Whether a layer takes the kernel for few rows; its multiplications are the CUDA cores', so the tensor
// cores overtake it where there are many.  Measured, us, this kernel against quantisation and product
// (columns x K): 1 row 2048 x 2048 3.3 / 6.3, 4096 x 4096 6.7 / 9.7, 8192 x 8192 25.7 / 16.7; 2 rows 4096 x 4096
// 8.0 / 9.8; 3 rows 4096 x 4096 11.3 / 9.8; 4 rows 2048 x 2048 4.9 / 6.6.
bool few_rows(int M, int N, int K) { return M <= MH3A_FP8_FEW_ROWS && (long long)M * N * K <= 40LL << 20; }

// Layout of mh3a_fp8_linear's scratch: x quantised, then its scales.
long long q_stride(int K) { return (K + 15LL) / 16 * 16; }
size_t q_bytes(int M, int K) { return ((size_t)M * q_stride(K) + 255) / 256 * 256; }

mh3a_status check_product(const void* a, const float* sa, const void* b, long long bs, const float* sb, int b_block_rows,
                          int M, int N, int K, const float* bias, int out_dtype, const void* out, long long os) {
    if (!a || !sa || !b || !sb || !out || !dtype_ok(out_dtype)) return MH3A_ERR_INVALID_ARG;
    if (b_block_rows != 1 && b_block_rows != kBlock) return MH3A_ERR_INVALID_ARG;
    if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return MH3A_ERR_SHAPE;
    if (!stored_ok(b, bs, K) || !aligned(sb, 4) || !aligned(sa, 4) || !aligned(bias, 4)) return MH3A_ERR_INVALID_ARG;
    if (os < N || !aligned(out, elem(out_dtype))) return MH3A_ERR_INVALID_ARG;
    if (blocks(M) * ((N + 15LL) / 16) > kMostSize) return MH3A_ERR_SHAPE;
    return MH3A_OK;
}

}  // namespace

int launch_few_rows(const FewRowsArgs& a, int dtype, cudaStream_t s) {
    switch (dtype) {
        case MH3A_DTYPE_F32: return few<float>(a, s);
        case MH3A_DTYPE_F16: return few<__half>(a, s);
        default: return few<__nv_bfloat16>(a, s);
    }
}

}  // namespace fp8
}  // namespace mh3a

using namespace mh3a;
using namespace mh3a::fp8;

extern "C" MH3A_API mh3a_status mh3a_fp8_quantize(const void* x, int dtype, int rows, int cols, long long x_stride,
                                                  int block_rows, int transpose, void* q, long long qs, float* scale,
                                                  void* stream) {
    if (!x || !scale || !dtype_ok(dtype) || x_stride < 0) return MH3A_ERR_INVALID_ARG;
    if ((block_rows != 1 && block_rows != kBlock) || (transpose != 0 && transpose != 1)) return MH3A_ERR_INVALID_ARG;
    if (!size_ok(rows) || !size_ok(cols)) return MH3A_ERR_SHAPE;
    if (!aligned(x, elem(dtype)) || !aligned(scale, 4) || !stored_ok(q, qs, transpose ? rows : cols)) return MH3A_ERR_INVALID_ARG;
    const long long grid = block_rows == 1 && !transpose ? blocks(cols) * ((rows + 31LL) / 32) : blocks(cols) * blocks(rows);
    if (grid > kMostSize) return MH3A_ERR_SHAPE;
    QuantArgs a{x, x_stride, static_cast<unsigned char*>(q), qs, scale, rows, cols, 0, 0};
    a.vec = aligned(x, 4 * elem(dtype)) && x_stride % 4 == 0;
    a.vec16 = elem(dtype) == 2 && aligned(x, 16) && x_stride % 8 == 0;
    return launch_quantize(a, dtype, block_rows, transpose, static_cast<cudaStream_t>(stream)) < 0 ? launch_failed("mh3a_fp8_quantize")
                                                                                                   : MH3A_OK;
}

extern "C" MH3A_API mh3a_status mh3a_fp8_matmul(const void* a, long long a_stride, const float* a_scale, const void* b,
                                                long long b_stride, const float* b_scale, int b_block_rows, int M, int N,
                                                int K, const float* bias, int out_dtype, void* out, long long out_stride,
                                                void* stream) {
    const mh3a_status st = check_product(a, a_scale, b, b_stride, b_scale, b_block_rows, M, N, K, bias, out_dtype, out, out_stride);
    if (st != MH3A_OK) return st;
    if (!stored_ok(a, a_stride, K)) return MH3A_ERR_INVALID_ARG;
    const MatmulArgs m{a, a_stride, a_scale, b, b_stride, b_scale, b_block_rows, M, N, K, bias, out, out_stride, out_dtype};
    return launch_matmul(m, static_cast<cudaStream_t>(stream)) < 0 ? launch_failed("mh3a_fp8_matmul") : MH3A_OK;
}

extern "C" MH3A_API size_t mh3a_fp8_linear_workspace(int M, int N, int K) {
    if (!size_ok(M) || !size_ok(N) || !size_ok(K) || few_rows(M, N, K)) return 0;
    return q_bytes(M, K) + (size_t)blocks(K) * M * 4;
}

extern "C" MH3A_API mh3a_status mh3a_fp8_linear(const void* x, int dtype, long long x_stride, const void* w,
                                                long long w_stride, const float* w_scale, int w_block_rows, int M, int N,
                                                int K, const float* bias, void* y, long long y_stride, void* workspace,
                                                size_t workspace_bytes, void* stream) {
    const mh3a_status st = check_product(x, w_scale, w, w_stride, w_scale, w_block_rows, M, N, K, bias, dtype, y, y_stride);
    if (st != MH3A_OK) return st;
    if (x_stride < 0 || !aligned(x, elem(dtype))) return MH3A_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (few_rows(M, N, K)) {
        const FewRowsArgs f{x, x_stride, static_cast<const unsigned char*>(w), w_stride, w_scale, w_block_rows, M, N, K, bias, y, y_stride};
        return launch_few_rows(f, dtype, s) < 0 ? launch_failed("mh3a_fp8_linear") : MH3A_OK;
    }
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < mh3a_fp8_linear_workspace(M, N, K)) return MH3A_ERR_INVALID_ARG;
    unsigned char* q = static_cast<unsigned char*>(workspace);
    float* scale = reinterpret_cast<float*>(q + q_bytes(M, K));
    const mh3a_status sq = mh3a_fp8_quantize(x, dtype, M, K, x_stride, 1, 0, q, q_stride(K), scale, stream);
    if (sq != MH3A_OK) return sq;
    return mh3a_fp8_matmul(q, q_stride(K), scale, w, w_stride, w_scale, w_block_rows, M, N, K, bias, dtype, y, y_stride, stream);
}
