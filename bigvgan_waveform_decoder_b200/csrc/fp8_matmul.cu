// fp8_matmul.cu -- out = a b^T for fp8 (e4m3) matrices with one scale for each block of 128 values
// along K, on the tensor cores.
//
//   out[m, n] = sum_kb sa[m, kb] sb[n, kb] (sum_{k in block kb} a[m, k] b[n, k]) + bias[n]
//
// A 128-byte row of a tile is exactly one block, so every K step of 128 is one scale: four
// tcgen05.mma (kind::f8f6f4, K = 32) into a tensor-memory buffer, which the epilogue warps then add
// into fp32 registers times the step's scales while the tensor core fills the next buffer.  So the
// scaling costs no extra pass, and no accumulator in the tensor core sees more than one block.
//
// Warps: 0 loads tiles by TMA (128-byte swizzle, rows beyond the matrix and the short last block
// filled with zeros), 1 issues the MMAs, 4.. are the epilogue (2 and 3 only fill up the warpgroup,
// since a warp reads the quarter of tensor memory of its number modulo 4).  Persistent: a block takes
// tiles blockIdx.x, + gridDim.x, ...
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "fp8_kernels.cuh"

namespace mh3a {
namespace fp8 {
namespace {

constexpr int kM = 128;  // tile rows (tensor-memory lanes)

struct MatmulParams {
    const float* sa;    // [KB][M]
    const float* sb;    // [KB][NB]
    const float* bias;
    void* out;
    long long os;
    int M, N, KB, NB;
    int mt, tiles;      // row tiles, all tiles
    int vec_out;        // rows of `out` can be written 16 bytes at a time
};

template <int NT>
struct Cfg {
    static constexpr int EW = NT >= 128 ? 8 : 4;          // epilogue warps
    static constexpr int CW = NT / (EW / 4);              // columns of an epilogue warp
    static constexpr int kThreads = 128 + 32 * EW;
    static constexpr int kAcc = NT == 256 ? 2 : 4;        // tensor-memory buffers
    static constexpr int kCols = kAcc * NT < 32 ? 32 : kAcc * NT;
    static constexpr int kStageBytes = (kM + NT) * kBlock;
    static constexpr int kPitch = 144;                    // staging row of 128 bytes, conflict-free
    static constexpr int kStaging = EW * 32 * kPitch;
    static constexpr int kStages = std::min(8, (200 * 1024 - kStaging) / kStageBytes);
    static constexpr int kSmem = kStages * kStageBytes + kStaging + 1024 + 256 + (CW * 4 * 2 * EW);
};

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            ptx::smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(ptx::smem_u32(bar))
        : "memory");
}

// K-major operand of 128-byte rows with the 128-byte swizzle: 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}

// D[tmem] (+)= A B^T, e4m3 operands (kind::f8f6f4), four K steps of 32 bytes: one block of K.
__device__ __forceinline__ void mma_block_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t.reg .b32 r;\n\t.reg .b64 a1, b1;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, 0, 0;\n\t"
        "setp.eq.b32 q, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 b1, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t"
        "add.s64 a1, %1, 4;\n\tadd.s64 b1, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t"
        "add.s64 a1, %1, 6;\n\tadd.s64 b1, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc)
        : "memory");
}

// 32 lanes x 32 bits, W consecutive columns; the values are there after tmem_wait().
template <int W>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[W]);
template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_ld<32>(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Writes a warp's 32 x CW results: 128 bytes of each row at a time go through shared memory, so that
// global memory gets whole lines.
template <typename O, int CW>
__device__ __forceinline__ void write_out(const MatmulParams& p, const float2 (&acc)[CW / 2], unsigned char* stage, int m0, int n0) {
    constexpr int kPitch = 144;
    constexpr int kStep = 128 / sizeof(O) < CW ? 128 / sizeof(O) : CW;  // columns at a time
    constexpr int kVecs = kStep * sizeof(O) / 16;                       // 16-byte pieces of a row
    const int lane = threadIdx.x & 31;
    O* out = static_cast<O*>(p.out);
#pragma unroll
    for (int c0 = 0; c0 < CW; c0 += kStep) {
        unsigned char* to = stage + lane * kPitch;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            constexpr int kPer = 16 / sizeof(O);
            float f[kPer];
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                const int c = c0 + v * kPer + i;
                f[i] = acc[c / 2].x;
                f[i + 1] = acc[c / 2].y;
                if (p.bias) {
                    f[i] += n0 + c < p.N ? __ldg(p.bias + n0 + c) : 0.f;
                    f[i + 1] += n0 + c + 1 < p.N ? __ldg(p.bias + n0 + c + 1) : 0.f;
                }
            }
            uint4 q;
            if constexpr (sizeof(O) == 4) {
                q = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
            } else {
                uint32_t* w = &q.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (std::is_same<O, __half>::value) {
                        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                }
            }
            *reinterpret_cast<uint4*>(to + v * 16) = q;
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int at = k * 32 + lane, row = at / kVecs, v = at % kVecs;
            const int n = n0 + c0 + v * (int)(16 / sizeof(O)), left = p.N - n;
            if (m0 + row < p.M && left > 0) {
                const unsigned char* from = stage + row * kPitch + v * 16;
                O* dst = out + (long long)(m0 + row) * p.os + n;
                if (p.vec_out && left >= (int)(16 / sizeof(O))) {
                    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(from);
                } else {
                    for (int i = 0; i < min(left, (int)(16 / sizeof(O))); ++i) dst[i] = reinterpret_cast<const O*>(from)[i];
                }
            }
        }
        __syncwarp();
    }
}

// WIDE: b's blocks span 128 rows (one scale for a warp's columns), else every column has its own.
template <typename O, int NT, bool WIDE>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 1)
k_fp8_matmul(const MatmulParams p, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b) {
    using C = Cfg<NT>;
    extern __shared__ unsigned char raw[];
    unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char* staging = tiles + C::kStages * C::kStageBytes;
    float* cols = reinterpret_cast<float*>(staging + C::kStaging);  // [EW][2][CW]: column scales
    uint64_t* full = reinterpret_cast<uint64_t*>(cols + C::EW * 2 * C::CW);
    uint64_t* empty = full + C::kStages;
    uint64_t* done = empty + C::kStages;  // accumulator buffer filled
    uint64_t* freed = done + C::kAcc;     // and read again
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(freed + C::kAcc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < C::kAcc; ++i) {
            ptx::mbar_init(done + i, 1);
            ptx::mbar_init(freed + i, C::EW);
        }
        ptx::fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_a) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_b) : "memory");
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, C::kCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
                const int m0 = (t % p.mt) * kM, n0 = (t / p.mt) * NT;
                for (int kb = 0; kb < p.KB; ++kb, ++it) {
                    const int s = it % C::kStages;
                    if (it >= C::kStages) ok = ptx::mbar_wait(empty + s, ((it / C::kStages) & 1) ^ 1);
                    if (!ok) break;
                    unsigned char* to = tiles + s * C::kStageBytes;
                    ptx::mbar_arrive_expect_tx(full + s, C::kStageBytes);
                    tma_load_2d(to, &map_a, kb * kBlock, m0, full + s);
                    tma_load_2d(to + kM * kBlock, &map_b, kb * kBlock, n0, full + s);
                }
            }
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);  // e4m3, fp32 sums
        int it = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
            for (int kb = 0; kb < p.KB; ++kb, ++it) {
                const int s = it % C::kStages, b = it % C::kAcc;
                if (it >= C::kAcc) ok = ptx::mbar_wait(freed + b, ((it / C::kAcc) & 1) ^ 1);
                ok = ok && ptx::mbar_wait(full + s, (it / C::kStages) & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t at = ptx::smem_u32(tiles + s * C::kStageBytes);
                mma_block_elect(tmem + b * NT, desc_sw128(at), desc_sw128(at + kM * kBlock), idesc);
                ptx::mma_commit_elect(empty + s);
                ptx::mma_commit_elect(done + b);
            }
        }
    } else if (warp >= 4) {
        const int e = warp - 4, quarter = warp & 3, half = e >> 2;
        const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + half * C::CW;
        float* my_cols = cols + e * 2 * C::CW;
        int it = 0;
        for (int t = blockIdx.x; t < p.tiles; t += gridDim.x) {
            const int m0 = (t % p.mt) * kM + quarter * 32, n0 = (t / p.mt) * NT + half * C::CW;
            const int row = min(m0 + lane, p.M - 1);
            float2 acc[C::CW / 2];
#pragma unroll
            for (int i = 0; i < C::CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            // the scales of step 0; those of the next step are loaded while a step is added up
            const int nb = min(n0, p.N - 1) / kBlock;
            constexpr int kPer = (C::CW + 31) / 32;  // column scales a lane fetches
            float sa = __ldg(p.sa + row), sb = 0.f, sc[kPer];
            auto fetch_cols = [&](int kb) {
                if constexpr (WIDE) {
                    sb = __ldg(p.sb + (long long)kb * p.NB + nb);
                } else {
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const int c = i * 32 + lane;
                        sc[i] = __ldg(p.sb + (long long)kb * p.NB + min(n0 + c, p.N - 1));
                    }
                }
            };
            fetch_cols(0);
            bool ok = true;
            for (int kb = 0; kb < p.KB; ++kb, ++it) {
                const int b = it % C::kAcc;
                float* now = my_cols + (kb & 1) * C::CW;
                const float s1 = WIDE ? sa * sb : sa;
                if constexpr (!WIDE) {
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        if (i * 32 + lane < C::CW) now[i * 32 + lane] = sc[i];
                    __syncwarp();
                }
                if (kb + 1 < p.KB) {
                    sa = __ldg(p.sa + (long long)(kb + 1) * p.M + row);
                    fetch_cols(kb + 1);
                }
                ok = ok && ptx::mbar_wait(done + b, (it / C::kAcc) & 1);
                ptx::tc_fence_after();
                const float2 s2 = make_float2(s1, s1);
                constexpr int kLd = C::CW >= 32 ? 32 : 16;
#pragma unroll
                for (int c = 0; c < C::CW; c += kLd) {
                    uint32_t v[kLd];
                    tmem_ld<kLd>(mine + b * NT + c, v);
                    tmem_wait();
                    if (c + kLd == C::CW) {  // the buffer is read: the tensor core may fill it again
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(freed + b);
                    }
#pragma unroll
                    for (int i = 0; i < kLd / 2; ++i) {
                        float2 f = make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                        if constexpr (!WIDE) f = __fmul2_rn(f, *reinterpret_cast<const float2*>(now + c + 2 * i));
                        acc[c / 2 + i] = __ffma2_rn(f, s2, acc[c / 2 + i]);
                    }
                }
            }
            if (!ok) {  // never expected: a wait ran out of time; NaN rather than a partial sum
#pragma unroll
                for (int i = 0; i < C::CW / 2; ++i) acc[i] = make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
            }
            write_out<O, C::CW>(p, acc, staging + e * 32 * C::kPitch, m0, n0);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::kCols);
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) != cudaSuccess ||
            st != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// [rows, cols] bytes, boxes of 128 bytes x box_rows.
bool make_map(CUtensorMap* map, const void* base, int rows, int cols, long long stride, int box_rows) {
    const EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {kBlock, (cuuint32_t)box_rows};
    const cuuint32_t one[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename O, int NT, bool WIDE>
int launch(const MatmulArgs& m, cudaStream_t s) {
    using C = Cfg<NT>;
    static_assert(C::kSmem <= 227 * 1024 && C::kStages >= 2, "shared memory");
    MatmulParams p{};
    p.sa = m.sa;
    p.sb = m.sb;
    p.bias = m.bias;
    p.out = m.out;
    p.os = m.os;
    p.M = m.M;
    p.N = m.N;
    p.KB = (m.K + kBlock - 1) / kBlock;
    p.NB = (int)((m.N + (long long)m.b_block_rows - 1) / m.b_block_rows);
    p.mt = (m.M + kM - 1) / kM;
    p.tiles = p.mt * ((m.N + NT - 1) / NT);
    p.vec_out = aligned(m.out, 16) && m.os * sizeof(O) % 16 == 0;
    CUtensorMap ma, mb;
    if (!make_map(&ma, m.a, m.M, m.K, m.as, kM) || !make_map(&mb, m.b, m.N, m.K, m.bs, NT)) return -1;
    auto kern = k_fp8_matmul<O, NT, WIDE>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return -1;
    const int grid = std::min(p.tiles, kSms);
    return launch_dependent(kern, dim3(grid), dim3(C::kThreads), C::kSmem, s, p, ma, mb) == cudaSuccess ? 1 : -1;
}

template <typename O, bool WIDE>
int launch_nt(const MatmulArgs& m, cudaStream_t s) {
    // The widest tile that still gives every SM one; narrower ones read the operands more often.
    const long long mt = (m.M + kM - 1LL) / kM;
    auto tiles = [&](int nt) { return mt * ((m.N + nt - 1LL) / nt); };
    if (tiles(256) >= kSms) return launch<O, 256, WIDE>(m, s);
    if (tiles(128) >= kSms) return launch<O, 128, WIDE>(m, s);
    if (tiles(64) >= kSms / 2) return launch<O, 64, WIDE>(m, s);
    if (tiles(32) >= kSms / 2) return launch<O, 32, WIDE>(m, s);
    return launch<O, 16, WIDE>(m, s);
}

template <typename O>
int launch_wide(const MatmulArgs& m, cudaStream_t s) {
    return m.b_block_rows == kBlock ? launch_nt<O, true>(m, s) : launch_nt<O, false>(m, s);
}

}  // namespace

int launch_matmul(const MatmulArgs& m, cudaStream_t s) {
    switch (m.out_dtype) {
        case MH3A_DTYPE_F32: return launch_wide<float>(m, s);
        case MH3A_DTYPE_F16: return launch_wide<__half>(m, s);
        default: return launch_wide<__nv_bfloat16>(m, s);
    }
}

}  // namespace fp8
}  // namespace mh3a
