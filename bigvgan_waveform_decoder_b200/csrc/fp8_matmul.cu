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
// filled with zeros), 1 issues the MMAs, 2 copies column scales to shared memory a few steps ahead
// where every column has its own, 4.. are the epilogue (3 only fills up the warpgroup, since a warp
// reads the quarter of tensor memory of its number modulo 4).  The other scales are fetched into
// registers steps ahead: a load that a step waits for costs more than the step.  Persistent: a
// block takes tiles blockIdx.x, + gridDim.x, ...
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "fp8_kernels.cuh"

namespace mh3a {
namespace fp8 {
namespace {

constexpr int kM = 128;     // tile rows (tensor-memory lanes)
constexpr int kPitch = 80;  // staging row of 64 bytes: 16-byte accesses of 8 rows meet no bank twice

struct MatmulParams {
    const float* sa;    // [KB][M]
    const float* sb;    // [KB][NB]
    const float* bias;
    void* out;
    long long os;
    int M, N, KB, NB;
    int mt, tiles;      // row tiles, all tiles
    int vec_out;        // rows of `out` can be written 16 bytes at a time
    int step_bytes;     // what the two copies of a step bring
};

template <int NT>
struct Cfg {
    static constexpr int EW = NT >= 128 ? 8 : 4;          // epilogue warps
    static constexpr int CW = NT / (EW / 4);              // columns of an epilogue warp
    static constexpr int kThreads = 128 + 32 * EW;
    // Steps of K between two handshakes of the tensor core and the epilogue, each with columns of its own:
    // a wait costs as much as adding up a narrow tile.
    static constexpr int kStep = NT == 256 ? 1 : NT == 128 ? 2 : 4;
    static constexpr int kAcc = std::min(4, 512 / (kStep * NT));  // tensor-memory buffers
    static constexpr int kCols = kAcc * kStep * NT;
    static constexpr int kAhead = kStep == 1 ? 3 : 2 * kStep;  // steps that scales are fetched ahead
    static constexpr int kScaleSlots = kStep == 1 ? 4 : 2 * kStep;
    // Steps of K in one stage of shared memory: their copies are announced, waited for and given back
    // together, since each of these costs the issuing warp 60 to 150 cycles.
    static constexpr int kPer = NT == 256 ? 1 : 2;
    static constexpr int kStepBytes = (kM + NT) * kBlock;
    static constexpr int kStageBytes = kPer * kStepBytes;
    static constexpr int kStaging = EW * 32 * kPitch;
    static constexpr int kOther = kStaging + kScaleSlots * NT * 4 + 1024 + 512;
    static constexpr int kStages = std::min(8, (227 * 1024 - kOther) / kStageBytes);
    static constexpr int kSmem = kStages * kStageBytes + kOther;
    // 128 columns of sums and two buffers of 32 do not fit an even share of the registers.  (With column scales
    // the compiler spills a few values from 64 columns on: 48 to 92 bytes a thread with tiles of 64 and 128
    // columns, 4 with 256.)
    static constexpr bool kSplitRegs = CW == 128;
};

// Whether a barrier's phase has completed, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(ptx::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok;
}

// The thread's earlier cp.async copies count as one arrival on the barrier once they are done.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}

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

// 32 lanes x 32 bits, 16 consecutive columns; the values are there after tmem_wait().
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// Waits for every load before it; the values pass through, so that no use of them moves ahead.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
template <int W>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[W / 16][16]) {
#pragma unroll
    for (int i = 0; i < W / 16; ++i) tmem_ld(addr + 16 * i, r[i]);
}
template <int W>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[W / 16][16]) {
#pragma unroll
    for (int i = 0; i < W / 16; ++i) tmem_wait(r[i]);  // the second finds nothing left to wait for
}

// 16 lanes x 256 bits, W consecutive columns of 8: lane t gets, for columns 8 i + 2 (t % 4) + {0, 1}, row
// t / 4 in r[4 i], r[4 i + 1] and row t / 4 + 8 in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void tmem_ld_frag(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

// Two neighbouring results as they are stored.
template <typename O>
struct Out2 {
    using Raw = typename std::conditional<sizeof(O) == 4, uint2, uint32_t>::type;
    static __device__ __forceinline__ Raw pack(float2 f) {
        if constexpr (sizeof(O) == 4) {
            return make_uint2(__float_as_uint(f.x), __float_as_uint(f.y));
        } else if constexpr (std::is_same<O, __half>::value) {
            const __half2 h = __floats2half2_rn(f.x, f.y);
            return *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
            return *reinterpret_cast<const uint32_t*>(&h);
        }
    }
};

// Writes a warp's 32 x CW results: 64 bytes of each row at a time go through shared memory, so that
// global memory gets whole sectors.
// FRAG: the sums lie as tmem_ld_frag leaves them, acc[4 i + r / 8] for row t / 4 + r; else acc[c / 2] of row t.
template <typename O, int CW, bool FRAG>
__device__ __forceinline__ void write_out(const MatmulParams& p, const float2 (&acc)[CW / 2], unsigned char* stage, int m0, int n0) {
    constexpr int kStep = 64 / sizeof(O) < CW ? 64 / sizeof(O) : CW;  // columns at a time
    constexpr int kVecs = kStep * sizeof(O) / 16;                     // 16-byte pieces of a row
    using Raw = typename Out2<O>::Raw;
    const int lane = threadIdx.x & 31;
    O* out = static_cast<O*>(p.out);
#pragma unroll
    for (int c0 = 0; c0 < CW; c0 += kStep) {
        if constexpr (FRAG) {
            unsigned char* to = stage + (lane >> 2) * kPitch + (lane & 3) * sizeof(Raw);
#pragma unroll
            for (int i = 0; i < kStep / 8; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<Raw*>(to + r * 8 * kPitch + i * 4 * sizeof(Raw)) = Out2<O>::pack(acc[(c0 / 8 + i) * 4 + r]);
        } else {
            unsigned char* to = stage + lane * kPitch;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                Raw q[16 / sizeof(Raw)];
#pragma unroll
                for (int i = 0; i < (int)(16 / sizeof(Raw)); ++i) q[i] = Out2<O>::pack(acc[c0 / 2 + v * (16 / sizeof(Raw)) + i]);
                *reinterpret_cast<uint4*>(to + v * 16) = *reinterpret_cast<const uint4*>(q);
            }
        }
        __syncwarp();
        if (p.vec_out && n0 + c0 + kStep <= p.N) {
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const int at = k * 32 + lane, row = at / kVecs, v = at % kVecs;
                if (m0 + row < p.M)
                    *reinterpret_cast<uint4*>(out + (long long)(m0 + row) * p.os + n0 + c0 + v * (int)(16 / sizeof(O))) =
                        *reinterpret_cast<const uint4*>(stage + row * kPitch + v * 16);
            }
        } else {  // rows that do not start on 16 bytes, the matrix's edge: neighbouring lanes, neighbouring elements
            const int col = lane % kStep;
#pragma unroll 4
            for (int row = lane / kStep; row < 32; row += 32 / kStep)
                if (m0 + row < p.M && n0 + c0 + col < p.N)
                    out[(long long)(m0 + row) * p.os + n0 + c0 + col] = reinterpret_cast<const O*>(stage + row * kPitch)[col];
        }
        __syncwarp();
    }
}

// WIDE: b's blocks span 128 rows (one scale for a warp's columns), else every column has its own.
template <typename O, int NT, bool WIDE>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 1)
k_fp8_matmul(const MatmulParams p, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b) {
    using C = Cfg<NT>;
    constexpr int kStep = C::kStep, kPer = C::kPer, kAhead = C::kAhead, kScaleSlots = C::kScaleSlots;
    extern __shared__ unsigned char raw[];
    unsigned char* tiles = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    unsigned char* staging = tiles + C::kStages * C::kStageBytes;
    float* scales = reinterpret_cast<float*>(staging + C::kStaging);  // [slot][NT]: column scales
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + kScaleSlots * NT);
    uint64_t* empty = full + C::kStages;
    uint64_t* done = empty + C::kStages;  // accumulator buffer filled
    uint64_t* freed = done + C::kAcc;     // and read again
    uint64_t* sfull = freed + C::kAcc;    // scales of a step are there
    uint64_t* sempty = sfull + kScaleSlots;
    uint64_t* drain = sempty + kScaleSlots;  // the last MMAs
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < C::kAcc; ++i) {
            ptx::mbar_init(done + i, WIDE ? 1 : 2);  // the MMAs; and the step's column scales
            ptx::mbar_init(freed + i, C::EW);
        }
        ptx::mbar_init(drain, 1);
        for (int i = 0; i < kScaleSlots; ++i) {
            ptx::mbar_init(sfull + i, 32);
            ptx::mbar_init(sempty + i, C::EW);
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

    // Split registers: 128 x 80 + 256 x 208 of the 384 x 168 at launch.
    if (warp < 4) {
        if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 0 && lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
                const int m0 = (t % p.mt) * kM, n0 = (t / p.mt) * NT;
                for (int kb = 0; kb < p.KB; kb += kPer, ++it) {
                    const int s = it % C::kStages;
                    if (it >= C::kStages) ok = ptx::mbar_wait(empty + s, ((it / C::kStages) & 1) ^ 1);
                    if (!ok) break;
                    unsigned char* to = tiles + s * C::kStageBytes;
                    const int steps = kPer == 1 ? 1 : min(kPer, p.KB - kb);
                    ptx::mbar_arrive_expect_tx(full + s, steps * p.step_bytes);
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        if (j < steps) {
                            tma_load_2d(to + j * C::kStepBytes, &map_a, (kb + j) * kBlock, m0, full + s);
                            tma_load_2d(to + j * C::kStepBytes + kM * kBlock, &map_b, (kb + j) * kBlock, n0, full + s);
                        }
                    }
                }
            }
            // the block's shared memory outlives the copies on their way, also where another warp gave up
            for (int j = max(0, it - C::kStages); j < it; ++j) ptx::mbar_wait(full + j % C::kStages, (j / C::kStages) & 1);
        } else if (warp == 1) {
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);  // e4m3, fp32 sums
            int it = 0, round = 0, column = 0;  // stages, handshakes, steps with column scales
            bool ok = true, there = false;  // there: the next stage's copies are known to have arrived
            for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
                for (int k0 = 0; k0 < p.KB && ok; k0 += kStep, ++round) {
                    const int b = round % C::kAcc, steps = kStep == 1 ? 1 : min(kStep, p.KB - k0);
                    if (round >= C::kAcc) ok = warp_wait(freed + b, ((round / C::kAcc) & 1) ^ 1);
#pragma unroll
                    for (int j = 0; j < kStep; j += kPer) {
                        if (j >= steps || !ok) break;
                        const int s = it % C::kStages;
                        if (!there) ok = warp_wait(full + s, (it / C::kStages) & 1);
                        if (!ok) break;
                        ++it;
                        there = __all_sync(0xffffffffu, mbar_test(full + it % C::kStages, (it / C::kStages) & 1));
                        ptx::tc_fence_after();
                        const uint32_t at = ptx::smem_u32(tiles + s * C::kStageBytes);
#pragma unroll
                        for (int i = 0; i < kPer; ++i) {
                            if (i == 0 || j + i < steps)
                                mma_block_elect(tmem + (b * kStep + j + i) * NT, desc_sw128(at + i * C::kStepBytes),
                                                desc_sw128(at + i * C::kStepBytes + kM * kBlock), idesc);
                        }
                        ptx::mma_commit_elect(empty + s);
                    }
                    if (!ok) break;
                    ptx::mma_commit_elect(done + b);
                    if (!WIDE) {
                        for (int i = 0; i < steps; ++i, ++column)
                            ok = ok && warp_wait(sfull + column % kScaleSlots, (column / kScaleSlots) & 1);
                        if (ok && lane == 0) ptx::mbar_arrive(done + b);
                    }
                }
            }
            // the MMAs on their way end before tensor memory is given back, also where another warp gave up
            ptx::mma_commit_elect(drain);
            warp_wait(drain, 0);
        } else if (warp == 2 && !WIDE) {
            int it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
                const int n0 = (t / p.mt) * NT;
                for (int kb = 0; kb < p.KB; ++kb, ++it) {
                    const int s = it % kScaleSlots;
                    if (it >= kScaleSlots) ok = warp_wait(sempty + s, ((it / kScaleSlots) & 1) ^ 1);
                    if (!ok) break;
                    float* to = scales + s * NT;
                    const float* sb = p.sb + (long long)kb * p.NB;
#pragma unroll
                    for (int i = 0; i < NT; i += 32)
                        if (i + lane < NT) ptx::cp_async4(to + i + lane, sb + min(n0 + i + lane, p.NB - 1));
                    cp_async_arrive(sfull + s);
                }
            }
            ptx::cp_async_wait_all();
        }
    } else {
        if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int e = warp - 4, quarter = warp & 3, half = e >> 2;
        const uint32_t mine = tmem + ((uint32_t)(quarter * 32) << 16) + half * C::CW;
        int it = 0, round = 0;  // steps with column scales; handshakes
        // A warp whose wait ran out of time, never expected, hands nothing back any more: the warps it works with
        // then run into limits of their own instead of over data that others still read.
        bool ok = true;
        for (int t = blockIdx.x; t < p.tiles; t += gridDim.x) {
            const int m0 = (t % p.mt) * kM + quarter * 32, n0 = (t / p.mt) * NT + half * C::CW;
            float2 acc[C::CW / 2];
#pragma unroll
            for (int i = 0; i < C::CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            if (p.bias) {
                if constexpr (WIDE) {  // lane l holds columns 32 j + l; a shuffle hands each to all rows
#pragma unroll
                    for (int j = 0; j < C::CW; j += 32) {
                        const float v = __ldg(p.bias + min(n0 + j + lane, p.N - 1));
#pragma unroll
                        for (int i = 0; i < (C::CW < 32 ? C::CW : 32); i += 2)
                            acc[(j + i) / 2] = make_float2(__shfl_sync(0xffffffffu, v, i), __shfl_sync(0xffffffffu, v, i + 1));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < C::CW / 8; ++i) {
                        const int n = n0 + 8 * i + 2 * (lane & 3);
                        const float2 v = make_float2(__ldg(p.bias + min(n, p.N - 1)), __ldg(p.bias + min(n + 1, p.N - 1)));
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[4 * i + r] = v;
                    }
                }
            }
            // scales of rows: its own (WIDE), or the four of the fragments
            constexpr int kRows = WIDE ? 1 : 4;
            const float* psa[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) psa[r] = p.sa + min(m0 + (WIDE ? lane : (lane >> 2) + 8 * r), p.M - 1);
            const float* psb = p.sb + min(n0 / kBlock, p.NB - 1);
            float sa[kAhead][kRows], sb[kAhead];
            auto fetch = [&](int slot, int kb) {
                const bool there = kb < p.KB;
#pragma unroll
                for (int r = 0; r < kRows; ++r) sa[slot][r] = there ? __ldg(psa[r] + (long long)kb * p.M) : 0.f;
                sb[slot] = WIDE && there ? __ldg(psb + (long long)kb * p.NB) : 1.f;
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(i, i);
            for (int k0 = 0; k0 < p.KB && ok; k0 += kStep, ++round) {
                const int b = round % C::kAcc, steps = kStep == 1 ? 1 : min(kStep, p.KB - k0);
                float s1[kStep][kRows];
#pragma unroll
                for (int j = 0; j < kStep; ++j)
#pragma unroll
                    for (int r = 0; r < kRows; ++r) s1[j][r] = sa[j][r] * sb[j];
#pragma unroll
                for (int i = 0; i + kStep < kAhead; ++i) {
#pragma unroll
                    for (int r = 0; r < kRows; ++r) sa[i][r] = sa[i + kStep][r];
                    sb[i] = sb[i + kStep];
                }
#pragma unroll
                for (int j = 0; j < kStep; ++j) fetch(kAhead - kStep + j, k0 + kAhead + j);
                ok = warp_wait(done + b, (round / C::kAcc) & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                // the next columns are on their way while a piece is added up
                constexpr int kLd = C::CW >= 32 ? 32 : 16, kPieces = C::CW / kLd;
                const uint32_t buf = mine + b * kStep * NT;
                auto hand_back = [&]() {  // the buffer is read: the tensor core may fill it again
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(freed + b);
                };
                // FULL: all kStep steps, which the compiler can then lay out in one go
                auto add_up = [&](auto full) {
                    constexpr bool FULL = decltype(full)::value;
                    const int count = FULL ? kStep : steps;
                    if constexpr (WIDE) {
                        uint32_t v[2][kLd / 16][16];
                        tmem_ld<kLd>(buf, v[0]);
#pragma unroll
                        for (int c = 0; c < kStep * kPieces; ++c) {
                            const int j = c / kPieces, next = c + 1;
                            if (FULL || j < count) {
                                tmem_wait<kLd>(v[c & 1]);
                                if (next < count * kPieces) tmem_ld<kLd>(buf + next / kPieces * NT + next % kPieces * kLd, v[next & 1]);
                                else hand_back();
                                const float2 s2 = make_float2(s1[j][0], s1[j][0]);
#pragma unroll
                                for (int i = 0; i < kLd / 2; ++i) {
                                    const uint32_t* w = &v[c & 1][i / 8][2 * (i % 8)];
                                    float2& to = acc[c % kPieces * kLd / 2 + i];
                                    to = __ffma2_rn(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), s2, to);
                                }
                            }
                        }
                    } else {
                        // Column scales: a lane of the fragments needs a quarter of them, where a lane that holds a
                        // whole row would read all from shared memory, 512 bytes a load and four columns (12 %
                        // slower at 2048 x 2048 x 6400 in tiles of 128 columns).
                        uint32_t v[2][2][kLd / 2];
                        auto load = [&](int c) {
                            const uint32_t from = buf + c / kPieces * NT + c % kPieces * kLd;
                            tmem_ld_frag(from, v[c & 1][0]);
                            tmem_ld_frag(from + (16u << 16), v[c & 1][1]);
                        };
                        load(0);
#pragma unroll
                        for (int c = 0; c < kStep * kPieces; ++c) {
                            const int j = c / kPieces, next = c + 1;
                            if (FULL || j < count) {
                                const float* cs = scales + (it + j) % kScaleSlots * NT + half * C::CW + 2 * (lane & 3);
                                float2 k2[kLd / 8];  // while the sums are on their way
#pragma unroll
                                for (int i = 0; i < kLd / 8; ++i) k2[i] = *reinterpret_cast<const float2*>(cs + c % kPieces * kLd + 8 * i);
                                tmem_wait(v[c & 1][0]);
                                tmem_wait(v[c & 1][1]);
                                if (next < count * kPieces) load(next);
                                else hand_back();
#pragma unroll
                                for (int i = 0; i < kLd / 8; ++i) {
#pragma unroll
                                    for (int r = 0; r < 4; ++r) {
                                        const uint32_t* w = &v[c & 1][r / 2][4 * i + 2 * (r % 2)];
                                        const float2 f = __fmul2_rn(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), k2[i]);
                                        float2& to = acc[(c % kPieces * kLd / 8 + i) * 4 + r];
                                        to = __ffma2_rn(f, make_float2(s1[j][r], s1[j][r]), to);
                                    }
                                }
                            }
                        }
                    }
                };
                if (kStep == 1 || steps == kStep) add_up(std::true_type{});
                else add_up(std::false_type{});
                if (!WIDE) {
                    __syncwarp();
                    if (lane == 0)
                        for (int j = 0; j < steps; ++j) ptx::mbar_arrive(sempty + (it + j) % kScaleSlots);
                    it += steps;
                }
            }
            if (!ok) {  // NaN rather than a partial sum
#pragma unroll
                for (int i = 0; i < C::CW / 2; ++i) acc[i] = make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
            }
            write_out<O, C::CW, !WIDE>(p, acc, staging + e * 32 * kPitch, m0, n0);
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
    // Boxes no higher than the matrix: what stands in the tile's other rows of shared memory only reaches
    // results that are not written.  (Boxes of 128 rows of a matrix of 9 to 15: 29 us, 16 rows and more 19,
    // at 8192 x 8192.)
    const int a_rows = std::min(m.M, kM), b_rows = std::min(m.N, NT);
    p.step_bytes = (a_rows + b_rows) * kBlock;
    CUtensorMap ma, mb;
    if (!make_map(&ma, m.a, m.M, m.K, m.as, a_rows) || !make_map(&mb, m.b, m.N, m.K, m.bs, b_rows)) return -1;
    auto kern = k_fp8_matmul<O, NT, WIDE>;
    if (!allow_smem<k_fp8_matmul<O, NT, WIDE>>(C::kSmem)) return -1;
    const int grid = std::min(p.tiles, kSms);
    return launch_dependent(kern, dim3(grid), dim3(C::kThreads), C::kSmem, s, p, ma, mb) == cudaSuccess ? 1 : -1;
}

template <typename O, bool WIDE>
int launch_nt(const MatmulArgs& m, cudaStream_t s) {
    // Rounds of tiles over the SMs, times what a round takes with tiles of that width.  At K = 2048 a round takes
    // 9.4, 6.0, 3.7, 3.1 and 3.1 us, of one round 0.2 us less with 16 columns than with 32; the weights below
    // were fitted when the narrow tiles took longer, and choose what these times choose in all but one of 7936
    // cases (128 to 12800 rows, 64 to 8192 columns).  K is left out: it stretches a round of every width.
    // Measured there, us with 256 / 128 / 64 / 32 / 16 columns: 64 x 2048: 10.6 / 7.4 / 5.9 / 5.5 / 5.3; 800 x
    // 1024: 11.9 / 8.2 / 6.8 / 9.0 / 14.5; 800 x 2048: 12.1 / 8.6 / 10.4 / 15.1 / 23.3; 2048 x 2048: 12.9 / 14.5 /
    // 17.8 / 24.6 / 44.6.
    const long long mt = (m.M + kM - 1LL) / kM;
    auto cost = [&](int nt, long long round) { return (mt * ((m.N + nt - 1LL) / nt) + kSms - 1) / kSms * round; };
    const long long c256 = cost(256, 17), c128 = cost(128, 11), c64 = cost(64, 8), c32 = cost(32, 7), c16 = cost(16, 6);
    const long long least = std::min({c256, c128, c64, c32, c16});
    if (c256 == least) return launch<O, 256, WIDE>(m, s);
    if (c128 == least) return launch<O, 128, WIDE>(m, s);
    if (c64 == least) return launch<O, 64, WIDE>(m, s);
    return c32 == least ? launch<O, 32, WIDE>(m, s) : launch<O, 16, WIDE>(m, s);
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
