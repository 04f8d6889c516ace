// norm_resident.cuh -- group norm with its tensors read from global memory once.
//
// A cluster of S blocks owns one item's slab of channels (whole groups, at least 64 bytes of a row
// where the tensor has them); each block keeps a chunk of the slab's rows in shared memory, so the
// statistics and the elementwise pass read global memory once and write it once.  The S blocks
// exchange their partial sums through distributed shared memory: each block stores its own into every
// peer's inbox with st.async, which counts the bytes on the peer's mbarrier (a cluster barrier with
// loads from the peers in its place took 0.9 us more at [2, 2000, 512]).  A thread reads back only what it
// copied itself (its channels are fixed, its rows are every TY-th), so no barrier stands between the
// copies and their use, and the statistics of the rows that have arrived are formed while the later
// ones are on their way.
#pragma once

#include "norm_kernels.cuh"

namespace mh3a {
namespace norm {

constexpr int kResThreads = 256;

// How a resident launch divides the tensor.
struct Resident {
    int S;      // blocks per cluster (row chunks per slab)
    int rows;   // rows per chunk
    int W;      // channels per slab
    int slabs;  // slabs per row
    int smem;   // dynamic shared memory, bytes
    FastDiv ty;    // rows of threads
    FastDiv w;     // vectors per slab row
    FastDiv D;     // channels per group
    FastDiv span;  // partial sums per group and row of threads
};

struct ResPlace {
    int b, c0, rank, w, tx, ty, TY, c;
    bool live;
};

template <int V>
__device__ __forceinline__ ResPlace res_place(const Resident& r) {
    ResPlace p;
    p.rank = blockIdx.x;
    p.c0 = blockIdx.y * r.W;
    p.w = r.w.d;
    p.ty = threadIdx.x / r.w;
    p.tx = threadIdx.x - p.ty * p.w;
    p.TY = r.ty.d;
    p.b = blockIdx.z;
    p.live = p.ty < p.TY;
    p.c = p.c0 + p.tx * V;
    return p;
}

__device__ __forceinline__ void cp_async16_to(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kParts = 4;  // copy groups whose arrival is waited for one by one

// Statistics of `n` values: mean = hi + lo, m2 the sum of squared deviations.
struct alignas(16) Part {
    float hi, lo, m2, n;
};

// Shared memory behind the data: one Part per thread (and channel, where vectors straddle groups),
// an inbox of one Part per peer and group with its mbarrier, and the final (mean, rstd).
__host__ __device__ constexpr int res_fwd_extra(int W, int D, int V, int S) {
    return kResThreads * (D % V ? V : 1) * 16 + (W / D) * (16 * S + 8) + 16;
}

__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, int rank) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(addr), "r"(rank));
    return to;
}
// 16 bytes into a peer's shared memory, counted on the peer's mbarrier.
__device__ __forceinline__ void send16(uint32_t to, uint32_t bar, float4 v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}
// Waits (up to a second) for the bytes that the peers send to this block's mbarrier.  A thread whose wait
// succeeded may read the inbox; a thread that gave up must not use it.
__device__ __forceinline__ bool wait_for_peers(uint64_t* bar, uint64_t limit_ns = 1000000000ull) {
    const uint64_t t0 = ptx::globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i) {
            uint32_t ok;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(ptx::smem_u32(bar))
                : "memory");
            if (ok) return true;
        }
        if (ptx::globaltimer_ns() - t0 > limit_ns) return false;
    }
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The end of a block, `arrived` the same in all its threads.  After a wait that succeeded nothing is on its way
// to this block any more.  After one that was given up (never expected) the block's shared memory has to
// outlive what the peers still send: it stays until every peer has ended or has come here too (each within
// limits of its own; the barrier does not count blocks that have ended), and what they sent has landed.
__device__ __forceinline__ void leave_peers(bool arrived, uint64_t* bar, uint64_t limit_ns = 1000000000ull) {
    if (arrived) return;
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    wait_for_peers(bar, limit_ns);
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Where the threads' statistics lie: rows of threads by vectors, or by channels, those of one place in the
// vector side by side (a thread that stored its channels one behind the other would meet the banks of
// its neighbours: 1900 cycles against 100 for 200 channels).
template <int V, bool WHOLE>
__device__ __forceinline__ int part_index(int row, int i, int w) {
    return WHOLE ? row * w + i : (row * V + i % V) * w + i / V;
}

// The block's statistics of one group (the result is in all lanes of the warp), from `rows` rows of threads
// and the entries first .. first + span of each, about the first one's mean, in fp64: one pass, and nothing
// to lose but its distance from the group's mean, squared, in 53 bits.  inv = 1 / n.
template <int V, bool WHOLE>
__device__ __forceinline__ Part group_stats(const Part* part, int rows, int w, int first, FastDiv span, float n, double inv) {
    const int lane = threadIdx.x & 31, m = rows * span.d;
    const Part ref = part[part_index<V, WHOLE>(0, first, w)];
    double s = 0.0, q = 0.0;
    float m2 = 0.f;
#pragma unroll 4
    for (int i = lane; i < m; i += 32) {
        const int row = (unsigned)i / span;
        const Part v = part[part_index<V, WHOLE>(row, first + i - row * (int)span.d, w)];
        const double d = (v.hi - ref.hi) + (v.lo - ref.lo), nd = d * v.n;
        s += nd;
        q = fma(nd, d, q);
        m2 += v.m2;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, off);
        q += __shfl_xor_sync(0xffffffffu, q, off);
        m2 += __shfl_xor_sync(0xffffffffu, m2, off);
    }
    if (!(n > 0.f)) return Part{0.f, 0.f, 0.f, 0.f};
    const double d = s * inv, mean = (double)ref.hi + ((double)ref.lo + d);
    const float hi = (float)mean;
    return Part{hi, (float)(mean - hi), (float)(m2 + (q - s * d)), n};
}

// WHOLE: no vector straddles two groups (D is a multiple of V).
template <typename T, int V, int ACT, bool WHOLE>
__global__ void __launch_bounds__(kResThreads) k_norm_resident(const NormArgs a, const Resident r) {
    constexpr bool kPrecise = sizeof(T) == 4;
    constexpr int H = V / 2;
    constexpr int P = WHOLE ? 1 : H;  // pairs of partial sums a thread keeps
    constexpr bool kSnake = ACT == MH3A_ACT_SNAKE_BETA;
    extern __shared__ __align__(16) unsigned char smem[];
    const ResPlace p = res_place<V>(r);
    const int r0 = min(p.rank * r.rows, a.T), r1 = min(r0 + r.rows, a.T);
    Part* part = reinterpret_cast<Part*>(smem + (size_t)r.rows * r.W * sizeof(T));
    Part* inbox = part + kResThreads * (WHOLE ? 1 : V);  // [S][ng]
    const int ng = (unsigned)r.W / r.D;
    uint64_t* bar = reinterpret_cast<uint64_t*>(inbox + r.S * ng);
    float2* fin = reinterpret_cast<float2*>(bar + 2);  // (mean, rstd)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int next = p.TY * p.w;  // between a thread's rows in shared memory, in vectors
    if (threadIdx.x == 0) {
        ptx::mbar_init(bar, 1);
        ptx::fence_mbar_init();
        ptx::mbar_arrive_expect_tx(bar, r.S * ng * 16);
    }
    cluster_arrive();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int n = valid_rows(a, p.b);
    const int have = max(0, min(n, r1) - r0);  // valid rows of this chunk
    // this thread's rows: ty + TY k, k < mine; `per` of them in each copy group
    const int mine = p.live && have > p.ty ? (int)((unsigned)(have - p.ty + p.TY - 1) / r.ty) : 0;
    const int per = (mine + kParts - 1) / kParts;
    {
        const T* x = static_cast<const T*>(a.x) + p.b * a.xb + p.c + (long long)(r0 + p.ty) * a.xr;
        const long long step = (long long)p.TY * a.xr;
        uint32_t to = ptx::smem_u32(smem) + (p.tx + p.ty * p.w) * 16;
        int k = 0;
#pragma unroll
        for (int g = 0; g < kParts; ++g) {
#pragma unroll 4
            for (int e = min(mine, (g + 1) * per); k < e; ++k, x += step, to += next * 16) cp_async16_to(to, x);
            ptx::cp_async_commit();
        }
    }
    // what does not depend on the rows, while they arrive
    float2 w[H], bi[H], al[H], ib[H];
    if (p.live) {
        load_param_vec<V>(a.weight, p.c, 1.f, w);
        load_param_vec<V>(a.bias, p.c, 0.f, bi);
        if (kSnake) {
            load_param_vec<V>(a.alpha, p.c, 0.f, al);
            load_param_vec<V>(a.beta, p.c, 0.f, ib);
#pragma unroll
            for (int i = 0; i < H; ++i) ib[i] = make_float2(rcp_ftz(ib[i].x + 1e-9f), rcp_ftz(ib[i].y + 1e-9f));
        }
    }
    const float group_n = (float)have * a.D;  // the group's values here, and what they are divided by, here and in all
    const double inv_here = have > 0 ? 1.0 / ((double)have * a.D) : 0.0, inv_count = n > 0 ? 1.0 / ((double)n * a.D) : 0.0;
    const Pack<T, V>* mydata = reinterpret_cast<const Pack<T, V>*>(smem) + p.tx + p.ty * p.w;

    // Sums of deviations from a value near the thread's mean: the mean of its first rows.  An
    // outlier among them moves it by a fraction only, so the squares cancel by a factor of
    // rows / 16 at worst.
    float2 sh[P], s[P], q[P];
#pragma unroll
    for (int i = 0; i < P; ++i) sh[i] = s[i] = q[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int g = 0; g < kParts; ++g) {
        if (g == 0) cp_async_wait_group<kParts - 1>();
        if (g == 1) cp_async_wait_group<kParts - 2>();
        if (g == 2) cp_async_wait_group<kParts - 3>();
        if (g == 3) cp_async_wait_group<kParts - 4>();
        if (g == 0 && mine > 0) {
            const int m = min(per, 4);
            for (int k = 0; k < m; ++k) {
                float2 f[H];
                unpack_pairs<T, V>(mydata[k * next], f);
#pragma unroll
                for (int i = 0; i < H; ++i) sh[WHOLE ? 0 : i] = __fadd2_rn(sh[WHOLE ? 0 : i], f[i]);
            }
            const float im = -rcp_ftz((float)(WHOLE ? m * V : m));
            if (WHOLE) sh[0].x = sh[0].y = sh[0].x + sh[0].y;
#pragma unroll
            for (int i = 0; i < P; ++i) sh[i] = __fmul2_rn(sh[i], make_float2(im, im));
        }
        const Pack<T, V>* at = mydata + g * per * next;
#pragma unroll 2
        for (int k = min(mine, (g + 1) * per) - g * per; k > 0; --k, at += next) {
            float2 f[H];
            unpack_pairs<T, V>(*at, f);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int j = WHOLE ? 0 : i;
                const float2 d = __fadd2_rn(f[i], sh[j]);
                s[j] = __fadd2_rn(s[j], d);
                q[j] = __ffma2_rn(d, d, q[j]);
            }
        }
    }
    if (p.live) {
        const float cnt = (float)(WHOLE ? mine * V : mine), ic = mine > 0 ? rcp_ftz(cnt) : 0.f;
        if (WHOLE) {
            const float sum = s[0].x + s[0].y, lo = sum * ic;
            part[p.ty * p.w + p.tx] = Part{-sh[0].x, lo, q[0].x + q[0].y - sum * lo, cnt};
        } else {
            Part* to = part + p.ty * r.W + p.tx;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                to[2 * i * p.w] = Part{-sh[i].x, s[i].x * ic, q[i].x - s[i].x * s[i].x * ic, cnt};
                to[(2 * i + 1) * p.w] = Part{-sh[i].y, s[i].y * ic, q[i].y - s[i].y * s[i].y * ic, cnt};
            }
        }
    }
    __syncthreads();
    cluster_wait();  // the peers' mbarriers are initialised
    for (int g = warp; g < ng; g += kResThreads / 32) {
        const Part o = group_stats<V, WHOLE>(part, min(p.TY, have), p.w, g * r.span.d, r.span, group_n, inv_here);
        if (lane < r.S)
            send16(peer_smem(ptx::smem_u32(inbox + p.rank * ng + g), lane), peer_smem(ptx::smem_u32(bar), lane),
                   make_float4(o.hi, o.lo, o.m2, o.n));
    }
    const bool arrived = wait_for_peers(bar);
    for (int g = warp; g < ng; g += kResThreads / 32) {
        Part o{0.f, 0.f, 0.f, 0.f};
        if (lane < r.S) o = inbox[lane * ng + g];
        const Part ref = inbox[g];  // the first block has rows if any has
        const double from = (double)(o.hi - ref.hi) + (double)o.lo;
        double s1 = o.n > 0.f ? from * o.n : 0.0, s2 = o.n > 0.f ? fma(s1, from, (double)o.m2) : 0.0;
#pragma unroll
        for (int off = 8; off; off >>= 1) {
            s1 += __shfl_xor_sync(0xffffffffu, s1, off);
            s2 += __shfl_xor_sync(0xffffffffu, s2, off);
        }
        if (lane == 0) {
            const double d = s1 * inv_count, mean = (double)ref.hi + d, var = s2 * inv_count - d * d;
            // Equal values leave a variance within rounding of 0, on either side (NaN stays).  A wait that ran
            // out of time, never expected, gives NaN rather than stale sums.
            const float root = sqrtf((float)((var < 0.0 ? 0.0 : var) + (double)a.eps)), nan = __int_as_float(0x7fffffff);
            const float2 f = arrived ? make_float2((float)mean, 1.0f / root) : make_float2(nan, nan);
            fin[g] = f;
            if (p.rank == 0) {
                const long long at = (long long)p.b * a.G + p.c0 / a.D + g;
                a.mean[at] = f.x;
                a.rstd[at] = f.y;
            }
        }
    }
    const bool all_arrived = __syncthreads_and(arrived);

    if (p.live) {
        float2 mu[H], sc[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 f = fin[(unsigned)(p.tx * V + (WHOLE ? 0 : 2 * i)) / r.D];
            const float2 h = WHOLE ? f : fin[(unsigned)(p.tx * V + 2 * i + 1) / r.D];
            mu[i] = make_float2(-f.x, -h.x);
            sc[i] = __fmul2_rn(w[i], make_float2(f.y, h.y));
        }
        T* y = static_cast<T*>(a.out) + ((long long)p.b * a.T + r0 + p.ty) * a.C + p.c;
        const long long step = (long long)p.TY * a.C;
        const Pack<T, V>* at = mydata;
#pragma unroll 2
        for (int k = 0; k < mine; ++k, at += next, y += step) {
            float2 f[H];
            unpack_pairs<T, V>(*at, f);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 u = __ffma2_rn(__fadd2_rn(f[i], mu[i]), sc[i], bi[i]);
                f[i] = act_fwd<ACT, kPrecise>(u, kSnake ? al[i] : u, kSnake ? ib[i] : u);
            }
            store_pairs<T, V>(y, f);
        }
        const Pack<T, V> zero{};  // rows behind the item's length
        for (int k = mine; p.ty + k * p.TY < r1 - r0; ++k, y += step) *reinterpret_cast<Pack<T, V>*>(y) = zero;
    }
    leave_peers(all_arrived, bar);
}

// Backward: shared memory behind x and dy: the threads' per-channel sums (one row for each warp where
// shuffles put the warp's rows together, else for each row of threads), the inbox of every peer's sums,
// their totals, and the groups' two means.
__host__ __device__ constexpr int res_bwd_extra(int W, int D, int V, int S, int ns) {
    return kResThreads * V * ns * 4 + (S + 1) * W * ns * 4 + (W / D) * 8 + 16;
}

// dx and the per-channel sums of one item's slab.  `a.ws` takes the item's totals [B][C][NS]; with one
// item they are the parameter gradients already.
template <typename T, int V, int ACT, bool WHOLE>
__global__ void __launch_bounds__(kResThreads) k_norm_bwd_resident(const NormArgs a, const Resident r) {
    constexpr bool kPrecise = sizeof(T) == 4;
    constexpr int H = V / 2, NS = kSums<ACT>, M = WHOLE ? 1 : H;
    constexpr bool kSnake = ACT == MH3A_ACT_SNAKE_BETA;
    extern __shared__ __align__(16) unsigned char smem[];
    const ResPlace p = res_place<V>(r);
    const int r0 = min(p.rank * r.rows, a.T), r1 = min(r0 + r.rows, a.T);
    const int ng = (unsigned)r.W / r.D, cols = r.W * NS;
    const uint32_t bytes = (uint32_t)r.rows * r.W * sizeof(T);
    float* red = reinterpret_cast<float*>(smem + 2 * (size_t)bytes);
    float* inbox = red + kResThreads * V * NS;  // [S][cols]
    float* total = inbox + r.S * cols;
    uint64_t* bar = reinterpret_cast<uint64_t*>(total + cols);
    float2* fin = reinterpret_cast<float2*>(bar + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int next = p.TY * p.w;
    if (threadIdx.x == 0) {
        ptx::mbar_init(bar, 1);
        ptx::fence_mbar_init();
        ptx::mbar_arrive_expect_tx(bar, r.S * cols * 4);
    }
    cluster_arrive();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int n = valid_rows(a, p.b);
    const int have = max(0, min(n, r1) - r0);
    const int mine = p.live && have > p.ty ? (int)((unsigned)(have - p.ty + p.TY - 1) / r.ty) : 0;
    const int per = (mine + kParts - 1) / kParts;
    const int first = p.tx + p.ty * p.w;
    {
        const T* x = static_cast<const T*>(a.x) + p.b * a.xb + p.c + (long long)(r0 + p.ty) * a.xr;
        const T* dy = static_cast<const T*>(a.dy) + p.b * a.gb + p.c + (long long)(r0 + p.ty) * a.gr;
        const long long xs = (long long)p.TY * a.xr, gs = (long long)p.TY * a.gr;
        uint32_t to = ptx::smem_u32(smem) + first * 16;
        int k = 0;
#pragma unroll
        for (int g = 0; g < kParts; ++g) {
#pragma unroll 2
            for (int e = min(mine, (g + 1) * per); k < e; ++k, x += xs, dy += gs, to += next * 16) {
                cp_async16_to(to, x);
                cp_async16_to(to + bytes, dy);
            }
            ptx::cp_async_commit();
        }
    }
    float2 mu[M], rs[M], w[H], bi[H], al[H], ib[H];
    if (p.live) {
        load_param_vec<V>(a.weight, p.c, 1.f, w);
        load_param_vec<V>(a.bias, p.c, 0.f, bi);
        if (kSnake) {
            load_param_vec<V>(a.alpha, p.c, 0.f, al);
            load_param_vec<V>(a.beta, p.c, 0.f, ib);
#pragma unroll
            for (int i = 0; i < H; ++i) ib[i] = make_float2(rcp_ftz(ib[i].x + 1e-9f), rcp_ftz(ib[i].y + 1e-9f));
        }
        const long long g0 = (long long)p.b * a.G + p.c0 / a.D;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const int ga = (unsigned)(p.tx * V + 2 * i) / r.D, gb = WHOLE ? ga : (unsigned)(p.tx * V + 2 * i + 1) / r.D;
            mu[i] = make_float2(-a.mean[g0 + ga], -a.mean[g0 + gb]);
            rs[i] = make_float2(a.rstd[g0 + ga], a.rstd[g0 + gb]);
        }
    }
    Pack<T, V>* myx = reinterpret_cast<Pack<T, V>*>(smem) + first;
    Pack<T, V>* myg = reinterpret_cast<Pack<T, V>*>(smem + bytes) + first;

    float2 acc[NS][H];
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) acc[j][i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int g = 0; g < kParts; ++g) {
        if (g == 0) cp_async_wait_group<kParts - 1>();
        if (g == 1) cp_async_wait_group<kParts - 2>();
        if (g == 2) cp_async_wait_group<kParts - 3>();
        if (g == 3) cp_async_wait_group<kParts - 4>();
        for (int k = g * per, e = min(mine, (g + 1) * per); k < e; ++k) {
            float2 f[H], d[H];
            unpack_pairs<T, V>(myx[k * next], f);
            unpack_pairs<T, V>(myg[k * next], d);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 xh = __fmul2_rn(__fadd2_rn(f[i], mu[WHOLE ? 0 : i]), rs[WHOLE ? 0 : i]);
                const float2 u = __ffma2_rn(xh, w[i], bi[i]);
                float2 pa, pb;
                const float2 du = __fmul2_rn(d[i], act_slope<ACT, kPrecise>(u, kSnake ? al[i] : u, kSnake ? ib[i] : u, &pa, &pb));
                acc[0][i] = __fadd2_rn(acc[0][i], du);
                acc[1][i] = __ffma2_rn(du, xh, acc[1][i]);
                if constexpr (NS == 4) {
                    acc[2][i] = __ffma2_rn(d[i], pa, acc[2][i]);
                    acc[3][i] = __ffma2_rn(d[i], pb, acc[3][i]);
                }
                if (kPrecise) d[i] = du;  // fp32: kept in dy's place, exactly what the second pass needs
            }
            if (kPrecise && ACT != MH3A_ACT_NONE) store_pairs<T, V>(reinterpret_cast<T*>(myg + k * next), d);
        }
    }
    // the block's sums: lanes that share channels first, where they stand a power of two apart
    const bool shuffled = p.w < 32 && (p.w & (p.w - 1)) == 0;
    int nrow = p.TY, row = p.ty;
    bool put = p.live;
    if (shuffled) {
        for (int off = 16; off >= p.w; off >>= 1) {
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    acc[j][i].x += __shfl_xor_sync(0xffffffffu, acc[j][i].x, off);
                    acc[j][i].y += __shfl_xor_sync(0xffffffffu, acc[j][i].y, off);
                }
        }
        nrow = kResThreads / 32;
        row = warp;
        put = lane < p.w;
    }
    if (put) {
        float* to = red + row * cols + p.tx * V;  // [sum][channel]
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int i = 0; i < H; ++i) *reinterpret_cast<float2*>(to + j * r.W + 2 * i) = acc[j][i];
    }
    __syncthreads();
    cluster_wait();
    for (int c = threadIdx.x * 4; c < cols; c += kResThreads * 4) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < nrow; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(red + k * cols + c);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        for (int peer = 0; peer < r.S; ++peer)
            send16(peer_smem(ptx::smem_u32(inbox + p.rank * cols + c), peer), peer_smem(ptx::smem_u32(bar), peer), s);
    }
    const bool arrived = wait_for_peers(bar);
    for (int c = threadIdx.x; c < cols; c += kResThreads) {
        float s = 0.f;
        for (int k = 0; k < r.S; ++k) s += inbox[k * cols + c];
        total[c] = arrived ? s : __int_as_float(0x7fffffff);
    }
    const bool all_arrived = __syncthreads_and(arrived);
    for (int g = warp; g < ng; g += kResThreads / 32) {
        float s1 = 0.f, s2 = 0.f;
        for (int i = lane; i < a.D; i += 32) {
            const int c = g * a.D + i;
            const float wc = a.weight ? __ldg(a.weight + p.c0 + c) : 1.f;
            s1 = fmaf(wc, total[c], s1);
            s2 = fmaf(wc, total[r.W + c], s2);
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        const float inv = n > 0 ? 1.0f / ((float)n * a.D) : 0.f;
        if (lane == 0) fin[g] = make_float2(-s1 * inv, -s2 * inv);
    }
    if (p.rank == 0) {
        for (int c = threadIdx.x; c < r.W; c += kResThreads) {
            const int at = p.c0 + c;
            if (a.B == 1) {
                if (a.dbias) a.dbias[at] = total[c];
                if (a.dweight) a.dweight[at] = total[r.W + c];
                if constexpr (NS == 4) {
                    if (a.dalpha) a.dalpha[at] = total[2 * r.W + c];
                    if (a.dbeta) {
                        const float v = 1.0f / (a.beta[at] + 1e-9f);
                        a.dbeta[at] = -total[3 * r.W + c] * v * v;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < NS; ++j) a.ws[((long long)p.b * a.C + at) * NS + j] = total[j * r.W + c];
            }
        }
    }
    __syncthreads();
    if (p.live) {
        float2 m1[M], m2[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const float2 f = fin[(unsigned)(p.tx * V + 2 * i) / r.D];
            const float2 h = WHOLE ? f : fin[(unsigned)(p.tx * V + 2 * i + 1) / r.D];
            m1[i] = make_float2(f.x, h.x);
            m2[i] = make_float2(f.y, h.y);
        }
        T* dx = static_cast<T*>(a.out) + ((long long)p.b * a.T + r0 + p.ty) * a.C + p.c;
        const long long step = (long long)p.TY * a.C;
        int k = 0;
        for (; k < mine; ++k, dx += step) {
            float2 f[H], d[H];
            unpack_pairs<T, V>(myx[k * next], f);
            unpack_pairs<T, V>(myg[k * next], d);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int j = WHOLE ? 0 : i;
                const float2 xh = __fmul2_rn(__fadd2_rn(f[i], mu[j]), rs[j]);
                float2 du = d[i];
                if (!kPrecise) {
                    const float2 u = __ffma2_rn(xh, w[i], bi[i]);
                    float2 pa, pb;
                    du = __fmul2_rn(du, act_slope<ACT, kPrecise>(u, kSnake ? al[i] : u, kSnake ? ib[i] : u, &pa, &pb));
                }
                f[i] = __fmul2_rn(rs[j], __ffma2_rn(xh, m2[j], __ffma2_rn(du, w[i], m1[j])));
            }
            store_pairs<T, V>(dx, f);
        }
        const Pack<T, V> zero{};
        for (; p.ty + k * p.TY < r1 - r0; ++k, dx += step) *reinterpret_cast<Pack<T, V>*>(dx) = zero;
    }
    leave_peers(all_arrived, bar);
}

}  // namespace norm
}  // namespace mh3a
