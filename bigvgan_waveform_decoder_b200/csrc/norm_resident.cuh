// norm_resident.cuh -- group norm with its tensors read from global memory once.
//
// A cluster of S blocks owns one item's slab of channels (whole groups, at least 64 bytes of a row
// where the tensor has them); each block keeps a chunk of the slab's rows in shared memory, so the
// statistics and the elementwise pass read global memory once and write it once.  The S blocks
// exchange their partial sums through distributed shared memory.  A thread reads back only what it
// copied itself (its channels are fixed, its rows are every TY-th), so no barrier stands between the
// copies and their use, and the statistics of the rows that have arrived are formed while the later
// ones are on their way.
#pragma once

#include <cooperative_groups.h>

#include "norm_kernels.cuh"

namespace mh3a {
namespace norm {

// How a resident launch divides the tensor.
struct Resident {
    int S;      // blocks per cluster (row chunks per slab)
    int rows;   // rows per chunk
    int W;      // channels per slab
    int slabs;  // slabs per row
    int smem;   // dynamic shared memory, bytes
};

struct ResPlace {
    int b, c0, rank, w, tx, ty, TY, c;
    bool live;
};

template <int V, int NT>
__device__ __forceinline__ ResPlace res_place(const Resident& r) {
    ResPlace p;
    p.rank = blockIdx.x % r.S;
    const unsigned unit = blockIdx.x / r.S;
    p.c0 = (int)(unit % r.slabs) * r.W;
    p.b = unit / r.slabs;
    p.w = r.W / V;
    p.tx = threadIdx.x % p.w;
    p.ty = threadIdx.x / p.w;
    p.TY = NT / p.w;
    p.live = p.ty < p.TY;
    p.c = p.c0 + p.tx * V;
    return p;
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
// then per group the block's Part and the final (mean, rstd).
__host__ __device__ constexpr int res_fwd_extra(int nt, int W, int D, int V) {
    return nt * (D % V ? V : 1) * 16 + (W / D) * 24;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The block's statistics of one group (the result is in all lanes of the warp): entries (row of
// threads, first .. first + span) of `part`, a few per lane, put together in fp64.
__device__ __forceinline__ Part group_stats(const Part* part, int ty_n, int width, int first, int span) {
    const int lane = threadIdx.x & 31, m = ty_n * span;
    float n = 0.f;
    double s = 0.0;
    for (int i = lane; i < m; i += 32) {
        const Part v = part[(i / span) * width + first + i % span];
        n += v.n;
        if (v.n > 0.f) s += ((double)v.hi + (double)v.lo) * v.n;
    }
    n = warp_sum(n);
    const double mean = n > 0.f ? warp_sum(s) / n : 0.0;
    double q = 0.0;
    for (int i = lane; i < m; i += 32) {
        const Part v = part[(i / span) * width + first + i % span];
        const double d = (double)v.hi + (double)v.lo - mean;
        if (v.n > 0.f) q += fma(v.n * d, d, (double)v.m2);
    }
    const float hi = (float)mean;
    return Part{hi, (float)(mean - hi), (float)warp_sum(q), n};
}

// WHOLE: no vector straddles two groups (D is a multiple of V).
template <typename T, int V, int ACT, bool WHOLE, int NT>
__global__ void __launch_bounds__(NT) k_norm_resident(const NormArgs a, const Resident r) {
    constexpr bool kPrecise = sizeof(T) == 4;
    constexpr int H = V / 2;
    constexpr int P = WHOLE ? 1 : H;  // pairs of partial sums a thread keeps
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) unsigned char smem[];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const ResPlace p = res_place<V, NT>(r);
    const int n = valid_rows(a, p.b);
    const int r0 = min(p.rank * r.rows, a.T), r1 = min(r0 + r.rows, a.T);
    const int have = max(0, min(n, r1) - r0);  // valid rows of this chunk
    Pack<T, V>* data = reinterpret_cast<Pack<T, V>*>(smem) + p.tx;
    Part* part = reinterpret_cast<Part*>(smem + (size_t)r.rows * r.W * sizeof(T));
    Part* loc = part + NT * (WHOLE ? 1 : V);
    const int ng = r.W / a.D;
    float2* fin = reinterpret_cast<float2*>(loc + ng);  // (mean, rstd)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // rows of this thread: ty + TY k, k < mine; `per` of them in each copy group
    const int mine = p.live ? (have - p.ty + p.TY - 1) / p.TY : 0;
    const int per = (mine + kParts - 1) / kParts;
    {
        const T* x = static_cast<const T*>(a.x) + p.b * a.xb + p.c + (long long)(r0 + p.ty) * a.xr;
        const long long step = (long long)p.TY * a.xr;
        int k = 0;
#pragma unroll
        for (int g = 0; g < kParts; ++g) {
            for (int e = min(mine, (g + 1) * per); k < e; ++k, x += step) ptx::cp_async16(data + (p.ty + k * p.TY) * p.w, x);
            ptx::cp_async_commit();
        }
    }
    // what does not depend on the rows, while they arrive
    const double inv_count = n > 0 ? 1.0 / ((double)n * a.D) : 0.0;
    float2 sc[H], bi[H], al[H], ib[H];
    if (p.live) {
        load_param<V>(a.weight, p.c, a.C, 1.f, reinterpret_cast<float(&)[V]>(sc));
        load_param<V>(a.bias, p.c, a.C, 0.f, reinterpret_cast<float(&)[V]>(bi));
        if (ACT == MH3A_ACT_SNAKE_BETA) {
            load_param<V>(a.alpha, p.c, a.C, 0.f, reinterpret_cast<float(&)[V]>(al));
            load_param<V>(a.beta, p.c, a.C, 0.f, reinterpret_cast<float(&)[V]>(ib));
#pragma unroll
            for (int i = 0; i < H; ++i) ib[i] = make_float2(1.0f / (ib[i].x + 1e-9f), 1.0f / (ib[i].y + 1e-9f));
        }
    }

    // Sums of deviations from a value near the thread's mean: the mean of its first rows.  An outlier
    // among them moves it by a fraction only, so the squares cancel by a factor of rows / 16 at worst.
    float2 sh[P], s[P], q[P];
#pragma unroll
    for (int i = 0; i < P; ++i) sh[i] = s[i] = q[i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int g = 0; g < kParts; ++g) {
        if (g == 0) cp_async_wait_group<3>();
        if (g == 1) cp_async_wait_group<2>();
        if (g == 2) cp_async_wait_group<1>();
        if (g == 3) cp_async_wait_group<0>();
        if (g == 0 && mine > 0) {
            const int m = min(per, 4);
            for (int k = 0; k < m; ++k) {
                float2 f[H];
                unpack_pairs<T, V>(data[(p.ty + k * p.TY) * p.w], f);
#pragma unroll
                for (int i = 0; i < H; ++i) sh[WHOLE ? 0 : i] = __fadd2_rn(sh[WHOLE ? 0 : i], f[i]);
            }
            if (WHOLE) {
                const float v = -(sh[0].x + sh[0].y) / (float)(m * V);
                sh[0] = make_float2(v, v);
            } else {
                const float v = -1.0f / (float)m;
#pragma unroll
                for (int i = 0; i < P; ++i) sh[i] = __fmul2_rn(sh[i], make_float2(v, v));
            }
        }
        for (int k = g * per, e = min(mine, (g + 1) * per); k < e; ++k) {
            float2 f[H];
            unpack_pairs<T, V>(data[(p.ty + k * p.TY) * p.w], f);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                constexpr int Z = 0;
                const int j = WHOLE ? Z : i;
                const float2 d = __fadd2_rn(f[i], sh[j]);
                s[j] = __fadd2_rn(s[j], d);
                q[j] = __ffma2_rn(d, d, q[j]);
            }
        }
    }
    const int width = WHOLE ? p.w : r.W;
    if (p.live) {
        if (WHOLE) {
            const float cnt = (float)mine * V, sum = s[0].x + s[0].y;
            const float lo = mine > 0 ? sum / cnt : 0.f;
            part[p.ty * width + p.tx] = Part{-sh[0].x, lo, q[0].x + q[0].y - sum * lo, cnt};
        } else {
            const float cnt = (float)mine, ic = mine > 0 ? 1.0f / cnt : 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                part[p.ty * width + p.tx * V + 2 * i] = Part{-sh[i].x, s[i].x * ic, q[i].x - s[i].x * s[i].x * ic, cnt};
                part[p.ty * width + p.tx * V + 2 * i + 1] = Part{-sh[i].y, s[i].y * ic, q[i].y - s[i].y * s[i].y * ic, cnt};
            }
        }
    }
    __syncthreads();
    const int span = WHOLE ? a.D / V : a.D;  // entries per group and row of threads
    for (int g = warp; g < ng; g += NT / 32) {
        const Part v = group_stats(part, p.TY, width, g * span, span);
        if (lane == 0) loc[g] = v;
    }
    if (r.S > 1) cg::this_cluster().sync();
    else __syncthreads();
    for (int g = warp; g < ng; g += NT / 32) {
        Part o{0.f, 0.f, 0.f, 0.f};
        if (r.S > 1) {
            if (lane < r.S) o = *cg::this_cluster().map_shared_rank(loc + g, lane);
        } else if (lane == 0) {
            o = loc[g];
        }
        const double m = (double)o.hi + (double)o.lo;
        double sum = o.n > 0.f ? m * o.n : 0.0;
#pragma unroll
        for (int off = 8; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const double mean = sum * inv_count, d = m - mean;
        double m2 = o.n > 0.f ? (double)o.m2 + d * d * o.n : 0.0;
#pragma unroll
        for (int off = 8; off; off >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, off);
        if (lane == 0) {
            const float rstd = 1.0f / sqrtf((float)(m2 * inv_count + (double)a.eps));
            fin[g] = make_float2((float)mean, rstd);
            if (p.rank == 0) {
                const long long at = (long long)p.b * a.G + p.c0 / a.D + g;
                a.mean[at] = (float)mean;
                a.rstd[at] = rstd;
            }
        }
    }
    __syncthreads();
    if (r.S > 1) cg::this_cluster().barrier_arrive();

    if (p.live) {
        float2 mu[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 f = fin[(p.tx * V + 2 * i) / a.D], h = WHOLE ? f : fin[(p.tx * V + 2 * i + 1) / a.D];
            mu[i] = make_float2(-f.x, -h.x);
            sc[i] = __fmul2_rn(sc[i], make_float2(f.y, h.y));
        }
        T* y = static_cast<T*>(a.out) + ((long long)p.b * a.T + r0) * a.C + p.c;
        for (int t = p.ty; t < r1 - r0; t += p.TY) {
            float f[V];
            if (t < have) {
                float2 f2[H];
                unpack_pairs<T, V>(data[t * p.w], f2);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 u = __ffma2_rn(__fadd2_rn(f2[i], mu[i]), sc[i], bi[i]);
                    constexpr bool kSnake = ACT == MH3A_ACT_SNAKE_BETA;
                    f[2 * i] = act_fwd<ACT, kPrecise>(u.x, kSnake ? al[i].x : 0.f, kSnake ? ib[i].x : 0.f);
                    f[2 * i + 1] = act_fwd<ACT, kPrecise>(u.y, kSnake ? al[i].y : 0.f, kSnake ? ib[i].y : 0.f);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = 0.f;
            }
            store_pack<T, V>(y + (long long)t * a.C, f);
        }
    }
    if (r.S > 1) cg::this_cluster().barrier_wait();  // peers may still read this block's sums
}

}  // namespace norm
}  // namespace mh3a
