// norm_ops.cu -- group norm with an activation over channels-last frames, and its gradient.
//
//   mean, rstd over an item's valid rows and a group's channels;  u = (x - mean) rstd w + b;
//   y = act(u).                                     (formulas at the entry points in mh3a.h)
//
// Both directions are bound by memory: a handful of operations an element against 4 to 12 bytes.
//
// Tensors up to 100 MB take the resident form (norm_resident.cuh), one pass over global memory.
//
// The general form takes any size and alignment, in passes over global memory: per-channel partial
// sums of a chunk of rows, their combination in fixed order, then the elementwise pass.  Rows are
// channels wide, so a warp reads whole rows (512 bytes) and every thread keeps one fixed run of V
// channels: its statistics stay per channel in registers, and groups of any width, also ones that end
// inside a vector, are put together only at the end.  None of its kernels lets the next one in early:
// grids that fill every SM once then start on SMs that still hold the blocks before them, and the
// uneven start costs more (101 against 93 us for sixteen 20 s items) than the launch it hides.
#include <algorithm>
#include <initializer_list>

#include "norm_kernels.cuh"
#include "norm_resident.cuh"
#include "ops_common.cuh"

namespace mh3a {
namespace norm {

constexpr int kThreads = 256;

// One block's place: item b, channel tile, row chunk.
struct Place {
    int b, c, ch, ty, TY;
    bool live;  // the thread's channels exist
};

template <int V>
__device__ __forceinline__ Place place(const NormArgs& a, unsigned id) {
    Place p;
    p.ch = id % a.chunks;
    id /= a.chunks;
    const int ct = id % a.ctiles;
    p.b = id / a.ctiles;
    const int tx = threadIdx.x & (a.tx - 1);
    p.ty = threadIdx.x / a.tx;
    p.TY = kThreads / a.tx;
    const long long c = ((long long)ct * a.tx + tx) * V;
    p.live = c < a.C;
    p.c = p.live ? (int)c : 0;
    return p;
}

// A thread's rows of N tensors, streamed through shared memory: kRing rows, in pairs, are on their way while
// one is worked on, with no registers held.  Only the thread itself reads its slots, so no barrier is needed.
// Element types that cp.async cannot copy (2 bytes) are loaded where they are used.
template <typename T, int V, int N>
struct Stream {
    static constexpr int kBytes = sizeof(T) * V;
    static constexpr bool kAsync = kBytes >= 4;
    static constexpr int kRing = kBytes * N > 16 ? 4 : 8;  // 32 KB a block at most
    static constexpr size_t kSmem = kAsync ? (size_t)kRing * N * kThreads * kBytes : 16;
    const T* at[N];
    long long step[N];
    Pack<T, V>* slots;
    int mine, issued, taken;

    __device__ __forceinline__ void fetch_pair() {
#pragma unroll
        for (int j = 0; j < 2; ++j, ++issued) {
            if (issued < mine) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const uint32_t to = ptx::smem_u32(slots + ((issued & (kRing - 1)) * N + i) * kThreads);
                    if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(at[i]) : "memory");
                    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(at[i]), "n"(kBytes < 4 ? 4 : kBytes) : "memory");
                    at[i] += step[i];
                }
            }
        }
        ptx::cp_async_commit();
    }
    __device__ __forceinline__ void start(void* smem, int rows) {
        slots = static_cast<Pack<T, V>*>(smem) + threadIdx.x;
        mine = rows;
        issued = taken = 0;
        if constexpr (kAsync) {
#pragma unroll
            for (int k = 0; k < kRing / 2; ++k) fetch_pair();
        }
    }
    // Calls f(rows of the N tensors) for every row in turn.
    template <typename F>
    __device__ __forceinline__ void run(F f) {
        if constexpr (kAsync) {
            for (; taken < mine; taken += 2) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kRing / 2 - 1) : "memory");
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (taken + j < mine) {
                        Pack<T, V> r[N];
#pragma unroll
                        for (int i = 0; i < N; ++i) r[i] = slots[(((taken + j) & (kRing - 1)) * N + i) * kThreads];
                        f(r);
                    }
                }
                fetch_pair();
            }
            ptx::cp_async_wait_all();
        } else {
            for (; taken < mine; ++taken) {
                Pack<T, V> r[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    r[i] = load_pack<T, V>(at[i]);
                    at[i] += step[i];
                }
                f(r);
            }
        }
    }
    // The sum of the first rows (up to four), which stay to be run over: f(row) for each; their number.
    template <typename F>
    __device__ __forceinline__ int peek(F f) {
        const int n = min(mine, 4);
        if constexpr (kAsync) asm volatile("cp.async.wait_group %0;" ::"n"(kRing / 2 - 2) : "memory");
        for (int k = 0; k < n; ++k) {
            if constexpr (kAsync) f(slots[k * N * kThreads]);
            else f(load_pack<T, V>(at[0] + k * step[0]));
        }
        return n;
    }
};

// Partial statistics of one channel: mean as hi + lo, and the sum of squared deviations from it.
// Means that lie far from zero would otherwise round away what tells them apart.
struct Stat {
    float hi, lo, m2;
};

// Merge of two partial statistics (Chan et al.), n the count of `s`, f = nb / (n + nb).
__device__ __forceinline__ void merge_stats(Stat& s, float n, const Stat& o, float f) {
    const float d = (o.hi - s.hi) + (o.lo - s.lo);
    const float t = fmaf(d, f, s.lo);
    const float hi = s.hi + t;  // Knuth's two-sum: hi + lo = s.hi + t exactly
    const float back = hi - s.hi;
    s.lo = (s.hi - (hi - back)) + (t - back);
    s.hi = hi;
    s.m2 += o.m2 + d * d * (n * f);
}

// Adds up V values of a row (as pairs where V is even).
template <int V>
struct Acc {
    static constexpr int H = V == 1 ? 1 : V / 2;
    float2 v[H];
};
template <typename T, int V>
__device__ __forceinline__ void unpack_acc(const Pack<T, V>& p, Acc<V>& f) {
    if constexpr (V == 1) f.v[0] = make_float2(to_f<T>(p.v[0]), 0.f);
    else unpack_pairs<T, V>(p, f.v);
}

// Statistics of one chunk of rows, per group.  A thread adds up deviations per channel from the mean of
// its first rows, so neither a large offset nor an outlier (which moves that mean by a quarter) costs
// accuracy; threads, warps, channels and chunks are merged as (mean, squared deviations).
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 4) k_norm_partial(const NormArgs a) {
    constexpr int H = Acc<V>::H;
    ptx::grid_dep_wait();
    const Place p = place<V>(a, blockIdx.x);
    const int n = valid_rows(a, p.b);
    const int r0 = min(p.ch * a.rows, n), r1 = min(r0 + a.rows, n);
    const T* x = static_cast<const T*>(a.x) + p.b * a.xb + p.c + (long long)(r0 + p.ty) * a.xr;
    const long long step = (long long)p.TY * a.xr;
    const int mine = p.live && r1 - r0 > p.ty ? (r1 - r0 - p.ty + p.TY - 1) / p.TY : 0;
    Acc<V> sh, s, q;
#pragma unroll
    for (int i = 0; i < H; ++i) sh.v[i] = s.v[i] = q.v[i] = make_float2(0.f, 0.f);
    auto add = [&](const Pack<T, V>& in) {
        Acc<V> f;
        unpack_acc<T, V>(in, f);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 d = __fadd2_rn(f.v[i], sh.v[i]);
            s.v[i] = __fadd2_rn(s.v[i], d);
            q.v[i] = __ffma2_rn(d, d, q.v[i]);
        }
    };
    constexpr size_t kMerge = sizeof(Stat) * (kThreads / 32) * 32 * V + 4 * kThreads;
    __shared__ __align__(16) unsigned char smem[Stream<T, V, 1>::kSmem > kMerge ? Stream<T, V, 1>::kSmem : kMerge];
    Stream<T, V, 1> rows;
    rows.at[0] = x;
    rows.step[0] = step;
    rows.start(smem, mine);
    const int m = rows.peek([&](const Pack<T, V>& in) {
        Acc<V> f;
        unpack_acc<T, V>(in, f);
#pragma unroll
        for (int i = 0; i < H; ++i) sh.v[i] = __fadd2_rn(sh.v[i], f.v[i]);
    });
    if (m > 0) {
        const float f = -1.0f / m;
#pragma unroll
        for (int i = 0; i < H; ++i) sh.v[i] = __fmul2_rn(sh.v[i], make_float2(f, f));
    }
    rows.run([&](const Pack<T, V>(&in)[1]) { add(in[0]); });
    __syncthreads();  // the rows' slots are used again below
    float cnt = (float)mine;
    Stat st[V];
    {
        const float ic = mine > 0 ? 1.0f / cnt : 0.f;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            st[V == 1 ? 0 : 2 * i] = Stat{-sh.v[i].x, s.v[i].x * ic, q.v[i].x - s.v[i].x * s.v[i].x * ic};
            if constexpr (V > 1) st[2 * i + 1] = Stat{-sh.v[i].y, s.v[i].y * ic, q.v[i].y - s.v[i].y * s.v[i].y * ic};
        }
    }
    // lanes of a warp that share the channels
    for (int off = 16; off >= a.tx; off >>= 1) {
        const float nb = __shfl_xor_sync(0xffffffffu, cnt, off);
        const float f = nb > 0.f ? nb / (cnt + nb) : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Stat o;
            o.hi = __shfl_xor_sync(0xffffffffu, st[i].hi, off);
            o.lo = __shfl_xor_sync(0xffffffffu, st[i].lo, off);
            o.m2 = __shfl_xor_sync(0xffffffffu, st[i].m2, off);
            merge_stats(st[i], cnt, o, f);
        }
        cnt += nb;
    }
    Stat(*sm)[32 * V] = reinterpret_cast<Stat(*)[32 * V]>(smem);
    float(*sn)[32] = reinterpret_cast<float(*)[32]>(smem + sizeof(Stat) * (kThreads / 32) * 32 * V);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    sn[warp][lane] = cnt;
#pragma unroll
    for (int i = 0; i < V; ++i) sm[warp][lane * V + i] = st[i];
    __syncthreads();
    if (warp == 0 && lane < a.tx && p.live) {
        for (int w = 1; w < kThreads / 32; ++w) {
            const float nb = sn[w][lane];
            const float f = nb > 0.f ? nb / (cnt + nb) : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) merge_stats(st[i], cnt, sm[w][lane * V + i], f);
            cnt += nb;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sm[0][lane * V + i] = st[i];
    }
    __syncthreads();
    // The tile's channels of each group it meets.  A group that two tiles share has an entry in each:
    // entry g + tile, since the next tile begins with this tile's last group or the one after.
    const int wide = a.tx * V, tile = blockIdx.x / a.chunks % a.ctiles;
    const int c0 = tile * wide, c1 = min(a.C, c0 + wide);
    const double n_rows = r1 - r0;
    float4* out = reinterpret_cast<float4*>(a.ws) + ((long long)p.b * a.chunks + p.ch) * (a.G + a.ctiles) + tile;
    const int g0 = c0 / a.D, g1 = (c1 - 1) / a.D;
    // sums about the first channel's mean, in fp64: no second pass, and nothing to lose but its distance
    // from the group's mean, squared, in 53 bits
    auto add_channel = [&](const Stat& v, const Stat& ref, double& s0, double& q0) {
        const double d = (double)(v.hi - ref.hi) + (double)(v.lo - ref.lo);
        s0 += d;
        q0 += fma(d * n_rows, d, (double)v.m2);
    };
    auto put = [&](int g, const Stat& ref, double s0, double q0, int channels) {
        const double d = s0 / channels, mean = (double)ref.hi + (double)ref.lo + d;
        const float hi = (float)mean;
        out[g] = make_float4(hi, (float)(mean - hi), (float)(q0 - n_rows * s0 * d), (float)(n_rows * channels));
    };
    if (a.D <= 32) {  // a thread a group
        for (int g = g0 + threadIdx.x; g <= g1; g += kThreads) {
            const int first = max(g * a.D, c0), last = min((g + 1) * a.D, c1);
            const Stat ref = sm[0][first - c0];
            double s0 = 0.0, q0 = 0.0;
            for (int c = first; c < last; ++c) add_channel(sm[0][c - c0], ref, s0, q0);
            put(g, ref, s0, q0, last - first);
        }
    } else {  // a warp a group
        for (int g = g0 + warp; g <= g1; g += kThreads / 32) {
            const int first = max(g * a.D, c0), last = min((g + 1) * a.D, c1);
            const Stat ref = sm[0][first - c0];
            double s0 = 0.0, q0 = 0.0;
            for (int c = first + lane; c < last; c += 32) add_channel(sm[0][c - c0], ref, s0, q0);
            s0 = warp_sum(s0);
            q0 = warp_sum(q0);
            if (lane == 0) put(g, ref, s0, q0, last - first);
        }
    }
}

constexpr int kStatThreads = 128;

// mean and rstd of one (item, group) from the entries of its chunks and channel tiles (of `wide`
// channels), in fp64.  `tx` threads (a power of two) stand along the tiles, the others along the chunks.
__global__ void __launch_bounds__(kStatThreads) k_norm_stats(const NormArgs a, int wide, int tx) {
    ptx::grid_dep_wait();
    __shared__ double sh[2][kStatThreads / 32];
    const int b = blockIdx.x / a.G, g = blockIdx.x % a.G;
    const int n = valid_rows(a, b);
    const float4* part = reinterpret_cast<const float4*>(a.ws) + (long long)b * a.chunks * (a.G + a.ctiles) + g;
    const int used = (n + a.rows - 1) / a.rows;
    const int t0 = (int)((long long)g * a.D / wide), t1 = (int)((((long long)g + 1) * a.D - 1) / wide);
    const long long step = a.G + a.ctiles;
    const int lx = threadIdx.x & (tx - 1), ly = threadIdx.x / tx, ny = kStatThreads / tx;
    // about the first entry's mean, as in k_norm_partial
    const float4 first = n > 0 ? part[t0] : make_float4(0.f, 0.f, 0.f, 0.f);
    const double ref = (double)first.x + (double)first.y;
    double s = 0, q = 0;
    for (int t = t0 + lx; t <= t1; t += tx) {
#pragma unroll 4
        for (int ch = ly; ch < used; ch += ny) {
            const float4 v = part[ch * step + t];
            const double d = (double)v.x + (double)v.y - ref;
            s += d * v.w;
            q += fma(d * v.w, d, (double)v.z);
        }
    }
    s = warp_sum(s);
    q = warp_sum(q);
    if ((threadIdx.x & 31) == 0) {
        sh[0][threadIdx.x >> 5] = s;
        sh[1][threadIdx.x >> 5] = q;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kStatThreads / 32; ++w) {
            s += sh[0][w];
            q += sh[1][w];
        }
        const double inv = n > 0 ? 1.0 / ((double)n * a.D) : 0.0, d = s * inv;
        const double var = q * inv - d * d;
        a.mean[blockIdx.x] = (float)(ref + d);
        a.rstd[blockIdx.x] = 1.0f / sqrtf((float)((var > 0.0 ? var : var == var ? 0.0 : var) + (double)a.eps));
    }
}

// y = act((x - mean) rstd w + b), zeros behind the valid rows.  Blocks go through the tensor from its
// end: what the statistics pass read last is still in L2.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 4) k_norm_apply(const NormArgs a) {
    constexpr bool kPrecise = sizeof(T) == 4, kSnake = ACT == MH3A_ACT_SNAKE_BETA;
    constexpr int H = Acc<V>::H;
    ptx::grid_dep_wait();
    const Place p = place<V>(a, gridDim.x - 1 - blockIdx.x);
    if (!p.live) return;
    const int n = valid_rows(a, p.b);
    const int r0 = min(p.ch * a.rows, a.T), r1 = min(r0 + a.rows, a.T);
    float mu[2 * H], sc[2 * H], bi[2 * H], al[2 * H], ib[2 * H];
#pragma unroll
    for (int i = 0; i < 2 * H; ++i) {
        const int c = min(p.c + i, a.C - 1), g = p.b * a.G + c / a.D;
        mu[i] = -a.mean[g];
        sc[i] = a.rstd[g] * (a.weight ? __ldg(a.weight + c) : 1.f);
        bi[i] = a.bias ? __ldg(a.bias + c) : 0.f;
        al[i] = kSnake ? __ldg(a.alpha + c) : 0.f;
        ib[i] = kSnake ? rcp_ftz(__ldg(a.beta + c) + 1e-9f) : 0.f;
    }
    const T* x = static_cast<const T*>(a.x) + p.b * a.xb + p.c + (long long)(r0 + p.ty) * a.xr;
    T* y = static_cast<T*>(a.out) + ((long long)p.b * a.T + r0 + p.ty) * a.C + p.c;
    const long long xs = (long long)p.TY * a.xr, ys = (long long)p.TY * a.C;
    const int top = min(n, r1) - r0;
    const int mine = top > p.ty ? (top - p.ty + p.TY - 1) / p.TY : 0;
    auto put = [&](const Pack<T, V>& in, T* to) {
        Acc<V> f;
        unpack_acc<T, V>(in, f);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 u = __ffma2_rn(__fadd2_rn(f.v[i], make_float2(mu[2 * i], mu[2 * i + 1])), make_float2(sc[2 * i], sc[2 * i + 1]),
                                        make_float2(bi[2 * i], bi[2 * i + 1]));
            f.v[i] = act_fwd<ACT, kPrecise>(u, make_float2(al[2 * i], al[2 * i + 1]), make_float2(ib[2 * i], ib[2 * i + 1]));
        }
        if constexpr (V == 1) *to = from_f<T>(f.v[0].x);
        else store_pairs<T, V>(to, f.v);
    };
    __shared__ __align__(16) unsigned char smem[Stream<T, V, 1>::kSmem];
    Stream<T, V, 1> rows;
    rows.at[0] = x;
    rows.step[0] = xs;
    rows.start(smem, mine);
    rows.run([&](const Pack<T, V>(&in)[1]) {
        put(in[0], y);
        y += ys;
    });
    int k = mine;
    const Pack<T, V> zero{};
    for (; p.ty + k * p.TY < r1 - r0; ++k, y += ys) *reinterpret_cast<Pack<T, V>*>(y) = zero;
}

// --------------------------------------------------------------------------------- backward

// The per-channel parameters of a thread, as pairs.
template <int V, int ACT>
struct BwdParams {
    static constexpr int H = Acc<V>::H;
    float2 mu[H], rs[H], w[H], bi[H], al[H], ib[H];

    __device__ __forceinline__ void load(const NormArgs& a, int b, int c0) {
        float* f[6] = {&mu[0].x, &rs[0].x, &w[0].x, &bi[0].x, &al[0].x, &ib[0].x};
#pragma unroll
        for (int i = 0; i < 2 * H; ++i) {
            const int c = min(c0 + i, a.C - 1);
            const long long g = (long long)b * a.G + c / a.D;
            f[0][i] = -a.mean[g];
            f[1][i] = a.rstd[g];
            f[2][i] = a.weight ? __ldg(a.weight + c) : 1.f;
            f[3][i] = a.bias ? __ldg(a.bias + c) : 0.f;
            if (ACT == MH3A_ACT_SNAKE_BETA) {
                f[4][i] = __ldg(a.alpha + c);
                f[5][i] = rcp_ftz(__ldg(a.beta + c) + 1e-9f);
            }
        }
    }
    __device__ __forceinline__ float2 xhat(float2 x, int i) const { return __fmul2_rn(__fadd2_rn(x, mu[i]), rs[i]); }
    template <bool PRECISE>
    __device__ __forceinline__ float2 slope(float2 xh, int i, float2* pa, float2* pb) const {
        constexpr bool kSnake = ACT == MH3A_ACT_SNAKE_BETA;
        const float2 u = __ffma2_rn(xh, w[i], bi[i]);
        return act_slope<ACT, PRECISE>(u, kSnake ? al[i] : u, kSnake ? ib[i] : u, pa, pb);
    }
};

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 2) k_norm_bwd_partial(const NormArgs a) {
    constexpr bool kPrecise = sizeof(T) == 4;
    constexpr int NS = kSums<ACT>, H = Acc<V>::H;
    ptx::grid_dep_wait();
    const Place p = place<V>(a, blockIdx.x);
    const int n = valid_rows(a, p.b);
    const int r0 = min(p.ch * a.rows, n), r1 = min(r0 + a.rows, n);
    constexpr size_t kMerge = sizeof(float) * (kThreads / 32) * 32 * V * NS;
    __shared__ __align__(16) unsigned char smem[Stream<T, V, 2>::kSmem > kMerge ? Stream<T, V, 2>::kSmem : kMerge];
    float2 acc[NS][H];
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int i = 0; i < H; ++i) acc[j][i] = make_float2(0.f, 0.f);
    if (p.live) {
        BwdParams<V, ACT> prm;
        prm.load(a, p.b, p.c);
        const T* x = static_cast<const T*>(a.x) + p.b * a.xb + p.c + (long long)(r0 + p.ty) * a.xr;
        const T* dy = static_cast<const T*>(a.dy) + p.b * a.gb + p.c + (long long)(r0 + p.ty) * a.gr;
        const long long xs = (long long)p.TY * a.xr, gs = (long long)p.TY * a.gr;
        const int mine = r1 - r0 > p.ty ? (r1 - r0 - p.ty + p.TY - 1) / p.TY : 0;
        auto add = [&](const Pack<T, V>& in, const Pack<T, V>& gr) {
            Acc<V> f, g;
            unpack_acc<T, V>(in, f);
            unpack_acc<T, V>(gr, g);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 xh = prm.xhat(f.v[i], i);
                float2 pa, pb;
                const float2 du = __fmul2_rn(g.v[i], prm.template slope<kPrecise>(xh, i, &pa, &pb));
                acc[0][i] = __fadd2_rn(acc[0][i], du);
                acc[1][i] = __ffma2_rn(du, xh, acc[1][i]);
                if constexpr (NS == 4) {
                    acc[2][i] = __ffma2_rn(g.v[i], pa, acc[2][i]);
                    acc[3][i] = __ffma2_rn(g.v[i], pb, acc[3][i]);
                }
            }
        };
        Stream<T, V, 2> rows;
        rows.at[0] = x;
        rows.at[1] = dy;
        rows.step[0] = xs;
        rows.step[1] = gs;
        rows.start(smem, mine);
        rows.run([&](const Pack<T, V>(&in)[2]) { add(in[0], in[1]); });
    }
    __syncthreads();  // the rows' slots are used again below
    for (int off = 16; off >= a.tx; off >>= 1) {
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int i = 0; i < H; ++i) {
                acc[j][i].x += __shfl_xor_sync(0xffffffffu, acc[j][i].x, off);
                acc[j][i].y += __shfl_xor_sync(0xffffffffu, acc[j][i].y, off);
            }
    }
    float(*sm)[32 * V * NS] = reinterpret_cast<float(*)[32 * V * NS]>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto part = [&](int i, int j) { return V == 1 || i % 2 == 0 ? acc[j][i / 2].x : acc[j][i / 2].y; };
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < NS; ++j) sm[warp][(i * NS + j) * 32 + lane] = part(i, j);
    __syncthreads();
    if (warp == 0 && lane < a.tx && p.live) {
        float* out = a.ws + (((long long)p.b * a.chunks + p.ch) * a.C + p.c) * NS;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                float s = 0.f;
#pragma unroll
                for (int w2 = 0; w2 < kThreads / 32; ++w2) s += sm[w2][(i * NS + j) * 32 + lane];
                out[i * NS + j] = s;
            }
    }
}

// Per (item, channel): the chunks' sums in fixed order.  32 x 8 threads, one column of sums each.
__global__ void __launch_bounds__(256) k_norm_bwd_sum(const NormArgs a, float* sums, int ns, int tiles) {
    ptx::grid_dep_wait();
    __shared__ double sh[8][33];
    const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const long long width = (long long)a.C * ns, j = (long long)tile * 32 + lane;
    const int n = valid_rows(a, b);
    const int used = (n + a.rows - 1) / a.rows;
    double s = 0;
    if (j < width) {
        const float* from = a.ws + (long long)b * a.chunks * width + j;
#pragma unroll 8
        for (int ch = row; ch < used; ch += 8) s += from[ch * width];
    }
    sh[row][lane] = s;
    __syncthreads();
    if (row == 0 && j < width) {
        for (int r = 1; r < 8; ++r) s += sh[r][lane];
        sums[b * width + j] = (float)s;
    }
}

// The first `group_blocks` blocks: the two group means of dx, a warp an (item, group).  Blocks behind
// them: parameter gradients, the items' sums in fixed order, 32 x 8 threads, one column of sums each.
__global__ void __launch_bounds__(256) k_norm_bwd_final(const NormArgs a, const float* sums, float2* means, int ns,
                                                        int group_blocks) {
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    if ((int)blockIdx.x < group_blocks) {
        const long long bg = (long long)blockIdx.x * 8 + row;
        if (bg >= (long long)a.B * a.G) return;
        const int b = (int)(bg / a.G), g = (int)(bg % a.G);
        double s1 = 0, s2 = 0;
#pragma unroll 4
        for (int c = lane; c < a.D; c += 32) {
            const long long ch = (long long)g * a.D + c;
            const double w = a.weight ? (double)__ldg(a.weight + ch) : 1.0;
            const float* s = sums + ((long long)b * a.C + ch) * ns;
            s1 += w * s[0];
            s2 += w * s[1];
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (lane == 0) {
            const int n = valid_rows(a, b);
            const double inv = n > 0 ? 1.0 / ((double)n * a.D) : 0.0;
            means[bg] = make_float2((float)(s1 * inv), (float)(s2 * inv));
        }
        return;
    }
    __shared__ double sh[8][33];
    const long long width = (long long)a.C * ns, j = (long long)(blockIdx.x - group_blocks) * 32 + lane;
    double s = 0;
    if (j < width) {
#pragma unroll 4
        for (int b = row; b < a.B; b += 8) s += sums[b * width + j];
    }
    sh[row][lane] = s;
    __syncthreads();
    if (row != 0 || j >= width) return;
    for (int r = 1; r < 8; ++r) s += sh[r][lane];
    const int c = (int)(j / ns), k = (int)(j % ns);
    float* const out = k == 0 ? a.dbias : k == 1 ? a.dweight : k == 2 ? a.dalpha : a.dbeta;
    if (!out) return;
    if (k == 3) {
        const double ib = 1.0 / (double)(a.beta[c] + 1e-9f);
        s = -s * ib * ib;
    }
    out[c] = (float)s;
}

// dx, from the tensor's end as in k_norm_apply.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 3) k_norm_bwd_apply(const NormArgs a, const float2* means) {
    constexpr bool kPrecise = sizeof(T) == 4;
    constexpr int H = Acc<V>::H;
    ptx::grid_dep_wait();
    const Place p = place<V>(a, gridDim.x - 1 - blockIdx.x);
    if (!p.live) return;
    const int n = valid_rows(a, p.b);
    const int r0 = min(p.ch * a.rows, a.T), r1 = min(r0 + a.rows, a.T);
    BwdParams<V, ACT> prm;
    prm.load(a, p.b, p.c);
    float2 m1[H], m2[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const float2 f = means[(long long)p.b * a.G + min(p.c + 2 * i, a.C - 1) / a.D];
        const float2 h = means[(long long)p.b * a.G + min(p.c + 2 * i + 1, a.C - 1) / a.D];
        m1[i] = make_float2(-f.x, -h.x);
        m2[i] = make_float2(-f.y, -h.y);
    }
    const T* x = static_cast<const T*>(a.x) + p.b * a.xb + p.c + (long long)(r0 + p.ty) * a.xr;
    const T* dy = static_cast<const T*>(a.dy) + p.b * a.gb + p.c + (long long)(r0 + p.ty) * a.gr;
    T* dx = static_cast<T*>(a.out) + ((long long)p.b * a.T + r0 + p.ty) * a.C + p.c;
    const long long xs = (long long)p.TY * a.xr, gs = (long long)p.TY * a.gr, os = (long long)p.TY * a.C;
    const int top = min(n, r1) - r0;
    const int mine = top > p.ty ? (top - p.ty + p.TY - 1) / p.TY : 0;
    auto put = [&](const Pack<T, V>& in, const Pack<T, V>& gr, T* to) {
        Acc<V> f, g;
        unpack_acc<T, V>(in, f);
        unpack_acc<T, V>(gr, g);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 xh = prm.xhat(f.v[i], i);
            float2 pa, pb;
            const float2 du = __fmul2_rn(g.v[i], prm.template slope<kPrecise>(xh, i, &pa, &pb));
            f.v[i] = __fmul2_rn(prm.rs[i], __ffma2_rn(xh, m2[i], __ffma2_rn(du, prm.w[i], m1[i])));
        }
        if constexpr (V == 1) *to = from_f<T>(f.v[0].x);
        else store_pairs<T, V>(to, f.v);
    };
    __shared__ __align__(16) unsigned char smem[Stream<T, V, 2>::kSmem];
    Stream<T, V, 2> rows;
    rows.at[0] = x;
    rows.at[1] = dy;
    rows.step[0] = xs;
    rows.step[1] = gs;
    rows.start(smem, mine);
    rows.run([&](const Pack<T, V>(&in)[2]) {
        put(in[0], in[1], dx);
        dx += os;
    });
    int k = mine;
    const Pack<T, V> zero{};
    for (; p.ty + k * p.TY < r1 - r0; ++k, dx += os) *reinterpret_cast<Pack<T, V>*>(dx) = zero;
}

// ------------------------------------------------------------------------------------- host
// Blocks for each SM, and the most rows of a thread.
struct Split {
    int per_sm, most_rows;
};
constexpr Split kFwdSplit{4, 80}, kBwdSplit{8, 128};

int pow2_ceil(long long n, int most) {
    int p = 1;
    while (p < n && p < most) p <<= 1;
    return p;
}

// Threads, channel tiles and row chunks for vectors of V channels.  Chunks are as many as give every
// SM `per_sm` blocks, but of 4 to `most_rows` rows a thread.  The upper end bounds what rounding does to a
// thread's fp32 sums: with outliers of 10^5 deviations among a thread's first rows, rstd is off by 18
// units of 2^-24 at most with 80 rows, 43 with 128, 8000 with 1250 (100 fp32 items of [20000, 256]).  Short
// chunks also even out the last round of blocks: there forward 1021 us with 80 rows, 1042 with 128, 1225 with
// no bound; backward (plain sums) bf16 [1200, 8000, 256] 3829 with 64, 3662 with 128, 3740 with no bound.
// Blocks for each SM, measured on sixteen 20 s items (256 channels, bf16): forward 100 us with 4, 106 with 8, 110 with 12; backward with unequal lengths, where blocks
// behind an item's end have nothing to do, 117, 112 and 115.
void plan_general(NormArgs* a, int V, Split split) {
    const long long cvecs = ((long long)a->C + V - 1) / V;
    a->tx = pow2_ceil(cvecs, 32);
    a->ctiles = (int)((cvecs + a->tx - 1) / a->tx);
    const int ty = kThreads / a->tx;
    const long long want = std::max<long long>(1, (long long)split.per_sm * kSms / std::max<long long>(1, (long long)a->ctiles * a->B));
    const long long most = std::max<long long>(1, ((long long)a->T + 4 * ty - 1) / (4 * ty));
    const long long least = ((long long)a->T + split.most_rows * ty - 1) / (split.most_rows * ty);
    a->chunks = (int)std::max(std::min(want, most), least);
    a->rows = (a->T + a->chunks - 1) / a->chunks;
    a->chunks = (a->T + a->rows - 1) / a->rows;
}

long long grid_general(const NormArgs& a) { return (long long)a.B * a.ctiles * a.chunks; }

template <typename F, typename... Args>
bool go(F kern, long long grid, int threads, cudaStream_t s, Args... args) {
    return launch_dependent(kern, dim3((unsigned)grid), dim3(threads), 0, s, args...) == cudaSuccess;
}

// Shared memory of a resident block: two blocks an SM where the slab allows, else one.
constexpr int kResTwo = 112 * 1024, kResOne = 224 * 1024;
// Larger tensors take the general form: a cluster's slab is a 64- or 128-byte piece of every row, and
// once clusters drift apart the pieces of a row reach DRAM at different times.  Measured (bf16, forward,
// T = 10000, C = 256): 41 MB 27 us against 33 us in the general form, 164 MB (T = 20000) 101 against 100;
// backward (x and dy) 82 MB 62 against 82 us, 164 MB 145 against 125.
constexpr long long kResMax = 100000000LL;

// The largest cluster (16, 8, 4, 2 or 1 blocks, each with an SM's shared memory to itself) that a device can
// place; 0: not asked yet.  A whole B200 places 16; a process that is given only some of its SMs may not.
std::atomic<int> cluster_limits[64];

// That of the current device, asked once; 16 where there is none, since sizes may be asked for without one.
int cluster_limit() {
    int dev = 0;
    const bool there = cudaGetDevice(&dev) == cudaSuccess;
    std::atomic<int>& known = cluster_limits[there ? dev & 63 : 0];
    int n = known.load(std::memory_order_relaxed);
    if (n) return n;
    if (!there) {
        cudaGetLastError();
        return 16;
    }
    constexpr auto kern = k_norm_bwd_resident<float, 4, MH3A_ACT_SNAKE_BETA, true>;  // all take the same shared memory
    for (n = allow_smem<kern>(kResOne, true) ? 16 : 1; n > 1; n /= 2) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(n);
        cfg.blockDim = dim3(kResThreads);
        cfg.dynamicSmemBytes = kResOne;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = n;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess) cudaGetLastError();  // no error of the call
        else if (clusters > 0) break;
    }
    known.store(n, std::memory_order_relaxed);
    return n;
}

FastDiv fast_div(unsigned d) { return FastDiv{d, (unsigned)(((1ull << 32) + d - 1) / d)}; }

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Divides a tensor for the resident form; false where it does not serve.  Slabs are whole groups and
// whole vectors.  `bytes_row` are kept per channel and row (x, or x and dy), `extra(W, S)` beside.
template <typename Extra>
bool plan_resident(const NormArgs& a, int V, int e, int bytes_row, Extra extra, Resident* r) {
    const long long unit_l = (long long)a.D / gcd(a.D, V) * V;
    if (unit_l > kResThreads * V || a.B > 65535 || (long long)a.B * a.C * a.T > kResMax / bytes_row) return false;
    const int unit = (int)unit_l, units = a.C / unit, most = kResThreads * V / unit, blocks = cluster_limit();
    for (int limit : {kResTwo, kResOne}) {
        for (int want : {128, 64}) {
            int k = 1;
            while (k < units && k <= most && (units % k || k * unit * e < want)) ++k;
            if (k > most) continue;  // wider than a row of threads
            const int W = k * unit;
            const int slabs = a.C / W;
            if (slabs > 65535) continue;
            // narrower slabs while whole clusters of wide ones would leave SMs idle
            if (want == 128 && k > 1 && (long long)a.B * slabs * 8 < 2 * kSms && a.T >= 128) continue;
            auto bytes = [&](int s) { return (long long)((a.T + s - 1) / s) * W * bytes_row + extra(W, s); };
            int S = 1;
            while (S < blocks && bytes(S) > limit) S *= 2;
            if (bytes(S) > limit) continue;
            while (S < std::min(8, blocks) && (long long)a.B * slabs * S * 2 <= 2 * kSms && (a.T + 2 * S - 1) / (2 * S) >= 16) S *= 2;
            *r = Resident{S, (a.T + S - 1) / S, W, slabs, (int)bytes(S), fast_div(kResThreads / (W / V)),
                          fast_div(W / V), fast_div(a.D), fast_div(a.D % V ? a.D : a.D / V)};
            return true;
        }
    }
    return false;
}

template <auto Kern>
bool go_resident(const NormArgs& a, const Resident& r, cudaStream_t s) {
    if (!allow_smem<Kern>(kResOne, true)) return false;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(r.S, r.slabs, a.B);
    cfg.blockDim = dim3(kResThreads);
    cfg.dynamicSmemBytes = r.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = r.S;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, Kern, a, r) == cudaSuccess;
}

// Vectors of the general form.  Backward takes 8 bytes at most of 16-bit types: twice as many channels'
// sums and parameters would halve the blocks an SM holds.
int general_width(int V, int backward) { return backward ? std::min(V, 4) : V; }

// Scratch of the general form with vectors of V channels.
size_t general_bytes(NormArgs a, int act, int backward, int V) {
    plan_general(&a, V, backward ? kBwdSplit : kFwdSplit);
    const long long ns = act == MH3A_ACT_SNAKE_BETA ? 4 : 2;
    long long floats = (long long)a.B * a.chunks * (backward ? a.C * ns : (a.G + a.ctiles) * 4LL);
    if (backward) floats += ((long long)a.B * a.C * ns + 3) / 4 * 4 + 2LL * a.B * a.G;
    return ((size_t)floats * 4 + 255) / 256 * 256;
}

// The way a call goes, by its sizes, the vectors of V channels that its pointers and strides allow, and
// whether the parameters are aligned to 16 bytes.
struct Way {
    bool resident;
    Resident r;
    size_t bytes;  // scratch
};

template <typename T>
Way way(const NormArgs& a, int act, int backward, int V, bool params) {
    Way w{};
    const int ns = act == MH3A_ACT_SNAKE_BETA ? 4 : 2;
    auto extra = [&](int W, int S) { return backward ? res_bwd_extra(W, a.D, V, S, ns) : res_fwd_extra(W, a.D, V, S); };
    w.resident = V == 16 / (int)sizeof(T) && params && plan_resident(a, V, sizeof(T), (backward ? 2 : 1) * sizeof(T), extra, &w.r);
    if (w.resident) w.bytes = backward && a.B > 1 ? ((size_t)a.B * a.C * ns * 4 + 255) / 256 * 256 : 0;
    else w.bytes = general_bytes(a, act, backward, general_width(V, backward));
    return w;
}

Way way(const NormArgs& a, int dtype, int act, int backward, int V, bool params) {
    switch (dtype) {
        case MH3A_DTYPE_F32: return way<float>(a, act, backward, V, params);
        case MH3A_DTYPE_F16: return way<__half>(a, act, backward, V, params);
        default: return way<__nv_bfloat16>(a, act, backward, V, params);
    }
}

bool scratch_ok(const void* workspace, size_t have, size_t need) {
    return need == 0 || (workspace && aligned(workspace, 16) && have >= need);
}

template <typename T, int V, int ACT>
bool forward_resident(const NormArgs& a, const Resident& r, cudaStream_t s) {
    return a.D % V == 0 ? go_resident<k_norm_resident<T, V, ACT, true>>(a, r, s)
                        : go_resident<k_norm_resident<T, V, ACT, false>>(a, r, s);
}

template <typename T, int V>
bool forward_general(const NormArgs& a, int act, cudaStream_t s) {
    const long long grid = grid_general(a);
    if (!go(k_norm_partial<T, V>, grid, kThreads, s, a)) return false;
    if (!go(k_norm_stats, (long long)a.B * a.G, kStatThreads, s, a, a.tx * V, pow2_ceil(a.tx * V % a.D ? (a.D - 1) / (a.tx * V) + 2 : 1, kStatThreads))) return false;
    switch (act) {
        case MH3A_ACT_SILU: return go(k_norm_apply<T, V, MH3A_ACT_SILU>, grid, kThreads, s, a);
        case MH3A_ACT_SNAKE_BETA: return go(k_norm_apply<T, V, MH3A_ACT_SNAKE_BETA>, grid, kThreads, s, a);
        default: return go(k_norm_apply<T, V, MH3A_ACT_NONE>, grid, kThreads, s, a);
    }
}

template <typename T>
bool forward(NormArgs& a, const Way& w, int act, int width, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (w.resident) {
        switch (act) {
            case MH3A_ACT_SILU: return forward_resident<T, V, MH3A_ACT_SILU>(a, w.r, s);
            case MH3A_ACT_SNAKE_BETA: return forward_resident<T, V, MH3A_ACT_SNAKE_BETA>(a, w.r, s);
            default: return forward_resident<T, V, MH3A_ACT_NONE>(a, w.r, s);
        }
    }
    plan_general(&a, general_width(width, 0), kFwdSplit);
    if constexpr (V == 8) {
        if (width == 8) return forward_general<T, 8>(a, act, s);
    }
    if (width == 4) return forward_general<T, 4>(a, act, s);
    return width == 2 ? forward_general<T, 2>(a, act, s) : forward_general<T, 1>(a, act, s);
}

template <typename T, int V, int ACT>
bool backward_general(const NormArgs& a, cudaStream_t s) {
    constexpr int NS = kSums<ACT>;
    const long long grid = grid_general(a);
    float* sums = a.ws + (long long)a.B * a.chunks * a.C * NS;
    float2* means = reinterpret_cast<float2*>(sums + ((long long)a.B * a.C * NS + 3) / 4 * 4);
    if (!go(k_norm_bwd_partial<T, V, ACT>, grid, kThreads, s, a)) return false;
    const int tiles = (int)(((long long)a.C * NS + 31) / 32);
    if (!go(k_norm_bwd_sum, (long long)a.B * tiles, 256, s, a, sums, NS, tiles)) return false;
    const int gblocks = (int)(((long long)a.B * a.G + 7) / 8);
    if (!go(k_norm_bwd_final, gblocks + tiles, 256, s, a, (const float*)sums, means, NS, gblocks)) return false;
    return go(k_norm_bwd_apply<T, V, ACT>, grid, kThreads, s, a, (const float2*)means);
}

template <typename T, int ACT>
bool backward_act(NormArgs& a, const Way& w, int width, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T), NS = kSums<ACT>;
    if (w.resident) {
        const bool ok = a.D % V == 0 ? go_resident<k_norm_bwd_resident<T, V, ACT, true>>(a, w.r, s)
                                     : go_resident<k_norm_bwd_resident<T, V, ACT, false>>(a, w.r, s);
        if (!ok || a.B == 1) return ok;
        return go(k_norm_bwd_final, ((long long)a.C * NS + 31) / 32, 256, s, a, (const float*)a.ws, (float2*)nullptr, NS, 0);
    }
    width = general_width(width, 1);
    plan_general(&a, width, kBwdSplit);
    if (width == 4) return backward_general<T, 4, ACT>(a, s);
    return width == 2 ? backward_general<T, 2, ACT>(a, s) : backward_general<T, 1, ACT>(a, s);
}

template <typename T>
bool backward(NormArgs& a, const Way& w, int act, int width, cudaStream_t s) {
    switch (act) {
        case MH3A_ACT_SILU: return backward_act<T, MH3A_ACT_SILU>(a, w, width, s);
        case MH3A_ACT_SNAKE_BETA: return backward_act<T, MH3A_ACT_SNAKE_BETA>(a, w, width, s);
        default: return backward_act<T, MH3A_ACT_NONE>(a, w, width, s);
    }
}

int elem_bytes(int dtype) { return dtype == MH3A_DTYPE_F32 ? 4 : 2; }

mh3a_status check(const mh3a_norm* p) {
    if (!p) return MH3A_ERR_INVALID_ARG;
    if (p->dtype < MH3A_DTYPE_F32 || p->dtype > MH3A_DTYPE_BF16) return MH3A_ERR_INVALID_ARG;
    if (p->act < MH3A_ACT_NONE || p->act > MH3A_ACT_SNAKE_BETA) return MH3A_ERR_INVALID_ARG;
    if (p->B < 1 || p->T < 1 || p->C < 1 || p->groups < 1 || p->C % p->groups) return MH3A_ERR_SHAPE;
    if (p->act == MH3A_ACT_SNAKE_BETA && (!p->alpha || !p->beta)) return MH3A_ERR_INVALID_ARG;
    // In 32 bits stay: row indices plus a block's stride; channels and groups plus a tile's width or a block's
    // threads, and the entries of a chunk (groups and channel tiles); grids, at most one block per item and channel, or
    // for 64 x 256 values.
    if (p->T > (1 << 30) || (long long)p->B * p->C >= (1LL << 30) || (long long)p->B * p->C * p->T >= (1LL << 40))
        return MH3A_ERR_SHAPE;
    return MH3A_OK;
}

NormArgs base_args(const mh3a_norm* p) {
    NormArgs a{};
    a.weight = p->weight;
    a.bias = p->bias;
    a.alpha = p->alpha;
    a.beta = p->beta;
    a.lengths = p->lengths;
    a.B = p->B;
    a.T = p->T;
    a.C = p->C;
    a.G = p->groups;
    a.D = p->C / p->groups;
    a.eps = p->eps;
    return a;
}

bool params_fit(const NormArgs& a) {
    return aligned(a.weight, 16) && aligned(a.bias, 16) && aligned(a.alpha, 16) && aligned(a.beta, 16);
}

// The widest vectors (16 bytes at most) that the channels, the pointers and the strides allow.
int vector_width(const NormArgs& a, int e, std::initializer_list<const void*> pointers, std::initializer_list<long long> strides) {
    int V = 16 / e;
    auto fits = [&]() {
        if (a.C % V) return false;
        for (const void* p : pointers)
            if (!aligned(p, (size_t)V * e)) return false;
        for (long long s : strides)
            if (s % V) return false;
        return true;
    };
    while (V > 1 && !fits()) V /= 2;
    return V;
}

}  // namespace norm
}  // namespace mh3a

using namespace mh3a;
using namespace mh3a::norm;

extern "C" MH3A_API size_t mh3a_group_norm_act_workspace(const mh3a_norm* p, int backward, int aligned_all) {
    if (check(p) != MH3A_OK) return 0;
    const NormArgs a = base_args(p);
    const int e = elem_bytes(p->dtype), V = vector_width(a, e, {}, {});
    size_t most = way(a, p->dtype, p->act, backward, V, true).bytes;
    if (!aligned_all)
        for (int v = V; v >= 1; v /= 2) most = std::max(most, way(a, p->dtype, p->act, backward, v, false).bytes);
    return most;
}

extern "C" MH3A_API mh3a_status mh3a_group_norm_act(const mh3a_norm* p, const void* x, long long x_batch_stride,
                                                    long long x_row_stride, void* y, float* mean, float* rstd,
                                                    void* workspace, size_t workspace_bytes, void* stream) {
    const mh3a_status st = check(p);
    if (st != MH3A_OK) return st;
    if (!x || !y || !mean || !rstd || x_batch_stride < 0 || x_row_stride < 0) return MH3A_ERR_INVALID_ARG;
    const int e = elem_bytes(p->dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(mean, 4) || !aligned(rstd, 4)) return MH3A_ERR_INVALID_ARG;
    NormArgs a = base_args(p);
    a.x = x;
    a.xb = x_batch_stride;
    a.xr = x_row_stride;
    a.out = y;
    a.mean = mean;
    a.rstd = rstd;
    a.ws = static_cast<float*>(workspace);
    const int V = vector_width(a, e, {x, y}, {a.xb, a.xr});
    const Way w = way(a, p->dtype, p->act, 0, V, params_fit(a));
    if (!scratch_ok(workspace, workspace_bytes, w.bytes)) return MH3A_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    bool ok;
    switch (p->dtype) {
        case MH3A_DTYPE_F32: ok = forward<float>(a, w, p->act, V, s); break;
        case MH3A_DTYPE_F16: ok = forward<__half>(a, w, p->act, V, s); break;
        default: ok = forward<__nv_bfloat16>(a, w, p->act, V, s);
    }
    return ok ? MH3A_OK : launch_failed("mh3a_group_norm_act");
}

extern "C" MH3A_API mh3a_status mh3a_group_norm_act_backward(const mh3a_norm* p, const void* x, long long x_batch_stride,
                                                             long long x_row_stride, const void* dy,
                                                             long long dy_batch_stride, long long dy_row_stride,
                                                             const float* mean, const float* rstd, void* dx,
                                                             float* dweight, float* dbias, float* dalpha, float* dbeta,
                                                             void* workspace, size_t workspace_bytes, void* stream) {
    const mh3a_status st = check(p);
    if (st != MH3A_OK) return st;
    if (!x || !dy || !dx || !mean || !rstd) return MH3A_ERR_INVALID_ARG;
    if (x_batch_stride < 0 || x_row_stride < 0 || dy_batch_stride < 0 || dy_row_stride < 0) return MH3A_ERR_INVALID_ARG;
    if (p->act != MH3A_ACT_SNAKE_BETA && (dalpha || dbeta)) return MH3A_ERR_INVALID_ARG;
    const int e = elem_bytes(p->dtype);
    if (!aligned(x, e) || !aligned(dy, e) || !aligned(dx, e)) return MH3A_ERR_INVALID_ARG;
    for (const float* f : {mean, rstd, static_cast<const float*>(dweight), static_cast<const float*>(dbias),
                           static_cast<const float*>(dalpha), static_cast<const float*>(dbeta)})
        if (!aligned(f, 4)) return MH3A_ERR_INVALID_ARG;
    NormArgs a = base_args(p);
    a.x = x;
    a.xb = x_batch_stride;
    a.xr = x_row_stride;
    a.dy = dy;
    a.gb = dy_batch_stride;
    a.gr = dy_row_stride;
    a.out = dx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dweight = dweight;
    a.dbias = dbias;
    a.dalpha = dalpha;
    a.dbeta = dbeta;
    a.ws = static_cast<float*>(workspace);
    const int V = vector_width(a, e, {x, dy, dx}, {a.xb, a.xr, a.gb, a.gr});
    const Way w = way(a, p->dtype, p->act, 1, V, params_fit(a));
    if (!scratch_ok(workspace, workspace_bytes, w.bytes)) return MH3A_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    bool ok;
    switch (p->dtype) {
        case MH3A_DTYPE_F32: ok = backward<float>(a, w, p->act, V, s); break;
        case MH3A_DTYPE_F16: ok = backward<__half>(a, w, p->act, V, s); break;
        default: ok = backward<__nv_bfloat16>(a, w, p->act, V, s);
    }
    return ok ? MH3A_OK : launch_failed("mh3a_group_norm_act_backward");
}
