// bounded_waits.cu -- the operators' waits with limits that run out.
//
// What a wait is for comes late or never here, because a thread of the test holds it back; every limit is
// milliseconds.  The kernels only use the library's own waiting code, and report what it answered.
#include "fp8_kernels.cuh"
#include "norm_resident.cuh"

using namespace mh3a;

namespace {

constexpr int kCluster = 4;

__device__ void hold(uint64_t ns) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < ns) {
    }
}

// One cluster.  Every block sends 16 bytes to every peer; block `slow` does so after 100 ms, or never.  The waits
// are given up after 1 ms.  out: [block] whether the whole block's wait succeeded, then [block][peer]
// what stands in the inbox when the block leaves.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(256) k_peers(int slow, int never, int* out) {
    __shared__ __align__(16) float4 inbox[kCluster];
    __shared__ uint64_t bar;
    const int rank = blockIdx.x, lane = threadIdx.x;
    if (lane < kCluster) inbox[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lane == 0) {
        ptx::mbar_init(&bar, 1);
        ptx::fence_mbar_init();
        ptx::mbar_arrive_expect_tx(&bar, kCluster * 16);
    }
    __syncthreads();
    norm::cluster_arrive();
    norm::cluster_wait();
    if (rank == slow && !never) hold(100000000);
    if (!(rank == slow && never) && lane < kCluster)
        norm::send16(norm::peer_smem(ptx::smem_u32(inbox + rank), lane), norm::peer_smem(ptx::smem_u32(&bar), lane),
                     make_float4(1.f + rank, 0.f, 0.f, 0.f));
    const bool arrived = __syncthreads_and(norm::wait_for_peers(&bar, 1000000));
    norm::leave_peers(arrived, &bar, 200000000);
    if (lane == 0) out[rank] = arrived;
    if (lane < kCluster) out[kCluster + rank * kCluster + lane] = (int)inbox[lane].x;
}

// The first warp waits on a barrier that the second completes after 100 ms; its even lanes would wait a second,
// its odd ones give up after a millisecond.
__global__ void __launch_bounds__(64) k_warp(int* out) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        ptx::mbar_init(&bar, 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        out[threadIdx.x] = fp8::warp_wait(&bar, 0, threadIdx.x % 2 ? 1000000 : 1000000000);
        out[32 + threadIdx.x] = fp8::warp_wait(&bar, 0);
    } else if (threadIdx.x == 32) {
        hold(100000000);
        ptx::mbar_arrive(&bar);
    }
}

}  // namespace

// `out`: device, 64 values: the lanes' answers of the wait that some of them give up, and of one after it.
extern "C" __attribute__((visibility("default"))) int run_warp(int* out) {
    k_warp<<<1, 64>>>(out);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : cudaDeviceSynchronize();
}

// `out`: device, 20 values.  The CUDA error of the launch and its end.
extern "C" __attribute__((visibility("default"))) int run_peers(int slow, int never, int* out) {
    k_peers<<<kCluster, 256>>>(slow, never, out);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : cudaDeviceSynchronize();
}
