// ops_common.cuh -- host helpers of the handle-free operators.
#pragma once

#include <atomic>

#include "mh3a_internal.cuh"

namespace mh3a {

constexpr int kSms = 148;  // streaming multiprocessors of a B200: what the plans fill

inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// The status of an entry point whose launch failed; the CUDA error's text goes to mh3a_last_error().
inline mh3a_status launch_failed(const char* what) {
    const cudaError_t e = cudaGetLastError();
    try {
        set_last_error(std::string(what) + ": " + cudaGetErrorString(e));
    } catch (...) {  // no exception leaves the C boundary
    }
    return MH3A_ERR_CUDA;
}

// Lets Kern use `smem` bytes of dynamic shared memory (and clusters of 16) on the current device; the
// driver is asked once per kernel and device.
template <auto Kern>
bool allow_smem(int smem, bool wide_clusters = false) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return false;
    if (wide_clusters && cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return false;
    if (dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

}  // namespace mh3a
