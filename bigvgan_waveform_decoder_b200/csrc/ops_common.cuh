// ops_common.cuh -- host helpers of the handle-free operators.
#pragma once

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

}  // namespace mh3a
