// cluster_limit.cu -- the group norm as it goes on a device that can place smaller clusters only.
#include "norm_ops.cu"

namespace mh3a {
void set_last_error(const std::string&) {}
}  // namespace mh3a

// What every device is said to place from now on; 0: each is asked.
extern "C" MH3A_API void set_cluster_limit(int n) {
    for (auto& known : mh3a::norm::cluster_limits) known = n;
}
extern "C" MH3A_API int get_cluster_limit() { return mh3a::norm::cluster_limit(); }
