// launch_evict.hip -- launcher of the eviction from the paged cache.
#include "hybrid_launch.hpp"

namespace bdssm_host {

void launch_kv_evict(const EvictArgs &a, int64_t batch, hipStream_t st) {
    const int n = a.max_pages;
    const auto go = [&](auto threads, auto per) {
        constexpr int kThreads = decltype(threads)::value, kPer = decltype(per)::value;
        hipLaunchKernelGGL((kv_evict_kernel<kThreads, kPer>), dim3((unsigned)batch), dim3(kThreads), 0, st, a);
    };
    if (n <= 320) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 5>{});
    else if (n <= 1024) go(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    else if (n <= 4096) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
    else if (n <= 8192) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
    else if (n <= 20480) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 20>{});
    else go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 0>{});
}

}  // namespace bdssm_host
