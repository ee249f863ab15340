// launch_evict.hip -- launcher of the eviction from the paged cache.
#include "hybrid_launch.hpp"

namespace bdssm_host {

void launch_kv_evict(const EvictArgs &a, int64_t batch, hipStream_t st) {
    const int n = a.max_pages;
    const auto go = [&](auto threads, auto per) {
        constexpr int kThreads = decltype(threads)::value, kPer = decltype(per)::value;
        const int turns = kPer > 0 ? kPer : (n + kThreads - 1) / kThreads;
        hipLaunchKernelGGL((kv_evict_kernel<kThreads, kPer>), dim3((unsigned)batch), dim3(kThreads), (size_t)turns * (kThreads / 64) * 8, st, a);
    };
    // sixteen values a thread; a single wave, without barriers, for rows of up to 1,024
    // pages.  The longest rows held in registers are those of 262,144 tokens in pages
    // of 16, with room for what is to come.
    if (n <= 1024) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
    else if (n <= 4096) go(std::integral_constant<int, 256>{}, std::integral_constant<int, 16>{});
    else if (n <= 8192) go(std::integral_constant<int, 512>{}, std::integral_constant<int, 16>{});
    else if (n <= 20480) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 20>{});
    else go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 0>{});
}

}  // namespace bdssm_host
