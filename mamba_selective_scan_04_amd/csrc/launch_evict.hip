// launch_evict.hip -- launcher of the eviction from the paged cache.
#include "hybrid_launch.hpp"

namespace bdssm_host {

void launch_kv_evict(const EvictArgs &a, int64_t batch, hipStream_t st) {
    const int n = a.max_pages;
    const auto go = [&](auto threads, auto per) {
        constexpr int kThreads = decltype(threads)::value, kPer = decltype(per)::value;
        hipLaunchKernelGGL((kv_evict_kernel<kThreads, kPer>), dim3((unsigned)batch), dim3(kThreads), 0, st, a);
    };
    // As few waves as hold the row with few values each: a single wave needs no barrier,
    // but each value adds to its time (64 rows of 258 pages, one wave: 6.4 us with five
    // values a lane, 11.6 with sixteen; four waves with four 9.1).  The longest rows held
    // in registers are those of 262,144 tokens in pages of 16, with room for what is to
    // come; longer ones read their weights again for each count.  Four rows at the ends of
    // the three longest layouts, and their like beyond, us by pages:
    //   8,192: 10.7   8,193: 13.6   16,386: 20.2   20,480: 21.7   20,481: 61 to 126 by how
    //   soon a trial parts the row   37,502 (two rows): 89 to 131
    if (n <= 320) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 5>{});
    else if (n <= 1024) go(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    else if (n <= 4096) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
    else if (n <= 8192) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
    else if (n <= 20480) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 20>{});
    else go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 0>{});
}

}  // namespace bdssm_host
