// host_checks.hpp -- argument checks shared by the entry points' sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "bdssm.h"

namespace bdssm_host {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range { const void *p; size_t n; };

inline bool overlaps(Range a, Range b) {
    if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

constexpr int64_t kMost = (int64_t)1 << 40;   // elements of one tensor
constexpr int64_t kMostGroups = 0xffffff;     // workgroups along a grid's axis: its 256 threads each are counted in 32 bits

inline bool product_fits(std::initializer_list<int64_t> f) {
    int64_t n = 1;
    for (int64_t x : f) {
        if (x == 0) return true;
        if (x > kMost / n) return false;
        n *= x;
    }
    return true;
}

inline bool all_aligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned16(p)) return false;
    return true;
}

// No output may overlap an input or another output.
inline bool distinct(std::initializer_list<Range> ins, std::initializer_list<Range> outs) {
    for (const Range &o : outs) {
        for (const Range &i : ins)
            if (overlaps(o, i)) return false;
        for (const Range &p : outs)
            if (&p != &o && overlaps(o, p)) return false;
    }
    return true;
}

inline int launch_status() {
    hipError_t e = hipGetLastError();
    return e == hipSuccess ? BDSSM_OK : BDSSM_ERR_HIP;
}

}  // namespace bdssm_host
