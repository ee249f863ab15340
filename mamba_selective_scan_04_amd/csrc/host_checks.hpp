// host_checks.hpp -- argument checks shared by the entry points' sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "bdssm.h"

namespace bdssm_host {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range { const void *p; size_t n; };

inline bool overlaps(Range a, Range b) {
    if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

inline int launch_status() {
    hipError_t e = hipGetLastError();
    return e == hipSuccess ? BDSSM_OK : BDSSM_ERR_HIP;
}

}  // namespace bdssm_host
