// launch_norm.hip -- launchers of the norm's kernels.
// Compiled once per stream type (BDSSM_TIN = float, or uint16_t for bf16).
#include "layer_launch.hpp"

#ifndef BDSSM_TIN
#error "compiled once per stream type: -DBDSSM_TIN=float or -DBDSSM_TIN=uint16_t"
#endif

namespace bdssm_host {

template <typename T, typename R>
NormArgs<T, R> norm_args(const NormCall &c) {
    NormArgs<T, R> a{};
    a.x = (const T *)c.x;
    a.res = (const R *)c.res;
    a.w = c.w;
    a.eps = c.eps;
    a.inv_ch = 1. / c.ch;
    a.y = (T *)c.y;
    a.codes = c.codes;
    a.scales = c.scales;
    a.group = (int)c.group;
    a.h = (R *)c.h;
    a.rstd = c.rstd;
    a.rows = c.rows;
    a.ch = c.ch;
    a.dy = (const T *)c.dy;
    a.dh = (const R *)c.dh;
    a.dx = (T *)c.dx;
    a.dres = (R *)c.dres;
    a.parts = c.parts;
    return a;
}

template <int kThreads_, int kV_, int kVecs_>
struct Row {
    static constexpr int kThreads = kThreads_, kV = kV_, kVecs = kVecs_;
};

// calls f with the threads and vectors of a row of ch channels, at most kNormHeld.
// Up to 1,024 channels a wave in vectors of four, whose lanes are all in use at 256,
// 512, 768 and 1,024 (in vectors of eight, a quarter idle at 768: 32,768 rows of 768 50
// and 84 us instead of 36 and 34; 65,536 rows of 1,024 to e4m3 188 instead of 160).
// Above, a workgroup in vectors of eight, all of whose lanes are in use at 2,048, 4,096
// and 8,192.  Idle ones cost little there: forward and gradients of 25.2 million values
// in bf16 (201 MB each), us by channels:
//   1,536: 38.5 36.5   2,048: 38.6 35.3   2,560: 36.4 44.3   4,096: 37.2 43.0
//   5,120: 42.5 41.6   6,144: 41.8 44.2   8,192: 42.6 47.8
template <typename F>
void with_row(int ch, F &&f) {
    if (ch <= 256) f(Row<64, 4, 1>{});
    else if (ch <= 512) f(Row<64, 4, 2>{});
    else if (ch <= 768) f(Row<64, 4, 3>{});
    else if (ch <= 1024) f(Row<64, 4, 4>{});
    else if (ch <= 2048) f(Row<256, 8, 1>{});
    else if (ch <= 4096) f(Row<256, 8, 2>{});
    else f(Row<1024, 8, 1>{});
}

template <typename T, typename R>
void norm_k(const NormCall &c, hipStream_t st) {
    const NormArgs<T, R> a = norm_args<T, R>(c);
    if (c.ch > kNormHeld) {
        const dim3 g((unsigned)c.groups), t(1024);
        if (c.code == kE4m3) hipLaunchKernelGGL((norm_wide_kernel<T, R, kE4m3>), g, t, 0, st, a);
        else if (c.code == kI8) hipLaunchKernelGGL((norm_wide_kernel<T, R, kI8>), g, t, 0, st, a);
        else hipLaunchKernelGGL((norm_wide_kernel<T, R, kOutStream>), g, t, 0, st, a);
        return;
    }
    with_row(c.ch, [&](auto row) {
        using W = decltype(row);
        constexpr int kThreads = W::kThreads;
        const dim3 g((unsigned)c.groups), t(kThreads > 256 ? kThreads : 256);
        if (c.code == kE4m3) hipLaunchKernelGGL((norm_kernel<T, R, kE4m3, kThreads, W::kV, W::kVecs>), g, t, 0, st, a);
        else if (c.code == kI8) hipLaunchKernelGGL((norm_kernel<T, R, kI8, kThreads, W::kV, W::kVecs>), g, t, 0, st, a);
        else hipLaunchKernelGGL((norm_kernel<T, R, kOutStream, kThreads, W::kV, W::kVecs>), g, t, 0, st, a);
    });
}

template <typename T, typename R>
void norm_bwd_k(const NormCall &c, hipStream_t st) {
    const NormArgs<T, R> a = norm_args<T, R>(c);
    if (c.groups == 0) return;
    if (c.ch > kNormHeld) {
        hipLaunchKernelGGL((norm_wide_bwd_kernel<T, R>), dim3((unsigned)c.groups), dim3(1024), 0, st, a);
        return;
    }
    with_row(c.ch, [&](auto row) {
        using W = decltype(row);
        constexpr int kThreads = W::kThreads;
        hipLaunchKernelGGL((norm_bwd_kernel<T, R, kThreads, W::kV, W::kVecs>), dim3((unsigned)c.groups), dim3(kThreads > 256 ? kThreads : 256), 0, st, a);
    });
}

template <>
void launch_norm<BDSSM_TIN>(const NormCall &c, hipStream_t st) {
    using T = BDSSM_TIN;
    if constexpr (sizeof(T) == 2) {
        if (c.wide) return norm_k<T, float>(c, st);
    }
    norm_k<T, T>(c, st);
}

template <>
void launch_norm_bwd<BDSSM_TIN>(const NormCall &c, hipStream_t st) {
    using T = BDSSM_TIN;
    bool done = false;
    if constexpr (sizeof(T) == 2) {
        if (c.wide) {
            norm_bwd_k<T, float>(c, st);
            done = true;
        }
    }
    if (!done) norm_bwd_k<T, T>(c, st);
    hipLaunchKernelGGL((parts_sum_kernel<16>), dim3((unsigned)((c.ch + 63) / 64)), dim3(1024), 0, st, c.parts, c.groups, 1, 0, c.ch, c.dw,
                       nullptr);
}

}  // namespace bdssm_host
