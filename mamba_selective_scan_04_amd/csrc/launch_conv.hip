// launch_conv.hip -- launchers of the short convolution's kernels.
// Compiled once per stream type (BDSSM_TIN = float, or uint16_t for bf16).
#include "layer_launch.hpp"

#ifndef BDSSM_TIN
#error "compiled once per stream type: -DBDSSM_TIN=float or -DBDSSM_TIN=uint16_t"
#endif

namespace bdssm_host {

template <typename T>
ConvArgs<T> conv_args(const ConvCall &c) {
    ConvArgs<T> a{};
    a.u = (const T *)c.u;
    a.ld = c.ld;
    a.batch_ld = c.batch_ld;
    a.w = c.w;
    a.bias = c.bias;
    a.lens = c.lens;
    a.starts = c.starts;
    a.c_init = (const T *)c.c_init;
    a.y = (T *)c.y;
    a.c_final = (T *)c.c_final;
    a.T_tokens = (int)c.T;
    a.jobs = c.plan.jobs;
    a.chunk = c.plan.chunk;
    a.chunks = (int)c.plan.chunks;
    a.ch = c.ch;
    a.lanes = c.plan.lanes;
    a.silu = c.silu;
    return a;
}

// calls f with the convolution's width, whether it is a plain one and has starts
template <typename F>
void with_width(const ConvCall &c, F &&f) {
    const auto kind = [&](auto width) {
        const bool plain = c.ch % kConvLane == 0 && c.silu;
        if (c.starts == nullptr) {
            if (plain) f(width, std::true_type{}, std::false_type{});
            else f(width, std::false_type{}, std::false_type{});
        } else {
            if (plain) f(width, std::true_type{}, std::true_type{});
            else f(width, std::false_type{}, std::true_type{});
        }
    };
    if (c.width == 4) kind(std::integral_constant<int, 4>{});
    else if (c.width == 3) kind(std::integral_constant<int, 3>{});
    else kind(std::integral_constant<int, 2>{});
}

template <>
void launch_conv<BDSSM_TIN>(const ConvCall &c, hipStream_t st) {
    using T = BDSSM_TIN;
    constexpr int kN = kConvLane;
    const ConvArgs<T> a = conv_args<T>(c);
    const dim3 g((unsigned)((c.plan.jobs + c.plan.block - 1) / c.plan.block)), t(c.plan.block);
    with_width(c, [&](auto width, auto plain, auto starts) {
        hipLaunchKernelGGL((conv_kernel<T, decltype(width)::value, kN, decltype(plain)::value, decltype(starts)::value>), g, t, 0, st, a);
    });
}

template <>
void launch_conv_bwd<BDSSM_TIN>(const ConvCall &c, hipStream_t st) {
    using T = BDSSM_TIN;
    constexpr int kN = kConvLane;
    ConvArgs<T> a = conv_args<T>(c);
    a.dy = (const T *)c.dy;
    a.dc_final = (const T *)c.dc_final;
    a.du = (T *)c.du;
    a.dc_init = (T *)c.dc_init;
    a.du_ld = c.du_ld;
    a.du_batch_ld = c.du_batch_ld;
    a.parts = c.parts;
    a.row_lanes = c.plan.row_lanes;
    a.rows = c.plan.chunks * c.batch;
    a.groups = c.plan.groups;
    a.n_parts = c.plan.n_parts;
    const dim3 g((unsigned)(c.plan.groups * c.plan.n_parts)), t(256);
    if (c.plan.n_parts > 0) {
        with_width(c, [&](auto width, auto plain, auto starts) {
            hipLaunchKernelGGL((conv_bwd_kernel<T, decltype(width)::value, kN, decltype(plain)::value, decltype(starts)::value>), g, t, 0, st, a);
        });
    }
    const int64_t cols = (int64_t)(c.width + 1) * c.ch;
    hipLaunchKernelGGL((parts_sum_kernel<16>), dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, st, c.parts, c.plan.n_parts, c.width, 1,
                       c.ch, c.dw, c.dbias);
}

}  // namespace bdssm_host
