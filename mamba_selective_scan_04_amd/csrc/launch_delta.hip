// launch_delta.hip -- launchers of the gated delta rule's kernels.
// Compiled once per stream type (BDSSM_TIN = float, or uint16_t for bf16).
#include "hybrid_launch.hpp"

#ifndef BDSSM_TIN
#error "compiled once per stream type: -DBDSSM_TIN=float or -DBDSSM_TIN=uint16_t"
#endif

namespace bdssm_host {

template <typename T, int kDk>
void launch_scan_k(const DeltaCall &c, hipStream_t st) {
    constexpr int kOut = Stream<T>::kOutParts;
    const dim3 gp((unsigned)c.d.chunks, (unsigned)c.d.hk, (unsigned)c.batch);
    if (c.d.chunks > 0)
        hipLaunchKernelGGL((delta_prep_kernel<T, kDk, kOut>), gp, dim3(kDeltaThreads), 0, st,
                           c.o != nullptr ? (const T *)c.q : (const T *)nullptr, (const T *)c.k, c.g, c.beta, (Mats<kOut> *)c.mats,
                           (double *)nullptr, c.d);
    ChainArgs<T> a{(const T *)c.q, (const T *)c.k, (const T *)c.v, (const Mats<kOut> *)c.mats, c.h_init, (T *)c.o, c.h_final, c.h_chunks,
                   c.agg, 1, c.d.chunks, 0, (int)(c.batch * c.d.hv), c.d};
    const auto grid = [&](int columns) { return dim3((unsigned)((a.groups + 7) / 8 * 8 * (columns / 64))); };
    if (c.segs > 1) {
        a.segs = c.segs;
        a.per = (c.d.chunks + c.segs - 1) / c.segs;
        a.groups *= c.segs;
        const bool chain = c.o != nullptr || c.h_chunks != nullptr;
        a.wanted = c.segs - (chain ? 1 : 0);   // the state behind the last comes from the chain
        hipLaunchKernelGGL((delta_chain_kernel<T, kDk, kAggregate, false>), grid(c.d.dv + kDk), dim3(kDeltaThreads), 0, st, a);
        // states alone: the join has the last
        const JoinArgs j{c.agg, c.h_init, chain ? c.h_seg : nullptr, chain ? nullptr : c.h_final, c.segs, c.d.dv, false};
        hipLaunchKernelGGL((delta_join_kernel<kDk>), dim3((unsigned)(c.d.dv / 16), (unsigned)(c.batch * c.d.hv)), dim3(kDk * 4), 0, st, j);
        if (!chain) return;
        a.h_init = c.h_seg;
    }
    const dim3 gc = grid(c.d.dv);
    // Two sets of tiles while there is a CU for each workgroup.  1,024 tokens of heads of
    // 128 by 128, us with two / one: 64 workgroups 72 / 77, 192: 88 / 94, 256: 95 / 106,
    // 288: 153 / 123, 512: 195 / 168 (the backward 160 / 169, 325 / 339, 411 / 428,
    // 530 / 478, 808 / 771).
    const bool two = sizeof(T) == 2 && (int64_t)a.groups * (c.d.dv / 64) <= 256;
    if (c.o != nullptr) {
        if constexpr (sizeof(T) == 2) {
            if (two) hipLaunchKernelGGL((delta_chain_kernel<T, kDk, kOutputs, true>), gc, dim3(kDeltaThreads), 0, st, a);
            else hipLaunchKernelGGL((delta_chain_kernel<T, kDk, kOutputs, false>), gc, dim3(kDeltaThreads), 0, st, a);
        } else {
            hipLaunchKernelGGL((delta_chain_kernel<T, kDk, kOutputs, false>), gc, dim3(kDeltaThreads), 0, st, a);
        }
    } else {
        hipLaunchKernelGGL((delta_chain_kernel<T, kDk, kStates, false>), gc, dim3(kDeltaThreads), 0, st, a);
    }
}

template <typename T, int kDk>
void launch_bwd_k(const DeltaCall &c, hipStream_t st) {
    const dim3 gp((unsigned)c.d.chunks, (unsigned)c.d.hk, (unsigned)c.batch);
    if (c.d.chunks > 0)
        hipLaunchKernelGGL((delta_prep_kernel<T, kDk, 3>), gp, dim3(kDeltaThreads), 0, st, (const T *)c.q, (const T *)c.k, c.g, c.beta,
                           (Mats<3> *)c.mats, c.G, c.d);
    AdjointArgs<T> a{(const T *)c.q, (const T *)c.k, (const T *)c.dout, (const Mats<3> *)c.mats, c.dh_final, c.dS, c.dh_init,
                     c.agg, nullptr, 1, c.d.chunks, (int)(c.batch * c.d.hv), c.d};
    const auto grid = [&](int columns) { return dim3((unsigned)((a.groups + 7) / 8 * 8 * (columns / 64))); };
    if (c.segs > 1) {
        a.segs = c.segs;
        a.per = (c.d.chunks + c.segs - 1) / c.segs;
        a.groups *= c.segs;
        hipLaunchKernelGGL((delta_adjoint_kernel<T, kDk, true, false>), grid(c.d.dv + kDk), dim3(kDeltaThreads), 0, st, a);
        const JoinArgs j{c.agg, c.dh_final, c.h_seg, nullptr, c.segs, c.d.dv, true};
        hipLaunchKernelGGL((delta_join_kernel<kDk>), dim3((unsigned)(c.d.dv / 16), (unsigned)(c.batch * c.d.hv)), dim3(kDk * 4), 0, st, j);
        a.h_seg = c.h_seg;
    }
    const dim3 gc = grid(c.d.dv);
    const bool two = sizeof(T) == 2 && (int64_t)a.groups * (c.d.dv / 64) <= 256;   // as the forward
    if constexpr (sizeof(T) == 2) {
        if (two) hipLaunchKernelGGL((delta_adjoint_kernel<T, kDk, false, true>), gc, dim3(kDeltaThreads), 0, st, a);
    }
    if (!two) hipLaunchKernelGGL((delta_adjoint_kernel<T, kDk, false, false>), gc, dim3(kDeltaThreads), 0, st, a);
    if (c.d.chunks == 0) return;
    const GradArgs<T> ga{(const T *)c.q, (const T *)c.k, (const T *)c.v, (const T *)c.dout, (const Mats<3> *)c.mats,
                         c.G, c.beta, c.h_chunks, c.dS, (T *)c.dq, (T *)c.dk_out, (T *)c.dv_out, c.dg, c.dbeta, c.d};
    const bool shared = c.d.group > 1;
    if (c.d.dv == 64) {
        if (shared) hipLaunchKernelGGL((delta_grad_kernel<T, kDk, 64, true>), gp, dim3(256), 0, st, ga);
        else hipLaunchKernelGGL((delta_grad_kernel<T, kDk, 64, false>), gp, dim3(256), 0, st, ga);
    } else {
        if (shared) hipLaunchKernelGGL((delta_grad_kernel<T, kDk, 128, true>), gp, dim3(512), 0, st, ga);
        else hipLaunchKernelGGL((delta_grad_kernel<T, kDk, 128, false>), gp, dim3(512), 0, st, ga);
    }
}

template <>
void launch_delta_bwd<BDSSM_TIN>(const DeltaCall &c, hipStream_t st) {
    if (c.dk == 64) launch_bwd_k<BDSSM_TIN, 64>(c, st);
    else launch_bwd_k<BDSSM_TIN, 128>(c, st);
}

template <>
void launch_delta_scan<BDSSM_TIN>(const DeltaCall &c, hipStream_t st) {
    if (c.dk == 64) launch_scan_k<BDSSM_TIN, 64>(c, st);
    else launch_scan_k<BDSSM_TIN, 128>(c, st);
}

// Tokens from which the step goes 16 at a time (bf16; fp32 streams go by token at any
// length).  64 rows of 16 heads of 128 by 128, read only / in place, in us: 4 tokens
// 19.5 / 26.1 by token and 19.7 / 30.8 by sixteen; 5: 21.9 / 28.0 and 20.0 / 31.1; 6:
// 24.5 / 30.1 and 20.1 / 31.4; 8: 29.6 / 35.0 and 20.6 / 31.9; 16: 48.9 / 54.5 and
// 22.3 / 33.9; 64: 163 / 168 and 62 / 71.  Less work (1 or 8 rows, or heads of 64) is
// the call's 10 to 11 us either way up to 8 tokens, and 16 tokens 12 to 18 by token.
constexpr int kBlockFrom = 6;

template <typename T>
void launch_step(const DeltaCall &c, hipStream_t st) {
    const StepArgs<T> a{(const T *)c.q, (const T *)c.k, (const T *)c.v, c.g, c.beta, c.h_init, (T *)c.o, c.h_final, c.d};
    const dim3 g((unsigned)(c.d.dv / 32), (unsigned)c.d.hv, (unsigned)c.batch);
    if constexpr (sizeof(T) == 2) {
        if (c.d.T >= kBlockFrom) {
            if (c.dk == 64) hipLaunchKernelGGL((delta_block_kernel<64>), g, dim3(64), 0, st, a);
            else hipLaunchKernelGGL((delta_block_kernel<128>), g, dim3(64), 0, st, a);
            return;
        }
    }
    if (c.dk == 64) hipLaunchKernelGGL((delta_step_kernel<T, 64>), g, dim3(64), 0, st, a);
    else hipLaunchKernelGGL((delta_step_kernel<T, 128>), g, dim3(64), 0, st, a);
}

template <>
void launch_delta_step<BDSSM_TIN>(const DeltaCall &c, hipStream_t st) { launch_step<BDSSM_TIN>(c, st); }

}  // namespace bdssm_host
