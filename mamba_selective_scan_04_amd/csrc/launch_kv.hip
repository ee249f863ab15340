// launch_kv.hip -- launchers of the paged 8-bit cache's kernels.
// Compiled once per stream type (BDSSM_TIN = float, or uint16_t for bf16).
#include "hybrid_launch.hpp"

#ifndef BDSSM_TIN
#error "compiled once per stream type: -DBDSSM_TIN=float or -DBDSSM_TIN=uint16_t"
#endif

namespace bdssm_host {

template <typename T, int kCode, int kD>
void commit_k(const KvCall &c, hipStream_t st) {
    const int64_t blocks = c.L / c.d.page_len, jobs = c.batch * blocks * c.d.heads_kv * 2;
    const CommitArgs<T> a{(const T *)c.k, (const T *)c.v, (uint8_t *)c.kc, (uint8_t *)c.vc, c.ks, c.vs, c.L,
                          (uint32_t)blocks, (uint32_t)jobs, c.d};
    const dim3 one((unsigned)((jobs + 3) / 4)), four((unsigned)jobs);
    switch (c.d.page_len * kD) {
    case 1024: hipLaunchKernelGGL((kv_commit_kernel<T, kCode, kD, 16, 1>), one, dim3(256), 0, st, a); break;
    case 2048: hipLaunchKernelGGL((kv_commit_kernel<T, kCode, kD, 32, 1>), one, dim3(256), 0, st, a); break;
    case 4096: hipLaunchKernelGGL((kv_commit_kernel<T, kCode, kD, 16, 4>), four, dim3(256), 0, st, a); break;
    case 8192: hipLaunchKernelGGL((kv_commit_kernel<T, kCode, kD, 32, 4>), four, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL((kv_commit_kernel<T, kCode, kD, 64, 4>), four, dim3(256), 0, st, a); break;
    }
}

template <typename T, int kCode, int kD>
void attn_k(const KvCall &c, hipStream_t st) {
    const AttnArgs<T> a{(const T *)c.q, (const T *)c.k, (const T *)c.v, (const uint8_t *)c.kc, (const uint8_t *)c.vc, c.ks, c.vs,
                        (T *)c.o, c.part_o, c.part_ml, c.L, c.Lq, c.plan.splits, c.plan.qtiles, c.causal,
                        c.scale * 1.44269504088896341f, c.batch * c.d.heads_kv * c.plan.splits, c.d};
    const dim3 g((unsigned)((a.jobs + 7) / 8 * 8 * c.plan.qtiles));
    bool two = false;
    if constexpr (sizeof(T) == 2 || kD == 64) {   // as kv_plan has it
        two = c.plan.tiles == 2;
        if (two) hipLaunchKernelGGL((kv_attn_kernel<T, kCode, kD, 2>), g, dim3(256), 0, st, a);
    }
    if (!two) hipLaunchKernelGGL((kv_attn_kernel<T, kCode, kD, 1>), g, dim3(256), 0, st, a);
    if (c.plan.splits > 1) {
        hipLaunchKernelGGL((kv_join_kernel<T, kD>), dim3((unsigned)(c.Lq * c.d.group), (unsigned)c.d.heads_kv, (unsigned)c.batch),
                           dim3(kD * 2), 0, st, c.part_o, c.part_ml, (T *)c.o, c.L, c.Lq, c.plan.splits, c.plan.qtiles,
                           c.plan.tiles * 16, c.d);
    }
}

template <>
void launch_kv_commit<BDSSM_TIN>(const KvCall &c, hipStream_t st) {
    using T = BDSSM_TIN;
    if (c.head_dim == 64) c.code == kE4m3 ? commit_k<T, kE4m3, 64>(c, st) : commit_k<T, kI8, 64>(c, st);
    else c.code == kE4m3 ? commit_k<T, kE4m3, 128>(c, st) : commit_k<T, kI8, 128>(c, st);
}

template <>
void launch_kv_attn<BDSSM_TIN>(const KvCall &c, hipStream_t st) {
    using T = BDSSM_TIN;
    if (c.head_dim == 64) c.code == kE4m3 ? attn_k<T, kE4m3, 64>(c, st) : attn_k<T, kI8, 64>(c, st);
    else c.code == kE4m3 ? attn_k<T, kE4m3, 128>(c, st) : attn_k<T, kI8, 128>(c, st);
}

}  // namespace bdssm_host
