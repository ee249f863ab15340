// launch_weights.hip -- launcher of the pages' attention weights.
// Compiled once per stream type (BDSSM_TIN = float, or uint16_t for bf16).
#include "hybrid_launch.hpp"

#ifndef BDSSM_TIN
#error "compiled once per stream type: -DBDSSM_TIN=float or -DBDSSM_TIN=uint16_t"
#endif

namespace bdssm_host {

template <typename T, int kCode, int kD>
void weights_k(const KvCall &c, hipStream_t st) {
    const WeightArgs<T> a{(const T *)c.q, c.lse, (const uint8_t *)c.kc, c.ks, c.mass, c.mass_out, c.Lq, c.scale * 1.44269504088896341f, c.d};
    const int64_t tokens = (int64_t)c.d.max_pages * c.d.page_len;
    hipLaunchKernelGGL((kv_weights_kernel<T, kCode, kD>), dim3((unsigned)((tokens + kWeightKeys - 1) / kWeightKeys), (unsigned)c.batch),
                       dim3(kWeightWaves * 64), 0, st, a);
}

template <>
void launch_kv_weights<BDSSM_TIN>(const KvCall &c, hipStream_t st) {
    using T = BDSSM_TIN;
    if (c.head_dim == 64) c.code == kE4m3 ? weights_k<T, kE4m3, 64>(c, st) : weights_k<T, kI8, 64>(c, st);
    else c.code == kE4m3 ? weights_k<T, kE4m3, 128>(c, st) : weights_k<T, kI8, 128>(c, st);
}

}  // namespace bdssm_host
