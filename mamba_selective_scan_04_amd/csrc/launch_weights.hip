// launch_weights.hip -- launcher of the pages' attention weights.
// Compiled once per stream type (BDSSM_TIN = float, or uint16_t for bf16).
#include "hybrid_launch.hpp"

#ifndef BDSSM_TIN
#error "compiled once per stream type: -DBDSSM_TIN=float or -DBDSSM_TIN=uint16_t"
#endif

namespace bdssm_host {

// Key tiles of a wave: four where there are more query rows than a tile (their queries
// are read for 64 keys at a time), else two, so that a wave goes over twice the heads.
// Microseconds of 2 / 4, 4 key heads (bf16 but the last; the host's side of a call is 9):
//   64 rows of up to 8,192 tokens, 64 channels    3 query rows: 19.1 / 22.2   48: 33.6 / 29.8
//   the same of 128 channels                      3: 38.0 / 43.4   12: 41.1 / 44.3   48: 67.3 / 56.1
//   1 row of 65,536, 128 channels                 4: 12.6 / 12.6   64: 23.4 / 16.9   256: 64.8 / 38.5
//   the same in fp32                              4: 12.7 / 12.9   64: 37.7 / 24.7
// (Eight: 15.2 for 65,536 tokens and 64 rows, but 62.8 for the second's 48 and more at
// 64 channels, where the registers leave two waves a SIMD.)
template <typename T, int kCode, int kD>
void weights_k(const KvCall &c, hipStream_t st) {
    const WeightArgs<T> a{(const T *)c.q, c.lse, (const uint8_t *)c.kc, c.ks, c.mass, c.mass_out, c.Lq, c.scale * 1.44269504088896341f, c.d};
    const int64_t tokens = (int64_t)c.d.max_pages * c.d.page_len;
    const dim3 g((unsigned)((tokens + kWeightKeys - 1) / kWeightKeys), (unsigned)c.batch);
    if (c.Lq * c.d.group <= 16) hipLaunchKernelGGL((kv_weights_kernel<T, kCode, kD, 2>), g, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((kv_weights_kernel<T, kCode, kD, 4>), g, dim3(256), 0, st, a);
}

template <>
void launch_kv_weights<BDSSM_TIN>(const KvCall &c, hipStream_t st) {
    using T = BDSSM_TIN;
    if (c.head_dim == 64) c.code == kE4m3 ? weights_k<T, kE4m3, 64>(c, st) : weights_k<T, kI8, 64>(c, st);
    else c.code == kE4m3 ? weights_k<T, kE4m3, 128>(c, st) : weights_k<T, kI8, 128>(c, st);
}

}  // namespace bdssm_host
