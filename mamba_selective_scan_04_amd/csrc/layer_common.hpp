// layer_common.hpp -- device helpers of the operators around the scans (short
// convolution, residual norm): runs of stream values in registers, and the sum
// of partial gradients.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hybrid_common.hpp"

namespace bdssm_dev {

// kN consecutive stream values in registers as they lie in memory.  Rows may
// start at any multiple of a value's size (odd channel counts, slices of a wider
// tensor): the loads and stores are declared so, and are one instruction of up to
// 16 bytes all the same.
template <typename T, int kN>
struct Vals {
    T v[kN];
    __device__ __forceinline__ void load(const T *p) { __builtin_memcpy(v, p, sizeof v); }
    __device__ __forceinline__ void store(T *p) const { __builtin_memcpy(p, v, sizeof v); }
    // the first n of them; the rest 0
    __device__ __forceinline__ void load(const T *p, int n) {
        if (n >= kN) return load(p);
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = i < n ? p[i] : T(0);
    }
    __device__ __forceinline__ void store(T *p, int n) const {
        if (n >= kN) return store(p);
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (i < n) p[i] = v[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = T(0);
    }
    __device__ __forceinline__ float at(int i) const { return v[i]; }
    __device__ __forceinline__ void put(const float *x) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = x[i];
    }
};
// bf16 in pairs: two of them a register
template <int kN>
struct Vals<uint16_t, kN> {
    uint32_t w[kN / 2];
    __device__ __forceinline__ void load(const uint16_t *p) { __builtin_memcpy(w, p, sizeof w); }
    __device__ __forceinline__ void store(uint16_t *p) const { __builtin_memcpy(p, w, sizeof w); }
    __device__ __forceinline__ void load(const uint16_t *p, int n) {
        if (n >= kN) return load(p);
#pragma unroll
        for (int i = 0; i < kN / 2; ++i)
            w[i] = (2 * i < n ? p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
    __device__ __forceinline__ void store(uint16_t *p, int n) const {
        if (n >= kN) return store(p);
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (i < n) p[i] = (uint16_t)(w[i / 2] >> i % 2 * 16);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const { return i % 2 ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]); }
    __device__ __forceinline__ void put(const float *x) {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) w[i] = pk_rne(x[2 * i], x[2 * i + 1]);
    }
};

// Sums a parameter's gradient over the workgroups that formed parts of it: parts
// [n_parts][taps + with_bias][ch], into dw [ch][taps] and dbias [ch] (null: not
// wanted).  A workgroup takes 64 columns, its waves the parts' ranges, joined in
// order: the sums do not depend on how the workgroups ran.  Bound by latency (of
// each wave's n_parts / kWaves loads, eight under way at a time): 1,024 parts of 768
// columns 5.8 us (16 under way 6.2, 32 21.8), 126 of 7,680 5.3 (5.4, 5.2).
template <int kWaves>
__global__ __launch_bounds__(kWaves * 64) void parts_sum_kernel(const float *parts, int n_parts, int taps, int with_bias, int ch, float *dw,
                                                                float *dbias) {
    __shared__ float red[kWaves][64];
    const int64_t cols = (int64_t)(taps + with_bias) * ch;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane;
    const int per = (n_parts + kWaves - 1) / kWaves, p0 = wave * per, p1 = p0 + per < n_parts ? p0 + per : n_parts;
    float s = 0.f;
    if (col < cols) {
#pragma unroll 8
        for (int p = p0; p < p1; ++p) s += parts[p * cols + col];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || col >= cols) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += red[w][lane];
    const int64_t j = col / ch, c = col % ch;
    if (j < taps) dw[c * taps + j] = s;
    else if (dbias != nullptr) dbias[c] = s;
}

}  // namespace bdssm_dev
