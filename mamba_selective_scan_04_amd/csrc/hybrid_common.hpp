// hybrid_common.hpp -- device helpers shared by the hybrid layer's operators
// (gated delta rule, attention over the paged 8-bit cache): matrix-instruction
// fragments, and fp32 operands split into bf16 parts.
//
// Matrix instruction.  v_mfma_f32_16x16x32_bf16: D[16x16] += A[16x32] B[32x16].
// Lane l holds row (A) or column (B) l % 16 and the eight k = 8 (l / 16) + j;
// of C and D it holds column l % 16 and rows 4 (l / 16) + r, r = 0..3.
//
// A product's result as the next product's B operand without a lane exchange:
// the k index is summed over, so any order of it will do as long as A and B
// agree.  Two result tiles (rows 0..15 and 16..31 of a 32-row slice) in the
// lane group g = l / 16 hold rows 4g..4g+3 and 16+4g..16+4g+3; taking those
// eight as k slots 8g..8g+7 makes them a B fragment as they are.  The A operand
// is then read as two runs of four: columns 4g.. and 16+4g.. of the slice
// ("paired order").
//
// Precision.  States, corrections and their adjoints are fp32.  A product with
// an fp32 operand runs on bf16 matrix instructions by splitting the operand
// into bf16 parts, each the rest rounded to nearest: three hold all 24 bits of an
// fp32 value (the second is at most 2^-8 of it, the third 2^-17), so a product with
// a bf16 operand is exact up to the fp32 accumulation at three instructions; two
// fp32 operands take the six products of parts i, j with i + j <= 2 (what is left
// out is at most 2^-24 + 2^-34 of the term, of either sign).  Two parts leave an
// error of at most 2^-17 of the value and serve where the result is rounded to bf16.
// (Parts cut by truncation cost the same and leave out up to 2^-21, all of one sign.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bdssm_dev {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// 16x16x4 in fp32: A and B hold k = l / 16; result as above
__device__ __forceinline__ f32x4 mfma32(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float as_f(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t as_u(float f) { return __builtin_bit_cast(uint32_t, f); }
__device__ __forceinline__ float bf_lo(uint32_t u) { return as_f(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return as_f(u & 0xffff0000u); }

// two fp32 values to a bf16 pair, rounded to nearest even (a in the low half)
__device__ __forceinline__ uint32_t pk_rne(float a, float b) {
    bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
// the high halves of two fp32 values (truncation)
__device__ __forceinline__ uint32_t pk_cut(float a, float b) {
    return __builtin_amdgcn_perm(as_u(b), as_u(a), 0x07060302u);
}

// a less the low (b less the high) bf16 of a pair, in one instruction: the dot
// product with (-1, 0) or (0, -1) on top of a.  Exact where the pair is (a, b)
// rounded.  The factors are kept in scalar registers: as inline constants of
// this instruction they came out as other values.
__device__ __forceinline__ float less_low(float a, uint32_t pair) {
    uint32_t f = 0x0000bf80u;
    asm("" : "+s"(f));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, f), a, false);
}
__device__ __forceinline__ float less_high(float b, uint32_t pair) {
    uint32_t f = 0xbf800000u;
    asm("" : "+s"(f));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, f), b, false);
}

// (a, b) as kParts packed bf16 pairs, each the rest rounded to nearest: three are
// exact.  kCut: cut instead (less than 2^-7 of the value is left for the second, 2^-15
// for the third), so that no finite value has an infinite part, nor a sum of the
// parts passes it.
template <int kParts, bool kCut = false>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t *out) {
    out[0] = kCut ? pk_cut(a, b) : pk_rne(a, b);
#pragma unroll
    for (int i = 1; i < kParts; ++i) {
        a = less_low(a, out[i - 1]);
        b = less_high(b, out[i - 1]);
        out[i] = kCut ? pk_cut(a, b) : pk_rne(a, b);
    }
}

// A fragment in kParts parts.
template <int kParts>
struct Frag {
    bf16x8 p[kParts];
};

__device__ __forceinline__ bf16x8 frag_of(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_bit_cast(bf16x8, make_uint4(a, b, c, d));
}

// two result tiles' registers -> a B fragment in paired order
template <int kParts, bool kCut = false>
__device__ __forceinline__ Frag<kParts> split_frag(f32x4 t0, f32x4 t1) {
    uint32_t w[4][kParts];
    split_pair<kParts, kCut>(t0[0], t0[1], w[0]);
    split_pair<kParts, kCut>(t0[2], t0[3], w[1]);
    split_pair<kParts, kCut>(t1[0], t1[1], w[2]);
    split_pair<kParts, kCut>(t1[2], t1[3], w[3]);
    Frag<kParts> f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) f.p[i] = frag_of(w[0][i], w[1][i], w[2][i], w[3][i]);
    return f;
}

// acc += A B over the parts i, j with i + j < max(kA, kB): the products below
// are the last part's own precision.  Smallest terms first.
template <int kA, int kB>
__device__ __forceinline__ f32x4 mma(const Frag<kA> &a, const Frag<kB> &b, f32x4 acc) {
    constexpr int kOrder = kA > kB ? kA : kB;
#pragma unroll
    for (int s = kOrder - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < kA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < kB) acc = mfma(a.p[i], b.p[j], acc);
        }
    return acc;
}

// The same for kN results at once, acc[i] += A_i B: consecutive instructions are
// independent, where one result's own chain would wait for each.
template <int kN, int kA, int kB>
__device__ __forceinline__ void mma_n(const Frag<kA> *a, const Frag<kB> &b, f32x4 *acc) {
    constexpr int kOrder = kA > kB ? kA : kB;
#pragma unroll
    for (int s = kOrder - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < kA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < kB) {
#pragma unroll
                for (int x = 0; x < kN; ++x) acc[x] = mfma(a[x].p[i], b.p[j], acc[x]);
            }
        }
}

// the first kTo parts
template <int kTo, int kFrom>
__device__ __forceinline__ Frag<kTo> first_parts(const Frag<kFrom> &f) {
    Frag<kTo> g;
#pragma unroll
    for (int i = 0; i < kTo; ++i) g.p[i] = f.p[i];
    return g;
}

// How a stream type (uint16_t: bf16 bits; float) enters products.
template <typename T>
struct Stream;
template <>
struct Stream<uint16_t> {
    static constexpr int kParts = 1;      // a bf16 value is one part
    static constexpr int kOutParts = 2;   // operands of results that are rounded to bf16
    __device__ static float load(const uint16_t *p) { return as_f((uint32_t)*p << 16); }
    __device__ static void store(uint16_t *p, float v) { *p = (uint16_t)pk_rne(v, v); }
};
template <>
struct Stream<float> {
    static constexpr int kParts = 3;
    static constexpr int kOutParts = 3;
    __device__ static float load(const float *p) { return *p; }
    __device__ static void store(float *p, float v) { *p = v; }
};

// A fragment of eight consecutive k of a row (both operands read from memory).
__device__ __forceinline__ Frag<1> load_straight(const uint16_t *p) {
    Frag<1> f;
    f.p[0] = __builtin_bit_cast(bf16x8, *(const uint4 *)p);
    return f;
}
__device__ __forceinline__ Frag<3> load_straight(const float *p) {
    return split_frag<3>(*(const f32x4 *)p, *(const f32x4 *)(p + 4));
}

// One wave's 64 x 16 bytes from memory straight into LDS: each lane's piece,
// `off` bytes behind the uniform src, to base + 16 * lane (base uniform).  By
// hand, for the compiler's own form made it wait for all such loads before the
// next read of LDS, whichever buffer that was from.  It writes no register; who
// reads the data waits by loads_done first.
typedef __attribute__((address_space(3))) void lds_ptr;
__device__ __forceinline__ void load_lds(const void *src, uint32_t off, void *base) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_ptr *)base);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(src), "s"(at) : "m0", "memory");
}
// ... from a lane's own address
__device__ __forceinline__ void load_lds(const void *src, void *base) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_ptr *)base);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(at) : "m0", "memory");
}
// Until no more than the kLater youngest memory operations of the wave are under
// way (they finish in order).
template <int kLater>
__device__ __forceinline__ void loads_done() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLater) : "memory");
}

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

}  // namespace bdssm_dev
