// kv_kernels.hpp -- the attention side of the hybrid's cache on gfx950: finished
// blocks of keys and values into a paged 8-bit cache, and the active block's
// queries over that cache and the block's own keys and values.
//
// Cache.  A page holds page_len tokens of every key/value head, with one scale
// for each page and head: value = code * scale.  Keys are kept by token
// ([page_len][d]), values by channel ([d][page_len]): both are then the A
// operand of their product in the order in which they lie in memory (scores: rows
// keys, sum over d; outputs: rows d, sum over keys), 16 bytes of codes a lane.  They
// go straight from memory into a buffer of each wave's own in LDS, a step ahead,
// and are read back as fragments.
#pragma once

#include <type_traits>

#include "hybrid_common.hpp"

namespace bdssm_dev {

constexpr int kE4m3 = 0, kI8 = 1;   // bdssm_code

struct KvDims {
    int heads_q, heads_kv, group, page_len, n_pages, max_pages;
    const int32_t *table;   // [batch, max_pages]
    const int32_t *ctx;     // [batch] tokens in the cache
    const int32_t *lens;    // [batch] active tokens, or null
};

// four values in the code's range -> their codes
template <int kCode>
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d) {
    if constexpr (kCode == kE4m3) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
        // 1.5 * 2^23 more, the sum's rounding is to whole numbers (ties to even) and
        // its lowest byte the number's
        const auto q = [](float x) { return as_u(x + 0x1.8p23f); };
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(q(d), q(c), 0x0c0c0400u), __builtin_amdgcn_perm(q(b), q(a), 0x0c0c0400u),
                                     0x05040100u);
    }
}

// ------------------------------------------------------------------ commit
//
// A unit is one head of one block of the call, of k or of v: its [page_len, d]
// values in registers, their largest magnitude, then the codes.  One wave takes a
// unit of up to 2,048 values, four waves a larger one; neighbouring waves take
// neighbouring heads.  Bound by memory: 2 or 4 bytes in, 1 out a value, if the
// arithmetic is kept short: 65,536 tokens of 4 heads of 128 in bf16, pages of 16,
// 32 us (6.2 TB/s read and written); with a workgroup to each unit and a plain
// division to each value it was 57.
//
// The quotient value / scale is the correctly rounded one at five operations a
// value, from r = 1 / scale correctly rounded once a unit: x r, then twice
// q += r (x - q scale) with the remainder exact.  The second makes a faithful q
// the correctly rounded one (Markstein, Computation of elementary functions on
// the IBM RISC System/6000 processor, 1990).  The remainder is exact while
// scale >= 2^-90 (x of less than scale / 2^11 is code 0 however it is rounded);
// other scales, and units with infinities or NaN, take plain divisions.
template <typename T>
struct CommitArgs {
    const T *k, *v;
    uint8_t *kc, *vc;
    float *ks, *vs;
    int64_t T_tokens;
    uint32_t blocks, jobs;   // whole blocks of T_tokens; units
    KvDims d;
};

// 8 stream values as they lie in memory
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
    uint4 w;
    __device__ __forceinline__ void load(const uint16_t *p) { w = *(const uint4 *)p; }
    __device__ __forceinline__ void values(float *x) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf_lo(u[j]);
            x[2 * j + 1] = bf_hi(u[j]);
        }
    }
    // the fp32 bits of the largest magnitude (those of infinities and NaN are larger than any value's)
    __device__ __forceinline__ uint32_t top() const {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        const auto mag = [](uint32_t u) { return __builtin_bit_cast(u16x2, u & 0x7fff7fffu); };
        const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(mag(w.x), mag(w.y)),
                                                  __builtin_elementwise_max(mag(w.z), mag(w.w)));
        return (uint32_t)(m.x > m.y ? m.x : m.y) << 16;
    }
};
template <>
struct Eight<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *(const f32x4 *)p;
        b = *(const f32x4 *)(p + 4);
    }
    __device__ __forceinline__ void values(float *x) const {
        *(f32x4 *)x = a;
        *(f32x4 *)(x + 4) = b;
    }
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t x = as_u(a[j]) & 0x7fffffffu, y = as_u(b[j]) & 0x7fffffffu;
            m = max(m, max(x, y));
        }
        return m;
    }
};

// kWaves waves a unit, kPer values a lane
template <typename T, int kCode, int kD, int kPer, int kWaves>
__global__ __launch_bounds__(256) void kv_commit_kernel(CommitArgs<T> a) {
    constexpr float kMax = kCode == kE4m3 ? 448.f : 127.f;
    constexpr int kThreads = kWaves * 64, kTotal = kPer * kThreads, kPage = kTotal / kD, kBytes = kD + 4;   // LDS row of codes
    constexpr int kVecs = kPer / 8;
    __shared__ uint32_t part[2][4];
    __shared__ __attribute__((aligned(16))) uint8_t room[4 / kWaves][kPage * kBytes];
    const KvDims &d = a.d;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tid = threadIdx.x % kThreads;
    const uint32_t job = blockIdx.x * (4 / kWaves) + wave / kWaves;
    if (job >= a.jobs) return;
    const int h = job % d.heads_kv;
    const bool is_v = job / d.heads_kv & 1;
    const uint32_t at_blk = job / d.heads_kv / 2, blk = at_blk % a.blocks, b = at_blk / a.blocks;
    int64_t n = a.T_tokens;
    if (d.lens != nullptr) n = d.lens[b] < n ? d.lens[b] : n;
    if ((int64_t)(blk + 1) * kPage > n) return;          // a block that is not whole
    const int64_t at = (int64_t)(d.ctx[b] < 0 ? 0 : d.ctx[b]) / kPage + blk;
    if (at >= d.max_pages) return;
    const int id = d.table[(int64_t)b * d.max_pages + at];
    if (id < 0 || id >= d.n_pages) return;
    const T *src = (is_v ? a.v : a.k) + (((int64_t)b * a.T_tokens + (int64_t)blk * kPage) * d.heads_kv + h) * kD;
    Eight<T> x[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int e = (tid + i * kThreads) * 8;
        x[i].load(src + (int64_t)(e / kD) * d.heads_kv * kD + e % kD);
    }
    // the largest of the unit's threads' values
    const auto largest = [&](uint32_t m, uint32_t (&to)[4]) {
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, s, 64));
        if constexpr (kWaves == 4) {
            if ((threadIdx.x & 63) == 0) to[wave] = m;
            __syncthreads();
            m = max(max(to[0], to[1]), max(to[2], to[3]));
        }
        return (uint32_t)__builtin_amdgcn_readfirstlane(m);
    };
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) top = max(top, x[i].top());
    top = largest(top, part[0]);
    const bool special = top >= 0x7f800000u;
    if (special) {   // of the finite ones then
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float y[8];
            x[i].values(y);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = as_u(y[j]) & 0x7fffffffu;
                m = u < 0x7f800000u ? max(m, u) : m;
            }
        }
        top = largest(m, part[1]);
    }
    const float scale = fmaxf(as_f(top) * (1.f / kMax), 0x1p-126f);
    const int64_t unit = (int64_t)id * d.heads_kv + h;
    if (tid == 0) (is_v ? a.vs : a.ks)[unit] = scale;
    uint8_t *out = (is_v ? a.vc : a.kc) + unit * kTotal;
    uint8_t *codes = room[wave / kWaves];
    const auto write = [&](auto &&quotient) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int e = (tid + i * kThreads) * 8;
            float y[8];
            x[i].values(y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = quotient(y[j]);
            const uint2 w = make_uint2(to_codes<kCode>(y[0], y[1], y[2], y[3]), to_codes<kCode>(y[4], y[5], y[6], y[7]));
            if (is_v) {
                *(uint32_t *)(codes + e / kD * kBytes + e % kD) = w.x;
                *(uint32_t *)(codes + e / kD * kBytes + e % kD + 4) = w.y;
            } else {
                *(uint2 *)(out + e) = w;
            }
        }
    };
    if (special || scale < 0x1p-90f) {
        write([&](float v) {
            const float z = v / scale;
            if (z != z) return kCode == kE4m3 ? z : 0.f;
            return fminf(fmaxf(z, -kMax), kMax);
        });
    } else {
        const float r = 1.f / scale;
        write([&](float v) {
            float q = v * r;
            q = fmaf(fmaf(-q, scale, v), r, q);
            return fmaf(fmaf(-q, scale, v), r, q);   // rounding makes it kMax at most
        });
    }
    if (!is_v) return;
    if constexpr (kWaves == 4) {
        __syncthreads();
    } else {   // a wave's LDS operations are done in order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    // by channel: 16 tokens of one channel a thread
#pragma unroll
    for (int e = tid; e < kTotal / 16; e += kThreads) {
        const int c = e % kD, t0 = e / kD * 16;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t *p = codes + (t0 + 4 * j) * kBytes + c;
            w[j] = p[0] | (uint32_t)p[kBytes] << 8 | (uint32_t)p[2 * kBytes] << 16 | (uint32_t)p[3 * kBytes] << 24;
        }
        *(uint4 *)(out + c * kPage + t0) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// --------------------------------------------------------------- attention
//
// A wave takes 32 keys at a time and kTiles * 16 queries: the rows of one
// key/value head's query heads and all query tokens, so that a key is read once
// for all of them.  Scores are formed as S^T = K Q^T (rows keys, columns
// queries), which makes each lane the owner of one query per tile (its maximum
// and sum need no exchange but over the four lane groups) and the probabilities
// the B operand of O^T = V^T P^T as they stand.  Score row 4 g + r of tile t
// is key 8 g + 4 t + r of the 32: lane group g then holds 8 consecutive keys,
// which lie in one page (one scale a lane) and are 8 consecutive codes of a
// channel's row.  32 keys are two pages at most, the same for the whole wave:
// their numbers and scales come by scalar loads.
//
// Probabilities enter their product in two bf16 parts (2^-17; fp32 streams: three,
// exact) after the page's value scale is multiplied in: in one part they would
// leave as much of an error as the output's own rounding (1.4 times the error of
// the whole for 2 us less at 65,536 tokens).  Scores, maxima, sums and
// outputs are fp32.  The running maximum moves only when a score passes it by
// 2^8: probabilities stay below 2^8 and the outputs are seldom rescaled.
//
// The keys of a row are cut into `splits` ranges (workgroups) and each range's
// 32-key steps go round its four waves; the waves join through LDS, the ranges
// through the workspace and kv_join_kernel.
//
// Measured at 128 channels, pages of 16, 64 query rows a key head (16 tokens of 4
// heads, two query tiles), with the join: 65,536 e4m3 tokens of 4 heads in 31 us (2.2
// TB/s), 4 rows of up to 262,144 int8 tokens in 215 to 256 us from one run to another
// (2.6 to 3.1 TB/s).  Registers leave two waves a
// SIMD, whose conversion of codes and softmax keep the vector units busy for 39% of
// the time (int8's codes take three times as many instructions as e4m3's: with one
// part 99 us against 83 for 4 rows of 65,536) and wait for the codes in the rest.
// At 64 channels and 3 query rows (64 rows of up to 8,192 int8 tokens, one tile):
// 46 to 50 us (3.4 to 3.7 TB/s; 42 where the same codes are read again), bound by
// memory and the rows' different ends.  fp32 streams: 42 us for the first (a tile of
// queries a wave, in three parts), 138 for 4 rows of 65,536 where bf16 takes 87.
template <typename T>
struct AttnArgs {
    const T *q, *k, *v;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    T *o;
    float *lse;                // [batch, Lq, heads_q] or null
    float *part_o, *part_ml;   // [unit][split][rows][d], [unit][split][rows][2]
    int64_t L, Lq;
    int splits, qtiles, causal;
    float scale;               // times log2(e)
    int64_t jobs;              // batch * heads_kv * splits
    KvDims d;
};

// log2 of a sum of powers of two over 2^top, as a natural logarithm; -inf without any
__device__ __forceinline__ float log_sum(float top, float sum) {
    return sum != 0.f ? (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f : -__builtin_inff();
}

constexpr float kNone = -3.4028235e38f;   // the maximum before any key: the lowest finite value

// 8 codes -> a fragment's eight bf16 values (exact)
template <int kCode>
__device__ __forceinline__ bf16x8 widen(uint32_t a, uint32_t b) {
    uint32_t w[4];
    if constexpr (kCode == kE4m3) {
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false));
        w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true));
        w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false));
        w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = (int)(i < 2 ? a : b) >> (i & 1) * 16;
            w[i] = pk_cut((float)(int8_t)s, (float)(int8_t)(s >> 8));   // 8 bits: cut is exact
        }
    }
    return frag_of(w[0], w[1], w[2], w[3]);
}

// A channel's values of eight active tokens as they lie in memory, and as a fragment.
// `seen` gathers whether any of them is an infinity or a NaN (two bf16 values an
// instruction, 0 times an fp32 value is a NaN), clear() makes those 0.
template <typename T>
struct Tokens;
template <>
struct Tokens<uint16_t> {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    struct Seen {
        u16x2 top = {0, 0};
        __device__ __forceinline__ bool special() const { return (top.x > top.y ? top.x : top.y) >= 0x7f80; }
    };
    uint32_t w[4];
    __device__ __forceinline__ void put(int j, const uint16_t *p) { w[j / 2] = j & 1 ? w[j / 2] | (uint32_t)*p << 16 : *p; }
    __device__ __forceinline__ void look(Seen &s) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) s.top = __builtin_elementwise_max(s.top, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
            if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
        }
    }
    __device__ __forceinline__ Frag<1> frag() const { return Frag<1>{{frag_of(w[0], w[1], w[2], w[3])}}; }
};
template <>
struct Tokens<float> {
    struct Seen {
        float zero = 0.f;
        __device__ __forceinline__ bool special() const { return zero != zero; }
    };
    f32x4 v[2];
    __device__ __forceinline__ void put(int j, const float *p) { v[j / 4][j % 4] = *p; }
    __device__ __forceinline__ void look(Seen &s) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) s.zero = fmaf(v[j / 4][j % 4], 0.f, s.zero);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!(fabsf(v[j / 4][j % 4]) < __builtin_inff())) v[j / 4][j % 4] = 0.f;
    }
    // Cut: a hidden token may hold fp32's largest value, which bf16 rounds to infinity.
    // With probabilities' parts rounded the products leave out less than 2^-22 of a term.
    __device__ __forceinline__ Frag<3> frag() const { return split_frag<3, true>(v[0], v[1]); }
};

// the probabilities' parts
template <typename T>
constexpr int kProbParts = sizeof(T) == 2 ? 2 : 3;

template <typename T, int kD, int kTiles>
struct AttnState {
    static constexpr int kIn = Stream<T>::kParts;
    f32x4 O[kD / 16][kTiles];
    float m[kTiles], l[kTiles];
    Frag<kIn> Q[kD / 32][kTiles];

    // scores S[t][nt] (already times scale, masked to -inf) of 32 keys; V(mt)
    // gives the values' fragment, vs their scale
    template <typename VFrag>
    __device__ __forceinline__ void step(f32x4 (&S)[2][kTiles], float vs, VFrag &&V) {
        float top[kTiles];
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
            float x = S[0][nt][0];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) x = fmaxf(x, S[t][nt][r]);
            top[nt] = x;
            raise |= x > m[nt] + 8.f;
        }
        if (__any(raise)) {
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt) {
                float x = fmaxf(top[nt], __shfl_xor(top[nt], 16, 64));
                x = fmaxf(x, __shfl_xor(x, 32, 64));
                x = fmaxf(x, m[nt]);
                const float f = __builtin_amdgcn_exp2f(m[nt] - x);
                m[nt] = x;
                l[nt] *= f;
#pragma unroll
                for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[mt][nt][r] *= f;
            }
        }
        Frag<kProbParts<T>> P[kTiles];
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = __builtin_amdgcn_exp2f(S[t][nt][r] - m[nt]);
                    l[nt] += p;
                    S[t][nt][r] = p * vs;
                }
            P[nt] = split_frag<kProbParts<T>>(S[0][nt], S[1][nt]);
        }
#pragma unroll
        for (int mt = 0; mt < kD / 16; ++mt) {
            const auto vf = V(mt);
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt) O[mt][nt] = mma(vf, P[nt], O[mt][nt]);
        }
    }
};

// A wave-uniform value that no kernel writes meanwhile, by a scalar load (a vector
// load would count among the loads into LDS that the waits below count).
template <typename T>
__device__ __forceinline__ T uniform_load(const T *p) {
    return *(const __attribute__((address_space(4))) T *)p;
}

template <typename T, int kCode, int kD, int kTiles>
__global__ __launch_bounds__(256, kTiles == 2 && (kD == 128 || sizeof(T) == 4) ? 2 : 3) void kv_attn_kernel(AttnArgs<T> a) {
    constexpr int kIn = Stream<T>::kParts, kRows = kTiles * 16, kChan = kD / 16, kORow = kD + 4;
    const KvDims &d = a.d;
    // the query tiles of one range of keys on one XCD, as the chains' column
    // blocks: the second finds the codes in its L2
    const int64_t place = blockIdx.x, job = place / 8 / a.qtiles * 8 + place % 8;
    if (job >= a.jobs) return;
    const int qt = (int)(place / 8 % a.qtiles), split = (int)(job % a.splits), h = (int)(job / a.splits % d.heads_kv);
    const int b = (int)(job / a.splits / d.heads_kv);
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, grp = lane >> 4;
    const int64_t unit = ((int64_t)b * d.heads_kv + h) * a.qtiles + qt;
    int64_t n = a.L;
    if (d.lens != nullptr) n = d.lens[b] < 0 ? 0 : d.lens[b] < n ? d.lens[b] : n;
    const int64_t nq = n < a.Lq ? n : a.Lq, rows = nq * d.group;   // the row's live queries
    int64_t ctx = d.ctx[b] < 0 ? 0 : d.ctx[b];
    const int64_t most = d.n_pages > 0 ? (int64_t)d.max_pages * d.page_len : 0;
    ctx = ctx < most ? ctx : most;
    const int64_t steps = (ctx + 31) / 32, per = (steps + a.splits - 1) / a.splits;
    const int64_t s0 = split * per, s1 = s0 + per < steps ? s0 + per : steps;
    const bool live = (int64_t)qt * kRows < rows, has_active = split == a.splits - 1;

    // Each wave's codes of two steps: of two key tiles 16 bytes a lane, as its
    // lanes use them, then the channels' rows of 32 keys.  Loaded straight from
    // memory a step ahead; a wave reads only what it loaded, so nothing but its
    // own wait is needed.  The waves' outputs take the room afterwards.
    constexpr int kKeyLoads = 2 * (kD / 64), kLoads = kKeyLoads + kD / 32;
    struct Codes {
        uint4 p[4][kLoads][64];
    };
    union Room {
        Codes c;
        float O[kRows * kORow];
    };
    __shared__ __attribute__((aligned(16))) Room r0;
    __shared__ __attribute__((aligned(16))) Codes r1;
    float *Ol = r0.O;
    __shared__ float ml[4][kRows][2];
    AttnState<T, kD, kTiles> st;
#pragma unroll
    for (int nt = 0; nt < kTiles; ++nt) {
        st.m[nt] = kNone;
        st.l[nt] = 0.f;
#pragma unroll
        for (int mt = 0; mt < kChan; ++mt) st.O[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (live) {
        // queries: k slot (step 2 t + x, group g, j) is channel 64 t + 16 g + 8 x + j
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
            const int64_t at = (int64_t)qt * kRows + nt * 16 + col, row = at < rows ? at : rows - 1;   // not stored
            const T *qp = a.q + (((int64_t)b * a.Lq + row / d.group) * d.heads_q + h * d.group + row % d.group) * kD;
#pragma unroll
            for (int s = 0; s < kD / 32; ++s) st.Q[s][nt] = load_straight(qp + s / 2 * 64 + grp * 16 + (s & 1) * 8);
        }
        // used here, so that no wait for them stays in the loop below (where it
        // would be one for the codes under way)
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
            for (int s = 0; s < kD / 32; ++s)
#pragma unroll
                for (int p = 0; p < kIn; ++p) asm volatile("" : "+v"(st.Q[s][nt].p[p]));
        const int32_t *table = d.table + (int64_t)b * d.max_pages;
        const int shift = 31 - __builtin_clz(d.page_len);
        // A step's two halves of 16 keys: their pages (-1: none) and scales.
        struct Pages {
            int id[2];
        };
        struct Scales {
            float k[2], v[2];
        };
        auto find = [&](int64_t step) {
            Pages p;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t key = step * 32 + i * 16;
                p.id[i] = key < ctx ? uniform_load(table + (key >> shift)) : -1;
                if (p.id[i] >= d.n_pages) p.id[i] = -1;
            }
            return p;
        };
        auto unit_of = [&](int id) { return (int64_t)(id < 0 ? 0 : id) * d.heads_kv + h; };
        auto scales = [&](Pages p) {
            const int64_t u0 = unit_of(p.id[0]), u1 = unit_of(p.id[1]);
            return Scales{{uniform_load(a.ks + u0), uniform_load(a.ks + u1)}, {uniform_load(a.vs + u0), uniform_load(a.vs + u1)}};
        };
        const int64_t page_bytes = (int64_t)kD * d.page_len;
        // a lane's offsets in a half's page: key row of its score row, channel row
        const bool khalf = col >= 8, vhalf = lane & 1;
        const uint32_t koff = ((col >> 2 & 1) * 8 + (col & 3)) * kD + grp * 16, voff = (lane >> 1) * d.page_len;
        auto fetch = [&](Codes &buf, int64_t step, Pages p) {
            const uint8_t *k0 = a.kc + unit_of(p.id[0]) * page_bytes, *k1 = a.kc + unit_of(p.id[1]) * page_bytes;
            const uint8_t *v0 = a.vc + unit_of(p.id[0]) * page_bytes, *v1 = a.vc + unit_of(p.id[1]) * page_bytes;
            const int in0 = (int)(step * 32 & (d.page_len - 1)), in1 = (int)((step * 32 + 16) & (d.page_len - 1));
            const uint8_t *kp = (khalf ? k1 + in1 * kD : k0 + in0 * kD) + koff, *vp = (vhalf ? v1 + in1 : v0 + in0) + voff;
            uint4(*to)[64] = buf.p[wave];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int s = 0; s < kD / 64; ++s) load_lds(kp + t * 4 * kD + s * 64, to[t * (kD / 64) + s]);
#pragma unroll
            for (int i = 0; i < kD / 32; ++i) load_lds(vp + i * 32 * d.page_len, to[kKeyLoads + i]);
        };
        auto use = [&](Codes &buf, int64_t step, Pages p, Scales sc) {
            uint4(*from)[64] = buf.p[wave];
            uint2 *vals = (uint2 *)from[kKeyLoads];   // of channel c, lane group g: 4 c + g
            const bool upper = grp >= 2;
            const float ks = (upper ? sc.k[1] : sc.k[0]) * a.scale;
            float vs = upper ? sc.v[1] : sc.v[0];
            f32x4 S[2][kTiles];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int nt = 0; nt < kTiles; ++nt) S[t][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kD / 64; ++s) {
                    const uint4 w = from[t * (kD / 64) + s][lane];
                    const Frag<1> k0{{widen<kCode>(w.x, w.y)}}, k1{{widen<kCode>(w.z, w.w)}};
#pragma unroll
                    for (int nt = 0; nt < kTiles; ++nt) S[t][nt] = mma(k0, st.Q[2 * s][nt], S[t][nt]);
#pragma unroll
                    for (int nt = 0; nt < kTiles; ++nt) S[t][nt] = mma(k1, st.Q[2 * s + 1][nt], S[t][nt]);
                }
#pragma unroll
                for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[t][nt][r] *= ks;
            }
            if (step * 32 + 32 > ctx || p.id[0] < 0 || p.id[1] < 0) {   // the context's end, or a page that is not there
                const int64_t left = ctx - (step * 32 + grp * 8);
                const int valid = (upper ? p.id[1] : p.id[0]) < 0 ? 0 : left < 8 ? (int)left : 8;   // of the lane's keys
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (4 * t + r >= valid) {
#pragma unroll
                            for (int nt = 0; nt < kTiles; ++nt) S[t][nt][r] = -__builtin_inff();
                        }
                // codes and scales behind the end may be anything (a NaN times 0 is a NaN)
                if (valid <= 0) vs = 0.f;
                const uint32_t k0 = valid >= 4 ? ~0u : valid <= 0 ? 0u : (1u << 8 * valid) - 1u;
                const uint32_t k1 = valid >= 8 ? ~0u : valid <= 4 ? 0u : (1u << 8 * (valid - 4)) - 1u;
#pragma unroll 1
                for (int mt = 0; mt < kChan; ++mt) {
                    uint2 &w = vals[(mt * 16 + col) * 4 + grp];
                    w = make_uint2(w.x & k0, w.y & k1);
                }
            }
            st.step(S, vs, [&](int mt) {
                const uint2 w = vals[(mt * 16 + col) * 4 + grp];
                return Frag<1>{{widen<kCode>(w.x, w.y)}};
            });
        };
        if (s0 + wave < s1) {
            int64_t s = s0 + wave;
            Pages p0 = find(s), p1 = find(s + 4);
            Scales c0 = scales(p0);
            fetch(r0.c, s, p0);
            // One turn: the next step's codes on their way (none behind the range:
            // then page 0's or the row's own, never used), then a wait until nothing
            // but those is: they are the wave's youngest kLoads memory operations.
            const auto turn = [&](Codes &now, Codes &next) {
                fetch(next, s + 4, p1);
                const Scales c1 = scales(p1);
                const Pages p2 = find(s + 8);
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
                use(now, s, p0, c0);
                p0 = p1;
                c0 = c1;
                p1 = p2;
                s += 4;
            };
            for (;;) {
                turn(r0.c, r1);
                if (s >= s1) break;
                turn(r1, r0.c);
                if (s >= s1) break;
            }
            // what is still on its way lands before the room is used again
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        if (has_active) {   // the active tokens' own keys and values
            const T *kb = a.k + ((int64_t)b * a.L * d.heads_kv + h) * kD, *vb = a.v + ((int64_t)b * a.L * d.heads_kv + h) * kD;
            const int64_t stride = (int64_t)d.heads_kv * kD;
            int64_t pos[kTiles];   // the last active token that a query sees
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt) {
                const int64_t row = (int64_t)qt * kRows + nt * 16 + col;
                pos[nt] = a.causal ? n - nq + row / d.group : n - 1;
            }
            for (int64_t s = wave; s * 32 < n; s += 4) {
                f32x4 S[2][kTiles];
                const int64_t kk = s * 32 + (col >> 2) * 8 + (col & 3), key0 = s * 32 + grp * 8;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int nt = 0; nt < kTiles; ++nt) S[t][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int x = 0; x < kD / 32; ++x) {
                        const int64_t key = kk + 4 * t < n ? kk + 4 * t : n - 1;   // repeated tokens are masked
                        const auto kf = load_straight(kb + key * stride + x / 2 * 64 + grp * 16 + (x & 1) * 8);
#pragma unroll
                        for (int nt = 0; nt < kTiles; ++nt) S[t][nt] = mma(kf, st.Q[x][nt], S[t][nt]);
                    }
#pragma unroll
                    for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int64_t key = key0 + 4 * t + r;
                            S[t][nt][r] = key < n && key <= pos[nt] ? S[t][nt][r] * a.scale : -__builtin_inff();
                        }
                }
                Tokens<T> vals[kChan];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const T *row = vb + (key0 + j < n ? key0 + j : n - 1) * stride + col;
#pragma unroll
                    for (int mt = 0; mt < kChan; ++mt) vals[mt].put(j, row + mt * 16);
                }
                // Infinities and NaN: 0 in the product (a probability of 0 times them, be
                // it a hidden token's or a part of a split one, is a NaN), then added
                typename Tokens<T>::Seen seen;
#pragma unroll
                for (int mt = 0; mt < kChan; ++mt) vals[mt].look(seen);
                const bool odd = __any(seen.special());
                if (odd) {
#pragma unroll
                    for (int mt = 0; mt < kChan; ++mt) vals[mt].clear();
                }
                st.step(S, 1.f, [&](int mt) { return vals[mt].frag(); });
                // the queries that see them get them as they are
#pragma unroll 1
                for (int j = 0; odd && j < 32 && s * 32 + j < n; ++j) {
                    const T *row = vb + (s * 32 + j) * stride + grp * 4;
#pragma unroll
                    for (int mt = 0; mt < kChan; ++mt)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            asm volatile("" ::: "memory");   // one at a time: registers before speed here
                            const float y = Stream<T>::load(row + mt * 16 + r);
#pragma unroll
                            for (int nt = 0; nt < kTiles; ++nt)
                                if (!(fabsf(y) < __builtin_inff()) && s * 32 + j <= pos[nt]) st.O[mt][nt][r] += y;
                        }
                }
            }
        }
    }
    // the four waves' outputs: to the largest maximum, then added in order (the
    // barrier behind the sums also ends every wave's use of the codes)
#pragma unroll
    for (int nt = 0; nt < kTiles; ++nt) {
        float l = st.l[nt];
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
        if (grp == 0) {
            ml[wave][nt * 16 + col][0] = st.m[nt];
            ml[wave][nt * 16 + col][1] = l;
        }
    }
    __syncthreads();
    float top[kTiles], sum[kTiles];
#pragma unroll
    for (int nt = 0; nt < kTiles; ++nt) {
        const int r = nt * 16 + col;
        top[nt] = fmaxf(fmaxf(ml[0][r][0], ml[1][r][0]), fmaxf(ml[2][r][0], ml[3][r][0]));
        sum[nt] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum[nt] = fmaf(ml[w][r][1], __builtin_amdgcn_exp2f(ml[w][r][0] - top[nt]), sum[nt]);
    }
    for (int w = 0; w < 4; ++w) {
        if (wave == w) {
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt) {
                const float f = __builtin_amdgcn_exp2f(st.m[nt] - top[nt]);
#pragma unroll
                for (int mt = 0; mt < kChan; ++mt) {
                    f32x4 *p = (f32x4 *)&Ol[(nt * 16 + col) * kORow + mt * 16 + grp * 4];
                    f32x4 x;
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[r] = st.O[mt][nt][r] * f;
                    if (w > 0) {
                        const f32x4 y = *p;
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] += y[r];
                    }
                    *p = x;
                }
            }
        }
        __syncthreads();
    }
    if (a.splits > 1) {
        const int64_t at = unit * a.splits + split;
        if (wave == 0 && grp == 0) {
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt) {
                a.part_ml[(at * kRows + nt * 16 + col) * 2] = top[nt];
                a.part_ml[(at * kRows + nt * 16 + col) * 2 + 1] = sum[nt];
            }
        }
        if (!live || (s0 >= s1 && !(has_active && n > 0))) return;   // no key: the sums say so
        for (int e = threadIdx.x; e < kRows * kD / 4; e += 256) {
            const int r = e / (kD / 4), c = e % (kD / 4) * 4;
            *(f32x4 *)(a.part_o + (at * kRows + r) * kD + c) = *(const f32x4 *)&Ol[r * kORow + c];
        }
        return;
    }
    // alone: the row's sums are in every wave's lanes; share them by row
    if (wave == 0 && grp == 0) {
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
            ml[0][nt * 16 + col][1] = sum[nt];
            const int64_t row = (int64_t)qt * kRows + nt * 16 + col;
            if (a.lse != nullptr && row < a.Lq * d.group)
                a.lse[((int64_t)b * a.Lq + row / d.group) * d.heads_q + h * d.group + row % d.group] =
                    log_sum(top[nt], row < rows ? sum[nt] : 0.f);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kRows * kD / 4; e += 256) {
        const int r = e / (kD / 4), c = e % (kD / 4) * 4;
        const int64_t row = (int64_t)qt * kRows + r;
        if (row >= a.Lq * d.group) continue;
        const float l = ml[0][r][1], inv = row < rows && l != 0.f ? 1.f / l : 0.f;
        const f32x4 x = *(const f32x4 *)&Ol[r * kORow + c];
        f32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = inv != 0.f ? x[i] * inv : 0.f;
        T *op = a.o + (((int64_t)b * a.Lq + row / d.group) * d.heads_q + h * d.group + row % d.group) * kD + c;
        if constexpr (sizeof(T) == 2) *(uint2 *)op = make_uint2(pk_rne(y[0], y[1]), pk_rne(y[2], y[3]));
        else *(f32x4 *)op = y;
    }
}

// Joins the ranges of one query row: a workgroup each.  The ranges' weights in LDS
// (kMaxSplits at a time), then eight groups of threads go round the ranges, four
// channels a thread.  5 to 7 us, most of it the launch.
constexpr int kMaxSplits = 1024;

template <typename T, int kD>
__global__ __launch_bounds__(kD * 2) void kv_join_kernel(const float *part_o, const float *part_ml, T *o, float *lse, int64_t L,
                                                         int64_t Lq, int splits, int qtiles, int kRows, KvDims d) {
    constexpr int kThreads = kD * 2, kLanes = kD / 4, kGroups = kThreads / kLanes;
    __shared__ float w[kMaxSplits];
    __shared__ float red[kThreads / 64][2];
    __shared__ __attribute__((aligned(16))) float acc[kGroups][kD];
    const int b = blockIdx.z, h = blockIdx.y;
    const int64_t row = blockIdx.x;
    int64_t n = L;
    if (d.lens != nullptr) n = d.lens[b] < 0 ? 0 : d.lens[b] < n ? d.lens[b] : n;
    const int64_t nq = n < Lq ? n : Lq;
    const int64_t query = ((int64_t)b * Lq + row / d.group) * d.heads_q + h * d.group + row % d.group;
    T *op = o + query * kD;
    const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes, c = lane * 4;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    float sum = 0.f, top = kNone;
    if (row < nq * d.group) {
        const int64_t unit = ((int64_t)b * d.heads_kv + h) * qtiles + row / kRows;
        const int64_t at = unit * splits * kRows + row % kRows;
        for (int s = threadIdx.x; s < splits; s += kThreads) top = fmaxf(top, part_ml[(at + (int64_t)s * kRows) * 2]);
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) top = fmaxf(top, __shfl_xor(top, i, 64));
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][0] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i) top = fmaxf(top, red[i][0]);
        for (int s0 = 0; s0 < splits; s0 += kMaxSplits) {
            const int m = splits - s0 < kMaxSplits ? splits - s0 : kMaxSplits;
            __syncthreads();
            for (int s = threadIdx.x; s < m; s += kThreads) {
                const float *p = part_ml + (at + (int64_t)(s0 + s) * kRows) * 2;
                const float f = p[1] != 0.f ? __builtin_amdgcn_exp2f(p[0] - top) : 0.f;
                w[s] = f;
                if (f != 0.f) sum = fmaf(p[1], f, sum);
            }
            __syncthreads();
#pragma unroll 4
            for (int s = grp; s < m; s += kGroups) {
                const float f = w[s];   // 0: no key in this range, and nothing written
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
                if (f != 0.f) x = *(const f32x4 *)(part_o + (at + (int64_t)(s0 + s) * kRows) * kD + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = fmaf(x[i], f, y[i]);
            }
        }
    }
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) sum += __shfl_xor(sum, i, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][1] = sum;
    *(f32x4 *)&acc[grp][c] = y;
    __syncthreads();
    if (grp > 0) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) sum += red[i][1];
    if (lse != nullptr && threadIdx.x == 0) lse[query] = log_sum(top, sum);
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v = 0.f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) v += acc[g][c + i];
        y[i] = inv != 0.f ? v * inv : 0.f;
    }
    if constexpr (sizeof(T) == 2) *(uint2 *)(op + c) = make_uint2(pk_rne(y[0], y[1]), pk_rne(y[2], y[3]));
    else *(f32x4 *)(op + c) = y;
}

}  // namespace bdssm_dev
