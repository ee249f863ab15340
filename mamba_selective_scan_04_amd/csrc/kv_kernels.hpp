// kv_kernels.hpp -- the attention side of the hybrid's cache on gfx950: finished
// blocks of keys and values into a paged 8-bit cache, and the active block's
// queries over that cache and the block's own keys and values.
//
// Cache.  A page holds page_len tokens of every key/value head, with one scale
// for each page and head: value = code * scale.  Keys are kept by token
// ([page_len][d]), values by channel ([d][page_len]): both are then the A
// operand of their product as they lie in memory (scores: rows keys, sum over
// d; outputs: rows d, sum over keys), 16 bytes of codes a lane, and no operand
// passes through LDS.
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

// two fp32 values in the code's range -> two codes in the low or high half
template <int kCode>
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d) {
    if constexpr (kCode == kE4m3) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
        const auto q = [](float x) { return (uint32_t)(int)rintf(x) & 255u; };   // NaN: 0
        return q(a) | q(b) << 8 | q(c) << 16 | q(d) << 24;
    }
}

// ------------------------------------------------------------------ commit
//
// One workgroup per (block of the call, head, row and tensor): the block's
// [page_len, d] values of one head in registers, their largest magnitude, then
// the codes.  Bound by memory: 2 or 4 bytes in, 1 out a value.
template <typename T>
struct CommitArgs {
    const T *k, *v;
    uint8_t *kc, *vc;
    float *ks, *vs;
    int64_t T_tokens;
    KvDims d;
};

template <typename T, int kCode, int kD, int kPerThread>
__global__ __launch_bounds__(256) void kv_commit_kernel(CommitArgs<T> a) {
    constexpr float kMax = kCode == kE4m3 ? 448.f : 127.f;
    constexpr int kBytes = kD + 4;                       // LDS row of codes
    __shared__ float part[4];
    __shared__ __attribute__((aligned(16))) uint8_t codes[kPerThread * 256 / kD * kBytes];
    const KvDims &d = a.d;
    const bool is_v = blockIdx.z & 1;
    const int b = blockIdx.z >> 1, h = blockIdx.y, page = d.page_len;
    const int64_t blk = blockIdx.x;
    int64_t n = a.T_tokens;
    if (d.lens != nullptr) n = d.lens[b] < n ? d.lens[b] : n;
    if ((blk + 1) * page > n) return;                    // a block that is not whole
    const int64_t at = (int64_t)(d.ctx[b] < 0 ? 0 : d.ctx[b]) / page + blk;
    if (at >= d.max_pages) return;
    const int id = d.table[(int64_t)b * d.max_pages + at];
    if (id < 0 || id >= d.n_pages) return;
    const T *src = (is_v ? a.v : a.k) + (((int64_t)b * a.T_tokens + blk * page) * d.heads_kv + h) * kD;
    constexpr int kVecs = (kPerThread + 7) / 8;
    float x[kVecs][8];
    float top = 0.f;
    const int total = page * kD;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int e = (threadIdx.x + i * 256) * 8;
        if (e < total) {
            const T *p = src + (int64_t)(e / kD) * d.heads_kv * kD + e % kD;
            if constexpr (sizeof(T) == 2) {
                const uint4 w = *(const uint4 *)p;
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][2 * j] = bf_lo(u[j]);
                    x[i][2 * j + 1] = bf_hi(u[j]);
                }
            } else {
                *(f32x4 *)&x[i][0] = *(const f32x4 *)p;
                *(f32x4 *)&x[i][4] = *(const f32x4 *)(p + 4);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = fabsf(x[i][j]);
                top = m < __builtin_inff() ? fmaxf(top, m) : top;   // the finite ones
            }
        }
    }
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) top = fmaxf(top, __shfl_xor(top, s, 64));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const float scale = fmaxf(top * (1.f / kMax), 0x1p-126f);
    const int64_t unit = (int64_t)id * d.heads_kv + h;
    if (threadIdx.x == 0) (is_v ? a.vs : a.ks)[unit] = scale;
    uint8_t *out = (is_v ? a.vc : a.kc) + unit * total;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int e = (threadIdx.x + i * 256) * 8;
        if (e < total) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float z = x[i][j] / scale;
                y[j] = z != z ? z : fminf(fmaxf(z, -kMax), kMax);
            }
            const uint2 w = make_uint2(to_codes<kCode>(y[0], y[1], y[2], y[3]), to_codes<kCode>(y[4], y[5], y[6], y[7]));
            if (is_v) {
                *(uint32_t *)(codes + e / kD * kBytes + e % kD) = w.x;
                *(uint32_t *)(codes + e / kD * kBytes + e % kD + 4) = w.y;
            } else {
                *(uint2 *)(out + e) = w;
            }
        }
    }
    if (!is_v) return;
    __syncthreads();
    // by channel: 16 tokens of one channel a thread
    for (int e = threadIdx.x; e < total / 16; e += 256) {
        const int c = e % kD, t0 = e / kD * 16;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t *p = codes + (t0 + 4 * j) * kBytes + c;
            w[j] = p[0] | (uint32_t)p[kBytes] << 8 | (uint32_t)p[2 * kBytes] << 16 | (uint32_t)p[3 * kBytes] << 24;
        }
        *(uint4 *)(out + c * page + t0) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// --------------------------------------------------------------- attention
//
// A wave takes 64 keys at a time and kTiles * 16 queries: the rows of one
// key/value head's query heads and all query tokens, so that a key is read once
// for all of them.  Scores are formed as S^T = K Q^T (rows keys, columns
// queries), which makes each lane the owner of one query per tile (its maximum
// and sum need no exchange but over the four lane groups) and the probabilities
// the B operand of O^T = V^T P^T as they stand.  Score row 4 g + r of tile t
// is key 16 g + 4 t + r of the 64: lane group g then holds 16 consecutive keys,
// which lie in one page (one scale a lane) and are 16 consecutive codes of a
// channel's row.
//
// Probabilities enter their product as bf16 (two parts for fp32 streams: three)
// after the page's value scale is multiplied in; scores, maxima, sums and
// outputs are fp32.  The running maximum moves only when a score passes it by
// 2^8: probabilities stay below 2^8 and the outputs are seldom rescaled.
//
// The keys of a row are cut into `splits` ranges (workgroups) and each range's
// 64-key steps go round its four waves; the waves join through LDS, the ranges
// through the workspace and kv_join_kernel.
template <typename T>
struct AttnArgs {
    const T *q, *k, *v;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    T *o;
    float *part_o, *part_ml;   // [unit][split][rows][d], [unit][split][rows][2]
    int64_t L, Lq;
    int splits, qtiles, causal;
    float scale;               // times log2(e)
    KvDims d;
};

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

// the probabilities' parts
template <typename T>
constexpr int kProbParts = sizeof(T) == 2 ? 1 : 3;

template <typename T, int kD, int kTiles>
struct AttnState {
    static constexpr int kIn = Stream<T>::kParts;
    f32x4 O[kD / 16][kTiles];
    float m[kTiles], l[kTiles];
    Frag<kIn> Q[kD / 32][kTiles];

    // scores S[t][nt] (already times scale, masked to -inf) of 64 keys; V(mt, u)
    // gives the values' fragment, vs their scale
    template <typename VFrag>
    __device__ __forceinline__ void step(f32x4 (&S)[4][kTiles], float vs, VFrag &&V) {
        float top[kTiles];
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
            float x = S[0][nt][0];
#pragma unroll
            for (int t = 0; t < 4; ++t)
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
        Frag<kProbParts<T>> P[2][kTiles];
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = __builtin_amdgcn_exp2f(S[t][nt][r] - m[nt]);
                    l[nt] += p;
                    S[t][nt][r] = p * vs;
                }
            P[0][nt] = split_frag<kProbParts<T>>(S[0][nt], S[1][nt]);
            P[1][nt] = split_frag<kProbParts<T>>(S[2][nt], S[3][nt]);
        }
#pragma unroll
        for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const auto vf = V(mt, u);
#pragma unroll
                for (int nt = 0; nt < kTiles; ++nt) O[mt][nt] = mma(vf, P[u][nt], O[mt][nt]);
            }
    }
};

template <typename T, int kCode, int kD, int kTiles>
__global__ __launch_bounds__(256) void kv_attn_kernel(AttnArgs<T> a) {
    constexpr int kIn = Stream<T>::kParts, kRows = kTiles * 16, kChan = kD / 16, kORow = kD + 4;
    const KvDims &d = a.d;
    const int split = blockIdx.x, h = blockIdx.y / a.qtiles, qt = blockIdx.y % a.qtiles, b = blockIdx.z;
    const int lane = lane_id(), wave = threadIdx.x >> 6, col = lane & 15, grp = lane >> 4;
    const int64_t unit = (int64_t)b * gridDim.y + blockIdx.y;
    int64_t n = a.L;
    if (d.lens != nullptr) n = d.lens[b] < 0 ? 0 : d.lens[b] < n ? d.lens[b] : n;
    const int64_t nq = n < a.Lq ? n : a.Lq, rows = nq * d.group;   // the row's live queries
    int64_t ctx = d.ctx[b] < 0 ? 0 : d.ctx[b];
    const int64_t most = d.n_pages > 0 ? (int64_t)d.max_pages * d.page_len : 0;
    ctx = ctx < most ? ctx : most;
    const int64_t steps = (ctx + 63) / 64, per = (steps + a.splits - 1) / a.splits;
    const int64_t s0 = split * per, s1 = s0 + per < steps ? s0 + per : steps;
    const bool live = (int64_t)qt * kRows < rows, has_active = split == a.splits - 1;

    __shared__ __attribute__((aligned(16))) float Ol[kRows * kORow];
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
            const int64_t row = (int64_t)qt * kRows + nt * 16 + col;
            const T *qp = a.q + (((int64_t)b * a.Lq + row / d.group) * d.heads_q + h * d.group + row % d.group) * kD;
#pragma unroll
            for (int s = 0; s < kD / 32; ++s) {
                if (row < rows) st.Q[s][nt] = load_straight(qp + s / 2 * 64 + grp * 16 + (s & 1) * 8);
                else st.Q[s][nt] = Frag<kIn>{};
            }
        }
        const int32_t *table = d.table + (int64_t)b * d.max_pages;
        // what a step needs of memory: codes of keys and values, and scales
        struct Step {
            uint4 k[4][kD / 64], v[kChan];
            float ks, vs;
            int valid;   // of the lane's 16 keys (its values and scores)
        };
        const int shift = 31 - __builtin_clz(d.page_len);
        auto page_of = [&](int64_t key, bool *ok) {
            const int64_t p = key >> shift;
            int id = -1;
            if (key < ctx) id = table[p];
            *ok = id >= 0 && id < d.n_pages;
            return *ok ? id : 0;
        };
        auto fetch = [&](Step &f, int64_t step) {
            bool ok;
            const int64_t key0 = step * 64 + grp * 16;
            const int64_t u = (int64_t)page_of(key0, &ok) * d.heads_kv + h;
            f.valid = !ok ? 0 : ctx - key0 < 16 ? (int)(ctx - key0) : 16;
            f.ks = a.ks[u];
            f.vs = ok ? a.vs[u] : 0.f;
            const uint8_t *vp = a.vc + u * (kD * d.page_len) + (key0 & (d.page_len - 1));
#pragma unroll
            for (int mt = 0; mt < kChan; ++mt) f.v[mt] = *(const uint4 *)(vp + (mt * 16 + col) * d.page_len);
            // score rows: lane row `col` of tile t is key 16 (col / 4) + 4 t + col % 4
            const int64_t kk = step * 64 + (col >> 2) * 16;
            bool okk;
            const int64_t uk = (int64_t)page_of(kk, &okk) * d.heads_kv + h;
            const uint8_t *kp = a.kc + uk * (kD * d.page_len) + ((kk & (d.page_len - 1)) + (col & 3)) * kD + grp * 16;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int s = 0; s < kD / 64; ++s) f.k[t][s] = *(const uint4 *)(kp + t * 4 * kD + s * 64);
        };
        auto use = [&](Step &f) {
            f32x4 S[4][kTiles];
            const float ks = f.ks * a.scale;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
#pragma unroll
                for (int nt = 0; nt < kTiles; ++nt) S[t][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kD / 64; ++s) {
                    const uint4 w = f.k[t][s];
                    const Frag<1> k0{{widen<kCode>(w.x, w.y)}}, k1{{widen<kCode>(w.z, w.w)}};
#pragma unroll
                    for (int nt = 0; nt < kTiles; ++nt) {
                        S[t][nt] = mma(k0, st.Q[2 * s][nt], S[t][nt]);
                        S[t][nt] = mma(k1, st.Q[2 * s + 1][nt], S[t][nt]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[t][nt][r] *= ks;
            }
            if (__any(f.valid < 16)) {   // the context's end, or a page that is not there
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (4 * t + r >= f.valid) {
#pragma unroll
                            for (int nt = 0; nt < kTiles; ++nt) S[t][nt][r] = -__builtin_inff();
                        }
                // codes behind the end may be anything (a NaN times 0 is a NaN)
                uint32_t keep[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int left = f.valid - 4 * i;
                    keep[i] = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << 8 * left) - 1u;
                }
#pragma unroll
                for (int mt = 0; mt < kChan; ++mt) {
                    f.v[mt].x &= keep[0];
                    f.v[mt].y &= keep[1];
                    f.v[mt].z &= keep[2];
                    f.v[mt].w &= keep[3];
                }
            }
            st.step(S, f.vs, [&](int mt, int u) {
                const uint4 w = f.v[mt];
                return u == 0 ? Frag<1>{{widen<kCode>(w.x, w.y)}} : Frag<1>{{widen<kCode>(w.z, w.w)}};
            });
        };
        Step f;
        for (int64_t s = s0 + wave; s < s1; s += 4) {
            fetch(f, s);
            use(f);
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
            for (int64_t s = wave; s * 64 < n; s += 4) {
                f32x4 S[4][kTiles];
                const int64_t kk = s * 64 + (col >> 2) * 16 + (col & 3), key0 = s * 64 + grp * 16;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
#pragma unroll
                    for (int nt = 0; nt < kTiles; ++nt) S[t][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int x = 0; x < kD / 32; ++x) {
                        Frag<kIn> kf{};
                        if (kk + 4 * t < n) kf = load_straight(kb + (kk + 4 * t) * stride + x / 2 * 64 + grp * 16 + (x & 1) * 8);
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
                st.step(S, 1.f, [&](int mt, int u) {
                    f32x4 x[2];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int64_t key = key0 + u * 8 + j;
                        x[j / 4][j % 4] = key < n ? Stream<T>::load(vb + key * stride + mt * 16 + col) : 0.f;
                    }
                    return split_frag<kIn>(x[0], x[1]);
                });
            }
        }
    }
    // the four waves' outputs: to the largest maximum, then added in order
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
        for (int nt = 0; nt < kTiles; ++nt) ml[0][nt * 16 + col][1] = sum[nt];
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

// Joins the splits: a thread per four channels of a query row.
template <typename T, int kD>
__global__ __launch_bounds__(256) void kv_join_kernel(const float *part_o, const float *part_ml, T *o, int64_t L, int64_t Lq,
                                                      int splits, int qtiles, int kRows, KvDims d) {
    const int b = blockIdx.z, h = blockIdx.y;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, row = e / (kD / 4);
    const int c = (int)(e % (kD / 4)) * 4;
    if (row >= Lq * d.group) return;
    int64_t n = L;
    if (d.lens != nullptr) n = d.lens[b] < 0 ? 0 : d.lens[b] < n ? d.lens[b] : n;
    const int64_t nq = n < Lq ? n : Lq;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    if (row < nq * d.group) {
        const int64_t unit = ((int64_t)b * d.heads_kv + h) * qtiles + row / kRows;
        const int64_t at = unit * splits * kRows + row % kRows;
        float top = kNone, sum = 0.f;
        for (int s = 0; s < splits; ++s) top = fmaxf(top, part_ml[(at + (int64_t)s * kRows) * 2]);
        for (int s = 0; s < splits; ++s) {
            const float *p = part_ml + (at + (int64_t)s * kRows) * 2;
            if (p[1] == 0.f) continue;   // no key in this range
            const float f = __builtin_amdgcn_exp2f(p[0] - top);
            sum = fmaf(p[1], f, sum);
            const f32x4 x = *(const f32x4 *)(part_o + (at + (int64_t)s * kRows) * kD + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = fmaf(x[i], f, y[i]);
        }
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = inv != 0.f ? y[i] * inv : 0.f;
    }
    T *op = o + (((int64_t)b * Lq + row / d.group) * d.heads_q + h * d.group + row % d.group) * kD + c;
    if constexpr (sizeof(T) == 2) *(uint2 *)op = make_uint2(pk_rne(y[0], y[1]), pk_rne(y[2], y[3]));
    else *(f32x4 *)op = y;
}

}  // namespace bdssm_dev
