// evict_kernels.hpp -- upkeep of the paged cache of kv_kernels.hpp: the attention
// weight that each page gets from the active queries, and the pages of least weight
// taken out of a row.
#pragma once

#include "kv_kernels.hpp"

namespace bdssm_dev {

// ------------------------------------------------------------------ weights
//
// mass[b, page] += sum over the row's queries i, heads h and the page's keys j of
// exp(scale q_ih . k_j - lse_ih), with lse what the attention returned: no maximum
// and no sum is carried here, and no values are read.
//
// Scores as in the attention, S^T = K Q^T: rows keys, columns queries.  A tile of 16
// keys lies in one page, so its page's scale is the tile's and everything a tile's
// lanes hold adds to one number.  A wave holds kKeyTiles tiles of one head's keys,
// widened once, and goes over the head's queries 16 at a time; half of the waves
// share a half of the workgroup's 128 keys, their heads in turn.  The sums over heads and
// tiles join in LDS in a fixed order.
//
// Bound by memory: the keys' codes, once (half of what the attention reads).
template <typename T>
struct WeightArgs {
    const T *q;
    const float *lse;          // [batch, Lq, heads_q], natural logarithms
    const uint8_t *kc;
    const float *ks;
    const float *mass;         // [batch, max_pages] or null
    float *out;
    int64_t Lq;
    float scale;               // times log2(e)
    KvDims d;
};

// Eight values of a row as they lie in memory, and as a fragment.
template <typename T>
struct Fragments;
template <>
struct Fragments<uint16_t> {
    typedef uint4 Raw;
    __device__ static __forceinline__ Raw read(const uint16_t *p) { return *(const uint4 *)p; }
    __device__ static __forceinline__ Frag<1> frag(const Raw &r) { return Frag<1>{{__builtin_bit_cast(bf16x8, r)}}; }
};
template <>
struct Fragments<float> {
    struct Raw {
        f32x4 a, b;
    };
    __device__ static __forceinline__ Raw read(const float *p) { return Raw{*(const f32x4 *)p, *(const f32x4 *)(p + 4)}; }
    __device__ static __forceinline__ Frag<3> frag(const Raw &r) { return split_frag<3>(r.a, r.b); }
};

constexpr int kWeightKeys = 128;   // of a workgroup: the longest page

constexpr int kWeightWaves = 8;

template <typename T, int kCode, int kD>
__global__ __launch_bounds__(kWeightWaves * 64, sizeof(T) == 2 ? 4 : 2) void kv_weights_kernel(WeightArgs<T> a) {
    constexpr int kIn = Stream<T>::kParts, kKeyTiles = 4, kSteps = kD / 32;
    constexpr float kLog2e = 1.44269504088896341f;
    __shared__ float part[kWeightWaves][kKeyTiles];
    const KvDims &d = a.d;
    const int b = blockIdx.y, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, grp = lane >> 4;
    const int half = wave & 1;
    int64_t nq = a.Lq;
    if (d.lens != nullptr) nq = d.lens[b] < 0 ? 0 : d.lens[b] < nq ? d.lens[b] : nq;
    const int64_t rows = nq * d.group;
    int64_t ctx = d.ctx[b] < 0 ? 0 : d.ctx[b];
    const int64_t most = d.n_pages > 0 ? (int64_t)d.max_pages * d.page_len : 0;
    ctx = ctx < most ? ctx : most;
    const int64_t key0 = (int64_t)blockIdx.x * kWeightKeys + half * (kKeyTiles * 16);
    const int shift = 31 - __builtin_clz(d.page_len);
    const int32_t *table = d.table + (int64_t)b * d.max_pages;
    float sum[kKeyTiles];
    int id[kKeyTiles];
    bool any = false;
#pragma unroll
    for (int t = 0; t < kKeyTiles; ++t) {
        sum[t] = 0.f;
        const int64_t key = key0 + t * 16;
        id[t] = key < ctx ? uniform_load(table + (key >> shift)) : -1;
        if (id[t] >= d.n_pages) id[t] = -1;
        any |= id[t] >= 0;
    }
    if (any && rows > 0) {
        for (int h = wave >> 1; h < d.heads_kv; h += kWeightWaves / 2) {
            Frag<1> K[kKeyTiles][kSteps];
            float ks[kKeyTiles];
#pragma unroll
            for (int t = 0; t < kKeyTiles; ++t) {
                const int64_t unit = (int64_t)(id[t] < 0 ? 0 : id[t]) * d.heads_kv + h;
                const int in = (int)((key0 + t * 16) & (d.page_len - 1)) + col;
                const uint8_t *kp = a.kc + (unit * d.page_len + in) * kD + grp * 16;
                ks[t] = uniform_load(a.ks + unit) * a.scale;
#pragma unroll
                for (int s = 0; s < kD / 64; ++s) {
                    const uint4 w = *(const uint4 *)(kp + s * 64);
                    K[t][2 * s].p[0] = widen<kCode>(w.x, w.y);
                    K[t][2 * s + 1].p[0] = widen<kCode>(w.z, w.w);
                }
            }
            // a tile of queries and the next one, on its way
            struct Queries {
                typename Fragments<T>::Raw raw[kSteps];
                float less;
            };
            const auto fetch = [&](Queries &to, int64_t r0) {
                // k slot (step 2 s + x, group g, j) is channel 64 s + 16 g + 8 x + j, as the keys lie
                const int64_t row = r0 + col < rows ? r0 + col : rows - 1;
                const int64_t at = ((int64_t)b * a.Lq + row / d.group) * d.heads_q + h * d.group + row % d.group;
                const T *qp = a.q + at * kD;
                to.less = a.lse[at];
#pragma unroll
                for (int s = 0; s < kSteps; ++s) to.raw[s] = Fragments<T>::read(qp + s / 2 * 64 + grp * 16 + (s & 1) * 8);
            };
            Queries now, next;
            fetch(now, 0);
            for (int64_t r0 = 0; r0 < rows; r0 += 16) {
                if (r0 + 16 < rows) fetch(next, r0 + 16);
                const float less = now.less * kLog2e;
                Frag<kIn> Q[kSteps];
#pragma unroll
                for (int s = 0; s < kSteps; ++s) Q[s] = Fragments<T>::frag(now.raw[s]);
                const bool live = r0 + col < rows && less != -__builtin_inff();   // -inf: a query that saw nothing
                f32x4 S[kKeyTiles];
#pragma unroll
                for (int t = 0; t < kKeyTiles; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int p = kIn - 1; p >= 0; --p)
#pragma unroll
                        for (int t = 0; t < kKeyTiles; ++t) S[t] = mfma(K[t][s].p[0], Q[s].p[p], S[t]);
#pragma unroll
                for (int t = 0; t < kKeyTiles; ++t) {
                    const int64_t left = ctx - (key0 + t * 16 + grp * 4);   // of the lane's four keys
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float p = __builtin_amdgcn_exp2f(fmaf(S[t][r], ks[t], -less));
                        sum[t] += live && r < left && id[t] >= 0 ? p : 0.f;
                    }
                }
                now = next;
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kKeyTiles; ++t) {
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) sum[t] += __shfl_xor(sum[t], s, 64);
        if (lane == 0) part[wave][t] = sum[t];
    }
    __syncthreads();
    const int pages = kWeightKeys >> shift, per = d.page_len / 16;   // of the workgroup; tiles of a page
    const int64_t page = (int64_t)blockIdx.x * pages + threadIdx.x;
    if ((int)threadIdx.x < pages && page < d.max_pages) {
        float s = 0.f;
        for (int i = 0; i < per; ++i) {
            const int t = threadIdx.x * per + i;   // of the eight
#pragma unroll
            for (int w = 0; w < kWeightWaves; w += 2) s += part[t / kKeyTiles + w][t % kKeyTiles];
        }
        const int64_t at = (int64_t)b * d.max_pages + page;
        a.out[at] = a.mass != nullptr ? a.mass[at] + s : s;
    }
}

// -------------------------------------------------------------------- evict
//
// A workgroup takes a row.  Of the whole pages in its context, budget stay; those of
// least weight among the ones that may leave go, at equal weight the one that lies
// first.  The row's order is kept: pages that stay, then those that left (free for the
// row's next blocks), then what lay behind the context.
//
// Weights become whole numbers of the same order (a NaN the largest).  The border is
// found bit by bit from the top: how many candidates lie below a trial value is
// counted by ballots, a compare and a population count a value, and a barrier each; it
// ends where a trial parts them exactly (after 18 to 20 bits for weights that differ),
// else at the value of which only the first few go.  Destinations are counted by
// ballots too, so nothing depends on an order of atomics.  Bound by one CU's issue
// slots and the barriers' latency (kPer values a thread in registers; 0: read again
// for every count, for longer rows).
struct EvictArgs {
    const int32_t *table, *ctx;
    const float *mass;
    int32_t *table_out, *ctx_out;
    float *mass_out;
    int max_pages, page_len, budget, sink, recent;
};

// Candidates are below kStays.
constexpr uint32_t kStays = ~0u;
__device__ __forceinline__ uint32_t weight_order(float m) {
    const uint32_t u = as_u(m + 0.f);   // -0 becomes 0
    return m != m ? kStays - 1 : u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kEvictMostPages = 1 << 18;   // of a row: its counts fit LDS

// exclusive sums of the n counts at `counts`, in place
template <int kThreads>
__device__ __forceinline__ void counts_scan(int *counts, int n, int *red) {
    const int lane = lane_id(), wave = threadIdx.x >> 6, per = (n + kThreads - 1) / kThreads, from = threadIdx.x * per;
    int own = 0;
    for (int i = 0; i < per; ++i)
        if (from + i < n) own += counts[from + i];
    int s = own;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
        const int x = __shfl_up(s, i, 64);
        if (lane >= i) s += x;
    }
    if (lane == 63) red[wave] = s;
    __syncthreads();
    int before = s - own;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) before += w < wave ? red[w] : 0;
    for (int i = 0; i < per; ++i) {
        if (from + i >= n) break;
        const int c = counts[from + i];
        counts[from + i] = before;
        before += c;
    }
    __syncthreads();
}

template <int kThreads, int kPer>
__global__ __launch_bounds__(kThreads) void kv_evict_kernel(EvictArgs a) {
    constexpr int kWaves = kThreads / 64;
    extern __shared__ int counts[];   // two of [turns][waves]
    __shared__ int red[2][kWaves];
    const int b = blockIdx.x, lane = lane_id(), wave = threadIdx.x >> 6, n = a.max_pages;
    const int turns = kPer > 0 ? kPer : (n + kThreads - 1) / kThreads;
    const float *mass = a.mass + (int64_t)b * n;
    const int32_t *table = a.table + (int64_t)b * n;
    int64_t ctx = a.ctx[b] < 0 ? 0 : a.ctx[b];
    const int64_t most = (int64_t)n * a.page_len;
    ctx = ctx < most ? ctx : most;
    const int shift = 31 - __builtin_clz(a.page_len), whole = (int)(ctx >> shift), used = (int)((ctx + a.page_len - 1) >> shift);
    const int gone = whole > a.budget ? whole - a.budget : 0, end = whole - a.recent;   // candidates: sink .. end - 1
    if (n == 0) {
        if (threadIdx.x == 0) a.ctx_out[b] = 0;
        return;
    }
    const auto weight = [&](int at) { return mass[at < n ? at : n - 1]; };   // no branch to a load
    const auto order = [&](int at, float m) {
        const uint32_t k = weight_order(m);
        return (at >= a.sink && at < end) ? k : kStays;
    };
    constexpr int kHeld = kPer > 0 ? kPer : 1;
    float held[kHeld];
    uint32_t key[kHeld];
#pragma unroll
    for (int i = 0; i < kPer; ++i) held[i] = weight(i * kThreads + threadIdx.x);
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = order(i * kThreads + threadIdx.x, held[i]);
    const auto weight_of = [&](int i) { return kPer > 0 ? held[i % kHeld] : weight(i * kThreads + threadIdx.x); };
    const auto key_of = [&](int i) {
        return kPer > 0 ? key[i % kHeld] : order(i * kThreads + threadIdx.x, weight(i * kThreads + threadIdx.x));
    };
    const auto each = [&](auto &&f) {
        if constexpr (kPer > 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) f(i);
        } else {
            for (int i = 0; i < turns; ++i) f(i);
        }
    };
    // fewer than `gone` candidates lie below border, or exactly as many (then none at it goes)
    uint32_t border = 0;
    int below = 0;
    if (gone > 0) {
#pragma unroll 1
        for (int bit = 31; bit >= 0 && below < gone; --bit) {
            const uint32_t trial = border | 1u << bit;
            int c = 0;
            each([&](int i) { c += __popcll(__ballot(key_of(i) < trial)); });
            if constexpr (kWaves > 1) {
                if (lane == 0) red[bit & 1][wave] = c;
                __syncthreads();
                c = 0;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) c += red[bit & 1][w];
                c = __builtin_amdgcn_readfirstlane(c);
            }
            if (c <= gone) {
                border = trial;
                below = c;
            }
        }
    }
    // in front of each turn's wave: candidates at the border (if some of them go, the
    // first gone - below), and pages that go
    int *ties = counts, *left = counts + turns * kWaves;
    const uint64_t before = (1ull << lane) - 1;
    const auto count = [&](int *to, auto &&flag) {
        each([&](int i) {
            const int c = __popcll(__ballot(flag(i)));
            if (lane == 0) to[i * kWaves + wave] = c;
        });
        __syncthreads();
        counts_scan<kThreads>(to, turns * kWaves, red[0]);
    };
    __syncthreads();   // red is read by the last count until here
    const bool tied = below < gone;
    if (tied) count(ties, [&](int i) { return key_of(i) == border; });
    const auto goes = [&](int i) {
        const uint32_t k = key_of(i);
        if (!tied) return k < border;
        const bool eq = k == border;
        const int rank = ties[i * kWaves + wave] + __popcll(__ballot(eq) & before);
        return k < border || (eq && rank < gone - below);
    };
    uint32_t mask = 0;   // of the held ones
    if constexpr (kPer > 0) each([&](int i) { mask |= goes(i) ? 1u << i : 0u; });
    const auto going = [&](int i) {
        if constexpr (kPer > 0) return (mask >> i & 1) != 0;
        else return goes(i);
    };
    count(left, going);
    int32_t *table_out = a.table_out + (int64_t)b * n;
    float *mass_out = a.mass_out + (int64_t)b * n;
    each([&](int i) {
        const bool go = going(i);
        const int rank = left[i * kWaves + wave] + __popcll(__ballot(go) & before), at = i * kThreads + threadIdx.x;
        if (at < n) {
            const int to = at >= used ? at : go ? used - gone + rank : at - rank;
            table_out[to] = table[at];
            mass_out[to] = go ? 0.f : weight_of(i);
        }
    });
    if (threadIdx.x == 0) a.ctx_out[b] = (int32_t)(ctx - (int64_t)gone * a.page_len);
}

}  // namespace bdssm_dev
