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
// Bound by memory (the keys' codes, half of what the attention reads) where query rows
// are few: 64 rows of up to 8,192 int8 tokens of 4 heads of 64, 3 query rows, 19 us (4.4
// TB/s).  65,536 e4m3 tokens of 4 heads of 128 and 64 query rows: 16 us (2.1 TB/s), start
// and latency of a short kernel: its waves, two a SIMD, wait for 54% of the time, for
// the table, then the codes, then each tile of queries.
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

// Sum over the wave, the same order whatever the lanes hold.
__device__ __forceinline__ float wave_sum(float v) {
    const auto add = [](float x, auto ror) {
        return x + as_f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u(x), 0x120 + decltype(ror)::value, 0xf, 0xf, false));
    };
    v = add(v, std::integral_constant<int, 8>{});   // around a row of 16 lanes
    v = add(v, std::integral_constant<int, 4>{});
    v = add(v, std::integral_constant<int, 2>{});
    v = add(v, std::integral_constant<int, 1>{});
    const auto row = [&](int r) { return as_f((uint32_t)__builtin_amdgcn_readlane((int)as_u(v), 16 * r)); };
    return (row(0) + row(1)) + (row(2) + row(3));
}

constexpr int kWeightKeys = 128;   // of a workgroup: the longest page

template <typename T, int kCode, int kD, int kKeyTiles>
__global__ __launch_bounds__(256) void kv_weights_kernel(WeightArgs<T> a) {
    constexpr int kIn = Stream<T>::kParts, kSteps = kD / 32;
    constexpr int kWaves = 4, kShares = kWeightKeys / 16 / kKeyTiles;   // waves; shares of the workgroup's keys
    constexpr float kLog2e = 1.44269504088896341f;
    __shared__ float part[kWaves][kKeyTiles];
    const KvDims &d = a.d;
    const int b = blockIdx.y, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, grp = lane >> 4;
    int nq = (int)a.Lq;
    if (d.lens != nullptr) nq = d.lens[b] < 0 ? 0 : d.lens[b] < nq ? d.lens[b] : nq;
    const int rows = nq * d.group;
    int ctx = d.ctx[b] < 0 ? 0 : d.ctx[b];
    const int most = d.n_pages > 0 ? d.max_pages * d.page_len : 0;
    ctx = ctx < most ? ctx : most;
    const int key0 = (int)blockIdx.x * kWeightKeys + wave % kShares * (kKeyTiles * 16);   // below 2^30 + 64: the host's limit of a row's positions
    const int shift = 31 - __builtin_clz(d.page_len);
    const int32_t *table = d.table + (int64_t)b * d.max_pages;
    float sum[kKeyTiles];
    int id[kKeyTiles], left[kKeyTiles];   // left: keys of the tile from the lane's first on
    bool any = false, whole = true;
#pragma unroll
    for (int t = 0; t < kKeyTiles; ++t) {
        sum[t] = 0.f;
        const int key = key0 + t * 16;
        id[t] = key < ctx ? uniform_load(table + (key >> shift)) : -1;
        if (id[t] >= d.n_pages) id[t] = -1;
        any |= id[t] >= 0;
        whole &= id[t] >= 0 && ctx - key >= 16;
        left[t] = id[t] < 0 ? 0 : ctx - key - grp * 4;
    }
    if (any && rows > 0) {
        for (int h = wave / kShares; h < d.heads_kv; h += kWaves / kShares) {
            struct Queries {
                typename Fragments<T>::Raw raw[kSteps];
                float less;
            };
            const auto fetch = [&](Queries &to, int r0) {
                // k slot (step 2 s + x, group g, j) is channel 64 s + 16 g + 8 x + j, as the keys lie
                const int row = r0 + col < rows ? r0 + col : rows - 1, tok = row / d.group;
                const int64_t at = ((int64_t)b * a.Lq + tok) * d.heads_q + h * d.group + (row - tok * d.group);
                const T *qp = a.q + at * kD;
                to.less = a.lse[at];
#pragma unroll
                for (int s = 0; s < kSteps; ++s) to.raw[s] = Fragments<T>::read(qp + s / 2 * 64 + grp * 16 + (s & 1) * 8);
            };
            Queries now;
            fetch(now, 0);
            Frag<1> K[kKeyTiles][kSteps];
            float ks[kKeyTiles];
#pragma unroll
            for (int t = 0; t < kKeyTiles; ++t) {
                const int64_t unit = (int64_t)(id[t] < 0 ? 0 : id[t]) * d.heads_kv + h;
                const int in = ((key0 + t * 16) & (d.page_len - 1)) + col;
                const uint8_t *kp = a.kc + (unit * d.page_len + in) * kD + grp * 16;
                ks[t] = uniform_load(a.ks + unit) * a.scale;
#pragma unroll
                for (int s = 0; s < kD / 64; ++s) {
                    const uint4 w = *(const uint4 *)(kp + s * 64);
                    K[t][2 * s].p[0] = widen<kCode>(w.x, w.y);
                    K[t][2 * s + 1].p[0] = widen<kCode>(w.z, w.w);
                }
            }
            for (int r0 = 0; r0 < rows; r0 += 16) {
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
                    float p[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[r] = __builtin_amdgcn_exp2f(fmaf(S[t][r], ks[t], -less));
                    if (!whole) {   // the context's end, or a page that is not there
#pragma unroll
                        for (int r = 0; r < 4; ++r) p[r] = r < left[t] ? p[r] : 0.f;
                    }
                    const float all = (p[0] + p[1]) + (p[2] + p[3]);
                    sum[t] += live ? all : 0.f;
                }
                if (r0 + 16 < rows) fetch(now, r0 + 16);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kKeyTiles; ++t) {
        sum[t] = wave_sum(sum[t]);
        if (lane == 0) part[wave][t] = sum[t];
    }
    __syncthreads();
    const int pages = kWeightKeys >> shift, per = d.page_len / 16;   // of the workgroup; tiles of a page
    const int page = (int)blockIdx.x * pages + threadIdx.x;
    if ((int)threadIdx.x < pages && page < d.max_pages) {
        float s = 0.f;
        for (int i = 0; i < per; ++i) {
            const int t = threadIdx.x * per + i;   // of the eight
#pragma unroll
            for (int w = 0; w < kWaves; w += kShares) s += part[t / kKeyTiles + w][t % kKeyTiles];
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
// Weights become whole numbers of the same order (a NaN the largest).  The border
// between those that stay and those that go is found bit by bit from the top: how many
// candidates lie below a trial value is a compare and a population count of the ballot
// for every 64 of them, and with several waves a barrier.  It ends where a trial parts
// the row exactly (after 18 to 20 bits for weights that differ), else at the value of
// which only the first few go.  Long rows count their top nine bits (a float's sign and
// exponent) in LDS instead, in kCopies places each, for many weights share one; of the
// candidates with the border's, if they are few, one wave finds the other bits.
// Destinations are counted by ballots.  All counts are whole numbers: no order of the
// atomics shows.  Bound by the issue slots of one CU and the latency of each step: 4
// rows of 16,386 pages 20 us (31 without the counts in LDS), 64 rows of 258 pages 6.5.
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

constexpr int kEvictMostPages = 1 << 18;   // of a row

template <int kThreads, int kPer>
__global__ __launch_bounds__(kThreads) void kv_evict_kernel(EvictArgs a) {
    constexpr int kWaves = kThreads / 64;
    constexpr bool kByTops = kThreads == 1024;
    constexpr int kLowBits = 23, kTops = 1 << (32 - kLowBits), kCopies = 4, kListed = 1024;
    __shared__ int tops[kByTops ? kTops * kCopies : 1], listed;
    __shared__ uint32_t list[kByTops ? kListed : 1];
    __shared__ int red[2][kWaves < 2 ? 2 : kWaves];
    const int b = blockIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = a.max_pages;
    // a wave's values: `turns` times 64 of the row, one behind the other
    const int turns = kPer > 0 ? kPer : (n + kThreads - 1) / kThreads, base = wave * turns * 64 + lane;
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
    int32_t page[kHeld];   // read now: between the stores at the end each load would be waited for
    uint32_t key[kHeld];
    const auto page_at = [&](int at) { return table[at < n ? at : n - 1]; };
#pragma unroll
    for (int i = 0; i < kPer; ++i) held[i] = weight(base + i * 64);
#pragma unroll
    for (int i = 0; i < kPer; ++i) page[i] = page_at(base + i * 64);
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = order(base + i * 64, held[i]);
    const auto key_of = [&](int i) { return kPer > 0 ? key[i % kHeld] : order(base + i * 64, weight(base + i * 64)); };
    const auto each = [&](auto &&f) {
        if constexpr (kPer > 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) f(i);
        } else {
            for (int i = 0; i < turns; ++i) f(i);
        }
    };
    // lanes of a ballot below this one
    const auto lower = [](uint64_t m) {
        return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
    };
    // fewer than `gone` candidates lie below border, or exactly as many (then none at it goes)
    uint32_t border = 0;
    int below = 0;
    // the bits from `bit` down, by counts over all candidates
    const auto search_all = [&](int bit) {
#pragma unroll 1
        for (; bit >= 0 && below < gone; --bit) {
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
    };
    if constexpr (!kByTops) {
        search_all(31);
    } else if (gone > 0) {
        for (int i = threadIdx.x; i < kTops * kCopies; i += kThreads) tops[i] = 0;
        if (threadIdx.x == 0) listed = 0;
        __syncthreads();
        each([&](int i) {
            const uint32_t k = key_of(i);
            if (k != kStays) atomicAdd(&tops[(k >> kLowBits) * kCopies + lane % kCopies], 1);
        });
        __syncthreads();
        // the copies' sums, then in every wave the top whose candidates hold the gone-th
        int sum = 0;
        if (threadIdx.x < kTops) {
#pragma unroll
            for (int j = 0; j < kCopies; ++j) sum += tops[threadIdx.x * kCopies + j];
        }
        __syncthreads();
        if (threadIdx.x < kTops) tops[threadIdx.x] = sum;
        __syncthreads();
        int c[8], own = 0;   // eight neighbours a lane
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = tops[lane * 8 + i];
            own += c[i];
        }
        int upto = own;
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) {
            const int x = __shfl_up(upto, i, 64);
            if (lane >= i) upto += x;
        }
        const int at = __builtin_ctzll(__ballot(upto >= gone));   // gone is at most the candidates' number
        int before = upto - own, top = lane * 8, many = c[0];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            if (before + many < gone) {
                before += many;
                many = c[i];
                top = lane * 8 + i;
            }
        top = __builtin_amdgcn_readlane(top, at);
        below = __builtin_amdgcn_readlane(before, at);
        many = __builtin_amdgcn_readlane(many, at);
        border = (uint32_t)top << kLowBits;
        if (below + many == gone) {
            border = top == kTops - 1 ? kStays : border + (1u << kLowBits);   // all with this top go
            below = gone;
        } else if (many <= kListed) {
            // in any order: only how many there are of each is asked
            const auto in_top = [&](int i) { return key_of(i) >> kLowBits == (uint32_t)top && key_of(i) != kStays; };
            int mine = 0;
            each([&](int i) { mine += __popcll(__ballot(in_top(i))); });
            int to = 0;
            if (lane == 0 && mine > 0) to = atomicAdd(&listed, mine);
            to = __builtin_amdgcn_readfirstlane(to);
            each([&](int i) {
                const uint64_t m = __ballot(in_top(i));
                if (in_top(i)) list[to + lower(m)] = key_of(i);
                to += __popcll(m);
            });
            __syncthreads();
            if (wave == 0) {
                uint32_t k[kListed / 64];
#pragma unroll
                for (int i = 0; i < kListed / 64; ++i) k[i] = i * 64 + lane < many ? list[i * 64 + lane] : kStays;
                const int less = below;   // of smaller tops
#pragma unroll 1
                for (int bit = kLowBits - 1; bit >= 0 && below < gone; --bit) {
                    const uint32_t trial = border | 1u << bit;
                    int c = less;
#pragma unroll
                    for (int i = 0; i < kListed / 64; ++i) c += __popcll(__ballot(k[i] < trial));
                    if (c <= gone) {
                        border = trial;
                        below = c;
                    }
                }
                if (lane == 0) {
                    red[0][0] = (int)border;
                    red[0][1] = below;
                }
            }
            __syncthreads();
            border = (uint32_t)__builtin_amdgcn_readfirstlane(red[0][0]);
            below = __builtin_amdgcn_readfirstlane(red[0][1]);
        } else {
            search_all(kLowBits - 1);
        }
    }
    // sum of the waves' counts in front of this one's
    const auto in_front = [&](int c, int set) {
        if constexpr (kWaves == 1) return 0;
        __syncthreads();   // the last counts are read
        if (lane == 0) red[set][wave] = c;
        __syncthreads();
        int s = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += w < wave ? red[set][w] : 0;
        return __builtin_amdgcn_readfirstlane(s);
    };
    // of the candidates at the border the first gone - below go
    const bool tied = below < gone;
    int ties = 0;
    if (tied) {
        each([&](int i) { ties += __popcll(__ballot(key_of(i) == border)); });
        ties = in_front(ties, 0);
    }
    // pages that go: of this wave in all (with a bit for each where they are held), then
    // in front of it
    int left = 0, seen = ties;
    uint32_t mask = 0;
    const auto goes = [&](int i) {
        const uint32_t k = key_of(i);
        if (!tied) return k < border;
        const uint64_t eq = __ballot(k == border);
        const bool go = k < border || (k == border && seen + lower(eq) < gone - below);
        seen += __popcll(eq);
        return go;
    };
    each([&](int i) {
        const bool go = goes(i);
        if constexpr (kPer > 0) mask |= go ? 1u << i : 0u;
        left += __popcll(__ballot(go));
    });
    left = in_front(left, 1);
    seen = ties;
    int32_t *table_out = a.table_out + (int64_t)b * n;
    float *mass_out = a.mass_out + (int64_t)b * n;
    each([&](int i) {
        const bool go = kPer > 0 ? (mask >> i & 1) != 0 : goes(i);
        const uint64_t going = __ballot(go);
        const int rank = left + lower(going), at = base + i * 64;
        left += __popcll(going);
        if (at < n) {
            const uint32_t to = at >= used ? at : go ? used - gone + rank : at - rank;
            table_out[to] = kPer > 0 ? page[i % kHeld] : page_at(at);
            mass_out[to] = go ? 0.f : kPer > 0 ? held[i % kHeld] : weight(at);
        }
    });
    if (threadIdx.x == 0) a.ctx_out[b] = (int32_t)(ctx - (int64_t)gone * a.page_len);
}

}  // namespace bdssm_dev
