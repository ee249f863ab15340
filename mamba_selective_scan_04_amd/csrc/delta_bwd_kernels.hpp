// delta_bwd_kernels.hpp -- gradients of the gated delta rule.
//
// In the notation of delta_kernels.hpp, with dO given and dS' the adjoint of
// the state after the chunk:
//   dU = P^T dO + diag(exp(G_C - G_j)) K dS'
//   X  = W^T dU            (= dR = dV)
//   dS = exp(G_C) dS' + scale Q^T E dO - K^T E X
// is a chain over the chunks from the last, with independent columns as in the
// forward: delta_adjoint_kernel writes dS' of every chunk, over a long row of few
// heads in segments that run at once, as in the forward: dS = M dS' + N over a
// segment, its maps by the same kernel (kAggregate).  All else follows per
// chunk from S, dS' (delta_grad_kernel).  With y = U / beta, Z = X / beta (the
// rows' prediction errors and their adjoints' sources):
//   dV = X,  dbeta_i = y_i.Z_i
//   dQ = scale E dO S^T + DP K,        DP_ij = scale D_ij dO_i.U_j  (j <= i)
//   dK = diag(exp(G_C - G_j)) U dS'^T - E X S^T + DP^T Q + (DA + DA^T) K,
//        DA_ij = -D_ij X_i.U_j  (j < i)
// A token's decay weighs what passes it, from a token (or the state) before it to
// it or a token (or the state) behind it:
//   dg_t = sum over j < t <= i of w_ij + sum over i >= t of r_i + sum over j < t of c_j
//          + exp(G_C) <S, dS'>,
//   w_ij = D_ij (scale (q_i.k_j) (dO_i.U_j) - (k_i.k_j) (X_i.U_j))
//   r_i  = exp(G_i) (scale (S^T q_i).dO_i - (S^T k_i).X_i)
//   c_j  = exp(G_C - G_j) (dS'^T k_j).U_j
// Each term is summed where it counts.  (As a difference of sums by row and by
// column, the terms that do not pass t would cancel in theory only, and leave their
// roundings in the small gradient of a strong decay.)  The sums need neither dQ nor
// dK: those may be computed to their own type's precision while dg and dbeta keep
// 32 bits, U and X in the products above three parts.
#pragma once

#include "delta_kernels.hpp"

namespace bdssm_dev {

template <typename T>
struct AdjointArgs {
    const T *q, *k, *dout;
    const Mats<3> *mats;
    const float *dh_final;            // null: zero
    float *dS;                        // [batch, chunks, hv, dv, dk]: dS' of each chunk
    float *dh_init;                   // null: not wanted
    float *agg;                       // kAgg: as the chain's
    const float *h_seg;               // null, or [batch, hv, segs, dk, dv]: dS' behind each segment
    int segs, per;                    // segments, and chunks of each
    int groups;                       // batch * segs * hv
    DeltaDims d;
};

template <typename T, int kDk>
struct AdjointStage {
    Tile<T, kDk> k, q;
    Tile<T, 64> o;
    Mats<3> m;
};

template <typename T, int kDk, bool kAgg>
struct Adjoint {
    static constexpr int kTiles = kDk / 16, kSteps = kDk / 32, kIn = Stream<T>::kParts;
    using Stage = AdjointStage<T, kDk>;
    f32x4 S[kTiles];   // the adjoint of the state
    const AdjointArgs<T> &a;
    const T *kp, *qp, *op;
    int64_t kstride, vstride, len;
    int hv, b, wave, col, grp, n;
    bool has_o;   // kAgg: not the identity's columns

    __device__ __forceinline__ int tokens(int c) const {
        const int64_t left = len - (int64_t)c * kChunk;
        return left < kChunk ? (int)left : kChunk;
    }
    typename Tile<T, kDk>::template Offsets<4> koff;
    typename Tile<T, 64>::template Offsets<4> voff;

    __device__ __forceinline__ void fill(Stage &l, int c) {
        const int64_t t0 = (int64_t)c * kChunk;
        l.k.template fill<4>(kp + t0 * kstride, koff);
        if (!kAgg || has_o) {
            l.q.template fill<4>(qp + t0 * kstride, koff);
            l.o.template fill<4>(op + t0 * vstride, voff);
        }
        fill_mats(a.mats + ((int64_t)b * a.d.hv + hv) * a.d.chunks + c, &l.m);
    }
    __device__ __forceinline__ void store_columns(float *out) {
        const uint32_t lane_off = (uint32_t)(n * kDk + grp * 8);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) *(f32x4 *)(out + state_row(t, 0, 0) + lane_off) = S[t];
    }
    // rows `ld` apart
    __device__ __forceinline__ void store_state(float *out, int ld) {
        const uint32_t lane_off = (uint32_t)(grp * 8 * ld + n);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) (out + state_row(t, 0, r) * ld)[lane_off] = S[t][r];
    }
    __device__ __forceinline__ void step(const Stage &l, int c) {
        const int m = tokens(c);
        f32x4 U[4], dO[4];
        {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) U[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const Frag<3> Sp = split_frag<3>(S[2 * s], S[2 * s + 1]);
                Frag<kIn> kf[4];
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) kf[mt] = l.k.row(mt * 16 + col, s, grp);
                mma_n<4>(kf, Sp, U);
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const f32x4 rest = *(const f32x4 *)(l.m.rest + mt * 16 + grp * 4);
                if (!kAgg || has_o) dO[mt] = l.o.values(mt, grp, wave * 16, col);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    U[mt][r] *= rest[r];
                    dO[mt][r] = mt * 16 + grp * 4 + r < m ? dO[mt][r] : 0.f;
                }
            }
        }
        if (!kAgg || has_o) upper_product<3, false, kIn>(l.m.P, dO, U);
        f32x4 X[4];
        upper_product<3>(l.m.W, U, X);
        const float last = l.m.e[kChunk - 1];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const f32x4 e = *(const f32x4 *)(l.m.e + mt * 16 + grp * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                X[mt][r] *= -e[r];
                if (!kAgg || has_o) dO[mt][r] *= a.d.scale * e[r];
            }
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] *= last;
        if (!kAgg || has_o) add_columns(l.q, dO, S);
        add_columns(l.k, X, S);
    }
};

// Bound as the forward's chain by a step's latency: 8 rows of 4,096 bf16 tokens of
// 12 heads of 128 (192 workgroups, one a CU, unsegmented) in 359 us, 5.6 us a
// chunk, 100 KB of it read and written by each workgroup.  kTwo as in the forward's
// chain.
template <typename T, int kDk, bool kAgg, bool kTwo>
__global__ __launch_bounds__(kDeltaThreads, kTwo || sizeof(T) == 4 ? 1 : 2) void delta_adjoint_kernel(AdjointArgs<T> a) {
    using C = Adjoint<T, kDk, kAgg>;
    __shared__ __attribute__((aligned(16))) typename C::Stage l0;
    __shared__ __attribute__((aligned(16))) typename std::conditional<kTwo, typename C::Stage, char>::type l1;
    const DeltaDims &d = a.d;
    const ChainPlace at = chain_place((d.dv + (kAgg ? kDk : 0)) / 64);
    if (at.group >= a.groups) return;
    C s{{}, a};
    s.hv = at.group % d.hv;
    s.b = at.group / d.hv / a.segs;
    const int seg = at.group / d.hv % a.segs, hk = s.hv / d.group, lane = lane_id();
    if (kAgg && seg == 0) return;   // nothing is in front of it
    s.wave = threadIdx.x >> 6;
    s.col = lane & 15;
    s.grp = lane >> 4;
    s.n = at.col * 64 + s.wave * 16 + s.col;
    s.has_o = !kAgg || at.col * 64 < d.dv;
    s.len = row_len(d, s.b);
    s.kstride = (int64_t)d.hk * kDk;
    s.vstride = (int64_t)d.hv * d.dv;
    const int64_t tok = (int64_t)s.b * d.T;
    s.kp = a.k + (tok * d.hk + hk) * kDk;
    s.qp = a.q + (tok * d.hk + hk) * kDk;
    s.op = a.dout + (tok * d.hv + s.hv) * d.dv + (s.has_o ? at.col * 64 : 0);
    const int chunks = (int)((s.len + kChunk - 1) / kChunk);   // the row's, of all segments
    const int c0 = seg * a.per, c1 = c0 + a.per < chunks ? c0 + a.per : chunks;
    const int64_t state = (int64_t)kDk * d.dv, head = (int64_t)s.b * d.hv + s.hv;
    const float *first = a.h_seg != nullptr ? a.h_seg + (head * a.segs + seg) * state : a.dh_final + head * state;
#pragma unroll
    for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) s.S[t][r] = kAgg && s.n - d.dv == state_row(t, s.grp, r) ? 1.f : 0.f;
    if (!kAgg && (a.h_seg != nullptr || a.dh_final != nullptr)) load_state<kDk>(first, d.dv, s.grp, s.n, s.S);
    auto keep = [&](int c) {
        if (!kAgg) s.store_columns(a.dS + (((int64_t)s.b * d.chunks + c) * d.hv + s.hv) * state);
    };
    int c = c1 - 1;
    s.koff.set(s.kstride, c >= c0 ? s.tokens(c) : kChunk);   // the last chunk's; the others are full
    s.voff.set(s.vstride, c >= c0 ? s.tokens(c) : kChunk);
    if constexpr (kTwo) {
        if (c >= c0) s.fill(l0, c);
        s.koff.set(s.kstride, kChunk);
        s.voff.set(s.vstride, kChunk);
        for (; c >= c0; c -= 2) {
            // l0 is filled, l1 is read; the state's stores came after the loads
            if (c < c1 - 1) loads_done<C::kTiles>();
            else loads_done<0>();
            __syncthreads();
            if (c > c0) s.fill(l1, c - 1);
            keep(c);
            s.step(l0, c);
            if (c == c0) break;
            loads_done<C::kTiles>();
            __syncthreads();
            if (c - 1 > c0) s.fill(l0, c - 2);
            keep(c - 1);
            s.step(l1, c - 1);
        }
    } else {
        for (; c >= c0; --c) {
            __syncthreads();
            s.fill(l0, c);
            s.koff.set(s.kstride, kChunk);
            s.voff.set(s.vstride, kChunk);
            keep(c);
            loads_done<0>();
            __syncthreads();
            s.step(l0, c);
        }
    }
    if (kAgg) {
        float *map = a.agg + (head * a.segs + seg) * kDk * (d.dv + kDk);
        if (s.has_o) s.store_state(map, d.dv);
        else store_map<kDk>(map + kDk * d.dv, s.grp, s.n - d.dv, s.S);
    } else if (a.dh_init != nullptr && seg == 0) s.store_state(a.dh_init + head * state, d.dv);
}

// ------------------------------------------------------------ chunk gradients

template <typename T>
struct GradArgs {
    const T *q, *k, *v, *dout;
    const Mats<3> *mats;
    const double *G;
    const float *beta, *S, *dS;   // S: h_chunks
    T *dq, *dk, *dv;
    float *dg, *dbeta;
    DeltaDims d;
};

// U and X between the two halves of the kernel, [64][dv] by rows: for bf16 streams
// two parts (the results are rounded to bf16) and the third in a tile of its own,
// for dg; fp32 else.
template <typename T, int kDv>
struct RowTile;
template <int kDv>
struct RowTile<uint16_t, kDv> {
    using Third = Tile<uint16_t, kDv>;
    Tile<uint16_t, kDv> p[2];
    __device__ __forceinline__ void put(int r, int c, float v, Third &third) {
        const uint32_t h = pk_rne(v, v);
        const float low = v - bf_lo(h);
        const uint32_t mid = pk_rne(low, low);
        const int at = (int)(p[0].piece(r, c / 8) - p[0].e) + c % 8;
        p[0].e[at] = (uint16_t)h;
        p[1].e[at] = (uint16_t)mid;
        third.e[at] = (uint16_t)pk_rne(low - bf_lo(mid), 0.f);
    }
    __device__ __forceinline__ Frag<2> get(int r, int s, int grp) const {
        return Frag<2>{{p[0].row(r, s, grp).p[0], p[1].row(r, s, grp).p[0]}};
    }
    __device__ __forceinline__ Frag<3> all(int r, int s, int grp, const Third &third) const {
        return Frag<3>{{p[0].row(r, s, grp).p[0], p[1].row(r, s, grp).p[0], third.row(r, s, grp).p[0]}};
    }
};
template <int kDv>
struct RowTile<float, kDv> {
    using Third = char;
    Tile<float, kDv> p;
    __device__ __forceinline__ void put(int r, int c, float v, Third &) { p.e[(int)(p.piece(r, c / 4) - p.e) + c % 4] = v; }
    __device__ __forceinline__ Frag<3> get(int r, int s, int grp) const { return p.row(r, s, grp); }
    __device__ __forceinline__ Frag<3> all(int r, int s, int grp, const Third &) const { return get(r, s, grp); }
};

// x of another lane of the row of 16 (0 where there is none), and x plus that
template <int kCtrl>
__device__ __forceinline__ float of_lane(float x) {
    return as_f(__builtin_amdgcn_update_dpp(0, as_u(x), kCtrl, 0xf, 0xf, false));
}
template <int kCtrl>
__device__ __forceinline__ float plus_lanes(float x) {
    return x + of_lane<kCtrl>(x);
}
// sums over a row's lanes up to each (row_shr:1, 2, 4, 8), and from each on (row_shl)
__device__ __forceinline__ float sums_to(float x) { return plus_lanes<0x118>(plus_lanes<0x114>(plus_lanes<0x112>(plus_lanes<0x111>(x)))); }
__device__ __forceinline__ float sums_from(float x) { return plus_lanes<0x108>(plus_lanes<0x104>(plus_lanes<0x102>(plus_lanes<0x101>(x)))); }
// x of the same lane in each of the four rows
__device__ __forceinline__ f32x4 of_rows(float x) {
    const auto h = __builtin_amdgcn_permlane16_swap(as_u(x), as_u(x), false, false);
    const auto even = __builtin_amdgcn_permlane32_swap(h[0], h[0], false, false);
    const auto odd = __builtin_amdgcn_permlane32_swap(h[1], h[1], false, false);
    return f32x4{as_f(even[0]), as_f(odd[0]), as_f(even[1]), as_f(odd[1])};
}
// Four values' sums over the 16 lanes of a row together, the values halved as the
// lanes: lane col < 4 of the row holds that of x[col].
__device__ __forceinline__ float sum_columns(f32x4 x, int col) {
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = plus_lanes<0xb1>(x[r]);            // lane ^ 1
    const bool odd = col & 1;
    const float a = plus_lanes<0x4e>(odd ? x[1] : x[0]), b = plus_lanes<0x4e>(odd ? x[3] : x[2]);   // lane ^ 2
    return plus_lanes<0x128>(plus_lanes<0x124>(col & 2 ? b : a));          // row_ror:4, row_ror:8
}

// eight consecutive fp32 values as parts
template <int kParts>
__device__ __forceinline__ Frag<kParts> load_state(const float *p) {
    return split_frag<kParts>(*(const f32x4 *)p, *(const f32x4 *)(p + 4));
}

template <typename T, int kDk, int kDv>
struct GradLds {
    static constexpr int kOut = Stream<T>::kOutParts;
    Tile<T, kDk> k, q;
    // dO, V (fp32 streams: from memory); V's room then holds U's third part
    typename std::conditional<sizeof(T) == 2, Tile<T, kDv>, char>::type o, v;
    union {
        Mats<3> m;
        struct {
            RowTile<T, kDv> U, X;
            union {
                uint4 pairs[8][kOut][64];   // B fragments of a token by token matrix: (column tile, step)
                struct {                    // of dg and dbeta, before the pairs
                    typename RowTile<T, kDv>::Third x;   // X's third part
                    float db[kDv / 16][kChunk];          // dbeta of a wave's columns
                    // of a 16 x 16 block of w: sums over its rows from each row on, over
                    // its columns before each column, and over all of it
                    float from[kBlocks][16], before[kBlocks][16], all[kBlocks];
                } g;
            };
        };
    };
    double G[kChunk];
    float e[kChunk], rest[kChunk], ib[kChunk];   // ib: 1 / beta
    float r[kDv / 16][kChunk], c[kDv / 16][kChunk];   // r_i and c_j of a wave's columns
    float ends[kDv / 16];
};

// One workgroup per (chunk, query/key head, batch) and a wave per 16 columns of
// v: each value head of the group in turn, dQ and dK summed over them in
// registers.  First by columns as in the chains (U, dU, X and the row products of
// r, c and dbeta), then the blocks of w for dg, a wave to each, then by rows: a wave takes 16 of dk (two such, or half the tokens,
// where waves and dk do not pair up) and forms dQ^T, dK^T as products over dv
// (rows of S, dS' from memory, each read once) and over the chunk's tokens.  The
// token by token matrices (DP for dQ, DP and DA + DA^T for dK) are formed in
// turn, two result tiles to a B fragment as they stand, and shared through LDS.
// One workgroup a CU: the tiles, the matrices and U, X take nearly all of its LDS,
// and the states are read straight into fragments.  8 rows of 4,096 bf16 tokens of
// 12 heads of 128: 828 us for 1.7 GB (2.1 TB/s), in which matrix instructions are
// busy for 162 us, LDS for 193 and other vector instructions for 249; its waves wait
// for memory or a barrier 47% of the time, most of it while a chunk is loaded.  The
// blocks of w are 65 us of it: their three parts of U and X are read for themselves.
// fp32 streams of 128 by 128 spill (10 vector registers, 43 with shared heads): the
// same training layer takes 3.4 ms in fp32.
template <typename T, int kDk, int kDv, bool kShared>
__global__ __launch_bounds__(kDv * 4, 1) void delta_grad_kernel(GradArgs<T> a) {
    using L = GradLds<T, kDk, kDv>;
    constexpr bool kBf16 = sizeof(T) == 2;
    constexpr int kThreads = kDv * 4, kWaves = kDv / 16, kSteps = kDk / 32, kVSteps = kDv / 32;
    constexpr int kIn = Stream<T>::kParts, kOut = Stream<T>::kOutParts;
    constexpr int kDkTiles = kDk / 16;
    constexpr int kMine = kDkTiles > kWaves ? kDkTiles / kWaves : 1;       // dk tiles of a wave
    constexpr int kToks = kWaves > kDkTiles ? 4 * kDkTiles / kWaves : 4;   // its token tiles
    __shared__ __attribute__((aligned(16))) L l;
    const DeltaDims &d = a.d;
    const int c = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t len = row_len(d, b), t0 = (int64_t)c * kChunk;
    const int rows = d.T - t0 < kChunk ? (int)(d.T - t0) : kChunk;
    const int m = len <= t0 ? 0 : len - t0 < kChunk ? (int)(len - t0) : kChunk;
    const int64_t kstride = (int64_t)d.hk * kDk, vstride = (int64_t)d.hv * kDv, state = (int64_t)kDk * kDv;
    const int64_t kat = (((int64_t)b * d.T + t0) * d.hk + hk) * kDk;
    const int dk0 = wave * kMine % kDkTiles, tk0 = kToks == 4 ? 0 : wave * kMine / kDkTiles * kToks;

    f32x4 dQ[kMine][kToks], dK[kMine][kToks];
    if (kShared || m == 0) {
#pragma unroll
        for (int i = 0; i < kMine; ++i)
#pragma unroll
            for (int j = 0; j < kToks; ++j) dQ[i][j] = dK[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (m > 0) {
        typename Tile<T, kDk>::template Offsets<kWaves> off;
        off.set(kstride, m);
        l.k.template fill<kWaves>(a.k + kat, off);
        l.q.template fill<kWaves>(a.q + kat, off);
    }
    for (int hv = hk * d.group; hv < (kShared ? (hk + 1) * d.group : hk + 1); ++hv) {
        // opaque to the compiler: it would keep some 200 lane addresses of the
        // loop's body in registers (and spill them) rather than form them again
        int lane = lane_id();
        asm volatile("" : "+v"(lane));
        const int col = lane & 15, grp = lane >> 4, n = wave * 16 + col;
        const int64_t at = ((int64_t)b * d.T + t0) * d.hv + hv;   // of the gates; times dv of v
        const int64_t unit = ((int64_t)b * d.hv + hv) * d.chunks + c;
        T *dvp = a.dv + at * kDv;
        const T *dop = a.dout + at * kDv, *vp = a.v + at * kDv;
        for (int e = threadIdx.x; e < (rows - m) * kDv; e += kThreads)
            Stream<T>::store(dvp + (m + e / kDv) * vstride + e % kDv, 0.f);
        for (int t = m + threadIdx.x; t < rows; t += kThreads) a.dg[at + (int64_t)t * d.hv] = a.dbeta[at + (int64_t)t * d.hv] = 0.f;
        if (m == 0) continue;
        const int64_t chunk_at = (((int64_t)b * d.chunks + c) * d.hv + hv) * state;
        const float *Sg = a.S + chunk_at, *dSg = a.dS + chunk_at;
        const uint32_t col_off = (uint32_t)(n * kDk + grp * 8);
        // the gates before all else: a wait for them is one for what was asked for earlier
        double g_sum = 0.;
        float beta = 1.f;
        if (threadIdx.x < kChunk) {
            const int t = (int)threadIdx.x < m ? threadIdx.x : m - 1;
            g_sum = a.G[unit * kChunk + threadIdx.x];
            beta = a.beta[at + (int64_t)t * d.hv];
        }
        __syncthreads();   // the last head's reads of LDS are done
        fill_mats<kWaves>(a.mats + unit, &l.m);
        if constexpr (kBf16) {
            typename Tile<T, kDv>::template Offsets<kWaves> off;
            off.set(vstride, m);
            l.o.template fill<kWaves>(dop, off);
            l.v.template fill<kWaves>(vp, off);
        }
        f32x4 raw[2 * kSteps];   // the state's columns, then its adjoint's, on their way
        const auto load_columns = [&](const float *p) {
#pragma unroll
            for (int t = 0; t < 2 * kSteps; ++t) raw[t] = *(const f32x4 *)(p + state_row(t, 0, 0) + col_off);
        };
        load_columns(Sg);
        if (threadIdx.x < kChunk) {
            const int t = threadIdx.x;
            l.G[t] = g_sum;
            l.ib[t] = t < m ? 1.f / strength(beta) : 1.f;
        }
        const auto value_tile = [&](int mt) {
            if constexpr (kBf16) {
                return l.v.values(mt, grp, wave * 16, col);
            } else {
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = mt * 16 + grp * 4 + r;
                    x[r] = vp[(t < m ? t : m - 1) * vstride + n];
                }
                return x;
            }
        };
        const auto dout_tile = [&](int mt) {
            f32x4 x;
            if constexpr (kBf16) x = l.o.values(mt, grp, wave * 16, col);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = mt * 16 + grp * 4 + r;
                if constexpr (!kBf16) x[r] = dop[(t < m ? t : m - 1) * vstride + n];
                x[r] = t < m ? x[r] : 0.f;
            }
            return x;
        };
        loads_done<0>();
        __syncthreads();
        if (threadIdx.x < kChunk) {   // these outlast the matrices
            l.e[threadIdx.x] = l.m.e[threadIdx.x];
            l.rest[threadIdx.x] = l.m.rest[threadIdx.x];
        }
        // by columns: R, U and the row products as they come
        f32x4 U[4], X[4], es[4];   // es: E K S
        {
            f32x4 R[4];
            {
                f32x4 ks[4], qs[4];
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) ks[mt] = qs[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const Frag<3> Sp = split_frag<3>(raw[2 * s], raw[2 * s + 1]);
                    Frag<kIn> f[4];
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) f[mt] = l.k.row(mt * 16 + col, s, grp);
                    mma_n<4>(f, Sp, ks);
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) f[mt] = l.q.row(mt * 16 + col, s, grp);
                    mma_n<4>(f, Sp, qs);
                    __builtin_amdgcn_sched_barrier(0);
                }
                load_columns(dSg);
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    const f32x4 e = *(const f32x4 *)(l.m.e + mt * 16 + grp * 4), v = value_tile(mt), dO = dout_tile(mt);
                    f32x4 x;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        es[mt][r] = e[r] * ks[mt][r];
                        R[mt][r] = v[r] - es[mt][r];
                        x[r] = d.scale * e[r] * qs[mt][r] * dO[r];
                    }
                    const float sum = sum_columns(x, col);
                    if (col < 4) l.r[wave][mt * 16 + grp * 4 + col] = sum;
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            lower_product<3>(l.m.W, R, U);
        }
        __builtin_amdgcn_sched_barrier(0);
        {
            f32x4 dU[4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) dU[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const Frag<3> Sp = split_frag<3>(raw[2 * s], raw[2 * s + 1]);
                Frag<kIn> kf[4];
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) kf[mt] = l.k.row(mt * 16 + col, s, grp);
                mma_n<4>(kf, Sp, dU);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const f32x4 rest = *(const f32x4 *)(l.m.rest + mt * 16 + grp * 4);
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dU[mt][r] *= rest[r];
                    x[r] = U[mt][r] * dU[mt][r];
                }
                const float sum = sum_columns(x, col);
                if (col < 4) l.c[wave][mt * 16 + grp * 4 + col] = sum;
            }
            __builtin_amdgcn_sched_barrier(0);
            {
                f32x4 dO[4];
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) dO[mt] = dout_tile(mt);
                upper_product<3, false, kIn>(l.m.P, dO, dU);
            }
            __builtin_amdgcn_sched_barrier(0);
            upper_product<3>(l.m.W, dU, X);
        }
        __syncthreads();   // the matrices are read: U and X take their place
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            f32x4 sr, sdb;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = mt * 16 + grp * 4 + r;
                const float u = U[mt][r], x = X[mt][r], ib = l.ib[t];
                sr[r] = -es[mt][r] * x;
                sdb[r] = u * ib * (x * ib);
                l.U.put(t, n, u, l.v);
                l.X.put(t, n, x, l.g.x);
                if (t < m) Stream<T>::store(dvp + t * vstride + n, ib == 0x1p64f ? 0.f : x);   // beta 0: as `strength` has it
            }
            const float sum = sum_columns(sr, col), db = sum_columns(sdb, col);
            if (col < 4) {
                l.r[wave][mt * 16 + grp * 4 + col] += sum;
                l.g.db[wave][mt * 16 + grp * 4 + col] = db;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
        const auto dout_row = [&](int r, int s) {
            if constexpr (kBf16) return l.o.row(r, s, grp);
            else return load_straight(dop + (r < m ? r : m - 1) * vstride + s * 32 + grp * 8);
        };
        // dg's blocks of w (rows i, columns j)
#pragma unroll 1
        for (int f = wave; f < kBlocks; f += kWaves) {
            int it, jt;
            block_of(f, &it, &jt);
            const int i0 = it * 16, j = jt * 16 + col;
            f32x4 ou = {0.f, 0.f, 0.f, 0.f}, xu[2] = {ou, ou}, qk = ou, kk = ou;   // xu: two sums side by side
#pragma unroll
            for (int s = 0; s < kVSteps; ++s) {
                const Frag<3> u = l.U.all(j, s, grp, l.v);
                ou = mma(dout_row(i0 + col, s), u, ou);
                xu[s & 1] = mma(l.X.all(i0 + col, s, grp, l.g.x), u, xu[s & 1]);
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const auto kj = l.k.row(j, s, grp);
                qk = mma(l.q.row(i0 + col, s, grp), kj, qk);
                kk = mma(l.k.row(i0 + col, s, grp), kj, kk);
            }
            f32x4 w;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = i0 + grp * 4 + r;
                w[r] = j < i && i < m ? decay(l.G[i] - l.G[j]) * (d.scale * qk[r] * ou[r] - kk[r] * (xu[0][r] + xu[1][r])) : 0.f;
            }
            // of each column, over the rows from its lane's on
            w[2] += w[3];
            w[1] += w[2];
            w[0] += w[1];
            const f32x4 g = of_rows(w[0]);   // the lane groups' sums
            const float last = grp < 3 ? g[3] : 0.f, behind = grp < 2 ? g[2] + last : last, rows_behind = grp < 1 ? g[1] + behind : behind;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                w[r] += rows_behind;
                if (it == jt && col >= grp * 4 + r) w[r] = 0.f;   // on the diagonal, columns before the row
            }
            const float from = sum_columns(w, col), to = sums_to((g[0] + g[1]) + (g[2] + g[3])), before = of_lane<0x111>(to);
            if (col < 4) l.g.from[f][grp * 4 + col] = from;
            if (grp == 0) l.g.before[f][col] = before;
            if (lane == 15) l.g.all[f] = to;
        }
        __syncthreads();
        float gate = 0.f, r_sum = 0.f, c_sum = 0.f;   // gate: dg of token threadIdx.x but for the state's way through the chunk
        if (threadIdx.x < kChunk) {
            const int t = threadIdx.x, tb = t >> 4;
            float db = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                r_sum += l.r[w][t];
                c_sum += l.c[w][t];
                db += l.g.db[w][t];
            }
            if (t < m) a.dbeta[at + (int64_t)t * d.hv] = db;
#pragma unroll
            for (int f = 0; f < kBlocks; ++f) {
                int it, jt;
                block_of(f, &it, &jt);
                if (it == tb) gate += l.g.from[f][t & 15];
                else if (jt == tb) gate += l.g.before[f][t & 15];
                else if (it > tb && jt < tb) gate += l.g.all[f];
            }
        }
        __syncthreads();   // read: the pairs take their place
        if (threadIdx.x < kChunk) {   // r from token t on, c before it
            const float from = sums_from(r_sum), to = sums_to(c_sum);
            const auto of = [](float x, int i) { return as_f(__builtin_amdgcn_readlane(as_u(x), i)); };   // a row's whole sum
            const float r3 = grp < 3 ? of(from, 48) : 0.f, r2 = grp < 2 ? of(from, 32) + r3 : r3;
            const float c0 = grp > 0 ? of(to, 15) : 0.f, c1 = grp > 1 ? of(to, 31) + c0 : c0;
            gate += from + (grp < 1 ? of(from, 16) + r2 : r2);
            gate += of_lane<0x111>(to) + (grp > 2 ? of(to, 47) + c1 : c1);
        }
        // by rows: products over dv
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int tile = dk0 + i;
            // row of dk in [dv][dk]: eight dv apart by rows
            const uint32_t r0 = (uint32_t)(grp * 8 * kDk + tile / 2 * 32 + col / 4 * 8 + (tile & 1) * 4 + col % 4);
            f32x4 so[kToks], sx[kToks], du[kToks], x[2], y[2];
#pragma unroll
            for (int j = 0; j < kToks; ++j) so[j] = sx[j] = du[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            const auto load_rows = [&](int s) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[h][r] = (Sg + (s * 32 + h * 4 + r) * kDk)[r0];
                        y[h][r] = (dSg + (s * 32 + h * 4 + r) * kDk)[r0];
                    }
            };
            load_rows(0);
#pragma unroll
            for (int s = 0; s < kVSteps; ++s) {
                const Frag<kOut> sf = split_frag<kOut>(x[0], x[1]), df = split_frag<kOut>(y[0], y[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) dot = fmaf(x[h][r], y[h][r], dot);
                if (s + 1 < kVSteps) load_rows(s + 1);
#pragma unroll
                for (int j = 0; j < kToks; ++j) {
                    const int t = (tk0 + j) * 16 + col;
                    so[j] = mma(sf, dout_row(t, s), so[j]);
                    sx[j] = mma(sf, l.X.get(t, s, grp), sx[j]);
                    du[j] = mma(df, l.U.get(t, s, grp), du[j]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < kToks; ++j) {
                const float et = l.e[(tk0 + j) * 16 + col], rt = l.rest[(tk0 + j) * 16 + col];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float q = d.scale * et * so[j][r], k = rt * du[j][r] - et * sx[j][r];
                    dQ[i][j][r] = kShared ? dQ[i][j][r] + q : q;
                    dK[i][j][r] = kShared ? dK[i][j][r] + k : k;
                }
            }
        }
        float end = tk0 == 0 ? l.e[kChunk - 1] * dot : 0.f;   // exp(G_C) <S, dS'>, each row of dk once
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) end += __shfl_xor(end, s, 64);
        if (lane == 0) l.ends[wave] = end;
        // products over the chunk's tokens.  kind 0: DP^T (rows j, columns i) for
        // dQ; 1: DP (rows i, columns j), 2: DA + DA^T, for dK.
        const auto pass = [&](auto which) {
            constexpr int kind = decltype(which)::value, frags = kind == 2 ? 8 : kFrags;
#pragma unroll 1
            for (int f = wave; f < frags; f += kWaves) {
                // column tile and step of the fragment
                const int ct = kind == 2 ? f / 2 : kind == 0 ? (f < 2 ? f : f / 2 + 1) : (f < 4 ? f / 2 : f - 2);
                const int st = kind == 2 ? f & 1 : kind == 0 ? (f < 2 ? 0 : f & 1) : (f < 4 ? f & 1 : 1);
                const int t = ct * 16 + col;
                f32x4 tile[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int rt = st * 2 + i;
                    f32x4 below = {0.f, 0.f, 0.f, 0.f}, above = below;   // rows before / behind the column's token
                    if (rt <= ct && kind != 1) {
#pragma unroll
                        for (int s = 0; s < kVSteps; ++s) {
                            if (kind == 0) below = mma(l.U.get(rt * 16 + col, s, grp), dout_row(t, s), below);
                            else below = mma(l.U.get(rt * 16 + col, s, grp), l.X.get(t, s, grp), below);
                        }
                    }
                    if (rt >= ct && kind != 0) {
#pragma unroll
                        for (int s = 0; s < kVSteps; ++s) {
                            if (kind == 1) above = mma(dout_row(rt * 16 + col, s), l.U.get(t, s, grp), above);
                            else above = mma(l.X.get(rt * 16 + col, s, grp), l.U.get(t, s, grp), above);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = rt * 16 + grp * 4 + r;
                        const float D = decay(j <= t ? l.G[t] - l.G[j] : l.G[j] - l.G[t]);
                        const bool in = j < m && t < m;   // repeated rows count for nothing
                        if (kind == 0) tile[i][r] = j <= t && in ? d.scale * D * below[r] : 0.f;
                        else if (kind == 1) tile[i][r] = j >= t && in ? d.scale * D * above[r] : 0.f;
                        else tile[i][r] = j == t || !in ? 0.f : -D * (j < t ? below[r] : above[r]);
                    }
                }
                const Frag<kOut> x = split_frag<kOut>(tile[0], tile[1]);
#pragma unroll
                for (int p = 0; p < kOut; ++p) l.pairs[f][p][lane] = __builtin_bit_cast(uint4, x.p[p]);
            }
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                Frag<kIn> x[kMine];
#pragma unroll
                for (int i = 0; i < kMine; ++i) x[i] = kind == 1 ? l.q.column(dk0 + i, s, grp, col) : l.k.column(dk0 + i, s, grp, col);
#pragma unroll
                for (int j = 0; j < kToks; ++j) {
                    // beyond the triangle: no fragment (with two token tiles a wave, both or none)
                    const int half = kToks == 4 ? j / 2 : tk0 / 2;
                    if (kind == 0 ? s > half : kind == 1 ? s < half : false) continue;
                    const int ct = tk0 + j, f = kind == 2 ? ct * 2 + s : kind == 0 ? frag_lower(ct, s) : ct < 2 ? ct * 2 + s : ct + 2;
                    Frag<kOut> y;
#pragma unroll
                    for (int p = 0; p < kOut; ++p) y.p[p] = __builtin_bit_cast(bf16x8, l.pairs[f][p][lane]);
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        if constexpr (kind == 0) dQ[i][j] = mma(x[i], y, dQ[i][j]);
                        else dK[i][j] = mma(x[i], y, dK[i][j]);
                    }
                }
            }
            __syncthreads();
        };
        pass(std::integral_constant<int, 0>{});
        pass(std::integral_constant<int, 1>{});
        pass(std::integral_constant<int, 2>{});
        if (threadIdx.x < kChunk) {
            const int t = threadIdx.x;
            float ends = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) ends += l.ends[w];
            if (t < m) a.dg[at + (int64_t)t * d.hv] = gate + ends;
        }
    }
    const int col = lane_id() & 15, grp = lane_id() >> 4;
#pragma unroll
    for (int j = 0; j < kToks; ++j) {
        const int t = (tk0 + j) * 16 + col;
        if (t >= rows) continue;
        T *dqp = a.dq + kat + t * kstride, *dkp = a.dk + kat + t * kstride;
        const f32x4 z = {0.f, 0.f, 0.f, 0.f};   // padding
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            store4(dqp + state_row(dk0 + i, grp, 0), t < m ? dQ[i][j] : z);
            store4(dkp + state_row(dk0 + i, grp, 0), t < m ? dK[i][j] : z);
        }
    }
}

}  // namespace bdssm_dev
