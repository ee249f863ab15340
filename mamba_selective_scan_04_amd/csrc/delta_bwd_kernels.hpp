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
// Every decay enters through G: reading tokens carry exp(G_i), writing tokens
// exp(-G_j), so its gradient is row products of what is at hand,
//   dG_i = dO_i.O_i - X_i.(V - y)_i - U_i.Z_i   (+ <S', dS'> at the last token),
//   dg_i = sum of dG_j over j >= i in the chunk,
// and needs neither dQ nor dK: those may be computed to their own type's
// precision while dg and dbeta keep 32 bits.
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
// 12 heads of 128 (192 workgroups, one a CU, unsegmented) in 390 to 408 us, 6.2 us a
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

// U and X between the two halves of the kernel, [64][dv] by rows: two parts for
// bf16 streams (their results are rounded to bf16), fp32 else.
template <typename T, int kDv>
struct RowTile;
template <int kDv>
struct RowTile<uint16_t, kDv> {
    Tile<uint16_t, kDv> p[2];
    __device__ __forceinline__ void put(int r, int c, float v) {
        const uint32_t h = pk_rne(v, v);
        const int at = (int)(p[0].piece(r, c / 8) - p[0].e) + c % 8;
        p[0].e[at] = (uint16_t)h;
        p[1].e[at] = (uint16_t)pk_rne(v - bf_lo(h), 0.f);
    }
    __device__ __forceinline__ Frag<2> get(int r, int s, int grp) const {
        return Frag<2>{{p[0].row(r, s, grp).p[0], p[1].row(r, s, grp).p[0]}};
    }
};
template <int kDv>
struct RowTile<float, kDv> {
    Tile<float, kDv> p;
    __device__ __forceinline__ void put(int r, int c, float v) { p.e[(int)(p.piece(r, c / 4) - p.e) + c % 4] = v; }
    __device__ __forceinline__ Frag<3> get(int r, int s, int grp) const { return p.row(r, s, grp); }
};

// eight consecutive fp32 values as parts
template <int kParts>
__device__ __forceinline__ Frag<kParts> load_state(const float *p) {
    return split_frag<kParts>(*(const f32x4 *)p, *(const f32x4 *)(p + 4));
}

template <typename T, int kDk, int kDv>
struct GradLds {
    static constexpr int kOut = Stream<T>::kOutParts;
    Tile<T, kDk> k, q;
    typename std::conditional<sizeof(T) == 2, Tile<T, kDv>, char>::type o, v;   // dO, V (fp32 streams: from memory)
    union {
        Mats<3> m;
        struct {
            RowTile<T, kDv> U, X;
            uint4 pairs[8][kOut][64];   // B fragments of a token by token matrix: (column tile, step)
        };
    };
    double G[kChunk];
    float e[kChunk], rest[kChunk], ib[kChunk];   // ib: 1 / beta
    float dG[kDv / 16][kChunk], db[kDv / 16][kChunk];
    float ends[kDv / 16];
};

// One workgroup per (chunk, query/key head, batch) and a wave per 16 columns of
// v: each value head of the group in turn, dQ and dK summed over them in
// registers.  First by columns as in the chains (U, O, dU, X and the row
// products), then by rows: a wave takes 16 of dk (two such, or half the tokens,
// where waves and dk do not pair up) and forms dQ^T, dK^T as products over dv
// (rows of S, dS' from memory, each read once) and over the chunk's tokens.  The
// token by token matrices (DP for dQ, DP and DA + DA^T for dK) are formed in
// turn, two result tiles to a B fragment as they stand, and shared through LDS.
// One workgroup a CU: the tiles, the matrices and U, X take nearly all of its LDS,
// and the states are read straight into fragments.  8 rows of 4,096 bf16 tokens of
// 12 heads of 128: 805 to 841 us for 1.7 GB (2.1 TB/s), in which matrix instructions are
// busy for 160 us, LDS for 200 and other vector instructions for 210; what it
// waits for is its own start (loading a chunk with nothing else to do: 40%).
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
        // by columns: R, U, O and dO's part of dG
        f32x4 U[4], X[4], dG[4];
        {
            f32x4 R[4], O[4];
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
                    const f32x4 e = *(const f32x4 *)(l.m.e + mt * 16 + grp * 4), v = value_tile(mt);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        R[mt][r] = fmaf(-e[r], ks[mt][r], v[r]);
                        O[mt][r] = d.scale * e[r] * qs[mt][r];
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            lower_product<3>(l.m.W, R, U);
            __builtin_amdgcn_sched_barrier(0);
            lower_product<3, false>(l.m.P, U, O);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const f32x4 dO = dout_tile(mt);
#pragma unroll
                for (int r = 0; r < 4; ++r) dG[mt][r] = dO[r] * O[mt][r];
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        float end = 0.f;   // <S, dS'> exp(G_C) (by rows, below) + sum of U (K dS') rows
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
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dU[mt][r] *= rest[r];
                    end = fmaf(U[mt][r], dU[mt][r], end);
                }
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
        float sdG[4], sdb[4];   // row sums over this wave's columns, lane r = col of each result row set
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const f32x4 v = value_tile(mt);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = mt * 16 + grp * 4 + r;
                const float u = U[mt][r], x = X[mt][r], ib = l.ib[t], y = u * ib, z = x * ib;
                sdG[r] = dG[mt][r] - x * (v[r] - y) - u * z;
                sdb[r] = y * z;
                l.U.put(t, n, u);
                l.X.put(t, n, x);
                if (t < m) Stream<T>::store(dvp + t * vstride + n, ib == 0x1p64f ? 0.f : x);   // beta 0: as `strength` has it
            }
            // four sums over 16 lanes together: halve the values as the lanes
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                sdG[r] += __shfl_xor(sdG[r], 1, 64);
                sdb[r] += __shfl_xor(sdb[r], 1, 64);
            }
            const bool odd = col & 1, two = col & 2;
            float g0 = odd ? sdG[1] : sdG[0], g1 = odd ? sdG[3] : sdG[2], b0 = odd ? sdb[1] : sdb[0], b1 = odd ? sdb[3] : sdb[2];
            g0 += __shfl_xor(g0, 2, 64);
            g1 += __shfl_xor(g1, 2, 64);
            b0 += __shfl_xor(b0, 2, 64);
            b1 += __shfl_xor(b1, 2, 64);
            float g = two ? g1 : g0, db = two ? b1 : b0;
            g += __shfl_xor(g, 4, 64);
            db += __shfl_xor(db, 4, 64);
            g += __shfl_xor(g, 8, 64);
            db += __shfl_xor(db, 8, 64);
            if (col < 4) {   // lane col holds row 2 (col / 2) + col % 2
                l.dG[wave][mt * 16 + grp * 4 + col] = g;
                l.db[wave][mt * 16 + grp * 4 + col] = db;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
        // by rows: products over dv
        const auto dout_row = [&](int r, int s) {
            if constexpr (kBf16) return l.o.row(r, s, grp);
            else return load_straight(dop + (r < m ? r : m - 1) * vstride + s * 32 + grp * 8);
        };
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
        if (tk0 == 0) end = fmaf(l.e[kChunk - 1], dot, end);   // each row of dk once
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
            float s = 0.f, db = 0.f, ends = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                s += l.dG[w][t];
                db += l.db[w][t];
                ends += l.ends[w];
            }
            if (t == kChunk - 1) s += ends;
#pragma unroll
            for (int w = 1; w < 64; w <<= 1) {
                const float up = __shfl_down(s, w, 64);
                if (t + w < 64) s += up;
            }
            if (t < m) {
                a.dg[at + (int64_t)t * d.hv] = s;
                a.dbeta[at + (int64_t)t * d.hv] = db;
            }
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
