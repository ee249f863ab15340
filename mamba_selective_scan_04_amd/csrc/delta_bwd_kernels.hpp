// delta_bwd_kernels.hpp -- gradients of the gated delta rule.
//
// In the notation of delta_kernels.hpp, with dO given and dS' the adjoint of
// the state after the chunk:
//   dU = P^T dO + diag(exp(G_C - G_j)) K dS'
//   X  = W^T dU            (= dR = dV)
//   dS = exp(G_C) dS' + scale Q^T E dO - K^T E X
// is a chain over the chunks from the last, with independent columns as in the
// forward: delta_adjoint_kernel writes dS' of every chunk.  All else follows per
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
    const double *G;
    const float *Wt, *dh_final;       // dh_final null: zero
    float *dS;                        // [batch, chunks, hv, dk, dv]: dS' of each chunk
    float *dh_init;                   // null: not wanted
    DeltaDims d;
};

template <typename T, int kDk>
struct AdjointLds {
    T k[kChunk * TileLoad<T, kDk>::kRow];
    T q[kChunk * TileLoad<T, kDk>::kRow];
    T kT[kTransSize<T, kDk>];
    T qT[kTransSize<T, kDk>];
    uint16_t Wt[3 * kChunk * kTri];
    uint16_t Pt[3 * kChunk * kTri];
    double G[kChunk];
    float e[kChunk], rest[kChunk];
};

template <typename T, int kDk>
__global__ __launch_bounds__(kDeltaThreads, 1) void delta_adjoint_kernel(AdjointArgs<T> a) {
    using L = AdjointLds<T, kDk>;
    constexpr int kRow = TileLoad<T, kDk>::kRow, kTiles = kDk / 16, kSteps = kDk / 32, kIn = Stream<T>::kParts;
    __shared__ __attribute__((aligned(16))) L l;
    const DeltaDims &d = a.d;
    const int hv = blockIdx.y, b = blockIdx.z, hk = hv / d.group;
    const int lane = lane_id(), wave = threadIdx.x >> 6, col = lane & 15, grp = lane >> 4;
    const int n = blockIdx.x * 64 + wave * 16 + col;
    const int64_t len = row_len(d, b);
    const int chunks = (int)((len + kChunk - 1) / kChunk);
    const int64_t kstride = (int64_t)d.hk * kDk, vstride = (int64_t)d.hv * d.dv, state = (int64_t)kDk * d.dv;
    const T *kp = a.k + ((int64_t)b * d.T * d.hk + hk) * kDk;
    const T *qp = a.q + ((int64_t)b * d.T * d.hk + hk) * kDk;
    const T *op = a.dout + ((int64_t)b * d.T * d.hv + hv) * d.dv + n;
    const double *Gp = a.G + ((int64_t)b * d.hv + hv) * d.chunks * kChunk;
    const float *Wp = a.Wt + ((int64_t)b * d.hv + hv) * d.chunks * kWFloats;
    zero_planes(l.Wt, 3);
    zero_planes(l.Pt, 3);

    f32x4 S[kTiles];   // the adjoint of the state
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[t][r] = a.dh_final == nullptr ? 0.f
                                            : a.dh_final[((int64_t)b * d.hv + hv) * state + (int64_t)(t * 16 + grp * 4 + r) * d.dv + n];
    TileLoad<T, kDk> kl, ql;
    WLoad<true> wl;
    T vr[16];
    double Gr = 0.;
    auto fetch = [&](int c) {
        const int64_t t0 = (int64_t)c * kChunk;
        const int m = len - t0 < kChunk ? (int)(len - t0) : kChunk;
        kl.load(kp + t0 * kstride, kstride, m);
        ql.load(qp + t0 * kstride, kstride, m);
        wl.load(Wp + (int64_t)c * kWFloats);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int t = i / 4 * 16 + grp * 4 + i % 4;
            vr[i] = t < m ? op[(t0 + t) * vstride] : T(0);
        }
        if (threadIdx.x < kChunk) Gr = Gp[(int64_t)c * kChunk + threadIdx.x];
    };
    if (chunks > 0) fetch(chunks - 1);

    for (int c = chunks - 1; c >= 0; --c) {
        __syncthreads();
        kl.store(l.k);
        ql.store(l.q);
        wl.store(l.Wt);
        const double *G = l.G;
        if (threadIdx.x < kChunk) {
            l.G[threadIdx.x] = Gr;
            l.e[threadIdx.x] = decay(Gr);
            l.rest[threadIdx.x] = decay(__shfl(Gr, 63, 64) - Gr);
        }
        f32x4 dO[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) dO[i / 4][i % 4] = Stream<T>::load(vr + i);
        __syncthreads();
        if (c > 0) fetch(c - 1);
        transpose_tile<kDk>(l.k, l.kT);
        transpose_tile<kDk>(l.q, l.qT);
        form_p<T, kDk, true, 3>(l.k, l.q, G, d.scale, l.Pt);
        {
            float *out = a.dS + (((int64_t)b * d.chunks + c) * d.hv + hv) * state + n;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) out[(int64_t)(t * 16 + grp * 4 + r) * d.dv] = S[t][r];
        }
        f32x4 U[4];   // dU
        {
            Frag<3> Sp[kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) Sp[s] = split_frag<3>(S[2 * s], S[2 * s + 1]);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    acc = mma(load_paired(l.k + (mt * 16 + col) * kRow + s * 32 + grp * 4), Sp[s], acc);
                const f32x4 e = *(const f32x4 *)(l.rest + mt * 16 + grp * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) U[mt][r] = e[r] * acc[r];
            }
        }
        __syncthreads();   // the transposes and P^T are written
        {
            Frag<kIn> Op[2] = {split_frag<kIn>(dO[0], dO[1]), split_frag<kIn>(dO[2], dO[3])};
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int s = mt / 2; s < 2; ++s)
                    U[mt] = mma(load_planes<3>(l.Pt + (mt * 16 + col) * kTri + s * 32 + grp * 4, kChunk * kTri), Op[s], U[mt]);
        }
        f32x4 X[4];
        {
            Frag<3> Up[2] = {split_frag<3>(U[0], U[1]), split_frag<3>(U[2], U[3])};
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = mt / 2; s < 2; ++s)
                    acc = mma(load_planes<3>(l.Wt + (mt * 16 + col) * kTri + s * 32 + grp * 4, kChunk * kTri), Up[s], acc);
                X[mt] = acc;
            }
        }
        const float last = l.e[kChunk - 1];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const f32x4 e = *(const f32x4 *)(l.e + mt * 16 + grp * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                X[mt][r] *= -e[r];
                dO[mt][r] *= d.scale * e[r];
            }
        }
        Frag<3> Xp[2] = {split_frag<3>(X[0], X[1]), split_frag<3>(X[2], X[3])};
        Frag<3> Op[2] = {split_frag<3>(dO[0], dO[1]), split_frag<3>(dO[2], dO[3])};
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] *= last;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                S[t] = mma(load_column<kDk>(l.q, l.qT, t * 16 + col, s, grp), Op[s], S[t]);
                S[t] = mma(load_column<kDk>(l.k, l.kT, t * 16 + col, s, grp), Xp[s], S[t]);
            }
        }
    }
    if (a.dh_init != nullptr) {
        float *out = a.dh_init + ((int64_t)b * d.hv + hv) * state + n;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) out[(int64_t)(t * 16 + grp * 4 + r) * d.dv] = S[t][r];
    }
}

// ------------------------------------------------------------ chunk gradients

template <typename T>
struct GradArgs {
    const T *q, *k, *v, *dout;
    const double *G;
    const float *beta, *W, *Wt, *S, *dS;   // S: h_chunks
    T *dq, *dk, *dv;
    float *dg, *dbeta;
    DeltaDims d;
};

// U and X between the two halves of the kernel, [64][dv]: parts in planes for
// bf16 streams (their results are rounded to bf16: two parts), fp32 else.
template <typename T, int kDv>
struct RowTile;
template <int kDv>
struct RowTile<uint16_t, kDv> {
    static constexpr int kRow = kDv + 8;
    uint16_t p[2][kChunk * kRow];
    __device__ void put(int row, int c, float v) {
        const uint32_t h = pk_rne(v, v);
        p[0][row * kRow + c] = (uint16_t)h;
        p[1][row * kRow + c] = (uint16_t)pk_rne(v - bf_lo(h), 0.f);
    }
    __device__ Frag<2> get(int row, int c) const {
        Frag<2> f;
        f.p[0] = load_straight(&p[0][row * kRow + c]).p[0];
        f.p[1] = load_straight(&p[1][row * kRow + c]).p[0];
        return f;
    }
};
template <int kDv>
struct RowTile<float, kDv> {
    static constexpr int kRow = kDv + 4;
    float p[kChunk * kRow];
    __device__ void put(int row, int c, float v) { p[row * kRow + c] = v; }
    __device__ Frag<3> get(int row, int c) const { return load_straight(&p[row * kRow + c]); }
};

// eight consecutive fp32 values as parts
template <int kParts>
__device__ __forceinline__ Frag<kParts> load_state(const float *p) {
    return split_frag<kParts>(*(const f32x4 *)p, *(const f32x4 *)(p + 4));
}

template <typename T, int kDk, int kDv>
struct GradLds {
    T k[kChunk * TileLoad<T, kDk>::kRow];
    T q[kChunk * TileLoad<T, kDk>::kRow];
    T kT[kTransSize<T, kDk>];
    T qT[kTransSize<T, kDk>];
    union {
        struct {
            uint16_t W[3 * kChunk * kTri];   // W, then W^T
            uint16_t P[3 * kChunk * kTri];   // P, then P^T
        };
        struct {
            RowTile<T, kDv> U, X;
        };
    };
    double G[kChunk];
    float e[kChunk], rest[kChunk], bt[kChunk];
    float dG[kDv / 16][kChunk], db[kDv / 16][kChunk];
    float ends[kDv / 16];
};

// One workgroup per (chunk, query/key head, batch) and a wave per 16 columns of
// v: each value head of the group in turn, dQ and dK summed over them in
// registers.  First by columns as in the chains (U, O, dU, X and the row
// products), then by rows: wave w takes token tile w % 4 and a share of dk, and
// forms dQ^T, dK^T as products over dv (S, dS' by rows from memory) and over
// the chunk's tokens (DP, DA formed as result tiles, which are B operands as
// they are).
template <typename T, int kDk, int kDv>
__global__ __launch_bounds__(kDv * 4, 1) void delta_grad_kernel(GradArgs<T> a) {
    using L = GradLds<T, kDk, kDv>;
    constexpr int kThreads = kDv * 4, kWaves = kDv / 16;
    constexpr int kRow = TileLoad<T, kDk>::kRow, kSteps = kDk / 32;
    constexpr int kIn = Stream<T>::kParts, kOut = Stream<T>::kOutParts;
    constexpr int kMine = kDk / 16 / (kWaves / 4);   // dk tiles of a wave
    __shared__ __attribute__((aligned(16))) L l;
    const DeltaDims &d = a.d;
    const int c = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
    const int lane = lane_id(), wave = threadIdx.x >> 6, col = lane & 15, grp = lane >> 4;
    const int64_t len = row_len(d, b), t0 = (int64_t)c * kChunk;
    const int rows = d.T - t0 < kChunk ? (int)(d.T - t0) : kChunk;
    const int m = len <= t0 ? 0 : len - t0 < kChunk ? (int)(len - t0) : kChunk;
    const int64_t kstride = (int64_t)d.hk * kDk, vstride = (int64_t)d.hv * kDv, state = (int64_t)kDk * kDv;
    const int64_t kat = (((int64_t)b * d.T + t0) * d.hk + hk) * kDk;
    const int tok = (wave & 3) * 16 + col, m0 = (wave >> 2) * kMine;   // by rows: this lane's token, first dk tile

    f32x4 dQ[kMine], dK[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) dQ[i] = dK[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (m > 0) {
        TileLoad<T, kDk, kThreads> kl, ql;
        kl.load(a.k + kat, kstride, m);
        ql.load(a.q + kat, kstride, m);
        kl.store(l.k);
        ql.store(l.q);
        __syncthreads();
        transpose_tile<kDk, kThreads>(l.k, l.kT);
        transpose_tile<kDk, kThreads>(l.q, l.qT);
    }
    for (int hv = hk * d.group; hv < (hk + 1) * d.group; ++hv) {
        const int64_t at = ((int64_t)b * d.T + t0) * d.hv + hv;   // of the gates; times dv of v
        T *dvp = a.dv + at * kDv;
        for (int e = threadIdx.x; e < (rows - m) * kDv; e += kThreads)
            Stream<T>::store(dvp + (m + e / kDv) * vstride + e % kDv, 0.f);
        for (int t = m + threadIdx.x; t < rows; t += kThreads) a.dg[at + (int64_t)t * d.hv] = a.dbeta[at + (int64_t)t * d.hv] = 0.f;
        if (m == 0) continue;
        const int64_t chunk_at = (((int64_t)b * d.chunks + c) * d.hv + hv) * state;
        const int64_t w_at = (((int64_t)b * d.hv + hv) * d.chunks + c) * kWFloats;
        const float *Sg = a.S + chunk_at, *dSg = a.dS + chunk_at;
        const int n = wave * 16 + col;
        __syncthreads();   // the last head's reads of U and X are done
        if (threadIdx.x < kChunk) l.G[threadIdx.x] = a.G[(((int64_t)b * d.hv + hv) * d.chunks + c) * kChunk + threadIdx.x];
        if (threadIdx.x < kChunk)
            l.bt[threadIdx.x] = (int)threadIdx.x < m ? strength(a.beta[at + (int64_t)threadIdx.x * d.hv]) : 1.f;
        zero_planes<kThreads>(l.W, 3);
        zero_planes<kThreads>(l.P, 3);
        __syncthreads();
        if (threadIdx.x < kChunk) {
            l.e[threadIdx.x] = decay(l.G[threadIdx.x]);
            l.rest[threadIdx.x] = decay(l.G[kChunk - 1] - l.G[threadIdx.x]);
        }
        {
            WLoad<false, kThreads> wl;
            wl.load(a.W + w_at);
            wl.store(l.W);
        }
        form_p<T, kDk, false, 3, kThreads>(l.k, l.q, l.G, d.scale, l.P);
        f32x4 v[4], dO[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int t = i / 4 * 16 + grp * 4 + i % 4;
            v[i / 4][i % 4] = t < m ? Stream<T>::load(a.v + at * kDv + t * vstride + n) : 0.f;
            dO[i / 4][i % 4] = t < m ? Stream<T>::load(a.dout + at * kDv + t * vstride + n) : 0.f;
        }
        __syncthreads();
        // by columns: R, O, U
        f32x4 R[4], O[4], U[4], X[4], Kd[4];
        float end = 0.f;   // <S, dS'> exp(G_C) + sum of U (K dS') rows
        {
            Frag<3> Sp[kSteps], Dp[kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                f32x4 x[2], y[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int64_t r0 = (int64_t)(s * 32 + i * 16 + grp * 4 + r) * kDv + n;
                        x[i][r] = Sg[r0];
                        y[i][r] = dSg[r0];
                        end = fmaf(x[i][r], y[i][r], end);
                    }
                Sp[s] = split_frag<3>(x[0], x[1]);
                Dp[s] = split_frag<3>(y[0], y[1]);
            }
            end *= l.e[kChunk - 1];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                f32x4 ks = {0.f, 0.f, 0.f, 0.f}, qs = ks, kd = ks;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const auto kf = load_paired(l.k + (mt * 16 + col) * kRow + s * 32 + grp * 4);
                    ks = mma(kf, Sp[s], ks);
                    kd = mma(kf, Dp[s], kd);
                    qs = mma(load_paired(l.q + (mt * 16 + col) * kRow + s * 32 + grp * 4), Sp[s], qs);
                }
                const f32x4 e = *(const f32x4 *)(l.e + mt * 16 + grp * 4), rest = *(const f32x4 *)(l.rest + mt * 16 + grp * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    R[mt][r] = fmaf(-e[r], ks[r], v[mt][r]);
                    O[mt][r] = d.scale * e[r] * qs[r];
                    Kd[mt][r] = rest[r] * kd[r];
                }
            }
        }
        {
            Frag<3> Rp[2] = {split_frag<3>(R[0], R[1]), split_frag<3>(R[2], R[3])};
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s <= mt / 2; ++s)
                    acc = mma(load_planes<3>(l.W + (mt * 16 + col) * kTri + s * 32 + grp * 4, kChunk * kTri), Rp[s], acc);
                U[mt] = acc;
            }
            Frag<3> Up[2] = {split_frag<3>(U[0], U[1]), split_frag<3>(U[2], U[3])};
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int s = 0; s <= mt / 2; ++s)
                    O[mt] = mma(load_planes<3>(l.P + (mt * 16 + col) * kTri + s * 32 + grp * 4, kChunk * kTri), Up[s], O[mt]);
        }
        __syncthreads();   // W and P are read: their transposes take their place
        zero_planes<kThreads>(l.W, 3);
        zero_planes<kThreads>(l.P, 3);
        __syncthreads();
        {
            WLoad<true, kThreads> wl;
            wl.load(a.Wt + w_at);
            wl.store(l.W);
        }
        form_p<T, kDk, true, 3, kThreads>(l.k, l.q, l.G, d.scale, l.P);
        __syncthreads();
        {
            f32x4 dU[4];
            Frag<kIn> Op[2] = {split_frag<kIn>(dO[0], dO[1]), split_frag<kIn>(dO[2], dO[3])};
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                dU[mt] = Kd[mt];
#pragma unroll
                for (int s = mt / 2; s < 2; ++s)
                    dU[mt] = mma(load_planes<3>(l.P + (mt * 16 + col) * kTri + s * 32 + grp * 4, kChunk * kTri), Op[s], dU[mt]);
            }
            Frag<3> Dp[2] = {split_frag<3>(dU[0], dU[1]), split_frag<3>(dU[2], dU[3])};
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = mt / 2; s < 2; ++s)
                    acc = mma(load_planes<3>(l.W + (mt * 16 + col) * kTri + s * 32 + grp * 4, kChunk * kTri), Dp[s], acc);
                X[mt] = acc;
            }
        }
        __syncthreads();   // W^T and P^T are read: U and X take their place
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = mt * 16 + grp * 4 + r;
                const float u = U[mt][r], x = X[mt][r], ib = 1.f / l.bt[t], y = u * ib, z = x * ib;
                end = fmaf(u, Kd[mt][r], end);
                float dG = dO[mt][r] * O[mt][r] - x * (v[mt][r] - y) - u * z, db = y * z;
#pragma unroll
                for (int s = 1; s < 16; s <<= 1) {
                    dG += __shfl_xor(dG, s, 64);
                    db += __shfl_xor(db, s, 64);
                }
                if (col == 0) {
                    l.dG[wave][t] = dG;
                    l.db[wave][t] = db;
                }
                l.U.put(t, n, u);
                l.X.put(t, n, x);
                if (t < m) Stream<T>::store(dvp + t * vstride + n, x);
            }
        }
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) end += __shfl_xor(end, s, 64);
        if (lane == 0) l.ends[wave] = end;
        __syncthreads();
        if (threadIdx.x < kChunk) {
            const int t = threadIdx.x;
            float dG = 0.f, db = 0.f, ends = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                dG += l.dG[w][t];
                db += l.db[w][t];
                ends += l.ends[w];
            }
            if (t == kChunk - 1) dG += ends;
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) {
                const float up = __shfl_down(dG, s, 64);
                if (t + s < 64) dG += up;
            }
            if (t < m) {
                a.dg[at + (int64_t)t * d.hv] = dG;
                a.dbeta[at + (int64_t)t * d.hv] = db;
            }
        }
        // by rows: products over dv
        const T *dop = a.dout + at * kDv;
        auto dout_frag = [&](int row, int c0) {
            if (row < m) return load_straight(dop + row * vstride + c0);
            Frag<kIn> z{};
            return z;
        };
        const float et = l.e[tok], rt = l.rest[tok];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            f32x4 so = {0.f, 0.f, 0.f, 0.f}, sx = so, du = so;
            const int64_t r0 = (int64_t)((m0 + i) * 16 + col) * kDv;
#pragma unroll
            for (int s = 0; s < kDv / 32; ++s) {
                const int c0 = s * 32 + grp * 8;
                const Frag<kOut> sf = load_state<kOut>(Sg + r0 + c0), df = load_state<kOut>(dSg + r0 + c0);
                so = mma(sf, dout_frag(tok, c0), so);
                sx = mma(sf, l.X.get(tok, c0), sx);
                du = mma(df, l.U.get(tok, c0), du);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dQ[i][r] = fmaf(d.scale * et, so[r], dQ[i][r]);
                dK[i][r] += rt * du[r] - et * sx[r];
            }
        }
        // products over the chunk's tokens: tiles rows `jt`, column this lane's token
        const double Gt = l.G[tok];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            f32x4 tq[2], tp[2], ta[2];   // DP^T (for dQ), DP and DA + DA^T (for dK)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int jt = s * 2 + i;
                f32x4 uo = {0.f, 0.f, 0.f, 0.f}, ou = uo, xu = uo, ux = uo;
#pragma unroll
                for (int x = 0; x < kDv / 32; ++x) {
                    const int c0 = x * 32 + grp * 8;
                    const auto uj = l.U.get(jt * 16 + col, c0), ut = l.U.get(tok, c0);
                    if (jt <= (wave & 3)) {
                        uo = mma(uj, dout_frag(tok, c0), uo);           // U_j.dO_t
                        ux = mma(uj, l.X.get(tok, c0), ux);             // U_j.X_t
                    }
                    if (jt >= (wave & 3)) {
                        ou = mma(dout_frag(jt * 16 + col, c0), ut, ou);   // dO_j.U_t
                        xu = mma(l.X.get(jt * 16 + col, c0), ut, xu);     // X_j.U_t
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = jt * 16 + grp * 4 + r;
                    const float below = j <= tok ? decay(Gt - l.G[j]) : 0.f, above = j >= tok ? decay(l.G[j] - Gt) : 0.f;
                    tq[i][r] = j <= tok ? d.scale * below * uo[r] : 0.f;
                    tp[i][r] = j >= tok ? d.scale * above * ou[r] : 0.f;
                    ta[i][r] = j < tok ? -below * ux[r] : j > tok ? -above * xu[r] : 0.f;
                }
            }
            const auto fq = split_frag<kOut>(tq[0], tq[1]), fp = split_frag<kOut>(tp[0], tp[1]), fa = split_frag<kOut>(ta[0], ta[1]);
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const auto kc = load_column<kDk>(l.k, l.kT, (m0 + i) * 16 + col, s, grp);
                dQ[i] = mma(kc, fq, dQ[i]);
                dK[i] = mma(load_column<kDk>(l.q, l.qT, (m0 + i) * 16 + col, s, grp), fp, dK[i]);
                dK[i] = mma(kc, fa, dK[i]);
            }
        }
    }
    if (tok < rows) {   // padding: m leaves zeros
        T *dqp = a.dq + kat + tok * kstride, *dkp = a.dk + kat + tok * kstride;
        const bool pad = tok >= m;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int at = (m0 + i) * 16 + grp * 4;
            const f32x4 z = {0.f, 0.f, 0.f, 0.f};
            store4(dqp + at, pad ? z : dQ[i]);
            store4(dkp + at, pad ? z : dK[i]);
        }
    }
}

}  // namespace bdssm_dev
