// delta_kernels.hpp -- the gated delta rule on gfx950.
//
// Per (batch, value head), with a_t = exp(g_t), state S [dk, dv] in fp32:
//   y_t = v_t - (a_t S_{t-1})^T k_t        the prediction's error
//   S_t = a_t S_{t-1} + k_t (beta_t y_t)^T,     o_t = scale S_t^T q_t
//
// Chunked form, C = 64 tokens.  G_i = sum of g over the chunk's tokens up to i,
// D_ij = exp(G_i - G_j), E = diag(exp(G_i)), S the state before the chunk:
//   R  = V - E K S                          (the chunk's tokens alone still missing)
//   U  = W R,  W = (I + diag(beta) A)^-1 diag(beta),  A_ij = D_ij k_i.k_j, j < i
//   O  = scale E Q S + P U,                 P_ij = scale D_ij q_i.k_j, j <= i
//   S' = exp(G_C) S + K^T (diag(exp(G_C - G_j)) U)
// W does not depend on the state: delta_prep_kernel forms it for all chunks at
// once.  The rest is a chain over chunks whose columns (dv) are independent:
// delta_chain_kernel gives each wave 16 columns and all dk rows, which keeps
// S, R and U in that wave's registers from one product to the next (see the
// paired order in hybrid_common.hpp).
//
// Log decays are summed in 64 bits: a decay of -inf (a reset at a document's
// start) is taken as -10000 per token, whose exponential is 0, and the
// differences of the tokens behind it keep their precision.
#pragma once

#include "hybrid_common.hpp"

namespace bdssm_dev {

constexpr int kChunk = 64;                 // BDSSM_DELTA_CHUNK
constexpr int kDeltaThreads = 256;
constexpr int kWBlocks = 10;               // 16x16 blocks on and below W's diagonal
constexpr int kWFloats = kWBlocks * 256;   // W of one chunk and head in the workspace
constexpr int kTri = kChunk + 8;           // row length of the 64x64 tiles' planes in LDS

struct DeltaDims {
    int64_t T;
    int hk, hv, group;   // group = hv / hk
    int dv;
    int chunks;          // ceil(T / 64)
    const int32_t *lens; // tokens of each row, or null
    float scale;
};

__device__ __forceinline__ int64_t row_len(const DeltaDims &d, int b) {
    if (d.lens == nullptr) return d.T;
    const int64_t n = d.lens[b];
    return n < 0 ? 0 : (n < d.T ? n : d.T);
}

// Inclusive sums of the chunk's log decays, by the first wave.
__device__ __forceinline__ void chunk_decays(const float *g, int64_t stride, int n, double *G) {
    if (threadIdx.x < 64) {
        const int t = threadIdx.x;
        double x = t < n ? (double)fmaxf(g[t * stride], -1e4f) : 0.0;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const double up = __shfl_up(x, s, 64);
            if (t >= s) x += up;
        }
        G[t] = x;
    }
}

// beta = 0 counts as 2^-64, which changes nothing in 32 bits and lets the
// backward divide by it.
__device__ __forceinline__ float strength(float beta) { return fabsf(beta) < 0x1p-64f ? 0x1p-64f : beta; }

__device__ __forceinline__ float decay(double d) { return __expf((float)d); }

// One [64, dk] tile of a token-major stream on its way to LDS: 16 bytes at a
// time in registers (issued a chunk ahead), zeros behind the row's length.
template <typename T, int kDk, int kThreads = kDeltaThreads>
struct TileLoad {
    static constexpr int kVec = 16 / sizeof(T);
    static constexpr int kPerRow = kDk / kVec;
    static constexpr int kN = kChunk * kPerRow / kThreads;
    static constexpr int kRow = kDk + (sizeof(T) == 2 ? 8 : 4);   // LDS row length
    uint4 r[kN];
    __device__ void load(const T *src, int64_t stride, int n) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = threadIdx.x + i * kThreads, row = at / kPerRow, c = at % kPerRow;
            r[i] = row < n ? *(const uint4 *)(src + row * stride + c * kVec) : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ void store(T *lds) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = threadIdx.x + i * kThreads, row = at / kPerRow, c = at % kPerRow;
            *(uint4 *)(lds + row * kRow + c * kVec) = r[i];
        }
    }
};

// LDS tile [64][dk] -> its transpose [dk][64] (row lengths TileLoad::kRow and
// kTransRow), bf16 by token pairs.
template <typename T>
constexpr int kTransRow = kChunk + (sizeof(T) == 2 ? 8 : 4);

template <int kDk, int kThreads = kDeltaThreads>
__device__ __forceinline__ void transpose_tile(const uint16_t *tile, uint16_t *out) {
    constexpr int kRow = TileLoad<uint16_t, kDk>::kRow;
    for (int at = threadIdx.x; at < 32 * (kDk / 8); at += kThreads) {
        const int tp = at % 32, c = at / 32 * 8;
        const uint4 a = *(const uint4 *)(tile + (2 * tp) * kRow + c);
        const uint4 b = *(const uint4 *)(tile + (2 * tp + 1) * kRow + c);
        const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *(uint32_t *)(out + (c + 2 * i) * kTransRow<uint16_t> + 2 * tp) = __builtin_amdgcn_perm(bv[i], av[i], 0x05040100u);
            *(uint32_t *)(out + (c + 2 * i + 1) * kTransRow<uint16_t> + 2 * tp) = __builtin_amdgcn_perm(bv[i], av[i], 0x07060302u);
        }
    }
}
// fp32 tiles keep no transposed copy: four-byte reads down a column are free of
// bank conflicts as they are.
template <int kDk, int kThreads = kDeltaThreads>
__device__ __forceinline__ void transpose_tile(const float *, float *) {}

template <typename T, int kDk>
constexpr int kTransSize = sizeof(T) == 2 ? kDk * kTransRow<T> : 4;

// Column `c` of a [64][dk] tile, tokens 32 s .. 32 s + 31 in paired order.
template <int kDk>
__device__ __forceinline__ Frag<1> load_column(const uint16_t *, const uint16_t *trans, int c, int s, int grp) {
    return load_paired(trans + c * kTransRow<uint16_t> + s * 32 + grp * 4);
}
template <int kDk>
__device__ __forceinline__ Frag<3> load_column(const float *tile, const float *, int c, int s, int grp) {
    constexpr int kRow = TileLoad<float, kDk>::kRow;
    f32x4 a, b;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        a[r] = tile[(s * 32 + grp * 4 + r) * kRow + c];
        b[r] = tile[(s * 32 + 16 + grp * 4 + r) * kRow + c];
    }
    return split_frag<3>(a, b);
}

// ------------------------------------------------------------------ W
//
// One workgroup per (chunk, query/key head, batch); K K^T once, then each
// value head of the group.  N = -diag(beta) A is strictly lower; (I - N)^-1 by
// 16x16 blocks: wave j inverts diagonal block j by substitution (a lane per
// column), then runs down block column j: X_i = inv_ii sum_k N_ik X_k, in fp32
// matrix instructions, X_k staying in registers.
template <typename T, int kDk>
__global__ __launch_bounds__(kDeltaThreads) void delta_prep_kernel(const T *__restrict__ k,
                                                                  const float *__restrict__ g,
                                                                  const float *__restrict__ beta,
                                                                  float *__restrict__ W, float *__restrict__ Wt,
                                                                  double *__restrict__ Gs, DeltaDims d) {
    constexpr int kRow = TileLoad<T, kDk>::kRow;
    __shared__ __attribute__((aligned(16))) T kt[kChunk * kRow];
    __shared__ __attribute__((aligned(16))) float gram[kChunk * 68], N[kChunk * 68];
    __shared__ __attribute__((aligned(16))) float inv[4 * 16 * 20];   // diagonal blocks' inverses
    __shared__ double G[kChunk];
    __shared__ float bt[kChunk];
    const int c = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int64_t t0 = (int64_t)c * kChunk, len = row_len(d, b);
    if (t0 >= len) return;
    const int n = len - t0 < kChunk ? (int)(len - t0) : kChunk;
    const int lane = lane_id(), wave = threadIdx.x >> 6, col = lane & 15, grp = lane >> 4;
    {
        TileLoad<T, kDk> kl;
        kl.load(k + (((int64_t)b * d.T + t0) * d.hk + h) * kDk, (int64_t)d.hk * kDk, n);
        kl.store(kt);
    }
    __syncthreads();
    for (int tile = wave; tile < kWBlocks; tile += 4) {
        const int it = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0, jt = tile - it * (it + 1) / 2;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < kDk / 32; ++s)
            acc = mma(load_straight(kt + (it * 16 + col) * kRow + s * 32 + grp * 8),
                      load_straight(kt + (jt * 16 + col) * kRow + s * 32 + grp * 8), acc);
#pragma unroll
        for (int r = 0; r < 4; ++r) gram[(it * 16 + grp * 4 + r) * 68 + jt * 16 + col] = acc[r];
    }
    for (int hv = h * d.group; hv < (h + 1) * d.group; ++hv) {
        const int64_t at = ((int64_t)b * d.T + t0) * d.hv + hv;
        chunk_decays(g + at, d.hv, n, G);
        if (threadIdx.x < kChunk) bt[threadIdx.x] = (int)threadIdx.x < n ? strength(beta[at + (int64_t)threadIdx.x * d.hv]) : 1.f;
        __syncthreads();
        for (int e = threadIdx.x; e < kChunk * kChunk; e += kDeltaThreads) {
            const int i = e / kChunk, j = e % kChunk;
            N[i * 68 + j] = j < i ? -bt[i] * (decay(G[i] - G[j]) * gram[i * 68 + j]) : 0.f;
        }
        __syncthreads();
        // diagonal block `wave`, column `col` of its inverse
        const int r0 = wave * 16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == col ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) s = fmaf(N[(r0 + i) * 68 + r0 + j], x[j], s);
            x[i] = s;
        }
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) inv[(r0 + i) * 20 + col] = x[i];
        }
        __syncthreads();
        float *Wc = W + (((int64_t)b * d.hv + hv) * d.chunks + c) * kWFloats;
        if (threadIdx.x < kChunk) Gs[(((int64_t)b * d.hv + hv) * d.chunks + c) * kChunk + threadIdx.x] = G[threadIdx.x];
        const float bj = bt[r0 + col];
        f32x4 X[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < wave) continue;
            if (i == wave) {
#pragma unroll
                for (int r = 0; r < 4; ++r) X[i][r] = inv[(r0 + grp * 4 + r) * 20 + col];
            } else {
                f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < i; ++kb) {
                    if (kb < wave) continue;
                    const f32x4 a = *(const f32x4 *)&N[(i * 16 + col) * 68 + kb * 16 + grp * 4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) t = mfma32(a[r], X[kb][r], t);
                }
                f32x4 y = {0.f, 0.f, 0.f, 0.f};
                const f32x4 a = *(const f32x4 *)&inv[(i * 16 + col) * 20 + grp * 4];
#pragma unroll
                for (int r = 0; r < 4; ++r) y = mfma32(a[r], t[r], y);
                X[i] = y;
            }
            float *blk = Wc + (i * (i + 1) / 2 + wave) * 256;
            f32x4 w;
#pragma unroll
            for (int r = 0; r < 4; ++r) w[r] = X[i][r] * bj;
#pragma unroll
            for (int r = 0; r < 4; ++r) blk[(grp * 4 + r) * 16 + col] = w[r];
            if (Wt != nullptr) *(f32x4 *)(Wt + (blk - W) + col * 16 + grp * 4) = w;
        }
        __syncthreads();
    }
}

// W's blocks (kTransposed: W^T's) from the workspace into three planes of bf16
// parts in LDS.
template <bool kTransposed, int kThreads = kDeltaThreads>
struct WLoad {
    static constexpr int kN = (kWFloats / 4 + kThreads - 1) / kThreads;
    f32x4 r[kN];
    __device__ void load(const float *W) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = threadIdx.x + i * kThreads;
            if (at < kWFloats / 4) r[i] = *(const f32x4 *)(W + at * 4);
        }
    }
    // row of the block at `at` and its column: element (row, col..col+3)
    __device__ static void place(int at, int *row, int *colm) {
        const int blk = at / 64, e = at % 64;
        const int it = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, jt = blk - it * (it + 1) / 2;
        *row = (kTransposed ? jt : it) * 16 + e / 4;
        *colm = (kTransposed ? it : jt) * 16 + e % 4 * 4;
    }
    __device__ void store(uint16_t *lds) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = threadIdx.x + i * kThreads;
            if (at < kWFloats / 4) {
                int row, c;
                place(at, &row, &c);
                uint32_t a[3], b[3];
                split_pair<3>(r[i][0], r[i][1], a);
                split_pair<3>(r[i][2], r[i][3], b);
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *(uint2 *)(lds + p * kChunk * kTri + row * kTri + c) = make_uint2(a[p], b[p]);
            }
        }
    }
};

// P_ij = scale exp(G_i - G_j) q_i.k_j (j <= i) in kParts planes: rows i, or rows
// j if kTransposed.  Each tile is formed with its rows as the product's
// columns, so that a lane stores four of a row.
template <typename T, int kDk, bool kTransposed, int kParts, int kThreads = kDeltaThreads>
__device__ __forceinline__ void form_p(const T *k, const T *q, const double *G, float scale, uint16_t *P) {
    constexpr int kRow = TileLoad<T, kDk>::kRow;
    const int lane = lane_id(), col = lane & 15, grp = lane >> 4;
    for (int tile = threadIdx.x >> 6; tile < kWBlocks; tile += kThreads / 64) {
        const int it = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0, jt = tile - it * (it + 1) / 2;
        const T *rows = kTransposed ? q + it * 16 * kRow : k + jt * 16 * kRow;
        const T *cols = kTransposed ? k + jt * 16 * kRow : q + it * 16 * kRow;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < kDk / 32; ++s)
            acc = mma(load_straight(rows + col * kRow + s * 32 + grp * 8), load_straight(cols + col * kRow + s * 32 + grp * 8), acc);
        const int row = (kTransposed ? jt : it) * 16 + col, c0 = (kTransposed ? it : jt) * 16 + grp * 4;
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = kTransposed ? c0 + r : row, j = kTransposed ? row : c0 + r;
            p[r] = j <= i ? scale * decay(G[i] - G[j]) * acc[r] : 0.f;
        }
        uint32_t w0[kParts], w1[kParts];
        split_pair<kParts>(p[0], p[1], w0);
        split_pair<kParts>(p[2], p[3], w1);
#pragma unroll
        for (int x = 0; x < kParts; ++x)
            *(uint2 *)(P + x * kChunk * kTri + row * kTri + c0) = make_uint2(w0[x], w1[x]);
    }
}

// Zero planes: the halves of 32-wide steps beyond W's and P's triangles are
// read but never written.
template <int kThreads = kDeltaThreads>
__device__ __forceinline__ void zero_planes(uint16_t *p, int planes) {
    for (int i = threadIdx.x; i < planes * kChunk * kTri / 2; i += kThreads) ((uint32_t *)p)[i] = 0;
}

// --------------------------------------------------------------- forward chain

template <typename T>
struct ChainArgs {
    const T *q, *k, *v;
    const double *G;      // the chunks' sums of log decays
    const float *W, *h_init;
    T *o;                 // null: states only
    float *h_final;       // null: not wanted
    float *h_chunks;      // null, or [batch, chunks, hv, dk, dv]
    DeltaDims d;
};

template <typename T, int kDk>
struct ChainLds {
    static constexpr int kOut = Stream<T>::kOutParts;
    T k[kChunk * TileLoad<T, kDk>::kRow];
    T q[kChunk * TileLoad<T, kDk>::kRow];
    T kT[kTransSize<T, kDk>];
    uint16_t W[3 * kChunk * kTri];
    uint16_t P[kOut * kChunk * kTri];
    double G[kChunk];
    float e[kChunk], rest[kChunk];
};

template <typename T, int kDk, bool kWithO>
__global__ __launch_bounds__(kDeltaThreads, 1) void delta_chain_kernel(ChainArgs<T> a) {
    using L = ChainLds<T, kDk>;
    constexpr int kRow = TileLoad<T, kDk>::kRow, kOut = L::kOut;
    constexpr int kTiles = kDk / 16, kSteps = kDk / 32;
    __shared__ __attribute__((aligned(16))) L l;
    const DeltaDims &d = a.d;
    const int hv = blockIdx.y, b = blockIdx.z, hk = hv / d.group;
    const int lane = lane_id(), wave = threadIdx.x >> 6, col = lane & 15, grp = lane >> 4;
    const int n = blockIdx.x * 64 + wave * 16 + col;   // this lane's state column
    const int64_t len = row_len(d, b);
    const int chunks = (int)((len + kChunk - 1) / kChunk);
    const int64_t kstride = (int64_t)d.hk * kDk, vstride = (int64_t)d.hv * d.dv;
    const T *kp = a.k + ((int64_t)b * d.T * d.hk + hk) * kDk;
    const T *qp = a.q + ((int64_t)b * d.T * d.hk + hk) * kDk;
    const T *vp = a.v + ((int64_t)b * d.T * d.hv + hv) * d.dv + n;
    const double *Gp = a.G + ((int64_t)b * d.hv + hv) * d.chunks * kChunk;
    const float *Wp = a.W + ((int64_t)b * d.hv + hv) * d.chunks * kWFloats;
    const int64_t state = (int64_t)kDk * d.dv;

    zero_planes(l.W, 3);
    zero_planes(l.P, kOut);

    f32x4 S[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[t][r] = a.h_init == nullptr ? 0.f
                                          : a.h_init[((int64_t)b * d.hv + hv) * state + (int64_t)(t * 16 + grp * 4 + r) * d.dv + n];

    TileLoad<T, kDk> kl, ql;
    WLoad<false> wl;
    T vr[16];         // as stored: nothing may wait for them here
    double Gr = 0.;   // threads 0..63
    auto fetch = [&](int c) {
        const int64_t t0 = (int64_t)c * kChunk;
        const int m = len - t0 < kChunk ? (int)(len - t0) : kChunk;
        kl.load(kp + t0 * kstride, kstride, m);
        if (kWithO) ql.load(qp + t0 * kstride, kstride, m);
        wl.load(Wp + (int64_t)c * kWFloats);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int t = i / 4 * 16 + grp * 4 + i % 4;
            vr[i] = t < m ? vp[(t0 + t) * vstride] : T(0);
        }
        if (threadIdx.x < kChunk) Gr = Gp[(int64_t)c * kChunk + threadIdx.x];
    };
    if (chunks > 0) fetch(0);

    for (int c = 0; c < chunks; ++c) {
        const int64_t t0 = (int64_t)c * kChunk;
        const int m = len - t0 < kChunk ? (int)(len - t0) : kChunk;
        __syncthreads();   // the last chunk's reads of LDS are done
        kl.store(l.k);
        if (kWithO) ql.store(l.q);
        wl.store(l.W);
        const double *G = l.G;
        if (threadIdx.x < kChunk) {   // one wave: the last token's sum is its last lane's
            l.G[threadIdx.x] = Gr;
            l.e[threadIdx.x] = decay(Gr);
            l.rest[threadIdx.x] = decay(__shfl(Gr, 63, 64) - Gr);
        }
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = Stream<T>::load(vr + i);
        __syncthreads();
        if (c + 1 < chunks) fetch(c + 1);
        transpose_tile<kDk>(l.k, l.kT);
        if (kWithO) {
            form_p<T, kDk, false, kOut>(l.k, l.q, G, d.scale, l.P);
        }
        if (a.h_chunks != nullptr) {
            float *out = a.h_chunks + (((int64_t)b * d.chunks + c) * d.hv + hv) * state + n;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) out[(int64_t)(t * 16 + grp * 4 + r) * d.dv] = S[t][r];
        }
        // R = V - E K S and the state's part of O
        f32x4 R[4], O[4];
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
                const f32x4 e = *(const f32x4 *)(l.e + mt * 16 + grp * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) R[mt][r] = fmaf(-e[r], acc[r], v[mt * 4 + r]);
                if (kWithO) {
                    f32x4 qs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        Frag<kOut> So;
#pragma unroll
                        for (int x = 0; x < kOut; ++x) So.p[x] = Sp[s].p[x];
                        qs = mma(load_paired(l.q + (mt * 16 + col) * kRow + s * 32 + grp * 4), So, qs);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[mt][r] = d.scale * e[r] * qs[r];
                }
            }
        }
        __syncthreads();   // kT and P are written
        f32x4 U[4];
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
        }
        if (kWithO) {
            Frag<kOut> Up[2] = {split_frag<kOut>(U[0], U[1]), split_frag<kOut>(U[2], U[3])};
            T *op = a.o + ((int64_t)b * d.T * d.hv + hv) * d.dv + n;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
                for (int s = 0; s <= mt / 2; ++s)
                    O[mt] = mma(load_planes<kOut>(l.P + (mt * 16 + col) * kTri + s * 32 + grp * 4, kChunk * kTri), Up[s], O[mt]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = mt * 16 + grp * 4 + r;
                    if (t < m) Stream<T>::store(op + (t0 + t) * vstride, O[mt][r]);
                }
            }
        }
        // the next state
        const float last = l.e[kChunk - 1];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const f32x4 e = *(const f32x4 *)(l.rest + mt * 16 + grp * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) U[mt][r] *= e[r];
        }
        Frag<3> Up[2] = {split_frag<3>(U[0], U[1]), split_frag<3>(U[2], U[3])};
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] *= last;
#pragma unroll
            for (int s = 0; s < 2; ++s)
                S[t] = mma(load_column<kDk>(l.k, l.kT, t * 16 + col, s, grp), Up[s], S[t]);
        }
    }
    if (a.h_final != nullptr) {
        float *out = a.h_final + ((int64_t)b * d.hv + hv) * state + n;
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) out[(int64_t)(t * 16 + grp * 4 + r) * d.dv] = S[t][r];
    }
    if (a.h_chunks != nullptr) {   // chunks of padding alone: the state stays
        for (int c = chunks; c < d.chunks; ++c) {
            float *out = a.h_chunks + (((int64_t)b * d.chunks + c) * d.hv + hv) * state + n;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) out[(int64_t)(t * 16 + grp * 4 + r) * d.dv] = S[t][r];
        }
    }
    if (kWithO) {   // padding: zeros
        T *op = a.o + ((int64_t)b * d.T * d.hv + hv) * d.dv + n;
        for (int64_t t = len + grp; t < d.T; t += 4) Stream<T>::store(op + t * vstride, 0.f);
    }
}

// ---------------------------------------------------------------- recurrent
//
// The recurrence as written, token by token, for the active block: one wave
// per 32 columns of one head's state, held in registers (a lane: 4 columns and
// dk / 8 consecutive rows), so the state is read once and written once however
// many tokens there are.  Both sums over the rows (S^T k and S^T q of the
// decayed state; o = S^T q + (k.q) u) fold over the 8 row groups together.
template <typename T>
struct StepArgs {
    const T *q, *k, *v;
    const float *g, *beta, *h;   // h null: zero state
    T *o;                        // null: the state alone
    float *h_out;                // null: the outputs alone; may be h
    DeltaDims d;
};

template <typename T, int kN>
__device__ __forceinline__ void load_run(const T *p, float *out) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < kN / 8; ++i) {
            const uint4 w = *(const uint4 *)(p + i * 8);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                out[i * 8 + 2 * j] = bf_lo(u[j]);
                out[i * 8 + 2 * j + 1] = bf_hi(u[j]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) *(f32x4 *)(out + i * 4) = *(const f32x4 *)(p + i * 4);
    }
}

__device__ __forceinline__ f32x4 load4(const uint16_t *p) {
    const uint2 w = *(const uint2 *)p;
    return f32x4{bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y)};
}
__device__ __forceinline__ f32x4 load4(const float *p) { return *(const f32x4 *)p; }
__device__ __forceinline__ void store4(uint16_t *p, f32x4 v) {
    *(uint2 *)p = make_uint2(pk_rne(v[0], v[1]), pk_rne(v[2], v[3]));
}
__device__ __forceinline__ void store4(float *p, f32x4 v) { *(f32x4 *)p = v; }

// sum over the 8 row groups (lanes 8 apart), in every lane
__device__ __forceinline__ float row_sum(float x) {
    x += __shfl_xor(x, 8, 64);
    x += __shfl_xor(x, 16, 64);
    x += __shfl_xor(x, 32, 64);
    return x;
}

template <typename T, int kDk>
__global__ __launch_bounds__(64) void delta_step_kernel(StepArgs<T> a) {
    constexpr int kR = kDk / 8;
    const DeltaDims &d = a.d;
    const int hv = blockIdx.y, b = blockIdx.z, hk = hv / d.group;
    const int lane = lane_id(), n = blockIdx.x * 32 + (lane & 7) * 4, r0 = (lane >> 3) * kR;
    const int64_t len = row_len(d, b), at0 = (int64_t)b * d.T;
    const int64_t state = (((int64_t)b * d.hv + hv) * kDk + r0) * d.dv + n;
    f32x4 S[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) S[i] = a.h == nullptr ? f32x4{0.f, 0.f, 0.f, 0.f} : *(const f32x4 *)(a.h + state + (int64_t)i * d.dv);
    for (int64_t t = 0; t < len; ++t) {
        float k[kR], q[kR];
        load_run<T, kR>(a.k + ((at0 + t) * d.hk + hk) * kDk + r0, k);
        if (a.o != nullptr) load_run<T, kR>(a.q + ((at0 + t) * d.hk + hk) * kDk + r0, q);
        const f32x4 v = load4(a.v + ((at0 + t) * d.hv + hv) * d.dv + n);
        const float al = __expf(a.g[(at0 + t) * d.hv + hv]), bt = a.beta[(at0 + t) * d.hv + hv];
        f32x4 p = {0.f, 0.f, 0.f, 0.f}, s = {0.f, 0.f, 0.f, 0.f};
        float kq = 0.f;
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                S[i][c] *= al;
                p[c] = fmaf(S[i][c], k[i], p[c]);
            }
        if (a.o != nullptr) {
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                kq = fmaf(k[i], q[i], kq);
#pragma unroll
                for (int c = 0; c < 4; ++c) s[c] = fmaf(S[i][c], q[i], s[c]);
            }
            kq = row_sum(kq);
        }
        f32x4 u;
#pragma unroll
        for (int c = 0; c < 4; ++c) u[c] = bt * (v[c] - row_sum(p[c]));
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) S[i][c] = fmaf(k[i], u[c], S[i][c]);
        if (a.o != nullptr) {
            f32x4 o;
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = d.scale * fmaf(kq, u[c], row_sum(s[c]));
            if (lane < 8) store4(a.o + ((at0 + t) * d.hv + hv) * d.dv + n, o);
        }
    }
    if (a.o != nullptr)
        for (int64_t t = len + (lane >> 3); t < d.T; t += 8)
            store4(a.o + ((at0 + t) * d.hv + hv) * d.dv + n, f32x4{0.f, 0.f, 0.f, 0.f});
    if (a.h_out != nullptr && !(len == 0 && a.h == a.h_out)) {
#pragma unroll
        for (int i = 0; i < kR; ++i) *(f32x4 *)(a.h_out + state + (int64_t)i * d.dv) = S[i];
    }
}

}  // namespace bdssm_dev
