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

#include <type_traits>

#include "hybrid_common.hpp"

namespace bdssm_dev {

constexpr int kChunk = 64;                 // BDSSM_DELTA_CHUNK
constexpr int kDeltaThreads = 256;
constexpr int kBlocks = 10;                // 16x16 blocks on and below the diagonal of a chunk's matrix
constexpr int kFrags = 6;                  // A fragments (16 x 32) that hold them

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

// Inclusive sums of kTokens log decays, by the first wave (g: the lane's own, 0
// behind the last token).
template <int kTokens = kChunk>
__device__ __forceinline__ void chunk_decays(float g, double *G) {
    if (threadIdx.x < 64) {
        const int t = threadIdx.x;
        double x = (double)fmaxf(g, -1e4f);
#pragma unroll
        for (int s = 1; s < kTokens; s <<= 1) {
            const double up = __shfl_up(x, s, 64);
            if (t >= s) x += up;
        }
        if (t < kTokens) G[t] = x;
    }
}

// beta = 0 counts as 2^-64, which changes nothing in 32 bits and lets the
// backward divide by it.
__device__ __forceinline__ float strength(float beta) { return fabsf(beta) < 0x1p-64f ? 0x1p-64f : beta; }

__device__ __forceinline__ float decay(double d) { return __expf((float)d); }

// ------------------------------------------------------------------- tiles
//
// A [64][kCols] tile of a token-major stream in LDS, filled by 16-byte loads
// straight from memory (no registers, any number in flight).  Such a load
// writes a wave's 64 pieces one after another, so rows cannot be padded;
// instead piece p of row r lies at place p ^ turn(r), which spreads the same
// piece of 16 rows over all banks.  Rows behind the chunk's last token repeat
// it: what they feed is multiplied by zero or not stored.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <typename T, int kCols>
struct Tile {
    static constexpr int kVec = 16 / sizeof(T);            // elements of a piece
    static constexpr int kPieces = kCols / kVec;           // of a row
    static constexpr int kBytes = kChunk * kCols * (int)sizeof(T);
    T e[kChunk * kCols];

    __device__ static int turn(int r) {
        return kPieces >= 16 ? r & 15 : r / (16 / kPieces) & (kPieces - 1);
    }
    __device__ __forceinline__ const T *piece(int r, int p) const { return e + r * kCols + (p ^ turn(r)) * kVec; }

    // Filled by kWaves waves.  A lane's offsets into the rows (stride elements
    // apart, of which m, at least 1, are tokens) do not change from one full
    // chunk to the next.
    template <int kWaves>
    struct Offsets {
        static constexpr int kLoads = kBytes / 1024 / kWaves;
        uint32_t off[kLoads];
        __device__ __forceinline__ void set(int64_t stride, int m) {
            const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int at = (wave * kLoads + i) * 64 + lane, r = at / kPieces, p = at % kPieces ^ turn(r);
                off[i] = ((uint32_t)(r < m ? r : m - 1) * (uint32_t)stride + (uint32_t)(p * kVec)) * (uint32_t)sizeof(T);
            }
        }
    };
    template <int kWaves>
    __device__ __forceinline__ void fill(const T *src, const Offsets<kWaves> &o) {
        constexpr int kLoads = Offsets<kWaves>::kLoads;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load_lds(src, o.off[i], (char *)e + (wave * kLoads + i) * 1024);
    }
    template <int kWaves>
    __device__ __forceinline__ void fill(const T *src, int64_t stride, int m) {
        Offsets<kWaves> o;
        o.set(stride, m);
        fill(src, o);
    }
    // eight consecutive elements of a row: columns 32 s + 8 grp ..
    __device__ __forceinline__ auto row(int r, int s, int grp) const {
        if constexpr (sizeof(T) == 2) {
            return load_straight(piece(r, s * 4 + grp));
        } else {
            return split_frag<3>(*(const f32x4 *)piece(r, s * 8 + grp * 2), *(const f32x4 *)piece(r, s * 8 + grp * 2 + 1));
        }
    }
    // four tokens t0 .. t0 + 3 of column c0 + 8 (col / 4) + col % 4 (by lane; the
    // 16 lanes of a group share t0).  bf16: the transposing read gives lane i of
    // a group column i of what the group's lanes address, 4 rows of 4 x 8 bytes.
    __device__ __forceinline__ uint2 quad(int t0, int c0, int col) const {
        static_assert(sizeof(T) == 2, "");
        const int r = t0 + col / 4, c = c0 + col % 4 * 8;
        const T *p = piece(r, c / kVec) + c % kVec;
        return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
    }
    // the same of 16 consecutive columns c0 + col
    __device__ __forceinline__ uint2 quad16(int t0, int c0, int col) const {
        const int r = t0 + col / 4, c = c0 + col % 4 * 4;
        const T *p = piece(r, c / kVec) + c % kVec;
        return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
    }
    __device__ __forceinline__ float at(int r, int c) const { return Stream<T>::load(piece(r, c / kVec) + c % kVec); }

    // A fragment of the tile's transpose: row `col` of state tile `tile`, tokens
    // 32 s .. in paired order.  State tiles come in pairs of 32 dk: row m of the
    // first is dk 8 (m / 4) + m % 4 of the 32, of the second 4 more, so that
    // lane group g's rows of a pair are dk 8g..8g+7.
    __device__ __forceinline__ auto column(int tile, int s, int grp, int col) const {
        const int c0 = tile / 2 * 32 + (tile & 1) * 4;
        if constexpr (sizeof(T) == 2) {
            const uint2 a = quad(s * 32 + grp * 4, c0, col), b = quad(s * 32 + 16 + grp * 4, c0, col);
            return Frag<1>{{frag_of(a.x, a.y, b.x, b.y)}};
        } else {
            const int c = c0 + col / 4 * 8 + col % 4;
            f32x4 a, b;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                a[r] = at(s * 32 + grp * 4 + r, c);
                b[r] = at(s * 32 + 16 + grp * 4 + r, c);
            }
            return split_frag<3>(a, b);
        }
    }
    // a result tile's registers (rows 16 mt + 4 grp + r, column c0 + col)
    __device__ __forceinline__ f32x4 values(int mt, int grp, int c0, int col) const {
        if constexpr (sizeof(T) == 2) {
            const uint2 w = quad16(mt * 16 + grp * 4, c0, col);
            return f32x4{bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y)};
        } else {
            f32x4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = at(mt * 16 + grp * 4 + r, c0 + col);
            return v;
        }
    }
};

// dk of register r of state tile `tile` (see Tile::column)
__device__ __forceinline__ int state_row(int tile, int grp, int r) { return tile / 2 * 32 + grp * 8 + (tile & 1) * 4 + r; }

// ------------------------------------------------------------- chunk matrices
//
// What the chains need of a chunk besides its tokens, laid out by
// delta_prep_kernel as they read it: W (in three parts) and P (in as many as its
// result needs) as A fragments in paired order, row tile mt, steps s <= mt / 2;
// then exp(G_i) and exp(G_C - G_i), 0 behind the last token.  The backward reads
// W^T and P^T out of the same fragments by transposing LDS reads.
template <int kPParts>
struct Mats {
    uint4 W[3][kFrags][64];
    float e[kChunk], rest[kChunk];
    float pad[128];               // whole kilobytes
    uint4 P[kPParts][kFrags][64]; // last: a chain without outputs stops here
};
__device__ __forceinline__ int frag_lower(int mt, int s) { return mt < 2 ? mt : mt * 2 - 2 + s; }

template <int kParts>
__device__ __forceinline__ Frag<kParts> mat_frag(const uint4 (*m)[kFrags][64], int f) {
    Frag<kParts> x;
#pragma unroll
    for (int i = 0; i < kParts; ++i) x.p[i] = __builtin_bit_cast(bf16x8, m[i][f][threadIdx.x & 63]);
    return x;
}
// Fragment of the transpose: row tile mt, step s >= mt / 2.  Block (it, mt) of the
// matrix holds four columns of a row in each lane's 8 bytes.
template <int kParts>
__device__ __forceinline__ Frag<kParts> mat_frag_t(const uint4 (*m)[kFrags][64], int mt, int s, int col, int grp) {
    const int at = (col & 3) * 16 + grp * 4 + (col >> 2);
    Frag<kParts> x;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        uint2 h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint2 *p = (const uint2 *)&m[i][frag_lower(2 * s + j, mt / 2)][at] + (mt & 1);
            h[j] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
        }
        x.p[i] = frag_of(h[0].x, h[0].y, h[1].x, h[1].y);
    }
    return x;
}
// four of a row into half h of its lane's 16 bytes
template <int kParts>
__device__ __forceinline__ void put_quad(uint4 (*m)[kFrags][64], int f, int lane, int h, const float *v) {
    uint32_t a[kParts], b[kParts];
    split_pair<kParts>(v[0], v[1], a);
    split_pair<kParts>(v[2], v[3], b);
#pragma unroll
    for (int i = 0; i < kParts; ++i) ((uint2 *)&m[i][f][lane])[h] = make_uint2(a[i], b[i]);
}

__device__ __forceinline__ void block_of(int tile, int *it, int *jt) {
    *it = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0;
    *jt = tile - *it * (*it + 1) / 2;
}

// One workgroup per (chunk, query/key head, batch): K K^T and Q K^T once, then
// each value head of the group.  N = -diag(beta) A is strictly lower; (I - N)^-1
// by 16x16 blocks: wave j inverts diagonal block j by substitution (a lane per
// column), then runs down block column j: X_i = inv_ii sum_k N_ik X_k, in fp32
// matrix instructions, X_k staying in registers.  Bound by memory where there are
// chunks enough: 65,536 bf16 tokens of 12 heads of 128 in 160 us, 0.76 GB of tokens
// in and matrices out at 4.7 TB/s; W in three parts, so that U keeps its 32 bits.
template <typename T, int kDk, int kPF>
__global__ __launch_bounds__(kDeltaThreads, sizeof(T) == 2 ? 3 : 1) void delta_prep_kernel(const T *__restrict__ q, const T *__restrict__ k,
                                                                  const float *__restrict__ g,
                                                                  const float *__restrict__ beta, Mats<kPF> *__restrict__ mats,
                                                                  double *__restrict__ Gs, DeltaDims d) {
    constexpr int kN = 68;
    __shared__ __attribute__((aligned(16))) union {
        struct {
            Tile<T, kDk> k, q;
        };
        struct {
            float N[kChunk * kN], inv[kChunk * 20];   // inv: the diagonal blocks' inverses
        };
    } l;
    __shared__ double G[kChunk];
    __shared__ float bt[kChunk];
    const int c = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int64_t t0 = (int64_t)c * kChunk, len = row_len(d, b);
    if (t0 >= len) return;
    const int n = len - t0 < kChunk ? (int)(len - t0) : kChunk;
    const int lane = lane_id(), wave = threadIdx.x >> 6, col = lane & 15, grp = lane >> 4;
    {
        const int64_t at = (((int64_t)b * d.T + t0) * d.hk + h) * kDk;
        l.k.template fill<4>(k + at, (int64_t)d.hk * kDk, n);
        if (q != nullptr) l.q.template fill<4>(q + at, (int64_t)d.hk * kDk, n);
    }
    // a head's gates, loaded a head ahead
    float gv = 0.f, bv = 1.f;
    const auto gates = [&](int hv) {
        const int64_t at = ((int64_t)b * d.T + t0 + threadIdx.x) * d.hv + hv;
        if ((int)threadIdx.x < n) {
            gv = g[at];
            bv = strength(beta[at]);
        }
    };
    gates(h * d.group);
    loads_done<0>();
    __syncthreads();
    f32x4 kk[3], kq[3];   // this wave's tiles: K K^T; K Q^T (rows j, columns i)
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        int it, jt;
        block_of(wave + 4 * x < kBlocks ? wave + 4 * x : 0, &it, &jt);
        kk[x] = kq[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < kDk / 32; ++s) {
            const auto ki = l.k.row(it * 16 + col, s, grp), kj = l.k.row(jt * 16 + col, s, grp);
            kk[x] = mma(ki, kj, kk[x]);
            kq[x] = mma(kj, l.q.row(it * 16 + col, s, grp), kq[x]);   // without q: not used
        }
    }
    __syncthreads();   // the tiles are read: N takes their place
    for (int hv = h * d.group; hv < (h + 1) * d.group; ++hv) {
        const int64_t unit = ((int64_t)b * d.hv + hv) * d.chunks + c;
        chunk_decays(gv, G);
        if (threadIdx.x < kChunk) bt[threadIdx.x] = bv;
        __syncthreads();
        if (hv + 1 < (h + 1) * d.group) gates(hv + 1);
        if (threadIdx.x < kChunk) {
            const int t = threadIdx.x;
            const float e = decay(G[t]), rest = t < n ? decay(G[kChunk - 1] - G[t]) : 0.f;
            mats[unit].e[t] = e;
            mats[unit].rest[t] = rest;
            if (Gs != nullptr) Gs[unit * kChunk + t] = G[t];
        }
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            if (wave + 4 * x >= kBlocks) continue;
            int it, jt;
            block_of(wave + 4 * x, &it, &jt);
            float pt[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = it * 16 + grp * 4 + r, j = jt * 16 + col;   // a result tile's rows and columns
                const bool in = i < n && j < n;                            // repeated rows count for nothing
                const float D = decay(G[i] - G[j]);
                l.N[i * kN + j] = j < i && in ? -bt[i] * (D * kk[x][r]) : 0.f;
                const int i2 = it * 16 + col, j2 = jt * 16 + grp * 4 + r;
                pt[r] = j2 <= i2 && i2 < n ? d.scale * decay(G[i2] - G[j2]) * kq[x][r] : 0.f;
            }
            if (q != nullptr) put_quad<kPF>(mats[unit].P, frag_lower(it, jt / 2), lane, jt & 1, pt);
        }
        // halves of the 32-wide steps beyond the triangle
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        if (wave < 2) {
            put_quad<3>(mats[unit].W, frag_lower(wave * 2, wave), lane, 1, zero);
            if (q != nullptr) put_quad<kPF>(mats[unit].P, frag_lower(wave * 2, wave), lane, 1, zero);
        }
        __syncthreads();
        // diagonal block `wave`, column `col` of its inverse
        const int r0 = wave * 16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == col ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; j += 4) {
                const f32x4 w = *(const f32x4 *)&l.N[(r0 + i) * kN + r0 + j];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (j + y < i) s = fmaf(w[y], x[j + y], s);
            }
            x[i] = s;
        }
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) l.inv[(r0 + i) * 20 + col] = x[i];
        }
        __syncthreads();
        const float bj = bt[r0 + col];
        f32x4 X[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < wave) continue;
            if (i == wave) {
#pragma unroll
                for (int r = 0; r < 4; ++r) X[i][r] = l.inv[(r0 + grp * 4 + r) * 20 + col];
            } else {
                f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < i; ++kb) {
                    if (kb < wave) continue;
                    const f32x4 a = *(const f32x4 *)&l.N[(i * 16 + col) * kN + kb * 16 + grp * 4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) t = mfma32(a[r], X[kb][r], t);
                }
                f32x4 y = {0.f, 0.f, 0.f, 0.f};
                const f32x4 a = *(const f32x4 *)&l.inv[(i * 16 + col) * 20 + grp * 4];
#pragma unroll
                for (int r = 0; r < 4; ++r) y = mfma32(a[r], t[r], y);
                X[i] = y;
            }
        }
        __syncthreads();   // N is read: W takes its place
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < wave) continue;
            float w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) w[r] = X[i][r] * bj;
#pragma unroll
            for (int r = 0; r < 4; ++r) l.N[(i * 16 + grp * 4 + r) * kN + wave * 16 + col] = w[r];
        }
        __syncthreads();
#pragma unroll
        for (int y = 0; y < 3; ++y) {
            if (wave + 4 * y >= kBlocks) continue;
            int it, jt;
            block_of(wave + 4 * y, &it, &jt);
            const f32x4 w = *(const f32x4 *)&l.N[(it * 16 + col) * kN + jt * 16 + grp * 4];
            const float v[4] = {w[0], w[1], w[2], w[3]};
            put_quad<3>(mats[unit].W, frag_lower(it, jt / 2), lane, jt & 1, v);
        }
        __syncthreads();
    }
}

// A chunk's matrices into LDS (kParts 0: all but P).
template <int kParts>
struct MatsUsed { using type = Mats<kParts>; };
template <>
struct MatsUsed<0> {
    struct type {
        uint4 W[3][kFrags][64];
        float e[kChunk], rest[kChunk];
        float pad[128];
    };
};
template <int kWaves = 4, typename M>
__device__ __forceinline__ void fill_mats(const void *src, M *dst) {
    constexpr int kLoads = (int)sizeof(M) / 1024;
    static_assert(sizeof(M) % 1024 == 0, "");
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lane = threadIdx.x & 63;
    for (int i = wave; i < kLoads; i += kWaves)
        load_lds((const char *)src + i * 1024, lane * 16, (char *)dst + i * 1024);
}

// out (+)= M x, or M^T x (kTransposed), for a chunk's lower triangular matrix in
// kParts parts and a [64 x 16] column slice x in result tiles.
template <int kParts, bool kZero, bool kTransposed, int kXParts>
__device__ __forceinline__ void tri_product(const uint4 (*m)[kFrags][64], const f32x4 *x, f32x4 *out) {
    const int col = lane_id() & 15, grp = lane_id() >> 4;
    const auto frag = [&](int mt, int s) {
        if constexpr (kTransposed) return mat_frag_t<kParts>(m, mt, s, col, grp);
        else return mat_frag<kParts>(m, frag_lower(mt, s));
    };
    if (kZero) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) out[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const Frag<kXParts> xp = split_frag<kXParts>(x[2 * s], x[2 * s + 1]);
        if ((s == 0) != kTransposed) {   // all four row tiles
            const Frag<kParts> f[4] = {frag(0, s), frag(1, s), frag(2, s), frag(3, s)};
            mma_n<4>(f, xp, out);
        } else {                         // the two at the far side
            constexpr int k0 = kTransposed ? 0 : 2;
            const Frag<kParts> f[2] = {frag(k0, s), frag(k0 + 1, s)};
            mma_n<2>(f, xp, out + k0);
        }
    }
}
template <int kParts, bool kZero = true>
__device__ __forceinline__ void lower_product(const uint4 (*m)[kFrags][64], const f32x4 *x, f32x4 *out) {
    tri_product<kParts, kZero, false, kParts>(m, x, out);
}
template <int kParts, bool kZero = true, int kXParts = kParts>
__device__ __forceinline__ void upper_product(const uint4 (*m)[kFrags][64], const f32x4 *x, f32x4 *out) {
    tri_product<kParts, kZero, true, kXParts>(m, x, out);
}

// S += tile^T x (rows dk, summed over the chunk's tokens), x in three parts
template <typename T, int kDk>
__device__ __forceinline__ void add_columns(const Tile<T, kDk> &tile, const f32x4 *x, f32x4 *S) {
    const int lane = lane_id(), col = lane & 15, grp = lane >> 4;
    constexpr int kTiles = kDk / 16;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const Frag<3> xp = split_frag<3>(x[2 * s], x[2 * s + 1]);
#pragma unroll
        for (int h = 0; h < kTiles; h += 4) {
            Frag<Stream<T>::kParts> f[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) f[t] = tile.column(h + t, s, grp, col);
            mma_n<4>(f, xp, S + h);
        }
    }
}

// --------------------------------------------------------------- forward chain
//
// Where batch, heads and columns are too few to fill the chip, the chunks are
// cut into segments that run at once.  A segment maps the state before it to
// the state behind it by S' = M S + N, the same for every column; the chain
// run from zero gives N, and run from the identity without V gives M
// (kAggregate).  delta_join_kernel goes through the segments once, and the
// chain proper starts each segment from the state it finds there.
enum ChainMode { kStates, kOutputs, kAggregate };

template <typename T>
struct ChainArgs {
    const T *q, *k, *v;
    const Mats<Stream<T>::kOutParts> *mats;
    const float *h_init;  // null: zero; with segments [batch, hv, segs, dk, dv]
    T *o;                 // kOutputs
    float *h_final;       // null: not wanted
    float *h_chunks;      // null, or [batch, chunks, hv, dv, dk]
    float *agg;           // kAggregate: [batch, hv, segs], N [dk, dv] and M (store_map)
    int segs, per;        // segments, and chunks of each
    int wanted;           // kAggregate: the segments whose maps are used
    int groups;           // batch * segs * hv
    DeltaDims d;
};

template <typename T, int kDk, int kMode>
struct ChainStage {
    Tile<T, kDk> k;
    typename std::conditional<kMode == kOutputs, Tile<T, kDk>, char>::type q;
    Tile<T, 64> v;
    typename MatsUsed<kMode == kOutputs ? Stream<T>::kOutParts : 0>::type m;
};

// A column's rows of a state [dk, dv] into its tiles.  (With a test for null at
// each load the compiler made as many branches, and the loads ran one by one.)
template <int kDk>
__device__ __forceinline__ void load_state(const float *h, int dv, int grp, int n, f32x4 *S) {
    const uint32_t lane_off = (uint32_t)(grp * 8 * dv + n);
#pragma unroll
    for (int t = 0; t < kDk / 16; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = (h + state_row(t, 0, r) * dv)[lane_off];
}

// Column j of a segment's M from its tiles, as the join reads it: A fragments (tile of
// rows, step of 32 columns), each in two halves of four floats a lane.  (By rows, each
// lane of the join's loads had a line of its own.)
template <int kDk>
__device__ __forceinline__ void store_map(float *M, int grp, int j, const f32x4 *S) {
    const int at = (j / 32 * 2 + (j % 8) / 4) * 256 + j % 32 / 8 * 64 + grp * 16 + j % 4;
#pragma unroll
    for (int t = 0; t < kDk / 16; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) M[at + t * (kDk / 32) * 512 + r * 4] = S[t][r];
}

template <typename T, int kDk, int kMode>
struct Chain {
    static constexpr bool kWithO = kMode == kOutputs;
    static constexpr int kOut = Stream<T>::kOutParts, kTiles = kDk / 16, kSteps = kDk / 32;
    using Stage = ChainStage<T, kDk, kMode>;
    using In = Frag<Stream<T>::kParts>;
    f32x4 S[kTiles];
    const ChainArgs<T> &a;
    const T *kp, *qp, *vp;
    T *op;
    int64_t kstride, vstride, len;
    int hv, b, lane, wave, col, grp, n;
    bool has_v;      // kAggregate: not the identity's columns
    uint32_t ooff;   // of this lane's outputs within a chunk's rows
    typename Tile<T, kDk>::template Offsets<4> koff;
    typename Tile<T, 64>::template Offsets<4> voff;

    __device__ __forceinline__ void fill(Stage &l, int c) {
        const int64_t t0 = (int64_t)c * kChunk;
        if (len - t0 < kChunk) {
            koff.set(kstride, (int)(len - t0));
            voff.set(vstride, (int)(len - t0));
        }
        l.k.template fill<4>(kp + t0 * kstride, koff);
        if constexpr (kWithO) l.q.template fill<4>(qp + t0 * kstride, koff);
        if (kMode != kAggregate || has_v) l.v.template fill<4>(vp + t0 * vstride, voff);
        fill_mats(a.mats + ((int64_t)b * a.d.hv + hv) * a.d.chunks + c, &l.m);
    }

    // the chunk states' layout, [dv][dk]: 16 bytes a lane and tile
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
        const DeltaDims &d = a.d;
        const int64_t t0 = (int64_t)c * kChunk;
        const int m = len - t0 < kChunk ? (int)(len - t0) : kChunk;
        // R = V - E K S and the state's part of O
        f32x4 R[4], O[4];
        {
            f32x4 ks[4], qs[4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) ks[mt] = qs[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const Frag<3> Sp = split_frag<3>(S[2 * s], S[2 * s + 1]);
                In kf[4], qf[4];
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    kf[mt] = l.k.row(mt * 16 + col, s, grp);
                    if constexpr (kWithO) qf[mt] = l.q.row(mt * 16 + col, s, grp);
                }
                mma_n<4>(kf, Sp, ks);
                if constexpr (kWithO) mma_n<4>(qf, first_parts<kOut>(Sp), qs);
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const f32x4 e = *(const f32x4 *)(l.m.e + mt * 16 + grp * 4);
                f32x4 v = {0.f, 0.f, 0.f, 0.f};
                if (kMode != kAggregate || has_v) v = l.v.values(mt, grp, wave * 16, col);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    R[mt][r] = fmaf(-e[r], ks[mt][r], v[r]);
                    O[mt][r] = d.scale * e[r] * qs[mt][r];
                }
            }
        }
        f32x4 U[4];
        lower_product<3>(l.m.W, R, U);
        // the next state
        {
            const float last = l.m.e[kChunk - 1];
            f32x4 Ur[4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const f32x4 rest = *(const f32x4 *)(l.m.rest + mt * 16 + grp * 4);
#pragma unroll
                for (int r = 0; r < 4; ++r) Ur[mt][r] = rest[r] * U[mt][r];
            }
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[t][r] *= last;
            add_columns(l.k, Ur, S);
        }
        if constexpr (kWithO) {
            T *out = op + t0 * vstride;
            lower_product<kOut, false>(l.m.P, U, O);
            if (m == kChunk) {   // uniform rows and a lane's own offset
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) Stream<T>::store(out + (mt * 16 + r) * vstride + ooff, O[mt][r]);
            } else {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (mt * 16 + grp * 4 + r < m) Stream<T>::store(out + (mt * 16 + r) * vstride + ooff, O[mt][r]);
            }
        }
    }
};

// A chain's workgroups in one dimension.  Consecutive workgroups go to the eight
// XCDs in turn; the column blocks of one head read the same keys and matrices
// and share an XCD's L2, so they take every eighth place.
struct ChainPlace {
    int col, group;   // column block; (row, segment, head), head fastest
};
__device__ __forceinline__ ChainPlace chain_place(int cols) {
    const int x = blockIdx.x % 8, r = blockIdx.x / 8;
    return ChainPlace{r % cols, r / cols * 8 + x};
}

// Bound by the latency of a step (products with the state, W, P, the state's
// update, each waiting for the one before) times the row's chunks: 3.3 us a step
// of 128 by 128 with outputs while workgroups have a CU of their own (5.9 where it
// writes its chunk states too).  Where workgroups fill the chip
// no unit is busy above 42% (65,536 bf16 tokens of 12 heads of 128: the aggregate
// pass in 373 us and the outputs in 355 us; matrix instructions 42% and 33% of the
// cycles, LDS 35% and 25%, other vector instructions 28% and 20%): 64 columns a workgroup, because 16 a
// wave is what its S, R, U, O and fragments leave room for at two workgroups a CU.
//
// kTwo: a second set of tiles in LDS, filled while a step computes: one
// workgroup a CU.  Else one set, and two workgroups a CU cover each other's
// waits: the faster of the two wherever there are enough workgroups.
template <typename T, int kDk, int kMode, bool kTwo>
__global__ __launch_bounds__(kDeltaThreads, kTwo || sizeof(T) == 4 ? 1 : 2) void delta_chain_kernel(ChainArgs<T> a) {
    using C = Chain<T, kDk, kMode>;
    constexpr bool kWithO = kMode == kOutputs;
    __shared__ __attribute__((aligned(16))) typename C::Stage l0;
    __shared__ __attribute__((aligned(16))) typename std::conditional<kTwo, typename C::Stage, char>::type l1;
    const DeltaDims &d = a.d;
    const ChainPlace at = chain_place((d.dv + (kMode == kAggregate ? kDk : 0)) / 64);
    if (at.group >= a.groups) return;
    C s{{}, a};
    s.hv = at.group % d.hv;
    s.b = at.group / d.hv / a.segs;
    const int seg = at.group / d.hv % a.segs, hk = s.hv / d.group;
    if (kMode == kAggregate && seg >= a.wanted) return;
    s.lane = lane_id();
    s.wave = threadIdx.x >> 6;
    s.col = s.lane & 15;
    s.grp = s.lane >> 4;
    s.n = at.col * 64 + s.wave * 16 + s.col;   // this lane's state column
    s.has_v = kMode != kAggregate || at.col * 64 < d.dv;
    s.len = row_len(d, s.b);
    s.kstride = (int64_t)d.hk * kDk;
    s.vstride = (int64_t)d.hv * d.dv;
    const int64_t tok = (int64_t)s.b * d.T;
    s.kp = a.k + (tok * d.hk + hk) * kDk;
    s.qp = kWithO ? a.q + (tok * d.hk + hk) * kDk : nullptr;
    s.vp = a.v + (tok * d.hv + s.hv) * d.dv + (s.has_v ? at.col * 64 : 0);
    s.op = kWithO ? a.o + (tok * d.hv + s.hv) * d.dv + at.col * 64 : nullptr;
    s.ooff = (uint32_t)(s.grp * 4 * s.vstride) + s.wave * 16 + s.col;
    s.koff.set(s.kstride, kChunk);
    s.voff.set(s.vstride, kChunk);
    const int chunks = (int)((s.len + kChunk - 1) / kChunk);   // the row's, of all segments
    const int c0 = seg * a.per, c1 = c0 + a.per < chunks ? c0 + a.per : chunks;
    const int64_t state = (int64_t)kDk * d.dv, head = (int64_t)s.b * d.hv + s.hv;
#pragma unroll
    for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            s.S[t][r] = kMode == kAggregate && s.n - d.dv == state_row(t, s.grp, r) ? 1.f : 0.f;
        }
    if (kMode != kAggregate && a.h_init != nullptr) load_state<kDk>(a.h_init + (head * a.segs + seg) * state, d.dv, s.grp, s.n, s.S);
    auto keep = [&](int c) {
        if (kMode != kAggregate && a.h_chunks != nullptr)
            s.store_columns(a.h_chunks + (((int64_t)s.b * d.chunks + c) * d.hv + s.hv) * state);
    };
    if constexpr (kTwo) {
        if (c0 < c1) s.fill(l0, c0);
        for (int c = c0; c < c1; c += 2) {
            // l0 is filled, l1 is read.  A full chunk's step ends with 16 stores of
            // its outputs; only the last is not full.
            if (kWithO && c > c0) loads_done<16>();
            else loads_done<0>();
            __syncthreads();
            if (c + 1 < c1) s.fill(l1, c + 1);
            keep(c);
            s.step(l0, c);
            if (c + 1 >= c1) break;
            loads_done<kWithO ? 16 : 0>();
            __syncthreads();
            if (c + 2 < c1) s.fill(l0, c + 2);
            keep(c + 1);
            s.step(l1, c + 1);
        }
    } else {
        for (int c = c0; c < c1; ++c) {
            __syncthreads();
            s.fill(l0, c);
            keep(c);
            loads_done<0>();
            __syncthreads();
            s.step(l0, c);
        }
    }
    if (kMode == kAggregate) {
        float *map = a.agg + (head * a.segs + seg) * kDk * (d.dv + kDk);
        if (s.has_v) s.store_state(map, d.dv);
        else store_map<kDk>(map + kDk * d.dv, s.grp, s.n - d.dv, s.S);
        return;
    }
    if (a.h_final != nullptr && seg == a.segs - 1) s.store_state(a.h_final + head * state, d.dv);
    // chunks of padding alone: the state stays
    const int end = c0 + a.per < d.chunks ? c0 + a.per : d.chunks;
    for (int c = c1 > c0 ? c1 : c0; c < end; ++c) keep(c);
    if (kWithO) {   // padding: zeros
        const int64_t t0 = s.len > (int64_t)c0 * kChunk ? s.len : (int64_t)c0 * kChunk;
        const int64_t t1 = (int64_t)end * kChunk < d.T ? (int64_t)end * kChunk : d.T;
        for (int64_t t = t0 + s.grp; t < t1; t += 4) Stream<T>::store(s.op + t * s.vstride + s.wave * 16 + s.col, 0.f);
    }
}

// Through the segments: h[0] = h_init, h[s + 1] = M_s h[s] + N_s (back: from the last
// segment to the first).  One workgroup per 16 columns and head: the state in LDS parts (B fragments of 32 dk), a wave to each
// 16 rows of M, read as its fragments (store_map).  Serial over the segments, 2 us
// each at 128 by 128 (16 segments of 12 heads: 33 us; with M by rows, whose loads
// touched a line for each lane, 49 where this took 35); the next two segments' maps are on their way
// meanwhile.
struct JoinArgs {
    const float *agg, *h_init;   // h_init null: zero
    float *h_seg;                // [batch, hv, segs, dk, dv] out, or null
    float *h_final;              // behind the last segment, or null
    int segs, dv;
    bool back;
};

template <int kDk>
__global__ __launch_bounds__(kDk * 4) void delta_join_kernel(JoinArgs a) {
    constexpr int kSteps = kDk / 32;
    __shared__ uint4 part[kSteps][3][64];
    const int lane = lane_id(), wave = threadIdx.x >> 6, col = lane & 15, grp = lane >> 4, n = blockIdx.x * 16 + col;
    const int64_t head = blockIdx.y, state = (int64_t)kDk * a.dv;
    const int64_t mine = (int64_t)state_row(wave, grp, 0) * a.dv + n;   // of the lane's four rows, dv apart
    f32x4 h = {0.f, 0.f, 0.f, 0.f};
    if (a.h_init != nullptr) {
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = a.h_init[head * state + mine + r * a.dv];
    }
    const auto store = [&](float *out) {
#pragma unroll
        for (int r = 0; r < 4; ++r) out[mine + r * a.dv] = h[r];
    };
    const auto at = [&](int s) { return head * a.segs + (a.back ? a.segs - 1 - s : s); };
    // a segment's N and the wave's 16 rows of M, loaded two segments ahead
    struct Map {
        f32x4 N, M[kSteps][2];
    } m0, m1;
    const auto fetch = [&](int s, Map &to) {
        const float *m = a.agg + at(s) * kDk * (a.dv + kDk);
#pragma unroll
        for (int r = 0; r < 4; ++r) to.N[r] = m[mine + r * a.dv];
#pragma unroll
        for (int x = 0; x < kSteps; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) to.M[x][y] = *(const f32x4 *)(m + kDk * a.dv + ((wave * kSteps + x) * 2 + y) * 256 + lane * 4);
    };
    const int last = a.h_final != nullptr ? a.segs : a.segs - 1;   // maps that are needed
    if (last > 0) fetch(0, m0);
    if (last > 1) fetch(1, m1);
    const auto turn = [&](int s, Map &now) {   // whether there is another
        if (a.h_seg != nullptr) store(a.h_seg + at(s) * state);
        if (s >= last) return false;
        __syncthreads();   // the parts of the segment before are read
        uint32_t lo[3], hi[3];
        split_pair<3>(h[0], h[1], lo);
        split_pair<3>(h[2], h[3], hi);
#pragma unroll
        for (int p = 0; p < 3; ++p) ((uint2 *)&part[wave / 2][p][lane])[wave & 1] = make_uint2(lo[p], hi[p]);
        Frag<3> mf[kSteps];
        h = now.N;
#pragma unroll
        for (int x = 0; x < kSteps; ++x) mf[x] = split_frag<3>(now.M[x][0], now.M[x][1]);
        if (s + 2 < last) fetch(s + 2, now);
        __syncthreads();
        f32x4 odd = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < kSteps; ++x) {
            Frag<3> y;
#pragma unroll
            for (int p = 0; p < 3; ++p) y.p[p] = __builtin_bit_cast(bf16x8, part[x][p][lane]);
            // two sums side by side: one of its own would wait for its last product
            if (x & 1) odd = mma(mf[x], y, odd);
            else h = mma(mf[x], y, h);
        }
        h += odd;
        return s + 1 < a.segs;
    };
    for (int s = 0; turn(s, m0) && turn(s + 1, m1); s += 2) {
    }
    if (a.h_final != nullptr) store(a.h_final + head * state);
}

// ---------------------------------------------------------------- recurrent
//
// The recurrence as written, token by token, for the active block: one wave
// per 32 columns of one head's state, held in registers (a lane: 4 columns and
// dk / 8 consecutive rows), so the state is read once and written once however
// many tokens there are.  Both sums over the rows (S^T k and S^T q of the
// decayed state; o = S^T q + (k.q) u) fold over the 8 row groups together.
// One token is bound by the launch (1 row of 16 heads: 3.9 us) or by memory (64
// rows of 16 heads of 128 by 128: 21.5 us with its launch, 6.2 TB/s); each further
// token adds 2 us there, three operations to each element of the state.  32 columns
// a wave: the sums' exchanges are shared by four columns a lane, and the state's 64
// registers leave three waves a SIMD.
template <typename T>
struct StepArgs {
    const T *q, *k, *v;
    const float *g, *beta, *h;   // h null: zero state
    T *o;                        // null: the state alone
    float *h_out;                // null: the outputs alone; may be h
    DeltaDims d;
};

// kN consecutive stream elements as they lie in memory, and as fp32
template <typename T, int kN>
struct Run {
    static constexpr int kWords = kN * (int)sizeof(T) / 16;
    uint4 w[kWords];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = ((const uint4 *)p)[i];
    }
    __device__ __forceinline__ void values(float *out) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 2) {
                    out[i * 8 + 2 * j] = bf_lo(u[j]);
                    out[i * 8 + 2 * j + 1] = bf_hi(u[j]);
                } else {
                    out[i * 4 + j] = as_f(u[j]);
                }
            }
        }
    }
};

template <typename T>
struct Four;
template <>
struct Four<uint16_t> {
    uint2 w;
    __device__ __forceinline__ void load(const uint16_t *p) { w = *(const uint2 *)p; }
    __device__ __forceinline__ f32x4 values() const { return f32x4{bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y)}; }
};
template <>
struct Four<float> {
    f32x4 w;
    __device__ __forceinline__ void load(const float *p) { w = *(const f32x4 *)p; }
    __device__ __forceinline__ f32x4 values() const { return w; }
};
__device__ __forceinline__ void store4(uint16_t *p, f32x4 v) {
    *(uint2 *)p = make_uint2(pk_rne(v[0], v[1]), pk_rne(v[2], v[3]));
}
__device__ __forceinline__ void store4(float *p, f32x4 v) { *(f32x4 *)p = v; }

// sum over the 8 row groups (lanes 8 apart), in every lane: by 8 within rows of
// 16 lanes, then by exchanging halves of 32 and of 64
__device__ __forceinline__ float row_sum(float x) {
    x += as_f(__builtin_amdgcn_update_dpp(0, as_u(x), 0x128, 0xf, 0xf, false));   // row_ror:8
    const auto h = __builtin_amdgcn_permlane16_swap(as_u(x), as_u(x), false, false);
    x = as_f(h[0]) + as_f(h[1]);
    const auto w = __builtin_amdgcn_permlane32_swap(as_u(x), as_u(x), false, false);
    return as_f(w[0]) + as_f(w[1]);
}

template <int kR>
__device__ __forceinline__ void scale_state(f32x4 (&S)[kR], float c) {
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) S[i][x] *= c;
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
    for (int i = 0; i < kR; ++i) S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.h != nullptr) {
#pragma unroll
        for (int i = 0; i < kR; ++i) S[i] = *(const f32x4 *)(a.h + state + (int64_t)i * d.dv);
    }
    // S holds the state divided by c, the product of the decays since S was last
    // scaled: a token's decay costs no pass over S.
    float c = 1.f;
    // a token's operands, on their way while the one before is worked on
    struct {
        Run<T, kR> k, q;
        Four<T> v;
        float g, beta;
    } next;
    const auto fetch = [&](int64_t t) {
        next.k.load(a.k + ((at0 + t) * d.hk + hk) * kDk + r0);
        if (a.o != nullptr) next.q.load(a.q + ((at0 + t) * d.hk + hk) * kDk + r0);
        next.v.load(a.v + ((at0 + t) * d.hv + hv) * d.dv + n);
        next.g = a.g[(at0 + t) * d.hv + hv];
        next.beta = a.beta[(at0 + t) * d.hv + hv];
    };
    if (len > 0) fetch(0);
    for (int64_t t = 0; t < len; ++t) {
        float k[kR], q[kR];
        next.k.values(k);
        if (a.o != nullptr) next.q.values(q);
        const f32x4 v = next.v.values();
        const float bt = next.beta;
        c *= __expf(next.g);
        if (t + 1 < len) fetch(t + 1);
        if (!(c >= 0x1p-30f && c <= 0x1p30f)) {
            scale_state(S, c);
            c = 1.f;
        }
        f32x4 p = {0.f, 0.f, 0.f, 0.f}, s = {0.f, 0.f, 0.f, 0.f};
        float kq = 0.f;
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) p[x] = fmaf(S[i][x], k[i], p[x]);
        if (a.o != nullptr) {
#pragma unroll
            for (int i = 0; i < kR; ++i) {
                kq = fmaf(k[i], q[i], kq);
#pragma unroll
                for (int x = 0; x < 4; ++x) s[x] = fmaf(S[i][x], q[i], s[x]);
            }
            kq = row_sum(kq);
        }
        const float ic = 1.f / c;
        f32x4 u, us;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            u[x] = bt * fmaf(-c, row_sum(p[x]), v[x]);
            us[x] = u[x] * ic;
        }
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) S[i][x] = fmaf(k[i], us[x], S[i][x]);
        if (a.o != nullptr) {
            f32x4 o;
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] = d.scale * fmaf(kq, u[x], c * row_sum(s[x]));
            if (lane < 8) store4(a.o + ((at0 + t) * d.hv + hv) * d.dv + n, o);
        }
    }
    if (c != 1.f) scale_state(S, c);
    if (a.o != nullptr)
        for (int64_t t = len + (lane >> 3); t < d.T; t += 8)
            store4(a.o + ((at0 + t) * d.hv + hv) * d.dv + n, f32x4{0.f, 0.f, 0.f, 0.f});
    if (a.h_out != nullptr && !(len == 0 && a.h == a.h_out)) {
#pragma unroll
        for (int i = 0; i < kR; ++i) *(f32x4 *)(a.h_out + state + (int64_t)i * d.dv) = S[i];
    }
}

// The same for blocks of bf16 tokens, 16 tokens at a time in the chunked form above
// with matrix instructions: the token by token kernel's three operations to each
// element of the state and token bound it from some tokens on.  One wave per 32
// columns of one head's state, in registers as the chains' (tile nt holds columns
// n + nt, so that a lane's pairs of columns are neighbours in memory).  U comes by
// substitution over the 16 tokens, (I + diag(beta) A) U = diag(beta) R, each
// token's row of U handed to the other lane groups in turn.  64 rows of 16 heads of
// 128 by 128 and 16 tokens in place: 34 us for 147 MB (4.3 TB/s; by token 54), bound by
// memory and a wave's start and end: two waves a SIMD, three spill and take 42.  The
// state goes on in three bf16 parts, so that it keeps its 32 bits.

// x of lane group kFrom (16 lanes) in all four
template <int kFrom>
__device__ __forceinline__ float of_group(float x) {
    const auto h = __builtin_amdgcn_permlane16_swap(as_u(x), as_u(x), false, false);
    const auto w = __builtin_amdgcn_permlane32_swap(h[kFrom & 1], h[kFrom & 1], false, false);
    return as_f(w[kFrom >> 1]);
}

// a wave's LDS operations are done in order: this one only keeps the compiler's
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int kDk>
__global__ __launch_bounds__(64, 2) void delta_block_kernel(StepArgs<uint16_t> a) {
    constexpr int kTiles = kDk / 16, kSteps = kDk / 32, kSub = 16;
    __shared__ __attribute__((aligned(16))) uint16_t K[kSub][kDk + 8];
    __shared__ __attribute__((aligned(16))) float L[kSub][kSub];   // [j][i]: beta_i A_ij
    __shared__ __attribute__((aligned(16))) float e[kSub], rest[kSub], strength_of[kSub];
    __shared__ double G[kSub];
    const DeltaDims &d = a.d;
    const int hv = blockIdx.y, b = blockIdx.z, hk = hv / d.group;
    const int lane = lane_id(), col = lane & 15, grp = lane >> 4, n = blockIdx.x * 32 + 2 * col;
    const int64_t len = row_len(d, b), at0 = (int64_t)b * d.T, state = ((int64_t)b * d.hv + hv) * kDk * d.dv + blockIdx.x * 32;
    const uint32_t lane_off = (uint32_t)(grp * 8 * d.dv) + 2 * col;   // of its pairs of columns in the state
    const bool with_o = a.o != nullptr;
    const uint16_t *qp = with_o ? a.q : a.k;   // without outputs: any
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 S[2][kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) S[0][t] = S[1][t] = zero;
    if (a.h != nullptr) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float2 w = *(const float2 *)(a.h + state + state_row(t, 0, r) * d.dv + lane_off);
                S[0][t][r] = w.x;
                S[1][t][r] = w.y;
            }
    }
    for (int64_t t0 = 0; t0 < len; t0 += kSub) {
        const int m = len - t0 < kSub ? (int)(len - t0) : kSub;
        const int64_t row = at0 + t0;
        const int64_t kat = ((row + (col < m ? col : m - 1)) * d.hk + hk) * kDk + grp * 8;   // tokens behind the last repeat it
        Frag<1> kf[kSteps], qf[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            kf[s] = load_straight(a.k + kat + s * 32);
            qf[s] = load_straight(qp + kat + s * 32);
        }
        uint32_t v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = grp * 4 + r;
            v[r] = *(const uint32_t *)(a.v + ((row + (i < m ? i : m - 1)) * d.hv + hv) * d.dv + n);
        }
        wave_order();   // the last 16 tokens' reads
        chunk_decays<kSub>(lane < m ? a.g[(row + lane) * d.hv + hv] : 0.f, G);
        if (lane < kSub) strength_of[lane] = lane < m ? a.beta[(row + lane) * d.hv + hv] : 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) *(uint4 *)&K[col][s * 32 + grp * 8] = __builtin_bit_cast(uint4, kf[s].p[0]);
        wave_order();
        const double end = G[kSub - 1], Gc = G[col];
        if (lane < kSub) {
            e[lane] = decay(Gc);
            rest[lane] = lane < m ? decay(end - Gc) : 0.f;
        }
        // rows k token 4 grp + r; columns k and q token
        f32x4 A = zero, P = zero;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            A = mma(kf[s], kf[s], A);
            P = mma(kf[s], qf[s], P);
        }
        const f32x4 bt = *(const f32x4 *)(strength_of + grp * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = grp * 4 + r;
            const double g = G[i];
            A[r] = col < i ? bt[r] * decay(g - Gc) * A[r] : 0.f;   // A is symmetric but for this
            P[r] = i <= col ? decay(Gc - g) * P[r] : 0.f;          // P_ji as the A operand of P U has it
        }
        *(f32x4 *)&L[col][grp * 4] = A;
        wave_order();
        f32x4 U[2] = {zero, zero}, O[2] = {zero, zero};
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const Frag<3> Sp = split_frag<3>(S[nt][2 * s], S[nt][2 * s + 1]);
                U[nt] = mma(kf[s], Sp, U[nt]);
                if (with_o) O[nt] = mma(qf[s], first_parts<2>(Sp), O[nt]);
            }
        const f32x4 ev = *(const f32x4 *)(e + grp * 4), rv = *(const f32x4 *)(rest + grp * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            U[0][r] = bt[r] * fmaf(-ev[r], U[0][r], bf_lo(v[r]));
            U[1][r] = bt[r] * fmaf(-ev[r], U[1][r], bf_hi(v[r]));
        }
        const auto eliminate = [&](auto from) {
            constexpr int g0 = decltype(from)::value;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 l = *(const f32x4 *)&L[g0 * 4 + j][grp * 4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const float u = of_group<g0>(U[nt][j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) U[nt][r] = fmaf(-l[r], u, U[nt][r]);
                }
            }
        };
        eliminate(std::integral_constant<int, 0>{});
        eliminate(std::integral_constant<int, 1>{});
        eliminate(std::integral_constant<int, 2>{});
        eliminate(std::integral_constant<int, 3>{});
        if (with_o) {
            const Frag<2> Pf = split_frag<2>(P, zero);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int r = 0; r < 4; ++r) O[nt][r] *= ev[r];
                O[nt] = mma(Pf, split_frag<2>(U[nt], zero), O[nt]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (grp * 4 + r < m)
                    *(uint32_t *)(a.o + ((row + grp * 4 + r) * d.hv + hv) * d.dv + n) = pk_rne(d.scale * O[0][r], d.scale * O[1][r]);
        }
        if (t0 + kSub >= len && a.h_out == nullptr) break;   // the state is not wanted
        const float last = decay(end);
        Frag<3> Up[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            f32x4 x;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = rv[r] * U[nt][r];
            Up[nt] = split_frag<3>(x, zero);
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const uint16_t *p = &K[grp * 4][t / 2 * 32 + col / 4 * 8 + (t & 1) * 4 + col % 4];
            constexpr int kRow = kDk + 8;
            const Frag<1> kt = {{frag_of(p[0] | (uint32_t)p[kRow] << 16, p[2 * kRow] | (uint32_t)p[3 * kRow] << 16, 0u, 0u)}};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[nt][t][r] *= last;
                S[nt][t] = mma(kt, Up[nt], S[nt][t]);
            }
        }
    }
    if (with_o)
        for (int64_t t = len + grp; t < d.T; t += 4) *(uint32_t *)(a.o + ((at0 + t) * d.hv + hv) * d.dv + n) = 0u;
    if (a.h_out != nullptr && !(len == 0 && a.h == a.h_out)) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *(float2 *)(a.h_out + state + state_row(t, 0, r) * d.dv + lane_off) = make_float2(S[0][t][r], S[1][t][r]);
    }
}

}  // namespace bdssm_dev
