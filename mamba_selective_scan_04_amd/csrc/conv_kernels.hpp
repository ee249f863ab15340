// conv_kernels.hpp -- the short causal convolution in front of a scan, for each
// channel by itself:
//   p_t = bias + sum_{j < W} w_j u_{t-W+1+j},   y_t = p_t or silu(p_t),
// and its gradients
//   dp_t = dy_t y'(p_t),  du_s = sum_{d < W} w_{W-1-d} dp_{s+d},
//   dw_j = sum_t dp_t u_{t-W+1+j},  dbias = sum_t dp_t.
// Inputs in front of the row come from its state (the last W - 1 inputs, kept as
// they are); a token that starts a document sees none but its own.
//
// Memory is the bound: 2 W + 4 operations a value against 4 bytes (bf16).  A lane
// takes four neighbouring channels and a chunk of consecutive tokens, keeping the last
// W - 1 inputs in registers, so that each input is read once but for the W - 1 in
// front of a chunk.  65,536 tokens of 2,048 channels in bf16, half of a projection: 104
// us a call (5.2 TB/s read and written; copies run at 4.9 to 5.2); 8 rows of 4,096 tokens
// of 1,536: 40 to 42 us.  Eight channels of bf16, 16 bytes a load: 109 and 42 us, 6.8
// instead of 6.0 for 64 rows of 16 tokens.  kPlain: every lane has its kN channels and
// y = silu(p); kStarts: there may be starts of documents.  Without kPlain, where all
// lanes are whole and only silu is asked for at run time, the first takes 106 us and the
// second 40; with 1,535 channels instead of 1,536, whose last lane's wave goes the whole
// lanes' way and the values' one by one for every token, 73.
// With kStarts the second takes 60 us: a token's byte of `starts` is loaded behind the
// store of the token in front of it, which for all that the compiler knows may have
// written it, and the wait for the byte is one for everything under way, the store and
// the tokens read ahead among it (waves wait for 68% of the time, without documents 39%).
#pragma once

#include "layer_common.hpp"

namespace bdssm_dev {

template <typename T>
struct ConvArgs {
    const T *u;
    int64_t ld, batch_ld;      // elements from a token to the next, from a row to the next
    const float *w, *bias;
    const int32_t *lens;       // [batch] or null
    const uint8_t *starts;     // [batch, T] or null
    const T *c_init;           // [batch, W - 1, ch] or null
    T *y, *c_final;            // either may be null
    int64_t jobs;              // lanes * chunks * batch
    int T_tokens, chunk, chunks;   // tokens of a row and of a chunk, chunks of a row
    int ch, lanes, silu;
    // backward
    const T *dy, *dc_final;
    T *du, *dc_init;
    int64_t du_ld, du_batch_ld;
    float *parts;              // [part][W + 1][ch]
    int row_lanes;             // lanes of a row of the workgroup (a power of two)
    int64_t rows;              // chunks in all
    int groups, n_parts;       // workgroups across the channels, and along the chunks
};

// 1 / (1 + exp(-p)).  exp as 2^x, whose argument's rounding moves it by |p| 2^-24 of
// itself at most; the sigmoid moves by as much where it is small (p far below 0) and
// by less elsewhere.
__device__ __forceinline__ float sigmoid(float p) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(p * -1.44269504088896341f));
}

// How many tokens behind the last document's start a token is, as far as taps care.
__device__ __forceinline__ int age_after(const uint8_t *starts, int t, int age) {
    return starts[t] ? 0 : age + 1;
}
constexpr int kOld = 1 << 30;   // at least as far; stays below 2^31 over a row

// The W - 1 inputs in front of token t0 (hist[0] the oldest) and their age.
template <typename T, int kW, int kN>
__device__ __forceinline__ int conv_history(const ConvArgs<T> &a, const uint8_t *starts, int64_t b, int t0, int c0, int n_ch, Vals<T, kN> (&hist)[kW - 1]) {
    const T *ub = a.u + b * a.batch_ld + c0;
#pragma unroll
    for (int j = 0; j < kW - 1; ++j) {
        const int t = t0 - (kW - 1) + j;
        if (t >= 0) hist[j].load(ub + (int64_t)t * a.ld, n_ch);
        else if (a.c_init != nullptr) hist[j].load(a.c_init + (b * (kW - 1) + t + kW - 1) * a.ch + c0, n_ch);
        else hist[j].zero();
    }
    int age = kOld;   // of token t0 - 1
    if (starts != nullptr) {
#pragma unroll
        for (int j = 0; j < kW - 1; ++j) {
            const int t = t0 - (kW - 1) + j;
            if (t >= 0) age = age_after(starts, t, age);
        }
    }
    return age;
}

template <int kW, int kN>
__device__ __forceinline__ void conv_weights(const float *w, const float *bias, int c0, int n_ch, float (&wt)[kN][kW], float (&bs)[kN]) {
    if (n_ch >= kN) {
        __builtin_memcpy(wt, w + (int64_t)c0 * kW, sizeof wt);
        if (bias != nullptr) __builtin_memcpy(bs, bias + c0, sizeof bs);
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
#pragma unroll
            for (int j = 0; j < kW; ++j) wt[i][j] = i < n_ch ? w[(int64_t)(c0 + i) * kW + j] : 0.f;
            bs[i] = i < n_ch && bias != nullptr ? bias[c0 + i] : 0.f;
        }
    }
    if (bias == nullptr) {
#pragma unroll
        for (int i = 0; i < kN; ++i) bs[i] = 0.f;
    }
}

// Tokens that a row has.
template <typename T>
__device__ __forceinline__ int conv_len(const ConvArgs<T> &a, int64_t b) {
    const int n = a.lens == nullptr ? a.T_tokens : a.lens[b];
    return n < 0 ? 0 : n < a.T_tokens ? n : a.T_tokens;
}

// The row's first chunk writes its last state: it alone has read the first one, which
// may lie in the same place.
template <typename T, int kW, int kN, bool kPlain, bool kStarts>
__global__ __launch_bounds__(256) void conv_kernel(ConvArgs<T> a) {
    constexpr int kAhead = 6;   // tokens read at a time: a multiple of W - 1, so that no input moves
    const int64_t job = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (job >= a.jobs) return;
    const int lane = (int)(job % a.lanes), chunk = (int)(job / a.lanes % a.chunks);
    const int64_t b = job / a.lanes / a.chunks;
    const int c0 = lane * kN, n_ch = kPlain ? kN : a.ch - c0, n = conv_len(a, b);
    const int t0 = chunk * a.chunk, t1 = a.T_tokens - t0 < a.chunk ? a.T_tokens : t0 + a.chunk;
    const int stop = t1 < n ? t1 : n;   // of the tokens that are read
    const uint8_t *starts = kStarts ? a.starts + b * a.T_tokens : nullptr;
    Vals<T, kN> hist[kW - 1];
    int age = kOld;
    if (a.y != nullptr && t0 < stop) age = conv_history<T, kW, kN>(a, starts, b, t0, c0, n_ch, hist);
    if (chunk == 0 && a.c_final != nullptr) {
        Vals<T, kN> last[kW - 1];
        const int old = conv_history<T, kW, kN>(a, starts, b, n, c0, n_ch, last);   // of token n - 1
#pragma unroll
        for (int j = 0; j < kW - 1; ++j) {
            if (kW - 2 - j > old) last[j].zero();   // a document started behind it
            last[j].store(a.c_final + (b * (kW - 1) + j) * a.ch + c0, n_ch);
        }
    }
    if (a.y == nullptr) return;
    T *yb = a.y + b * a.T_tokens * a.ch + c0;
    if (t0 < stop) {
        float wt[kN][kW], bs[kN];
        conv_weights<kW, kN>(a.w, a.bias, c0, n_ch, wt, bs);
        const T *ub = a.u + b * a.batch_ld + c0;
        const auto token = [&](int t, const Vals<T, kN> &x) {
            if (kStarts) {
                age = age_after(starts, t, age);
#pragma unroll
                for (int j = 0; j < kW - 1; ++j)
                    if (kW - 1 - j > age) hist[j].zero();
            }
            float p[kN];
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                p[e] = bs[e];
#pragma unroll
                for (int j = 0; j < kW - 1; ++j) p[e] = fmaf(wt[e][j], hist[j].at(e), p[e]);
                p[e] = fmaf(wt[e][kW - 1], x.at(e), p[e]);
            }
            if (kPlain || a.silu) {
#pragma unroll
                for (int e = 0; e < kN; ++e) p[e] *= sigmoid(p[e]);
            }
            Vals<T, kN> out;
            out.put(p);
            out.store(yb + (int64_t)t * a.ch, n_ch);
#pragma unroll
            for (int j = 0; j + 1 < kW - 1; ++j) hist[j] = hist[j + 1];
            hist[kW - 2] = x;
        };
        int t = t0;
        if (t + kAhead <= stop) {   // the next tokens on their way while these are worked on
            Vals<T, kN> x[kAhead], next[kAhead];
            const auto fetch = [&](Vals<T, kN> (&to)[kAhead], int t) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) to[i].load(ub + (int64_t)(t + i) * a.ld, n_ch);
            };
            fetch(x, t);
            for (; t + 2 * kAhead <= stop; t += kAhead) {
                fetch(next, t + kAhead);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) token(t + i, x[i]);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) x[i] = next[i];
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) token(t + i, x[i]);
            t += kAhead;
        }
        {   // fewer than kAhead are left
            Vals<T, kN> x[kAhead - 1];
#pragma unroll
            for (int i = 0; i < kAhead - 1; ++i)
                if (t + i < stop) x[i].load(ub + (int64_t)(t + i) * a.ld, n_ch);
#pragma unroll
            for (int i = 0; i < kAhead - 1; ++i)
                if (t + i < stop) token(t + i, x[i]);
        }
    }
    Vals<T, kN> none;
    none.zero();
    for (int t = stop > t0 ? stop : t0; t < t1; ++t) none.store(yb + (int64_t)t * a.ch, n_ch);
}

// Gradients.  A lane sweeps its chunk and the W - 1 tokens behind it forward in
// time, the inputs' last W - 1 values and the W - 1 unfinished sums of du in
// registers; du_s is whole once dp_{s+W-1} is there.  Tokens go kAhead at a time
// but at a row's ends (chunks are multiples of 6).  The parameters' sums of a
// workgroup's chunks join in LDS in a fixed order and go to `parts`.  Bound by memory
// and the vector units (57% of their slots): 8 rows of 4,096 tokens of 1,536 channels in
// bf16 66 to 71 us (4.3 to 4.6 TB/s; 84 with three tokens at a time).  With documents 92
// to 94: three tokens at a time, by registers, and for each the wait for its byte of
// `starts`, as above (waves wait for 60% of the time, without documents 39%).  1,535
// channels, whose last lane's wave walks both ways: 205.
template <typename T, int kW, int kN, bool kPlain, bool kStarts>
__global__ __launch_bounds__(256, 3) void conv_bwd_kernel(ConvArgs<T> a) {
    constexpr int kAhead = kPlain && !kStarts ? 6 : kW == 4 ? 3 : 2, kSums = kN * (kW + 1);
    static_assert(kAhead >= kW - 1 && 6 % kAhead == 0, "a chunk is whole groups; what its first one completes lies in front of it");
    __shared__ float sums[256 * kSums];
    const int group = blockIdx.x % a.groups, part = blockIdx.x / a.groups;
    const int lane = group * a.row_lanes + (int)(threadIdx.x & (a.row_lanes - 1));
    const int per = 256 / a.row_lanes;                        // chunks of the workgroup at a time
    const int c0 = lane * kN, n_ch = kPlain ? kN : a.ch - c0;
    float dw[kN][kW], db[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < kW; ++j) dw[e][j] = 0.f;
    }
    float wt[kN][kW], bs[kN];
    const bool there = lane < a.lanes;
    if (there) conv_weights<kW, kN>(a.w, a.bias, c0, n_ch, wt, bs);
    for (int64_t row = (int64_t)part * per + threadIdx.x / a.row_lanes; there && row < a.rows; row += (int64_t)a.n_parts * per) {
        const int chunk = (int)(row % a.chunks);
        const int64_t b = row / a.chunks;
        const int n = conv_len(a, b), t0 = chunk * a.chunk, t1 = a.T_tokens - t0 < a.chunk ? a.T_tokens : t0 + a.chunk;
        float open[kW - 1][kN];                               // open[d - 1]: du of token t - d
        Vals<T, kN> hist[kW - 1];
        const uint8_t *starts = kStarts ? a.starts + b * a.T_tokens : nullptr;
        int age = conv_history<T, kW, kN>(a, starts, b, t0, c0, n_ch, hist);
#pragma unroll
        for (int d = 0; d < kW - 1; ++d)
#pragma unroll
            for (int e = 0; e < kN; ++e) open[d][e] = 0.f;
        const T *ub = a.u + b * a.batch_ld + c0, *dyb = a.dy + b * a.T_tokens * a.ch + c0;
        T *dub = a.du + b * a.du_batch_ld + c0;
        // dp of token s, and what it adds to; own: the token is one of the chunk's
        const auto token = [&](int s, const Vals<T, kN> &x, const Vals<T, kN> &g, bool own, float (&dp)[kN]) {
            if (kStarts) {
                age = age_after(starts, s, age);
#pragma unroll
                for (int j = 0; j < kW - 1; ++j)
                    if (kW - 1 - j > age) hist[j].zero();
            }
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                dp[e] = g.at(e);
                if (kPlain || a.silu) {
                    float p = bs[e];
#pragma unroll
                    for (int j = 0; j < kW - 1; ++j) p = fmaf(wt[e][j], hist[j].at(e), p);
                    p = fmaf(wt[e][kW - 1], x.at(e), p);
                    const float sg = sigmoid(p);
                    dp[e] *= sg * fmaf(p, 1.f - sg, 1.f);
                }
            }
            if (own) {
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    db[e] += dp[e];
#pragma unroll
                    for (int j = 0; j < kW - 1; ++j) dw[e][j] = fmaf(dp[e], hist[j].at(e), dw[e][j]);
                    dw[e][kW - 1] = fmaf(dp[e], x.at(e), dw[e][kW - 1]);
                }
            }
#pragma unroll
            for (int d = 1; d < kW; ++d)
                if (!kStarts || d <= age) {
#pragma unroll
                    for (int e = 0; e < kN; ++e) open[d - 1][e] = fmaf(wt[e][kW - 1 - d], dp[e], open[d - 1][e]);
                }
#pragma unroll
            for (int j = 0; j + 1 < kW - 1; ++j) hist[j] = hist[j + 1];
            hist[kW - 2] = x;
        };
        // there: the token is one of the row's.  Of padding nothing is formed, not even
        // weights times 0, which an infinite weight would make a NaN
        const auto shift = [&](bool there, const float (&dp)[kN]) {
#pragma unroll
            for (int d = kW - 2; d > 0; --d)
#pragma unroll
                for (int e = 0; e < kN; ++e) open[d][e] = open[d - 1][e];
#pragma unroll
            for (int e = 0; e < kN; ++e) open[0][e] = there ? wt[e][kW - 1] * dp[e] : 0.f;
        };
        const int inside = t1 < n ? t1 : n, end = t1 + kW - 1;
        int t = t0;
        while (t < end) {
            // whole groups of the chunk's own tokens; the first one, whose first W - 1 tokens
            // complete none of the chunk's, only where they complete none of the state's either
            const bool first = t == t0 && (t0 > 0 || a.dc_init == nullptr);
            if (t + kAhead <= inside && (first || t >= t0 + kW - 1)) {
                Vals<T, kN> x[kAhead], g[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    x[i].load(ub + (int64_t)(t + i) * a.ld, n_ch);
                    g[i].load(dyb + (int64_t)(t + i) * a.ch, n_ch);
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    float dp[kN];
                    token(t + i, x[i], g[i], true, dp);
                    if (!first || i >= kW - 1) {
                        Vals<T, kN> out;
                        out.put(open[kW - 2]);
                        out.store(dub + (int64_t)(t + i - (kW - 1)) * a.du_ld, n_ch);
                    }
                    shift(true, dp);
                }
                t += kAhead;
                continue;
            }
            float dp[kN];
#pragma unroll
            for (int e = 0; e < kN; ++e) dp[e] = 0.f;
            if (t < n) {
                Vals<T, kN> x, g;
                x.load(ub + (int64_t)t * a.ld, n_ch);
                g.load(dyb + (int64_t)t * a.ch, n_ch);
                token(t, x, g, t < t1, dp);
            }
            // token t - (W - 1) is whole (in front of the row: an input of the state)
            const int at = t - (kW - 1);
            const bool state = at < 0 && a.dc_init != nullptr;
            if (at >= t0 || state) {
                if (t >= n && at < n && a.dc_final != nullptr && n - 1 - at <= age) {   // it is in the last state too
                    Vals<T, kN> dc;
                    dc.load(a.dc_final + (b * (kW - 1) + at - n + kW - 1) * a.ch + c0, n_ch);
#pragma unroll
                    for (int e = 0; e < kN; ++e) open[kW - 2][e] += dc.at(e);
                }
                Vals<T, kN> out;
                out.put(open[kW - 2]);
                if (state) out.store(a.dc_init + (b * (kW - 1) + at + kW - 1) * a.ch + c0, n_ch);
                else out.store(dub + (int64_t)at * a.du_ld, n_ch);
            }
            shift(t < n, dp);
            ++t;
        }
    }
#pragma unroll
    for (int e = 0; e < kN; ++e) {
#pragma unroll
        for (int j = 0; j < kW; ++j) sums[(e * (kW + 1) + j) * 256 + threadIdx.x] = dw[e][j];
        sums[(e * (kW + 1) + kW) * 256 + threadIdx.x] = db[e];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < a.row_lanes * kSums; o += 256) {
        // neighbouring threads take neighbouring channels of one tap
        const int wide = a.row_lanes * kN, j = o / wide, cc = o % wide, l = cc / kN, e = cc % kN;
        const int c = group * wide + cc;
        if (c >= a.ch) continue;
        float s = 0.f;
        for (int r = 0; r < per; ++r) s += sums[(e * (kW + 1) + j) * 256 + r * a.row_lanes + l];
        a.parts[((int64_t)part * (kW + 1) + j) * a.ch + c] = s;
    }
}

}  // namespace bdssm_dev
