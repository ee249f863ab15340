// norm_kernels.hpp -- root-mean-square norm with the residual's addition:
//   h = x + res (rounded to res's type),  r = 1 / sqrt(mean(h^2) + eps),  y = w (h r),
// to the stream's type or to 8-bit codes with scales, and its gradients:
//   g = w dy,  n = h r,  dh = r (g - n mean(g n)) + dh_out,  dw = sum over rows of dy n.
//
// Memory is the bound.  A row lies in the registers of kThreads threads (a wave for
// up to 1,024 channels), so that it is read once; a workgroup goes over several rows
// with the weights kept, the next row's loads on their way while one is worked on.
// 65,536 rows of 1,024 channels, bf16 with an fp32 residual, to e4m3: 160 us (4.6 TB/s
// read and written; copies run at 4.9 to 5.2).  32,768 rows of 768, all bf16: 36 to 38
// us and 34 to 36 for the gradients (5.3 to 5.9 TB/s, partly out of the last-level cache).
//
// Sums of squares are taken in 64 bits: another order of the lanes moves them by some
// 2^-52 of themselves, so that all but always they round to the same 32-bit r however a
// row is laid out (in about one row of 2^27 r's 64-bit value lies that near a border),
// and outputs, codes beside a border among them, come out the same.
#pragma once

#include "kv_kernels.hpp"
#include "layer_common.hpp"

namespace bdssm_dev {

template <typename T, typename R>
struct NormArgs {
    const T *x;
    const R *res;        // or null: h is x
    const float *w;
    double eps, inv_ch;  // inv_ch: 1 / ch
    T *y;                // or codes:
    uint8_t *codes;
    float *scales;       // [rows, groups]
    int group;           // channels that share a scale
    R *h;                // or null
    float *rstd;         // or null
    int64_t rows;
    int ch;
    // backward: h is read
    const T *dy;
    const R *dh;
    T *dx;
    R *dres;
    float *parts;        // [workgroup][ch]
};

// Sum over the kThreads threads that share a row.  Waves join through `red`, two
// sets of it in turn, so that one barrier a sum is enough.
template <int kThreads, typename V>
__device__ __forceinline__ V row_sum(V v, V (*red)[16], int &turn) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s, 64);
    if constexpr (kThreads > 64) {
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[turn][0];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) v += red[turn][i];
    }
    return v;
}
template <int kThreads>
__device__ __forceinline__ float row_max(float v, double (*red)[16], int &turn) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) v = fmaxf(v, __shfl_xor(v, s, 64));
    if constexpr (kThreads > 64) {
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = v;
        __syncthreads();
        v = (float)red[turn][0];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) v = fmaxf(v, (float)red[turn][i]);
    }
    return v;
}

// 1 / sqrt(m), to a few last bits of 64: two steps on the estimate.
__device__ __forceinline__ double inverse_root(double m) {
    if (!(m > 0x1p-1000 && m < 0x1p1000)) return 1. / sqrt(m);
    double y = __builtin_amdgcn_rsq(m);
    y *= fma(-0.5 * m * y, y, 1.5);
    return y * fma(-0.5 * m * y, y, 1.5);
}

// A vector of weights as floats, 0 behind the channels.
template <int kV>
__device__ __forceinline__ Vals<float, kV> weights_at(const float *w, int at, int left) {
    Vals<float, kV> v;
    v.zero();
    if (left > 0) v.load(w + at, left);
    return v;
}

template <int kCode>
constexpr float kCodeMax = kCode == kE4m3 ? 448.f : 127.f;

// the largest finite magnitude
template <int kV>
__device__ __forceinline__ float largest_of(const float (&y)[kV]) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        const float m = fabsf(y[e]);
        top = fmaxf(top, m < __builtin_inff() ? m : 0.f);
    }
    return top;
}

// y / scale to codes.  The correctly rounded quotient in five operations, as in the
// cache's commit, where the scale leaves its remainders exact; infinities become the
// largest code, NaN a NaN or 0.
template <int kCode, int kV>
__device__ __forceinline__ Vals<uint8_t, kV> codes_of(const float (&y)[kV], float scale) {
    float q[kV];
    if (scale < 0x1p-90f || !(scale < 0x1p90f)) {
#pragma unroll
        for (int e = 0; e < kV; ++e) q[e] = y[e] / scale;
    } else {
        const float r = 1.f / scale;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            float p = y[e] * r;
            p = fmaf(fmaf(-p, scale, y[e]), r, p);
            p = fmaf(fmaf(-p, scale, y[e]), r, p);
            q[e] = fabsf(y[e]) < __builtin_inff() ? p : y[e];
        }
    }
#pragma unroll
    for (int e = 0; e < kV; ++e) {
        if (kCode == kI8 && q[e] != q[e]) q[e] = 0.f;
        if (q[e] == q[e]) q[e] = fminf(fmaxf(q[e], -kCodeMax<kCode>), kCodeMax<kCode>);
    }
    Vals<uint8_t, kV> out;
#pragma unroll
    for (int e = 0; e < kV; e += 4) {
        const uint32_t c = to_codes<kCode>(q[e], q[e + 1], q[e + 2], q[e + 3]);
        __builtin_memcpy(out.v + e, &c, 4);
    }
    return out;
}

constexpr int kOutStream = -1;   // kCode of norms that write the stream's type

// kVecs vectors of kV channels a thread, vector i of thread t the channels from
// kV (i kThreads + t) on.  One row at a time for kThreads of more than a wave (of as
// many threads the workgroup), four (one a wave) otherwise.
template <typename T, typename R, int kCode, int kThreads, int kV, int kVecs>
__global__ __launch_bounds__(kThreads > 256 ? kThreads : 256) void norm_kernel(NormArgs<T, R> a) {
    __shared__ double red[2][16];
    int turn = 0;
    const int tid = kThreads == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int rows_at_once = kThreads == 64 ? 4 : 1;
    int64_t row = (int64_t)blockIdx.x * rows_at_once + (kThreads == 64 ? threadIdx.x >> 6 : 0);
    const int64_t step = (int64_t)gridDim.x * rows_at_once;
    Vals<float, kV> w[kVecs];
    Vals<T, kV> x[kVecs];
    Vals<R, kV> res[kVecs];
    int at[kVecs], left[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        at[i] = kV * (i * kThreads + tid);
        left[i] = a.ch - at[i];
        w[i] = weights_at<kV>(a.w, at[i], left[i]);
    }
    const auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (left[i] > 0) {
                x[i].load(a.x + r * a.ch + at[i], left[i]);
                if (a.res != nullptr) res[i].load(a.res + r * a.ch + at[i], left[i]);
            }
        }
    };
    if (row < a.rows) fetch(row);
    for (; row < a.rows; row += step) {
        float h[kVecs][kV];
        double sum = 0.;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
#pragma unroll
            for (int e = 0; e < kV; ++e) h[i][e] = left[i] > 0 ? x[i].at(e) : 0.f;
            if (a.res != nullptr && left[i] > 0) {
                Vals<R, kV> hr;
                float s[kV];
#pragma unroll
                for (int e = 0; e < kV; ++e) s[e] = h[i][e] + res[i].at(e);
                hr.put(s);
                hr.store(a.h + row * a.ch + at[i], left[i]);
#pragma unroll
                for (int e = 0; e < kV; ++e) h[i][e] = hr.at(e);
            }
#pragma unroll
            for (int e = 0; e < kV; ++e) sum = fma((double)h[i][e], (double)h[i][e], sum);
        }
        if (row + step < a.rows) fetch(row + step);
        sum = row_sum<kThreads>(sum, red, turn);
        const float r = (float)inverse_root(fma(sum, a.inv_ch, a.eps));
        if (a.rstd != nullptr && tid == 0) a.rstd[row] = r;
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
#pragma unroll
            for (int e = 0; e < kV; ++e) h[i][e] = (h[i][e] * r) * w[i].v[e];
            if constexpr (kCode == kOutStream) {
                Vals<T, kV> out;
                out.put(h[i]);
                if (left[i] > 0) out.store(a.y + row * a.ch + at[i], left[i]);
            }
        }
        if constexpr (kCode != kOutStream) {
            float big[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                big[i] = largest_of(h[i]);
                top = fmaxf(top, big[i]);
            }
            const bool whole = a.group == a.ch;
            if (whole) top = row_max<kThreads>(top, red, turn);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                float m = top;
                if (!whole) {   // 128 channels: neighbouring lanes' vectors
                    m = big[i];
#pragma unroll
                    for (int s = 1; s < 128 / kV; s <<= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
                }
                const float scale = fmaxf(m / kCodeMax<kCode>, 0x1p-126f);
                if (whole ? tid == 0 && i == 0 : (tid & (128 / kV - 1)) == 0 && left[i] > 0)
                    a.scales[whole ? row : row * (a.ch / 128) + at[i] / 128] = scale;
                const Vals<uint8_t, kV> out = codes_of<kCode, kV>(h[i], scale);
                if (left[i] > 0) out.store(a.codes + row * a.ch + at[i], left[i]);
            }
        }
    }
}

template <typename T, typename R, int kThreads, int kV, int kVecs>
__global__ __launch_bounds__(kThreads > 256 ? kThreads : 256) void norm_bwd_kernel(NormArgs<T, R> a) {
    __shared__ float red[2][16];
    __shared__ float joined[kThreads == 64 ? 4 : 1][kThreads == 64 ? 64 * kVecs * kV : 1];
    int turn = 0;
    const int tid = kThreads == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int rows_at_once = kThreads == 64 ? 4 : 1;
    int64_t row = (int64_t)blockIdx.x * rows_at_once + (kThreads == 64 ? threadIdx.x >> 6 : 0);
    const int64_t step = (int64_t)gridDim.x * rows_at_once;
    Vals<float, kV> w[kVecs];
    float dw[kVecs][kV];
    Vals<R, kV> h[kVecs], up[kVecs];
    Vals<T, kV> dy[kVecs];
    float r_next = 0.f;
    int at[kVecs], left[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        at[i] = kV * (i * kThreads + tid);
        left[i] = a.ch - at[i];
        w[i] = weights_at<kV>(a.w, at[i], left[i]);
        h[i].zero();
        up[i].zero();
        dy[i].zero();
#pragma unroll
        for (int e = 0; e < kV; ++e) dw[i][e] = 0.f;
    }
    const auto fetch = [&](int64_t r) {
        r_next = a.rstd[r];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (left[i] > 0) {
                h[i].load(a.h + r * a.ch + at[i], left[i]);
                dy[i].load(a.dy + r * a.ch + at[i], left[i]);
                if (a.dh != nullptr) up[i].load(a.dh + r * a.ch + at[i], left[i]);
            }
        }
    };
    if (row < a.rows) fetch(row);
    for (; row < a.rows; row += step) {
        float n[kVecs][kV], g[kVecs][kV], sum = 0.f;
        Vals<R, kV> more[kVecs];
        const float r = r_next;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            more[i] = up[i];
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                const float d = dy[i].at(e);
                n[i][e] = h[i].at(e) * r;
                g[i][e] = d * w[i].v[e];
                dw[i][e] = fmaf(d, n[i][e], dw[i][e]);
                sum = fmaf(g[i][e], n[i][e], sum);
            }
        }
        if (row + step < a.rows) fetch(row + step);
        const float mean = row_sum<kThreads>(sum, red, turn) / (float)a.ch;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (left[i] <= 0) continue;
#pragma unroll
            for (int e = 0; e < kV; ++e) {
                g[i][e] = r * fmaf(-n[i][e], mean, g[i][e]);
                if (a.dh != nullptr) g[i][e] += more[i].at(e);
            }
            Vals<T, kV> dx;
            dx.put(g[i]);
            dx.store(a.dx + row * a.ch + at[i], left[i]);
            if (a.dres != nullptr) {
                Vals<R, kV> out;
                out.put(g[i]);
                out.store(a.dres + row * a.ch + at[i], left[i]);
            }
        }
    }
    // the workgroup's part of dw: its waves' in order
    float *part = a.parts + (int64_t)blockIdx.x * a.ch;
    if constexpr (kThreads == 64) {
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int e = 0; e < kV; ++e) joined[wave][(i * kV + e) * 64 + tid] = dw[i][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.ch; c += 256) {
            const int o = (c / (64 * kV) * kV + c % kV) * 64 + c % (64 * kV) / kV;
            part[c] = joined[0][o] + joined[1][o] + joined[2][o] + joined[3][o];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (left[i] <= 0) continue;
            Vals<float, kV> out;
#pragma unroll
            for (int e = 0; e < kV; ++e) out.v[e] = dw[i][e];
            out.store(part + at[i], left[i]);
        }
    }
}

// Rows of more than kNormHeld channels: nothing of a row is kept, each pass over it
// reads it again (from L2; what a thread reads again it wrote itself).
constexpr int kNormHeld = 8192, kNormMost = 32768;

template <typename T, typename R, int kCode>
__global__ __launch_bounds__(1024) void norm_wide_kernel(NormArgs<T, R> a) {
    __shared__ double red[2][16];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t r0 = row * a.ch;
        double sum = 0.;
#pragma unroll 1
        for (int at = 8 * threadIdx.x; at < a.ch; at += 8 * 1024) {
            const int left = a.ch - at;
            Vals<T, 8> x;
            x.load(a.x + r0 + at, left);
            float h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = x.at(e);
            if (a.res != nullptr) {
                Vals<R, 8> hr;
                hr.load(a.res + r0 + at, left);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] += hr.at(e);
                hr.put(h);
                hr.store(a.h + r0 + at, left);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = hr.at(e);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fma((double)h[e], (double)h[e], sum);
        }
        sum = row_sum<1024>(sum, red, turn);
        const float r = (float)inverse_root(fma(sum, a.inv_ch, a.eps));
        if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = r;
        const auto output = [&](int at, int left, float (&y)[8]) {
            if (a.res != nullptr) {
                Vals<R, 8> h;
                h.load(a.h + r0 + at, left);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = h.at(e);
            } else {
                Vals<T, 8> h;
                h.load(a.x + r0 + at, left);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = h.at(e);
            }
            const Vals<float, 8> w = weights_at<8>(a.w, at, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = (y[e] * r) * w.v[e];
        };
        float top = 0.f;
        if (kCode != kOutStream && a.group == a.ch) {
#pragma unroll 1
            for (int at = 8 * threadIdx.x; at < a.ch; at += 8 * 1024) {
                float y[8];
                output(at, a.ch - at, y);
                top = fmaxf(top, largest_of(y));
            }
            top = row_max<1024>(top, red, turn);
        }
#pragma unroll 1
        for (int at = 8 * threadIdx.x; at < a.ch; at += 8 * 1024) {
            const int left = a.ch - at;
            float y[8];
            output(at, left, y);
            if constexpr (kCode == kOutStream) {
                Vals<T, 8> out;
                out.put(y);
                out.store(a.y + r0 + at, left);
            } else {
                float m = top;
                const bool whole = a.group == a.ch;
                if (!whole) {   // 128 channels: 16 lanes, all of them here (groups divide the row)
                    m = largest_of(y);
#pragma unroll
                    for (int s = 1; s < 16; s <<= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
                }
                const float scale = fmaxf(m / kCodeMax<kCode>, 0x1p-126f);
                if (whole ? at == 0 : (threadIdx.x & 15) == 0) a.scales[whole ? row : row * (a.ch / 128) + at / 128] = scale;
                codes_of<kCode, 8>(y, scale).store(a.codes + r0 + at, left);
            }
        }
    }
}

template <typename T, typename R>
__global__ __launch_bounds__(1024) void norm_wide_bwd_kernel(NormArgs<T, R> a) {
    __shared__ float red[2][16];
    __shared__ __attribute__((aligned(16))) float dw[kNormMost];   // each thread's own channels
    int turn = 0;
    for (int at = 8 * threadIdx.x; at < a.ch; at += 8 * 1024) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[at + e] = 0.f;
    }
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t r0 = row * a.ch;
        const float r = a.rstd[row];
        const auto terms = [&](int at, int left, float (&d)[8], float (&n)[8], float (&g)[8]) {
            Vals<R, 8> h;
            Vals<T, 8> dy;
            h.load(a.h + r0 + at, left);
            dy.load(a.dy + r0 + at, left);
            const Vals<float, 8> w = weights_at<8>(a.w, at, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                d[e] = dy.at(e);
                n[e] = h.at(e) * r;
                g[e] = d[e] * w.v[e];
            }
        };
        float sum = 0.f;
#pragma unroll 1
        for (int at = 8 * threadIdx.x; at < a.ch; at += 8 * 1024) {
            float d[8], n[8], g[8];
            terms(at, a.ch - at, d, n, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[at + e] = fmaf(d[e], n[e], dw[at + e]);
                sum = fmaf(g[e], n[e], sum);
            }
        }
        const float mean = row_sum<1024>(sum, red, turn) / (float)a.ch;
#pragma unroll 1
        for (int at = 8 * threadIdx.x; at < a.ch; at += 8 * 1024) {
            const int left = a.ch - at;
            float d[8], n[8], g[8];
            terms(at, left, d, n, g);
            Vals<R, 8> up;
            up.zero();
            if (a.dh != nullptr) up.load(a.dh + r0 + at, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = r * fmaf(-n[e], mean, g[e]) + up.at(e);
            Vals<T, 8> dx;
            dx.put(g);
            dx.store(a.dx + r0 + at, left);
            if (a.dres != nullptr) {
                up.put(g);
                up.store(a.dres + r0 + at, left);
            }
        }
    }
    float *part = a.parts + (int64_t)blockIdx.x * a.ch;
    for (int at = 8 * threadIdx.x; at < a.ch; at += 8 * 1024) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (at + e < a.ch) part[at + e] = dw[at + e];
    }
}

}  // namespace bdssm_dev
