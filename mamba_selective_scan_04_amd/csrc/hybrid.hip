// hybrid.hip -- C ABI and argument checks of the hybrid layer's operators: the
// gated delta rule and attention over the paged 8-bit cache.  As in bdssm.hip,
// every argument is checked on the host before the first HIP call.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <initializer_list>

#include "bdssm.h"
#include "host_checks.hpp"
#include "hybrid_launch.hpp"

using namespace bdssm_host;

namespace {

constexpr int64_t kMost = (int64_t)1 << 40;   // elements of one tensor

bool product_fits(std::initializer_list<int64_t> f) {
    int64_t n = 1;
    for (int64_t x : f) {
        if (x == 0) return true;
        if (x > kMost / n) return false;
        n *= x;
    }
    return true;
}

bool all_aligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned16(p)) return false;
    return true;
}

// No output may overlap an input or another output.
bool distinct(std::initializer_list<Range> ins, std::initializer_list<Range> outs) {
    for (const Range &o : outs) {
        for (const Range &i : ins)
            if (overlaps(o, i)) return false;
        for (const Range &p : outs)
            if (&p != &o && overlaps(o, p)) return false;
    }
    return true;
}

// ------------------------------------------------------------- delta rule

int check_delta(const bdssm_delta_shape *s, int64_t T) {
    if (s == nullptr) return BDSSM_ERR_NULL;
    if (s->dtype != BDSSM_F32 && s->dtype != BDSSM_BF16) return BDSSM_ERR_DTYPE;
    if (T < 0 || s->batch < 0 || s->batch > 65535 || s->heads_k < 1 || s->heads_v < 1 || s->heads_v > 65535)
        return BDSSM_ERR_SHAPE;
    if (s->heads_v % s->heads_k != 0) return BDSSM_ERR_SHAPE;
    if ((s->d_k != 64 && s->d_k != 128) || (s->d_v != 64 && s->d_v != 128)) return BDSSM_ERR_SHAPE;
    // 2^31 - 1 chunks at most in a launch, and every tensor's elements countable
    if (T > kMost || (T + 63) / 64 >= ((int64_t)1 << 31)) return BDSSM_ERR_SHAPE;
    if (!product_fits({s->batch, (T + 63) / 64, s->heads_v, s->d_k, s->d_v})) return BDSSM_ERR_SHAPE;
    return BDSSM_OK;
}

struct DeltaSizes {
    int64_t chunks;
    size_t qk, vo, gate, state, hchunks, W;
};

DeltaSizes delta_sizes(const bdssm_delta_shape *s, int64_t T) {
    const size_t e = s->dtype == BDSSM_BF16 ? 2 : 4;
    DeltaSizes z;
    z.chunks = (T + kChunk - 1) / kChunk;
    z.qk = (size_t)s->batch * T * s->heads_k * s->d_k * e;
    z.vo = (size_t)s->batch * T * s->heads_v * s->d_v * e;
    z.gate = (size_t)s->batch * T * s->heads_v * 4;
    z.state = (size_t)s->batch * s->heads_v * s->d_k * s->d_v * 4;
    z.hchunks = z.state * (size_t)z.chunks;
    z.W = (size_t)s->batch * s->heads_v * z.chunks * kWFloats * 4;
    return z;
}

DeltaCall delta_call(const bdssm_delta_shape *s, int64_t T, const void *q, const void *k, const void *v,
                     const float *g, const float *beta, float scale, const int32_t *lens) {
    DeltaCall c{};
    c.q = q;
    c.k = k;
    c.v = v;
    c.g = g;
    c.beta = beta;
    c.batch = s->batch;
    c.dk = (int)s->d_k;
    c.d.T = T;
    c.d.hk = (int)s->heads_k;
    c.d.hv = (int)s->heads_v;
    c.d.group = (int)(s->heads_v / s->heads_k);
    c.d.dv = (int)s->d_v;
    c.d.chunks = (int)((T + kChunk - 1) / kChunk);
    c.d.lens = lens;
    c.d.scale = scale;
    return c;
}

}  // namespace

extern "C" {

size_t bdssm_delta_workspace_bytes(const bdssm_delta_shape *s, int64_t T, int bwd) {
    if (check_delta(s, T) != BDSSM_OK) return (size_t)-1;
    const DeltaSizes z = delta_sizes(s, T);
    return bwd ? 2 * z.W + z.hchunks : z.W;   // W, W^T, the states' adjoints
}

int bdssm_delta_scan(const bdssm_delta_shape *s, int64_t T, const void *q, const void *k, const void *v,
                     const float *g, const float *beta, float scale, const int32_t *lens, const float *h_init,
                     void *o, float *h_final, float *h_chunks, void *ws, size_t ws_bytes, hipStream_t st) {
    const int rc = check_delta(s, T);
    if (rc) return rc;
    if (s->batch == 0) return BDSSM_OK;
    if (T > 0 && (!k || !v || !g || !beta || (o && !q))) return BDSSM_ERR_NULL;
    if (!all_aligned({q, k, v, g, beta, lens, h_init, o, h_final, h_chunks, ws})) return BDSSM_ERR_ALIGN;
    const DeltaSizes z = delta_sizes(s, T);
    const Range lr{lens, (size_t)s->batch * 4};
    if (!distinct({{o ? q : nullptr, z.qk}, {k, z.qk}, {v, z.vo}, {g, z.gate}, {beta, z.gate}, lr,
                   {h_init == h_final ? nullptr : h_init, z.state}},
                  {{o, z.vo}, {h_final, z.state}, {h_chunks, z.hchunks}, {ws, z.W}}))
        return BDSSM_ERR_ALIAS;
    if (h_init && h_init == h_final && !distinct({{h_init, z.state}}, {{o, z.vo}, {h_chunks, z.hchunks}, {ws, z.W}}))
        return BDSSM_ERR_ALIAS;
    if (z.W > 0 && (ws == nullptr || ws_bytes < z.W)) return BDSSM_ERR_WORKSPACE;
    if (!o && !h_final && !h_chunks) return BDSSM_OK;
    DeltaCall c = delta_call(s, T, q, k, v, g, beta, scale, lens);
    c.h_init = h_init;
    c.o = o;
    c.h_final = h_final;
    c.h_chunks = h_chunks;
    c.W = (float *)ws;
    (void)hipGetLastError();
    if (s->dtype == BDSSM_BF16) launch_delta_scan<uint16_t>(c, st);
    else launch_delta_scan<float>(c, st);
    return launch_status();
}

int bdssm_delta_scan_bwd(const bdssm_delta_shape *s, int64_t T, const void *q, const void *k, const void *v,
                         const float *g, const float *beta, float scale, const int32_t *lens, const float *h_chunks,
                         const void *dout, const float *dh_final, void *dq, void *dk, void *dv, float *dg, float *dbeta,
                         float *dh_init, void *ws, size_t ws_bytes, hipStream_t st) {
    const int rc = check_delta(s, T);
    if (rc) return rc;
    if (s->batch == 0) return BDSSM_OK;
    if (T > 0 && (!q || !k || !v || !g || !beta || !h_chunks || !dout || !dq || !dk || !dv || !dg || !dbeta))
        return BDSSM_ERR_NULL;
    if (!all_aligned({q, k, v, g, beta, lens, h_chunks, dout, dh_final, dq, dk, dv, dg, dbeta, dh_init, ws}))
        return BDSSM_ERR_ALIGN;
    const DeltaSizes z = delta_sizes(s, T);
    const size_t need = 2 * z.W + z.hchunks;
    if (!distinct({{q, z.qk}, {k, z.qk}, {v, z.vo}, {g, z.gate}, {beta, z.gate}, {lens, (size_t)s->batch * 4},
                   {h_chunks, z.hchunks}, {dout, z.vo}, {dh_final, z.state}},
                  {{dq, z.qk}, {dk, z.qk}, {dv, z.vo}, {dg, z.gate}, {dbeta, z.gate}, {dh_init, z.state}, {ws, need}}))
        return BDSSM_ERR_ALIAS;
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return BDSSM_ERR_WORKSPACE;
    DeltaCall c = delta_call(s, T, q, k, v, g, beta, scale, lens);
    c.h_chunks = const_cast<float *>(h_chunks);
    c.dout = dout;
    c.dh_final = dh_final;
    c.W = (float *)ws;
    c.Wt = c.W + z.W / 4;
    c.dS = c.Wt + z.W / 4;
    c.dq = dq;
    c.dk_out = dk;
    c.dv_out = dv;
    c.dg = dg;
    c.dbeta = dbeta;
    c.dh_init = dh_init;
    (void)hipGetLastError();
    if (s->dtype == BDSSM_BF16) launch_delta_bwd<uint16_t>(c, st);
    else launch_delta_bwd<float>(c, st);
    return launch_status();
}

int bdssm_delta_step(const bdssm_delta_shape *s, int64_t T, const float *h_cache, const void *q, const void *k,
                     const void *v, const float *g, const float *beta, float scale, const int32_t *lens, void *o,
                     float *h_out, hipStream_t st) {
    const int rc = check_delta(s, T);
    if (rc) return rc;
    if (s->batch == 0) return BDSSM_OK;
    if (T > 0 && (!k || !v || !g || !beta || (o && !q))) return BDSSM_ERR_NULL;
    if (!all_aligned({q, k, v, g, beta, lens, h_cache, o, h_out})) return BDSSM_ERR_ALIGN;
    const DeltaSizes z = delta_sizes(s, T);
    const Range lr{lens, (size_t)s->batch * 4};
    if (!distinct({{o ? q : nullptr, z.qk}, {k, z.qk}, {v, z.vo}, {g, z.gate}, {beta, z.gate}, lr,
                   {h_cache == h_out ? nullptr : h_cache, z.state}},
                  {{o, z.vo}, {h_out, z.state}}))
        return BDSSM_ERR_ALIAS;
    if (!o && !h_out) return BDSSM_OK;
    DeltaCall c = delta_call(s, T, q, k, v, g, beta, scale, lens);
    c.h_init = h_cache;
    c.o = o;
    c.h_final = h_out;
    (void)hipGetLastError();
    if (s->dtype == BDSSM_BF16) launch_delta_step<uint16_t>(c, st);
    else launch_delta_step<float>(c, st);
    return launch_status();
}

}  // extern "C"
