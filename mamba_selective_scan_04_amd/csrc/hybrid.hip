// hybrid.hip -- C ABI and argument checks of the hybrid layer's operators: the
// gated delta rule and attention over the paged 8-bit cache.  As in bdssm.hip,
// every argument is checked on the host before the first HIP call.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <stdlib.h>

#include <initializer_list>

#include "bdssm.h"
#include "host_checks.hpp"
#include "hybrid_launch.hpp"

using namespace bdssm_host;

namespace {

constexpr int64_t kCus = 256;
constexpr int64_t kMost = (int64_t)1 << 40;   // elements of one tensor
constexpr int64_t kMostGroups = 0xffffff;     // workgroups along a grid's axis: its 256 threads each are counted in 32 bits

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
    // up to 4 workgroups a chain, and of 512 threads a chunk, in a grid's axis; every
    // tensor's elements countable
    if (s->batch * s->heads_v > kMostGroups / 4 || T > kMost || (T + 63) / 64 > kMostGroups / 2) return BDSSM_ERR_SHAPE;
    if (!product_fits({s->batch, (T + 63) / 64, s->heads_v, s->d_k, s->d_v})) return BDSSM_ERR_SHAPE;
    return BDSSM_OK;
}

// Segments of a row's chunks (1: none).  A chain's step is a chunk's, whatever
// the batch; cutting the row costs the aggregate pass over d_v + d_k columns
// besides the chain's own d_v, and the join's step for each segment, so it pays
// from three segments of two chunks on.  No more than the aggregate pass runs at
// once (three workgroups of 64 columns a CU, two for fp32 streams): another round
// of them costs more than shorter segments give.  Nor more than makes the two
// chains' steps and the join's (a sixth of theirs) least: n^2 = 4 chunks is near
// that.  Backward the same of the adjoint's passes, whose larger stages leave room
// for two workgroups a CU (fp32: one).  Microseconds of the forward / the backward
// (the rule's counts in the last column), bf16, 128 by 128 but the last:
//   1 row of 65,536 tokens, 12 heads  1: 4071 / 7017  10: 1026 / 3125  16: 926 / 3075  24: 1060 / 3202   16 / 10
//   4 rows of 4,096 tokens, 16 heads  1: 312 / 956    3: 306 / 975     6: 338 / 1039   16: 409 / 1105    3 / 1
//   8 rows of 4,096 tokens, 12 heads  1: 348 / 1272   2: 420 / 1424    4: 465 / 1498                     1 / 1
//   1 row of 2,048 tokens, 2 heads    1: 119 / 188    4: 71 / 126      8: 56 / 100     24: 77 / 115      11 / 11
//   1 row of 1,024 tokens, 1 of 64    1: 50 / 85      4: 35 / 68       8: 30 / 58      12: 33 / 61       8 / 8
// BDSSM_DELTA_SEGMENTS forces a count (tests).
int delta_segments(const bdssm_delta_shape *s, int64_t chunks, bool bwd) {
    const int64_t blocks = s->batch * s->heads_v * ((s->d_v + s->d_k) / 64);
    int64_t n = blocks > 0 ? kCus * ((s->dtype == BDSSM_BF16 ? 3 : 2) - (bwd ? 1 : 0)) / blocks : 1;
    if (n > chunks / 2) n = chunks / 2;
    while (n * n > 4 * chunks) --n;
    if (n < 3) n = 1;
    const char *e = getenv("BDSSM_DELTA_SEGMENTS");
    if (e != nullptr && *e != 0) n = atoi(e);
    if (n > chunks) n = chunks;
    if (n * s->batch * s->heads_v > kMostGroups / 4) n = kMostGroups / 4 / (s->batch * s->heads_v);
    return n < 1 ? 1 : (int)n;
}

struct DeltaSizes {
    size_t qk, vo, gate, state, hchunks, units, map;   // map: a segment's, of every head
    bool bf16;
    int segs, segs_bwd;
    // the workspace: the chunks' matrices and the segments' maps; for the backward
    // the matrices, the summed log decays, the states' adjoints and the maps
    size_t mats() const { return units * (bf16 ? sizeof(Mats<2>) : sizeof(Mats<3>)); }
    size_t fwd() const { return mats() + (segs > 1 ? (map + state) * segs : 0); }
    size_t mats3() const { return units * sizeof(Mats<3>); }
    size_t sums() const { return units * kChunk * 8; }
    size_t bwd() const { return mats3() + sums() + hchunks + (segs_bwd > 1 ? (map + state) * segs_bwd : 0); }
};

DeltaSizes delta_sizes(const bdssm_delta_shape *s, int64_t T) {
    const size_t e = s->dtype == BDSSM_BF16 ? 2 : 4;
    const size_t chunks = (size_t)(T + kChunk - 1) / kChunk;
    DeltaSizes z;
    z.qk = (size_t)s->batch * T * s->heads_k * s->d_k * e;
    z.vo = (size_t)s->batch * T * s->heads_v * s->d_v * e;
    z.gate = (size_t)s->batch * T * s->heads_v * 4;
    z.state = (size_t)s->batch * s->heads_v * s->d_k * s->d_v * 4;
    z.hchunks = z.state * chunks;
    z.units = (size_t)s->batch * s->heads_v * chunks;
    z.bf16 = s->dtype == BDSSM_BF16;
    z.segs = delta_segments(s, (int64_t)chunks, false);
    z.segs_bwd = delta_segments(s, (int64_t)chunks, true);
    z.map = (size_t)s->batch * s->heads_v * s->d_k * (s->d_v + s->d_k) * 4;
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

// --------------------------------------------------- paged 8-bit cache

int check_kv(const bdssm_kv_shape *s, int64_t L) {
    if (s == nullptr) return BDSSM_ERR_NULL;
    if (s->dtype != BDSSM_F32 && s->dtype != BDSSM_BF16) return BDSSM_ERR_DTYPE;
    if (s->code != BDSSM_E4M3 && s->code != BDSSM_I8) return BDSSM_ERR_DTYPE;
    if (L < 0 || s->batch < 0 || s->batch > 32767 || s->heads_kv < 1 || s->heads_kv > 32767) return BDSSM_ERR_SHAPE;
    if (s->heads_q < 1 || s->heads_q > 32767 || s->heads_q % s->heads_kv != 0) return BDSSM_ERR_SHAPE;
    if (s->head_dim != 64 && s->head_dim != 128) return BDSSM_ERR_SHAPE;
    if (s->page_len != 16 && s->page_len != 32 && s->page_len != 64 && s->page_len != 128) return BDSSM_ERR_SHAPE;
    if (s->n_pages < 0 || s->n_pages > 0x7fffffff || s->max_pages < 0 || s->max_pages > 0x7fffffff / s->page_len)
        return BDSSM_ERR_SHAPE;   // token positions of a row fit 31 bits
    if (!product_fits({s->n_pages, s->heads_kv, s->page_len, s->head_dim}) || !product_fits({s->batch, s->max_pages}) ||
        !product_fits({s->batch, L, s->heads_q, s->head_dim}) || L > 0x7fffffff)
        return BDSSM_ERR_SHAPE;
    return BDSSM_OK;
}

int64_t kv_group(const bdssm_kv_shape *s) { return s->heads_q / s->heads_kv; }

struct KvSizes {
    size_t q, kv, cache, scale, table, row;
};

KvSizes kv_sizes(const bdssm_kv_shape *s, int64_t L, int64_t Lq) {
    const size_t e = s->dtype == BDSSM_BF16 ? 2 : 4;
    KvSizes z;
    z.q = (size_t)s->batch * Lq * s->heads_q * s->head_dim * e;
    z.kv = (size_t)s->batch * L * s->heads_kv * s->head_dim * e;
    z.cache = (size_t)s->n_pages * s->heads_kv * s->page_len * s->head_dim;
    z.scale = (size_t)s->n_pages * s->heads_kv * 4;
    z.table = (size_t)s->batch * s->max_pages * 4;
    z.row = (size_t)s->batch * 4;
    return z;
}

// A wave's query tiles: two where there are more than 16 rows (64 accumulators at
// 128 channels; four tiles' 128 made the compiler spill, and ran at half the
// speed), but one for fp32 streams of 128 channels, whose queries take three times
// the registers (4 rows of 65,536 tokens and 64 queries: 138 us; 190 with two
// tiles, which spilled, where one took 146).  Key ranges: 512 workgroups, two a CU,
// as many as the 66 KB of LDS of 128 channels leave room for (64 channels': three
// or four a CU, and no faster for it), but at least one step of 32 keys for each
// wave of a range; beyond that up to three times as many, of at least 2,048 keys,
// so that rows of different lengths (which only the GPU knows) even out.  The table's
// width stands for the context, so a table wider than the rows' contexts makes
// shorter ranges than these.  Microseconds by the number of ranges, the rule's in
// brackets:
//   64 rows of up to 8,192, 64 channels   2: 50   3: 45   [4: 42]   6: 44   8: 40   16: 45
//   16 rows of 8,192, 64 channels         2: 45   [4: 35]   6: 34   8: 36   16: 41   32: 55
//   16 rows of 8,192, 128 channels        2: 66   3: 60   [4: 50]   6: 60   8: 58   16: 73
//   1 row of 65,536, 128 channels         32: 38   48: 35   [64: 31]   96: 41   128: 41   256: 58
//   4 rows of up to 262,144, 128 channels 16: 257   32: 207   [48: 217]   96: 234   128: 249
//   1 row of 65,536 in a table of 4, 8 and 32 times its width: 41, 47 and 47
KvPlan kv_plan(const bdssm_kv_shape *s, int64_t Lq) {
    const int64_t rows = Lq * kv_group(s);
    KvPlan p;
    p.tiles = rows > 16 && !(s->dtype == BDSSM_F32 && s->head_dim == 128) ? 2 : 1;
    const int64_t qtiles = (rows + p.tiles * 16 - 1) / (p.tiles * 16);
    const int64_t units = s->batch * s->heads_kv * qtiles;
    const int64_t fill = 512;   // resident at once
    const int64_t steps = (s->max_pages * s->page_len + 31) / 32;
    int64_t n = units > 0 ? (fill + units - 1) / units : 1;
    int64_t even = units > 0 ? (3 * fill + units - 1) / units : 1;
    if (even > steps / 64) even = steps / 64;
    if (n < even) n = even;
    if (n > (steps + 3) / 4) n = (steps + 3) / 4;
    const char *e = getenv("BDSSM_KV_SPLITS");   // forces a count (tests)
    if (e != nullptr && *e != 0) n = atoi(e);
    p.qtiles = (int)qtiles;
    p.splits = (int)(n < 1 ? 1 : n);
    return p;
}

size_t kv_workspace(const bdssm_kv_shape *s, const KvPlan &p, size_t *part_o) {
    if (p.splits <= 1) return 0;
    const size_t rows = (size_t)s->batch * s->heads_kv * p.qtiles * p.splits * p.tiles * 16;
    *part_o = rows * s->head_dim * 4;
    return *part_o + rows * 8;
}

KvCall kv_call(const bdssm_kv_shape *s, int64_t L, const void *k, const void *v, const int32_t *table, const int32_t *ctx,
               const int32_t *lens) {
    KvCall c{};
    c.k = k;
    c.v = v;
    c.batch = s->batch;
    c.L = L;
    c.head_dim = (int)s->head_dim;
    c.code = s->code;
    c.d.heads_q = (int)s->heads_q;
    c.d.heads_kv = (int)s->heads_kv;
    c.d.group = (int)kv_group(s);
    c.d.page_len = (int)s->page_len;
    c.d.n_pages = (int)s->n_pages;
    c.d.max_pages = (int)s->max_pages;
    c.d.table = table;
    c.d.ctx = ctx;
    c.d.lens = lens;
    return c;
}

}  // namespace

extern "C" {

size_t bdssm_delta_workspace_bytes(const bdssm_delta_shape *s, int64_t T, int bwd) {
    if (check_delta(s, T) != BDSSM_OK) return (size_t)-1;
    const DeltaSizes z = delta_sizes(s, T);
    return bwd ? z.bwd() : z.fwd();
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
                  {{o, z.vo}, {h_final, z.state}, {h_chunks, z.hchunks}, {ws, z.fwd()}}))
        return BDSSM_ERR_ALIAS;
    if (h_init && h_init == h_final && !distinct({{h_init, z.state}}, {{o, z.vo}, {h_chunks, z.hchunks}, {ws, z.fwd()}}))
        return BDSSM_ERR_ALIAS;
    if (z.fwd() > 0 && (ws == nullptr || ws_bytes < z.fwd())) return BDSSM_ERR_WORKSPACE;
    if (!o && !h_final && !h_chunks) return BDSSM_OK;
    DeltaCall c = delta_call(s, T, q, k, v, g, beta, scale, lens);
    c.h_init = h_init;
    c.o = o;
    c.h_final = h_final;
    c.h_chunks = h_chunks;
    c.mats = ws;
    c.segs = z.segs;
    c.agg = (float *)((char *)ws + z.mats());
    c.h_seg = (float *)((char *)ws + z.mats() + z.map * z.segs);
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
    const size_t need = z.bwd();
    if (!distinct({{q, z.qk}, {k, z.qk}, {v, z.vo}, {g, z.gate}, {beta, z.gate}, {lens, (size_t)s->batch * 4},
                   {h_chunks, z.hchunks}, {dout, z.vo}, {dh_final, z.state}},
                  {{dq, z.qk}, {dk, z.qk}, {dv, z.vo}, {dg, z.gate}, {dbeta, z.gate}, {dh_init, z.state}, {ws, need}}))
        return BDSSM_ERR_ALIAS;
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return BDSSM_ERR_WORKSPACE;
    DeltaCall c = delta_call(s, T, q, k, v, g, beta, scale, lens);
    c.h_chunks = const_cast<float *>(h_chunks);
    c.dout = dout;
    c.dh_final = dh_final;
    char *w = (char *)ws;
    c.mats = w;
    c.G = (double *)(w + z.mats3());
    c.dS = (float *)(w + z.mats3() + z.sums());
    c.segs = z.segs_bwd;
    c.agg = (float *)(w + z.mats3() + z.sums() + z.hchunks);
    c.h_seg = (float *)(w + z.mats3() + z.sums() + z.hchunks + z.map * z.segs_bwd);
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

int bdssm_kv_commit(const bdssm_kv_shape *s, int64_t T, const void *k, const void *v, const int32_t *page_table,
                    const int32_t *ctx_lens, const int32_t *lens, void *k_cache, float *k_scale, void *v_cache,
                    float *v_scale, hipStream_t st) {
    const int rc = check_kv(s, T);
    if (rc) return rc;
    if (s->batch == 0 || T < s->page_len || s->n_pages == 0 || s->max_pages == 0) return BDSSM_OK;
    if (!k || !v || !page_table || !ctx_lens || !k_cache || !k_scale || !v_cache || !v_scale) return BDSSM_ERR_NULL;
    if (!all_aligned({k, v, page_table, ctx_lens, lens, k_cache, k_scale, v_cache, v_scale})) return BDSSM_ERR_ALIGN;
    if (!product_fits({s->batch, T / s->page_len, s->heads_kv}) ||
        s->batch * (T / s->page_len) * s->heads_kv > kMostGroups / 2)
        return BDSSM_ERR_SHAPE;
    const KvSizes z = kv_sizes(s, T, 0);
    if (!distinct({{k, z.kv}, {v, z.kv}, {page_table, z.table}, {ctx_lens, z.row}, {lens, z.row}},
                  {{k_cache, z.cache}, {k_scale, z.scale}, {v_cache, z.cache}, {v_scale, z.scale}}))
        return BDSSM_ERR_ALIAS;
    KvCall c = kv_call(s, T, k, v, page_table, ctx_lens, lens);
    c.kc = k_cache;
    c.ks = k_scale;
    c.vc = v_cache;
    c.vs = v_scale;
    (void)hipGetLastError();
    if (s->dtype == BDSSM_BF16) launch_kv_commit<uint16_t>(c, st);
    else launch_kv_commit<float>(c, st);
    return launch_status();
}

size_t bdssm_kv_workspace_bytes(const bdssm_kv_shape *s, int64_t Lq) {
    if (check_kv(s, Lq) != BDSSM_OK) return (size_t)-1;
    size_t part = 0;
    return kv_workspace(s, kv_plan(s, Lq), &part);
}

int bdssm_kv_attn_step(const bdssm_kv_shape *s, int64_t L, int64_t Lq, const void *q, const void *k, const void *v,
                       const void *k_cache, const float *k_scale, const void *v_cache, const float *v_scale,
                       const int32_t *page_table, const int32_t *ctx_lens, const int32_t *lens, int causal, float scale,
                       void *o, void *ws, size_t ws_bytes, hipStream_t st) {
    const int rc = check_kv(s, L);
    if (rc) return rc;
    if (Lq < 0 || Lq > L) return BDSSM_ERR_SHAPE;
    if (s->batch == 0 || Lq == 0) return BDSSM_OK;
    const bool cached = s->n_pages > 0 && s->max_pages > 0;
    if (!q || !k || !v || !o || !ctx_lens || (cached && (!k_cache || !k_scale || !v_cache || !v_scale || !page_table)))
        return BDSSM_ERR_NULL;
    if (!all_aligned({q, k, v, k_cache, k_scale, v_cache, v_scale, page_table, ctx_lens, lens, o, ws})) return BDSSM_ERR_ALIGN;
    const KvSizes z = kv_sizes(s, L, Lq);
    const KvPlan plan = kv_plan(s, Lq);
    if (!product_fits({s->batch, s->heads_kv, plan.splits, plan.qtiles}) ||
        s->batch * s->heads_kv * plan.splits * plan.qtiles > kMostGroups - 8 * plan.qtiles || Lq * kv_group(s) > kMostGroups)
        return BDSSM_ERR_SHAPE;
    size_t part = 0;
    const size_t need = kv_workspace(s, plan, &part);
    if (!distinct({{q, z.q}, {k, z.kv}, {v, z.kv}, {k_cache, z.cache}, {k_scale, z.scale}, {v_cache, z.cache}, {v_scale, z.scale},
                   {page_table, z.table}, {ctx_lens, z.row}, {lens, z.row}},
                  {{o, z.q}, {ws, need}}))
        return BDSSM_ERR_ALIAS;
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return BDSSM_ERR_WORKSPACE;
    KvCall c = kv_call(s, L, k, v, page_table, ctx_lens, lens);
    c.q = q;
    c.kc = const_cast<void *>(k_cache);
    c.ks = const_cast<float *>(k_scale);
    c.vc = const_cast<void *>(v_cache);
    c.vs = const_cast<float *>(v_scale);
    c.o = o;
    c.Lq = Lq;
    c.causal = causal != 0;
    c.scale = scale;
    c.plan = plan;
    c.part_o = (float *)ws;
    c.part_ml = (float *)((char *)ws + part);
    (void)hipGetLastError();
    if (s->dtype == BDSSM_BF16) launch_kv_attn<uint16_t>(c, st);
    else launch_kv_attn<float>(c, st);
    return launch_status();
}

}  // extern "C"
