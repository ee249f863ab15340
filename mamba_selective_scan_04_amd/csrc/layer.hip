// layer.hip -- C ABI, argument checks and plans of the operators around the scans:
// the short causal convolution and the residual norm.  As in bdssm.hip, every
// argument is checked on the host before the first HIP call.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "bdssm.h"
#include "host_checks.hpp"
#include "layer_launch.hpp"

using namespace bdssm_host;

namespace {

constexpr int64_t kCus = 256;

size_t value_bytes(int32_t dtype) { return dtype == BDSSM_BF16 ? 2 : 4; }

// ------------------------------------------------------------ convolution

// elements from the first to behind the last of rows of T tokens
bool extent(const bdssm_conv_shape *s, int64_t T, int64_t ld, int64_t batch_ld, int64_t *n) {
    *n = 0;
    if (s->batch == 0 || T == 0) return true;
    if (ld > kMost || batch_ld > kMost || !product_fits({T, T > 1 ? ld : 1}) || !product_fits({s->batch, s->batch > 1 ? batch_ld : 1}))
        return false;
    if (T > 1 && ld < s->channels) return false;
    const int64_t row = (T - 1) * ld + s->channels;
    if (s->batch > 1 && batch_ld < row) return false;
    *n = (s->batch - 1) * batch_ld + row;
    return true;
}

int check_conv(const bdssm_conv_shape *s, int64_t T) {
    if (s == nullptr) return BDSSM_ERR_NULL;
    if (s->dtype != BDSSM_F32 && s->dtype != BDSSM_BF16) return BDSSM_ERR_DTYPE;
    if (s->width < 2 || s->width > 4 || s->channels < 1 || s->channels > 0x7fffff00 || T < 0 || s->batch < 0) return BDSSM_ERR_SHAPE;
    if (!product_fits({s->batch, T, s->channels}) || !product_fits({s->batch, s->channels, 4}) || T > kConvMost) return BDSSM_ERR_SHAPE;
    int64_t n;
    return extent(s, T, s->u_stride, s->u_batch_stride, &n) ? BDSSM_OK : BDSSM_ERR_SHAPE;
}

// The gradients' parts are summed by workgroups of 1,024 threads, one for 64 columns.
int check_conv_bwd(const bdssm_conv_shape *s, int64_t T) {
    const int rc = check_conv(s, T);
    if (rc) return rc;
    return ((s->width + 1) * s->channels + 63) / 64 > kMostGroups / 4 ? BDSSM_ERR_SHAPE : BDSSM_OK;
}

int64_t within(int64_t x, int64_t low, int64_t high) { return x < low ? low : x > high ? high : x; }

int64_t power_from(int64_t x, int64_t low, int64_t high) {   // the least power of two from x on, within low .. high
    int64_t p = low;
    while (p < x && p < high) p *= 2;
    return p;
}

// Tokens of a lane: so many that about 16 waves a CU share the work, but 4 to 24 (each
// chunk reads the W - 1 tokens in front of its own again, from L2 or beyond).
// Microseconds by the least of them, and by the most:
//   64 rows of 16 tokens, 2,048 channels, bf16   6: 5.6   4: 6.0   12: 6.7
//   2 rows of 2,041, 1,021 channels, fp32        4: 11.2   6: 12.0   12: 14.6
//   1 row of 65,536, 2,048 channels, bf16        12: 111   24: 104   48: 108   66: 106
//   8 rows of 4,096, 1,536 channels, bf16        12: 43.6   24: 42.0   48: 44.3   66: 44.0
// One chunk where only the state is wanted.
ConvPlan conv_plan(const bdssm_conv_shape *s, int64_t T, bool state_only) {
    ConvPlan p{};
    p.lanes = (int)((s->channels + kConvLane - 1) / kConvLane);
    const int64_t most = kCus * 16 * 64, work = s->batch * T * p.lanes;
    p.chunk = (int)(state_only ? (T > 0 ? T : 1) : within((work + most - 1) / most, 4, 24));
    p.chunks = T > 0 ? (T + p.chunk - 1) / p.chunk : 1;
    p.jobs = s->batch * p.chunks * p.lanes;
    p.block = p.jobs < 256 * 256 ? 64 : 256;   // few lanes: spread over the CUs
    return p;
}

// Backward: as many workgroups as run at once (three a CU, by registers), and as many
// chunks as they take at a time, or as there are rows: a second round of a few would
// take as long as the first.  Each workgroup's sums of the parameters' gradients make
// a part.
ConvPlan conv_bwd_plan(const bdssm_conv_shape *s, int64_t T) {
    ConvPlan p{};
    p.lanes = (int)((s->channels + kConvLane - 1) / kConvLane);
    p.row_lanes = (int)power_from(p.lanes, 1, 64);
    p.groups = (p.lanes + p.row_lanes - 1) / p.row_lanes;
    const int64_t per = 256 / p.row_lanes, most = p.groups < kCus * 3 ? kCus * 3 / p.groups : 1;
    int64_t chunks = s->batch > 0 ? most * per / s->batch : 1;
    if (chunks < 1) chunks = 1;
    p.chunk = (int)((T + chunks - 1) / chunks + 5) / 6 * 6;   // whole groups, see conv_bwd_kernel
    if (p.chunk == 0) p.chunk = 6;
    p.chunks = T > 0 ? (T + p.chunk - 1) / p.chunk : 1;
    const int64_t parts = (s->batch * p.chunks + per - 1) / per;
    p.n_parts = (int)(parts < most ? parts : most);
    return p;
}

size_t conv_workspace(const bdssm_conv_shape *s, const ConvPlan &p) {
    return (size_t)p.n_parts * (s->width + 1) * s->channels * 4;
}

ConvCall conv_call(const bdssm_conv_shape *s, int64_t T, const void *u, const float *w, const float *bias, int silu, const int32_t *lens) {
    ConvCall c{};
    c.u = u;
    c.w = w;
    c.bias = bias;
    c.lens = lens;
    c.batch = s->batch;
    c.T = T;
    c.ld = s->u_stride;
    c.batch_ld = s->u_batch_stride;
    c.ch = (int)s->channels;
    c.width = (int)s->width;
    c.silu = silu != 0;
    return c;
}

bool aligned_value(const void *p, int32_t dtype) { return (reinterpret_cast<uintptr_t>(p) & (value_bytes(dtype) - 1)) == 0; }

int conv_forward(const bdssm_conv_shape *s, int64_t T, const void *u, const float *w, const float *bias, int silu, const int32_t *lens,
                 const uint8_t *starts, const void *c_init, void *y, void *c_final, hipStream_t st) {
    const int rc = check_conv(s, T);
    if (rc) return rc;
    if (s->batch == 0 || (!y && !c_final)) return BDSSM_OK;
    if ((T > 0 && !u) || !w) return BDSSM_ERR_NULL;
    if (!aligned_value(u, s->dtype) || !all_aligned({w, bias, lens, starts, c_init, y, c_final})) return BDSSM_ERR_ALIGN;
    const size_t e = value_bytes(s->dtype), out = (size_t)s->batch * T * s->channels * e, state = (size_t)s->batch * (s->width - 1) * s->channels * e;
    int64_t n;
    (void)extent(s, T, s->u_stride, s->u_batch_stride, &n);
    if (!distinct({{u, n * e}, {w, (size_t)s->channels * s->width * 4}, {bias, (size_t)s->channels * 4}, {lens, (size_t)s->batch * 4},
                   {starts, (size_t)s->batch * T}, {c_init == c_final ? nullptr : c_init, state}},
                  {{y, out}, {c_final, state}}))
        return BDSSM_ERR_ALIAS;
    ConvCall c = conv_call(s, T, u, w, bias, silu, lens);
    c.starts = starts;
    c.c_init = c_init;
    c.y = y;
    c.c_final = c_final;
    c.plan = conv_plan(s, T, !y);
    if ((c.plan.jobs + c.plan.block - 1) / c.plan.block > kMostGroups) return BDSSM_ERR_SHAPE;
    (void)hipGetLastError();
    if (s->dtype == BDSSM_BF16) launch_conv<uint16_t>(c, st);
    else launch_conv<float>(c, st);
    return launch_status();
}

// ------------------------------------------------------------------- norm

int check_norm(const bdssm_norm_shape *s) {
    if (s == nullptr) return BDSSM_ERR_NULL;
    if (s->dtype != BDSSM_F32 && s->dtype != BDSSM_BF16) return BDSSM_ERR_DTYPE;
    if (s->res_dtype != s->dtype && s->res_dtype != BDSSM_F32) return BDSSM_ERR_DTYPE;
    if (s->rows < 0 || s->channels < 1 || s->channels > kNormMost || !product_fits({s->rows, s->channels})) return BDSSM_ERR_SHAPE;
    return BDSSM_OK;
}

// Workgroups: rows go round them, so that each reads the weights once; for rows of up to
// 4,096 channels four waves a SIMD backward, eight forward, whose registers are fewer.
int norm_groups(const bdssm_norm_shape *s, bool bwd) {
    const int64_t at_once = s->channels <= 1024 ? 4 : 1, most = bwd ? 1024 : 2048;
    const int64_t n = (s->rows + at_once - 1) / at_once;
    return (int)(n < most ? n : most);
}

NormCall norm_call(const bdssm_norm_shape *s, const float *w, double eps, bool bwd) {
    NormCall c{};
    c.w = w;
    c.eps = eps;
    c.rows = s->rows;
    c.ch = (int)s->channels;
    c.wide = s->res_dtype != s->dtype;
    c.groups = norm_groups(s, bwd);
    c.code = kOutStream;
    return c;
}

int norm_forward(const bdssm_norm_shape *s, const void *x, const void *res, const float *w, double eps, int code, int64_t group, void *out,
                 size_t out_bytes, float *scales, size_t scale_bytes, void *h, float *rstd, hipStream_t st) {
    if (!(eps >= 0.) || eps > 1e300 || (!res && s->res_dtype != s->dtype)) return BDSSM_ERR_SHAPE;
    if (s->rows == 0) return BDSSM_OK;
    if (!x || !w || !out || (res && !h) || (!res && h) || (code != kOutStream && !scales)) return BDSSM_ERR_NULL;
    if (!all_aligned({x, res, w, out, scales, h, rstd})) return BDSSM_ERR_ALIGN;
    const size_t n = (size_t)s->rows * s->channels, in = n * value_bytes(s->dtype), hb = n * value_bytes(s->res_dtype);
    if (!distinct({{x, in}, {res == h ? nullptr : res, hb}, {w, (size_t)s->channels * 4}},
                  {{out, out_bytes}, {scales, scale_bytes}, {h, hb}, {rstd, (size_t)s->rows * 4}}))
        return BDSSM_ERR_ALIAS;
    NormCall c = norm_call(s, w, eps, false);
    c.x = x;
    c.res = res;
    c.h = h;
    c.rstd = rstd;
    c.code = code;
    c.group = group;
    if (code == kOutStream) c.y = out;
    else c.codes = (uint8_t *)out;
    c.scales = scales;
    (void)hipGetLastError();
    if (s->dtype == BDSSM_BF16) launch_norm<uint16_t>(c, st);
    else launch_norm<float>(c, st);
    return launch_status();
}

}  // namespace

extern "C" {

int bdssm_conv_scan(const bdssm_conv_shape *s, int64_t T, const void *u, const float *w, const float *bias, int silu, const int32_t *lens,
                    const uint8_t *starts, const void *c_init, void *y, void *c_final, hipStream_t st) {
    return conv_forward(s, T, u, w, bias, silu, lens, starts, c_init, y, c_final, st);
}

int bdssm_conv_step(const bdssm_conv_shape *s, int64_t T, const void *c_cache, const void *u, const float *w, const float *bias, int silu,
                    const int32_t *lens, void *y, void *c_out, hipStream_t st) {
    return conv_forward(s, T, u, w, bias, silu, lens, nullptr, c_cache, y, c_out, st);
}

int bdssm_conv_scan_bwd(const bdssm_conv_shape *s, int64_t T, const void *u, const float *w, const float *bias, int silu,
                        const int32_t *lens, const uint8_t *starts, const void *c_init, const void *dy, const void *dc_final, void *du,
                        int64_t du_stride, int64_t du_batch_stride, float *dw, float *dbias, void *dc_init, void *ws, size_t ws_bytes,
                        hipStream_t st) {
    const int rc = check_conv_bwd(s, T);
    if (rc) return rc;
    int64_t nu, ndu;
    (void)extent(s, T, s->u_stride, s->u_batch_stride, &nu);
    if (!extent(s, T, du_stride, du_batch_stride, &ndu)) return BDSSM_ERR_SHAPE;
    if (!w || !dw || (s->batch > 0 && T > 0 && (!u || !dy || !du))) return BDSSM_ERR_NULL;
    if (!aligned_value(u, s->dtype) || !aligned_value(du, s->dtype) ||
        !all_aligned({w, bias, lens, starts, c_init, dy, dc_final, dw, dbias, dc_init, ws}))
        return BDSSM_ERR_ALIGN;
    const ConvPlan plan = conv_bwd_plan(s, T);
    const size_t e = value_bytes(s->dtype), out = (size_t)s->batch * T * s->channels * e, state = (size_t)s->batch * (s->width - 1) * s->channels * e;
    const size_t wb = (size_t)s->channels * s->width * 4, bb = (size_t)s->channels * 4, need = conv_workspace(s, plan);
    if (!distinct({{u, nu * e}, {w, wb}, {bias, bb}, {lens, (size_t)s->batch * 4}, {starts, (size_t)s->batch * T}, {c_init, state},
                   {dy, out}, {dc_final, state}},
                  {{du, ndu * e}, {dw, wb}, {dbias, bb}, {dc_init, state}, {ws, need}}))
        return BDSSM_ERR_ALIAS;
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return BDSSM_ERR_WORKSPACE;
    ConvCall c = conv_call(s, T, u, w, bias, silu, lens);
    c.starts = starts;
    c.c_init = c_init;
    c.dy = dy;
    c.dc_final = dc_final;
    c.du = du;
    c.du_ld = du_stride;
    c.du_batch_ld = du_batch_stride;
    c.dw = dw;
    c.dbias = dbias;
    c.dc_init = dc_init;
    c.parts = (float *)ws;
    c.plan = plan;
    (void)hipGetLastError();
    if (s->dtype == BDSSM_BF16) launch_conv_bwd<uint16_t>(c, st);
    else launch_conv_bwd<float>(c, st);
    return launch_status();
}

size_t bdssm_conv_workspace_bytes(const bdssm_conv_shape *s, int64_t T) {
    if (check_conv_bwd(s, T) != BDSSM_OK) return (size_t)-1;
    return conv_workspace(s, conv_bwd_plan(s, T));
}

int bdssm_rms_norm(const bdssm_norm_shape *s, const void *x, const void *res, const float *w, double eps, void *y, void *h, float *rstd,
                   hipStream_t st) {
    const int rc = check_norm(s);
    if (rc) return rc;
    return norm_forward(s, x, res, w, eps, kOutStream, 0, y, (size_t)s->rows * s->channels * value_bytes(s->dtype), nullptr, 0, h, rstd, st);
}

int bdssm_rms_norm_codes(const bdssm_norm_shape *s, const void *x, const void *res, const float *w, double eps, int code, int64_t group,
                         void *codes, float *scales, void *h, hipStream_t st) {
    const int rc = check_norm(s);
    if (rc) return rc;
    if (code != BDSSM_E4M3 && code != BDSSM_I8) return BDSSM_ERR_DTYPE;
    if (group != 0 && (group != 128 || s->channels % 128 != 0)) return BDSSM_ERR_SHAPE;
    const int64_t per = group == 0 ? s->channels : group;
    return norm_forward(s, x, res, w, eps, code, per, codes, (size_t)s->rows * s->channels, scales,
                        (size_t)s->rows * (s->channels / per) * 4, h, nullptr, st);
}

int bdssm_rms_norm_bwd(const bdssm_norm_shape *s, const void *h, const float *w, const float *rstd, const void *dy, const void *dh, void *dx,
                       void *dres, float *dw, void *ws, size_t ws_bytes, hipStream_t st) {
    const int rc = check_norm(s);
    if (rc) return rc;
    if (!w || !dw || (s->rows > 0 && (!h || !rstd || !dy || !dx))) return BDSSM_ERR_NULL;
    if (!all_aligned({h, w, rstd, dy, dh, dx, dres, dw, ws})) return BDSSM_ERR_ALIGN;
    const size_t n = (size_t)s->rows * s->channels, in = n * value_bytes(s->dtype), hb = n * value_bytes(s->res_dtype);
    const size_t wb = (size_t)s->channels * 4, need = (size_t)norm_groups(s, true) * wb;
    if (!distinct({{h, hb}, {w, wb}, {rstd, (size_t)s->rows * 4}, {dy, in}, {dh, hb}}, {{dx, in}, {dres, hb}, {dw, wb}, {ws, need}}))
        return BDSSM_ERR_ALIAS;
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return BDSSM_ERR_WORKSPACE;
    NormCall c = norm_call(s, w, 0., true);
    c.h = const_cast<void *>(h);
    c.rstd = const_cast<float *>(rstd);
    c.dy = dy;
    c.dh = dh;
    c.dx = dx;
    c.dres = dres;
    c.dw = dw;
    c.parts = (float *)ws;
    (void)hipGetLastError();
    if (s->dtype == BDSSM_BF16) launch_norm_bwd<uint16_t>(c, st);
    else launch_norm_bwd<float>(c, st);
    return launch_status();
}

size_t bdssm_norm_workspace_bytes(const bdssm_norm_shape *s) {
    if (check_norm(s) != BDSSM_OK) return (size_t)-1;
    return (size_t)norm_groups(s, true) * s->channels * 4;
}

}  // extern "C"
