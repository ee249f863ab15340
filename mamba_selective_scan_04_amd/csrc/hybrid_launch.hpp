// hybrid_launch.hpp -- host-side launch arguments shared by the translation
// units of the hybrid layer's operators.  The launchers are defined in
// launch_delta.hip and launch_kv.hip (each compiled once per stream type) and
// called by the entry points in hybrid.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bdssm.h"
#include "delta_bwd_kernels.hpp"
#include "delta_kernels.hpp"
#include "kv_kernels.hpp"

namespace bdssm_host {

using namespace bdssm_dev;

struct DeltaCall {
    const void *q, *k, *v;
    const float *g, *beta, *h_init;
    void *o;
    float *h_final, *h_chunks;
    void *mats;   // the chunks' matrices (Mats)
    float *agg, *h_seg;   // the segments' maps and first states
    int segs;
    // backward
    const void *dout;
    const float *dh_final;
    float *dS, *dh_init, *dg, *dbeta;
    void *dq, *dk_out, *dv_out;
    double *G;
    int64_t batch;
    int dk;
    DeltaDims d;
};

template <typename T>
void launch_delta_scan(const DeltaCall &c, hipStream_t st);
template <typename T>
void launch_delta_step(const DeltaCall &c, hipStream_t st);
template <typename T>
void launch_delta_bwd(const DeltaCall &c, hipStream_t st);
template <> void launch_delta_bwd<float>(const DeltaCall &, hipStream_t);
template <> void launch_delta_bwd<uint16_t>(const DeltaCall &, hipStream_t);
template <> void launch_delta_scan<float>(const DeltaCall &, hipStream_t);
template <> void launch_delta_scan<uint16_t>(const DeltaCall &, hipStream_t);
template <> void launch_delta_step<float>(const DeltaCall &, hipStream_t);
template <> void launch_delta_step<uint16_t>(const DeltaCall &, hipStream_t);

// How the attention's work is cut: query rows (tokens x heads of a key/value
// head) in tiles of 16 a wave, keys in `splits` ranges.
struct KvPlan {
    int tiles, qtiles, splits;
};

struct KvCall {
    const void *q, *k, *v;
    void *kc, *vc, *o;
    float *ks, *vs, *part_o, *part_ml;
    int64_t batch, L, Lq;
    int head_dim, code, causal;
    float scale;
    KvPlan plan;
    KvDims d;
};

template <typename T>
void launch_kv_commit(const KvCall &c, hipStream_t st);
template <typename T>
void launch_kv_attn(const KvCall &c, hipStream_t st);
template <> void launch_kv_commit<float>(const KvCall &, hipStream_t);
template <> void launch_kv_commit<uint16_t>(const KvCall &, hipStream_t);
template <> void launch_kv_attn<float>(const KvCall &, hipStream_t);
template <> void launch_kv_attn<uint16_t>(const KvCall &, hipStream_t);

}  // namespace bdssm_host
