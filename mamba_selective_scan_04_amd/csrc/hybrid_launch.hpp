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

namespace bdssm_host {

using namespace bdssm_dev;

struct DeltaCall {
    const void *q, *k, *v;
    const float *g, *beta, *h_init;
    void *o;
    float *h_final, *h_chunks, *W;
    // backward
    const void *dout;
    const float *dh_final;
    float *Wt, *dS, *dh_init, *dg, *dbeta;
    void *dq, *dk_out, *dv_out;
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

}  // namespace bdssm_host
