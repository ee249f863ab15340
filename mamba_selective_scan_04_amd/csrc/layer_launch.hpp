// layer_launch.hpp -- host-side launch arguments shared by the translation units
// of the operators around the scans.  The launchers are defined in
// launch_conv.hip and launch_norm.hip (each compiled once per stream type) and
// called by the entry points in layer.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bdssm.h"
#include "conv_kernels.hpp"
#include "norm_kernels.hpp"

namespace bdssm_host {

using namespace bdssm_dev;

constexpr int kConvLane = 4;       // channels of a lane
constexpr int kConvMost = (1 << 30) - 1;   // tokens of a row

// How the convolution's work is cut: rows in `chunks` of `chunk` tokens; backward,
// workgroups of 256 / row_lanes chunks at a time.
struct ConvPlan {
    int64_t chunks, jobs;
    int chunk, lanes, block;                       // forward
    int row_lanes, groups, n_parts;          // backward
};

struct ConvCall {
    const void *u, *c_init, *dy, *dc_final;
    const float *w, *bias;
    const int32_t *lens;
    const uint8_t *starts;
    void *y, *c_final, *du, *dc_init;
    float *dw, *dbias, *parts;
    int64_t batch, T, ld, batch_ld, du_ld, du_batch_ld;
    int ch, width, silu;
    ConvPlan plan;
};

template <typename T>
void launch_conv(const ConvCall &c, hipStream_t st);
template <typename T>
void launch_conv_bwd(const ConvCall &c, hipStream_t st);
template <> void launch_conv<float>(const ConvCall &, hipStream_t);
template <> void launch_conv<uint16_t>(const ConvCall &, hipStream_t);
template <> void launch_conv_bwd<float>(const ConvCall &, hipStream_t);
template <> void launch_conv_bwd<uint16_t>(const ConvCall &, hipStream_t);

struct NormCall {
    const void *x, *res, *dy, *dh;
    const float *w;
    double eps;
    void *y, *h, *dx, *dres;
    uint8_t *codes;
    float *scales, *rstd, *dw, *parts;
    int64_t rows, group;
    int ch, code;          // code: kOutStream, or the codes'
    bool wide;             // res, h fp32 where the stream is bf16
    int groups;            // workgroups
};

template <typename T>
void launch_norm(const NormCall &c, hipStream_t st);
template <typename T>
void launch_norm_bwd(const NormCall &c, hipStream_t st);
template <> void launch_norm<float>(const NormCall &, hipStream_t);
template <> void launch_norm<uint16_t>(const NormCall &, hipStream_t);
template <> void launch_norm_bwd<float>(const NormCall &, hipStream_t);
template <> void launch_norm_bwd<uint16_t>(const NormCall &, hipStream_t);

}  // namespace bdssm_host
