// Launch parameters of the operators around the state update of a layer: RMS norm,
// causal convolution and gated scan (device pointers, strides in elements).
#pragma once

#include "kda_rows.cuh"

namespace kda {

struct NormParams {
    const void *x, *residual, *gate, *weight;
    long long x_stride, residual_stride, gate_stride;
    int weight_f32;
    long long rows;
    int D;
    float eps;
    void *y;             // element type of x, or e4m3 where `scales` is given
    void *residual_out;  // x + residual
    float *scales;
    int group;           // channels per scale
    int pow2;
};

struct NormBwdParams {
    const void *x, *dy, *gate, *dresidual, *weight;
    long long x_stride, dy_stride, gate_stride, dresidual_stride;
    int weight_f32;
    long long rows;
    int D;
    float eps;
    void *dx, *dgate, *dweight;
    float *partial;      // [slices, D]
};

struct ConvParams {
    RowSpan span;
    const void *x;
    long long x_stride;
    const float *w;      // [C, K]
    int C, K;
    const float *s0;     // [N, C, K] windows or null
    float *sT;
    void *y;
};

struct ConvBwdParams {
    RowSpan span;
    const void *x, *dy;
    long long x_stride, dy_stride;
    const float *w;
    int C, K;
    const float *s0, *dsT;
    void *dx;
    float *dw, *ds0;
    float *partial;      // [slices, K, C]
};

struct ConvStepParams {
    const void *x;
    long long x_stride;
    const float *w;
    float *state;
    void *y;
    int N, C, K;
};

// Scratch of a scan whose rows are cut into chunks.
struct ScanChain {
    int *status;         // 1: a wait gave up
    unsigned *ticket;
    unsigned *flags;     // [chunks, tiles]
    float2 *agg;         // [chunks, tiles, kTileChannels]: a chunk as the map c -> A c + H
    float *inc;          // [chunks / group, tiles, kTileChannels]: the state behind a group
    int chunks, tiles, group;
    int stall;           // test of the bounded waits
};

struct ScanParams {
    RowSpan span;
    const void *x, *g;
    long long x_stride, g_stride;
    int D;
    const float *s0;     // [N, D] or null
    float *sT;
    void *h;
    int has_lb;
    float lb;
    ScanChain chain;
};

struct ScanBwdParams {
    RowSpan span;
    const void *x, *g, *h, *dout;
    long long x_stride, g_stride, h_stride, dout_stride;
    int D;
    const float *s0, *dsT;
    void *dx, *dg;
    float *ds0;
    int has_lb;
    float lb;
    ScanChain chain;
};

struct ScanStepParams {
    const void *x, *g;
    long long x_stride, g_stride;
    const float *state;
    float *state_out;
    void *h;
    int N, D;
    int has_lb;
    float lb;
};

cudaError_t launch_rms_norm(const NormParams &p, bool bf16, cudaStream_t st);
size_t rms_norm_bwd_workspace_bytes(long long rows, int D, bool bf16, bool weight);
cudaError_t launch_rms_norm_bwd(const NormBwdParams &p, bool bf16, cudaStream_t st);

cudaError_t launch_conv(const ConvParams &p, bool bf16, cudaStream_t st);
size_t conv_bwd_workspace_bytes(int rows, int C, int K);
cudaError_t launch_conv_bwd(const ConvBwdParams &p, bool bf16, cudaStream_t st);
cudaError_t launch_conv_step(const ConvStepParams &p, bool bf16, cudaStream_t st);

size_t scan_workspace_bytes(int rows, int D, bool bf16, bool backward);
cudaError_t launch_scan(ScanParams p, bool bf16, bool sigmoid, void *workspace, cudaStream_t st);
cudaError_t launch_scan_bwd(ScanBwdParams p, bool bf16, bool sigmoid, void *workspace, cudaStream_t st);
cudaError_t launch_scan_step(const ScanStepParams &p, bool bf16, bool sigmoid, cudaStream_t st);

}  // namespace kda
