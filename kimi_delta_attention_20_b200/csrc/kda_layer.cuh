// Launch parameters of the operators around the state update of a layer: RMS norm,
// causal convolution and gated scan (device pointers, strides in elements).
#pragma once

#include "kda_walk.cuh"

namespace kda {

// Rows of a norm: `heads` rows of D channels back to back, `stride` between such groups
// (heads 1: evenly spaced rows).
struct NormRows {
    const void *at;
    long long stride;
    int heads;
};

struct NormParams {
    NormRows x, residual, gate;
    const void *weight;
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
    NormRows x, dy, gate, dresidual;
    const void *weight;
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
    int piece, pieces;   // rows of a walker, walkers of a channel unit
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
    float *partial;      // [pieces, K, C]
    int piece, pieces;
};

struct ConvStepParams {
    const void *x;
    long long x_stride;
    const float *w;
    float *state;
    void *y;
    int N, C, K;
};

// How a scan's rows are cut into pieces, one after another:
//   kCutBatch  `per` pieces of `rows` rows in each sequence of T rows (the last shorter)
//   kCutSeqs   a piece per sequence of cu
//   kCutRows   pieces of `rows` rows, wherever sequences begin
enum : int { kCutBatch = 0, kCutSeqs = 1, kCutRows = 2 };
struct ScanCut {
    int kind, pieces, per, rows;
    int lb;              // bytes of a lane
    int carries;         // whether a piece may continue a sequence of the one before
    void *maps;          // [pieces, channels of whole units] pairs (A, H): a piece as the map c -> A c + H;
                         // null where no piece carries
    float *carry;        // [pieces, channels of whole units] states before the pieces, or null
};

struct ScanParams {
    RowSpan span;
    const void *x, *g;
    long long x_stride, g_stride;
    int D;
    const float *s0;     // [N, D] or null
    float *sT;
    void *h;
    float lb;            // -inf without a bound
    ScanCut cut;
};

struct ScanBwdParams {
    RowSpan span;
    const void *x, *g, *h, *dout;
    long long x_stride, g_stride, h_stride, dout_stride;
    int D;
    const float *s0, *dsT;
    void *dx, *dg;
    float *ds0;
    float lb;            // -inf without a bound
    ScanCut cut;
};

struct ScanStepParams {
    const void *x, *g;
    long long x_stride, g_stride;
    const float *state;
    float *state_out;
    void *h;
    int N, D;
    float lb;            // -inf without a bound
};

cudaError_t launch_rms_norm(const NormParams &p, bool bf16, cudaStream_t st);
cudaError_t launch_rms_norm_quant(const NormParams &p, bool bf16, int g, cudaStream_t st);
size_t rms_norm_bwd_workspace_bytes(long long rows, int D, bool weight);
cudaError_t launch_rms_norm_bwd(const NormBwdParams &p, bool bf16, cudaStream_t st);

cudaError_t launch_conv(ConvParams p, bool bf16, cudaStream_t st);
size_t conv_bwd_workspace_bytes(int rows, int C, int K, bool bf16);
cudaError_t launch_conv_bwd(ConvBwdParams p, bool bf16, cudaStream_t st);
cudaError_t launch_conv_step(const ConvStepParams &p, bool bf16, cudaStream_t st);

size_t scan_workspace_bytes(const RowSpan &span, const int32_t *cu_host, int D, bool bf16);
cudaError_t launch_scan(ScanParams p, const int32_t *cu_host, bool bf16, bool sigmoid, void *workspace, cudaStream_t st);
cudaError_t launch_scan_bwd(ScanBwdParams p, const int32_t *cu_host, bool bf16, bool sigmoid, void *workspace, cudaStream_t st);
cudaError_t launch_scan_step(const ScanStepParams &p, bool bf16, bool sigmoid, cudaStream_t st);

}  // namespace kda
