// Entry points of the operators around the state update (RMS norm, causal convolution,
// gated scan): argument validation and launch. No allocation, no synchronisation.
#include <math.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_layer.cuh"

namespace kda {
void record_cuda_error(int e);      // kda_api.cu
bool token_conv_supported(int K);   // kda_token.cu
}  // namespace kda

namespace {

constexpr int kMaxNormDim = 16384;
constexpr int kMaxChannels = 1 << 28;

kda_status launched(cudaError_t e) {
    if (e == cudaSuccess) return KDA_OK;
    kda::record_cuda_error((int)e);
    return KDA_ERR_CUDA;
}

bool dtype_ok(int d) { return d == KDA_DTYPE_F32 || d == KDA_DTYPE_BF16; }
size_t size_of(kda_dtype d) { return d == KDA_DTYPE_BF16 ? 2 : 4; }

// Memory that a call reads or writes: `rows` rows of `cols` elements, `stride` apart.
struct Range {
    uintptr_t lo, hi;
};

// A tensor of the call, or none. `bad` is set where a required one is missing, misaligned,
// or has a stride below its row.
struct Checker {
    bool bad = false;
    Range in[8], out[8];
    int nin = 0, nout = 0;

    static Range range(const void *p, long long rows, long long cols, long long stride, size_t esz) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        const long long n = rows > 0 && cols > 0 ? (rows - 1) * stride + cols : 0;
        return {lo, lo + (uintptr_t)n * esz};
    }
    // Returns the stride with 0 resolved.
    long long input(const void *p, bool need, long long rows, long long cols, long long stride, size_t esz) {
        const long long s = stride == 0 ? cols : stride;
        if (!p) { bad |= need; return s; }
        if (s < cols || reinterpret_cast<uintptr_t>(p) % esz) { bad = true; return s; }
        in[nin++] = range(p, rows, cols, s, esz);
        return s;
    }
    void output(const void *p, bool need, long long rows, long long cols, size_t esz, size_t align = 0) {
        if (!p) { bad |= need; return; }
        if (reinterpret_cast<uintptr_t>(p) % (align ? align : esz)) { bad = true; return; }
        out[nout++] = range(p, rows, cols, cols, esz);
    }
    void scratch(const void *p, size_t need) {
        if (p && need) out[nout++] = range(p, 1, (long long)need, (long long)need, 1);
    }
    static bool overlap(const Range &a, const Range &b) { return a.lo < b.hi && b.lo < a.hi; }
    // Whether every output stands apart from the inputs and the other outputs.
    bool apart() const {
        for (int i = 0; i < nout; ++i) {
            for (int j = 0; j < nin; ++j)
                if (overlap(out[i], in[j])) return false;
            for (int j = 0; j < i; ++j)
                if (overlap(out[i], out[j])) return false;
        }
        return true;
    }
};

// Batch, lengths and offsets of packed sequences.
kda_status check_span(int B, int T, int N, const int32_t *cu, const int32_t *cu_host, kda::RowSpan *span) {
    if (B < 1 || T < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (!cu && cu_host) return KDA_ERR_INVALID_ARGUMENT;
    if (cu) {
        if (B != 1 || N < 1 || reinterpret_cast<uintptr_t>(cu) % 4) return KDA_ERR_INVALID_ARGUMENT;
    } else {
        if (N == 0) N = B;
        if (N != B) return KDA_ERR_INVALID_ARGUMENT;
    }
    // rows are 32-bit numbers, and chunks of rows reach a little beyond the last
    if ((long long)B * T > 0x7fffffffLL - 4096 || N > 0x7fffffff - 4096) return KDA_ERR_INVALID_ARGUMENT;
    if (cu_host) {
        if (cu_host[0] != 0 || cu_host[N] != T) return KDA_ERR_INVALID_ARGUMENT;
        for (int n = 0; n < N; ++n)
            if (cu_host[n + 1] < cu_host[n]) return KDA_ERR_INVALID_ARGUMENT;
    }
    span->cu = cu;
    span->T = T;
    span->N = N;
    span->R = B * T;
    return KDA_OK;
}

kda_status check_scan_gate(int gate, int has_lb, float lb) {
    if (gate != KDA_SCAN_GATE_LOG && gate != KDA_SCAN_GATE_SIGMOID) return KDA_ERR_INVALID_ARGUMENT;
    if (has_lb && (gate == KDA_SCAN_GATE_SIGMOID || !(lb < 0.f))) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

bool workspace_ok(const void *ws, size_t bytes, size_t need, size_t align) {
    return need == 0 || (ws && bytes >= need && reinterpret_cast<uintptr_t>(ws) % align == 0);
}

// The rows of a norm tensor; ones that follow one another are evenly spaced.
kda::NormRows norm_rows(const void *at, long long token_stride, int heads, int D) {
    if (token_stride == (long long)heads * D) return {at, D, 1};
    return {at, token_stride, heads};
}

kda_status check_norm_shape(int dtype, int weight_dtype, long long rows, int heads, int D, float eps) {
    if (!dtype_ok(dtype) || (weight_dtype != KDA_DTYPE_F32 && weight_dtype != dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (rows < 0 || heads < 0 || D < 1 || !(eps >= 0.f)) return KDA_ERR_INVALID_ARGUMENT;
    if (D > kMaxNormDim) return KDA_ERR_UNSUPPORTED;
    if (rows > (1LL << 40) / D) return KDA_ERR_INVALID_ARGUMENT;
    // rows of several heads are numbered in 32 bits
    if (heads > 1 && (rows % heads || rows > 0x7fffffffLL)) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

kda_status check_conv_shape(int dtype, int C, int K) {
    if (!dtype_ok(dtype) || C < 1 || C > kMaxChannels) return KDA_ERR_INVALID_ARGUMENT;
    if (!kda::token_conv_supported(K)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

template <typename Args> kda_status scan_shape(const Args *a, kda::RowSpan *span) {
    if (!dtype_ok(a->dtype) || a->D < 1 || a->D > kMaxChannels) return KDA_ERR_INVALID_ARGUMENT;
    kda_status s = check_scan_gate(a->gate, a->has_lower_bound, a->lower_bound);
    if (s != KDA_OK) return s;
    return check_span(a->B, a->T, a->N, a->cu_seqlens, a->cu_seqlens_host, span);
}

template <typename Args> kda_status scan_workspace(const Args *a, size_t *bytes) {
    if (!a || !bytes) return KDA_ERR_INVALID_ARGUMENT;
    kda::RowSpan span;
    kda_status s = scan_shape(a, &span);
    if (s != KDA_OK) return s;
    *bytes = kda::scan_workspace_bytes(span, a->cu_seqlens_host, a->D, a->dtype == KDA_DTYPE_BF16);
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_rms_norm(const kda_rms_norm_args *a, void *stream) {
    if (!a) return KDA_ERR_INVALID_ARGUMENT;
    kda_status s = check_norm_shape(a->dtype, a->weight_dtype, a->rows, a->heads, a->D, a->eps);
    if (s != KDA_OK) return s;
    if (a->group_size != 0 && a->group_size != 32 && a->group_size != 64 && a->group_size != 128) return KDA_ERR_UNSUPPORTED;
    if (a->residual && a->gate) return KDA_ERR_UNSUPPORTED;
    if (a->residual_out && !a->residual) return KDA_ERR_INVALID_ARGUMENT;
    if (a->rows == 0) return KDA_OK;
    const size_t esz = size_of(a->dtype);
    kda::NormParams p{};
    Checker c;
    const int heads = a->heads > 1 ? a->heads : 1;
    const long long tokens = a->rows / heads, width = (long long)heads * a->D;
    p.x = norm_rows(a->x, c.input(a->x, true, tokens, width, a->x_stride, esz), heads, a->D);
    p.residual = norm_rows(a->residual, c.input(a->residual, false, tokens, width, a->residual_stride, esz), heads, a->D);
    p.gate = norm_rows(a->gate, c.input(a->gate, false, tokens, width, a->gate_stride, esz), heads, a->D);
    c.input(a->weight, false, 1, a->D, 0, size_of(a->weight_dtype));
    const int group = a->group_size ? a->group_size : a->D;
    c.output(a->y, true, a->rows, a->D, a->scales ? 1 : esz);
    c.output(a->scales, false, a->rows, (a->D + group - 1) / group, 4);
    // every thread reads its channels of a row before it writes them, so the sum may replace a term
    const bool in_place = a->residual_out && ((a->residual_out == a->residual && p.residual.stride == a->D) ||
                                              (a->residual_out == a->x && p.x.stride == a->D));
    if (in_place) {
        for (int i = 0; i < c.nin; ++i)  // but no other input may lie there
            if (c.in[i].lo != reinterpret_cast<uintptr_t>(a->residual_out)) {
                Range r = Checker::range(a->residual_out, a->rows, a->D, a->D, esz);
                if (Checker::overlap(r, c.in[i])) return KDA_ERR_INVALID_ARGUMENT;
            } else if ((c.in[i].hi - c.in[i].lo) != (uintptr_t)a->rows * a->D * esz) {
                return KDA_ERR_INVALID_ARGUMENT;
            }
    } else {
        c.output(a->residual_out, false, a->rows, a->D, esz);
    }
    if (c.bad || !c.apart()) return KDA_ERR_INVALID_ARGUMENT;
    p.weight = a->weight;
    p.weight_f32 = a->weight_dtype == KDA_DTYPE_F32;
    p.rows = a->rows; p.D = a->D; p.eps = a->eps;
    p.y = a->y; p.residual_out = a->residual_out;
    p.scales = a->scales; p.group = group; p.pow2 = a->pow2_scales ? 1 : 0;
    return launched(kda::launch_rms_norm(p, a->dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

kda_status kda_rms_norm_bwd_workspace_size(const kda_rms_norm_bwd_args *a, size_t *bytes) {
    if (!a || !bytes) return KDA_ERR_INVALID_ARGUMENT;
    kda_status s = check_norm_shape(a->dtype, a->weight_dtype, a->rows, a->heads, a->D, a->eps);
    if (s != KDA_OK) return s;
    *bytes = kda::rms_norm_bwd_workspace_bytes(a->rows, a->D, a->dweight != nullptr);
    return KDA_OK;
}

kda_status kda_rms_norm_bwd(const kda_rms_norm_bwd_args *a, void *stream) {
    size_t need = 0;
    kda_status s = kda_rms_norm_bwd_workspace_size(a, &need);
    if (s != KDA_OK) return s;
    if (a->dresidual && a->gate) return KDA_ERR_UNSUPPORTED;
    const size_t esz = size_of(a->dtype), wsz = size_of(a->weight_dtype);
    kda::NormBwdParams p{};
    Checker c;
    const int heads = a->heads > 1 ? a->heads : 1;
    const long long tokens = a->rows / heads, width = (long long)heads * a->D;
    p.x = norm_rows(a->x, c.input(a->x, a->rows > 0, tokens, width, a->x_stride, esz), heads, a->D);
    p.dy = norm_rows(a->dy, c.input(a->dy, a->rows > 0, tokens, width, a->dy_stride, esz), heads, a->D);
    p.gate = norm_rows(a->gate, c.input(a->gate, false, tokens, width, a->gate_stride, esz), heads, a->D);
    p.dresidual = norm_rows(a->dresidual, c.input(a->dresidual, false, tokens, width, a->dresidual_stride, esz), heads, a->D);
    c.input(a->weight, false, 1, a->D, 0, wsz);
    c.output(a->dx, a->rows > 0, a->rows, a->D, esz);
    c.output(a->dgate, a->rows > 0 && a->gate, a->rows, a->D, esz);
    c.output(a->dweight, false, 1, a->D, wsz);
    c.scratch(a->workspace, need);
    if (c.bad || !c.apart() || (a->dgate && !a->gate) || (a->dweight && !a->weight)) return KDA_ERR_INVALID_ARGUMENT;
    if (a->rows == 0) {  // a sum over no rows
        if (!a->dweight) return KDA_OK;
        return launched(cudaMemsetAsync(a->dweight, 0, (size_t)a->D * wsz, static_cast<cudaStream_t>(stream)));
    }
    if (!workspace_ok(a->workspace, a->workspace_bytes, need, 16)) return KDA_ERR_WORKSPACE;
    p.weight = a->weight;
    p.weight_f32 = a->weight_dtype == KDA_DTYPE_F32;
    p.rows = a->rows; p.D = a->D; p.eps = a->eps;
    p.dx = a->dx; p.dgate = a->dgate; p.dweight = a->dweight;
    p.partial = need ? static_cast<float *>(a->workspace) : nullptr;
    return launched(kda::launch_rms_norm_bwd(p, a->dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

kda_status kda_causal_conv(const kda_conv_args *a, void *stream) {
    if (!a) return KDA_ERR_INVALID_ARGUMENT;
    kda::ConvParams p{};
    kda_status s = check_conv_shape(a->dtype, a->C, a->K);
    if (s == KDA_OK) s = check_span(a->B, a->T, a->N, a->cu_seqlens, a->cu_seqlens_host, &p.span);
    if (s != KDA_OK) return s;
    const size_t esz = size_of(a->dtype);
    const bool any = p.span.R > 0;
    Checker c;
    p.x_stride = c.input(a->x, any, p.span.R, a->C, a->x_stride, esz);
    c.input(a->conv_w, true, a->C, a->K, 0, 4);
    c.input(a->initial_state, false, p.span.N, (long long)a->C * a->K, 0, 4);
    c.output(a->y, any, p.span.R, a->C, esz);
    c.output(a->final_state, false, p.span.N, (long long)a->C * a->K, 4);
    if (c.bad || !c.apart()) return KDA_ERR_INVALID_ARGUMENT;
    if (!any && !a->final_state) return KDA_OK;
    p.x = a->x; p.w = a->conv_w; p.C = a->C; p.K = a->K;
    p.s0 = a->initial_state; p.sT = a->final_state; p.y = a->y;
    return launched(kda::launch_conv(p, a->dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

kda_status kda_causal_conv_step(const kda_conv_step_args *a, void *stream) {
    if (!a || a->N < 0) return KDA_ERR_INVALID_ARGUMENT;
    kda_status s = check_conv_shape(a->dtype, a->C, a->K);
    if (s != KDA_OK) return s;
    if (a->N == 0) return KDA_OK;
    if ((long long)a->N * a->C > (1LL << 36)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t esz = size_of(a->dtype);
    kda::ConvStepParams p{};
    Checker c;
    p.x_stride = c.input(a->x, true, a->N, a->C, a->x_stride, esz);
    c.input(a->conv_w, true, a->C, a->K, 0, 4);
    c.output(a->conv_state, true, a->N, (long long)a->C * a->K, 4);
    c.output(a->y, true, a->N, a->C, esz);
    if (c.bad || !c.apart()) return KDA_ERR_INVALID_ARGUMENT;
    p.x = a->x; p.w = a->conv_w; p.state = a->conv_state; p.y = a->y;
    p.N = a->N; p.C = a->C; p.K = a->K;
    return launched(kda::launch_conv_step(p, a->dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

kda_status kda_causal_conv_bwd_workspace_size(const kda_conv_bwd_args *a, size_t *bytes) {
    if (!a || !bytes) return KDA_ERR_INVALID_ARGUMENT;
    kda::RowSpan span;
    kda_status s = check_conv_shape(a->dtype, a->C, a->K);
    if (s == KDA_OK) s = check_span(a->B, a->T, a->N, a->cu_seqlens, a->cu_seqlens_host, &span);
    if (s != KDA_OK) return s;
    *bytes = a->dconv_w ? kda::conv_bwd_workspace_bytes(span.R, a->C, a->K, a->dtype == KDA_DTYPE_BF16) : 0;
    return KDA_OK;
}

kda_status kda_causal_conv_bwd(const kda_conv_bwd_args *a, void *stream) {
    size_t need = 0;
    kda_status s = kda_causal_conv_bwd_workspace_size(a, &need);
    if (s != KDA_OK) return s;
    kda::ConvBwdParams p{};
    check_span(a->B, a->T, a->N, a->cu_seqlens, nullptr, &p.span);
    const size_t esz = size_of(a->dtype);
    const bool any = p.span.R > 0;
    const long long state = (long long)a->C * a->K;
    Checker c;
    p.x_stride = c.input(a->x, any, p.span.R, a->C, a->x_stride, esz);
    p.dy_stride = c.input(a->dy, any, p.span.R, a->C, a->dy_stride, esz);
    c.input(a->conv_w, true, a->C, a->K, 0, 4);
    c.input(a->initial_state, false, p.span.N, state, 0, 4);
    c.input(a->dfinal_state, false, p.span.N, state, 0, 4);
    c.output(a->dx, any, p.span.R, a->C, esz);
    c.output(a->dconv_w, false, a->C, a->K, 4);
    c.output(a->dinitial_state, false, p.span.N, state, 4);
    c.scratch(a->workspace, need);
    if (c.bad || !c.apart()) return KDA_ERR_INVALID_ARGUMENT;
    if (!workspace_ok(a->workspace, a->workspace_bytes, need, 16)) return KDA_ERR_WORKSPACE;
    if (!any && !a->dconv_w && !a->dinitial_state) return KDA_OK;
    p.x = a->x; p.dy = a->dy; p.w = a->conv_w; p.C = a->C; p.K = a->K;
    p.s0 = a->initial_state; p.dsT = a->dfinal_state;
    p.dx = a->dx; p.dw = a->dconv_w; p.ds0 = a->dinitial_state;
    p.partial = need ? static_cast<float *>(a->workspace) : nullptr;
    return launched(kda::launch_conv_bwd(p, a->dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

kda_status kda_gated_scan_workspace_size(const kda_scan_args *a, size_t *bytes) { return scan_workspace(a, bytes); }

kda_status kda_gated_scan(const kda_scan_args *a, void *stream) {
    size_t need = 0;
    kda_status s = scan_workspace(a, &need);
    if (s != KDA_OK) return s;
    kda::ScanParams p{};
    check_span(a->B, a->T, a->N, a->cu_seqlens, nullptr, &p.span);
    const size_t esz = size_of(a->dtype);
    const bool any = p.span.R > 0;
    Checker c;
    p.x_stride = c.input(a->x, any, p.span.R, a->D, a->x_stride, esz);
    p.g_stride = c.input(a->g, any, p.span.R, a->D, a->g_stride, esz);
    c.input(a->initial_state, false, p.span.N, a->D, 0, 4);
    c.output(a->h, any, p.span.R, a->D, esz);
    c.output(a->final_state, false, p.span.N, a->D, 4);
    c.scratch(a->workspace, need);
    if (c.bad || !c.apart()) return KDA_ERR_INVALID_ARGUMENT;
    if (!workspace_ok(a->workspace, a->workspace_bytes, need, 16)) return KDA_ERR_WORKSPACE;
    if (!any && !a->final_state) return KDA_OK;
    p.x = a->x; p.g = a->g; p.D = a->D; p.s0 = a->initial_state; p.sT = a->final_state; p.h = a->h;
    p.lb = a->has_lower_bound ? a->lower_bound : -INFINITY;
    return launched(kda::launch_scan(p, a->cu_seqlens_host, a->dtype == KDA_DTYPE_BF16, a->gate == KDA_SCAN_GATE_SIGMOID, a->workspace,
                                     static_cast<cudaStream_t>(stream)));
}

kda_status kda_gated_scan_step(const kda_scan_step_args *a, void *stream) {
    if (!a || !dtype_ok(a->dtype) || a->N < 0 || a->D < 1 || a->D > kMaxChannels) return KDA_ERR_INVALID_ARGUMENT;
    kda_status s = check_scan_gate(a->gate, a->has_lower_bound, a->lower_bound);
    if (s != KDA_OK) return s;
    if (a->N == 0) return KDA_OK;
    if ((long long)a->N * a->D > (1LL << 36)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t esz = size_of(a->dtype);
    kda::ScanStepParams p{};
    Checker c;
    p.x_stride = c.input(a->x, true, a->N, a->D, a->x_stride, esz);
    p.g_stride = c.input(a->g, true, a->N, a->D, a->g_stride, esz);
    float *to = a->state_out ? a->state_out : a->state;
    if (to != a->state) c.input(a->state, true, a->N, a->D, 0, 4);
    c.output(to, true, a->N, a->D, 4);
    c.output(a->h, true, a->N, a->D, esz);
    if (c.bad || !a->state || !c.apart()) return KDA_ERR_INVALID_ARGUMENT;
    p.x = a->x; p.g = a->g; p.state = a->state; p.state_out = to; p.h = a->h;
    p.N = a->N; p.D = a->D;
    p.lb = a->has_lower_bound ? a->lower_bound : -INFINITY;
    return launched(kda::launch_scan_step(p, a->dtype == KDA_DTYPE_BF16, a->gate == KDA_SCAN_GATE_SIGMOID,
                                          static_cast<cudaStream_t>(stream)));
}

kda_status kda_gated_scan_bwd_workspace_size(const kda_scan_bwd_args *a, size_t *bytes) { return scan_workspace(a, bytes); }

kda_status kda_gated_scan_bwd(const kda_scan_bwd_args *a, void *stream) {
    size_t need = 0;
    kda_status s = scan_workspace(a, &need);
    if (s != KDA_OK) return s;
    kda::ScanBwdParams p{};
    check_span(a->B, a->T, a->N, a->cu_seqlens, nullptr, &p.span);
    const size_t esz = size_of(a->dtype);
    const bool any = p.span.R > 0, sig = a->gate == KDA_SCAN_GATE_SIGMOID;
    Checker c;
    p.x_stride = c.input(a->x, any && sig, p.span.R, a->D, a->x_stride, esz);
    p.g_stride = c.input(a->g, any, p.span.R, a->D, a->g_stride, esz);
    p.h_stride = c.input(a->h, any, p.span.R, a->D, a->h_stride, esz);
    p.dout_stride = c.input(a->dout, any, p.span.R, a->D, a->dout_stride, esz);
    c.input(a->initial_state, false, p.span.N, a->D, 0, 4);
    c.input(a->dfinal_state, false, p.span.N, a->D, 0, 4);
    c.output(a->dx, any, p.span.R, a->D, esz);
    c.output(a->dg, any, p.span.R, a->D, esz);
    c.output(a->dinitial_state, false, p.span.N, a->D, 4);
    c.scratch(a->workspace, need);
    if (c.bad || !c.apart()) return KDA_ERR_INVALID_ARGUMENT;
    if (!workspace_ok(a->workspace, a->workspace_bytes, need, 16)) return KDA_ERR_WORKSPACE;
    if (!any && !a->dinitial_state) return KDA_OK;
    p.x = a->x; p.g = a->g; p.h = a->h; p.dout = a->dout; p.D = a->D;
    p.s0 = a->initial_state; p.dsT = a->dfinal_state;
    p.dx = a->dx; p.dg = a->dg; p.ds0 = a->dinitial_state;
    p.lb = a->has_lower_bound ? a->lower_bound : -INFINITY;
    return launched(kda::launch_scan_bwd(p, a->cu_seqlens_host, a->dtype == KDA_DTYPE_BF16, sig, a->workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
