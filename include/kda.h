/*
 * kda.h -- C ABI of the Kimi Delta Attention (KDA) library for NVIDIA B200
 * (sm_100a). Plain pointers and sizes only; no C++ or framework types.
 *
 * The operator (page "atlas_core/kimi_k3/kda.rs", module doc and
 * `kda_recurrent_step`): per sequence and head, a state S of d_k x d_v fp32
 * values (row = key channel) evolves token by token as
 *     S     <- diag(exp(g_t)) S                 (decay on the key axis)
 *     delta <- sigmoid(beta_t) (v_t - S^T k_t)  (beta_t is a logit)
 *     S     <- S + k_t delta^T
 *     o_t   <- scale S^T q_t
 * with q_t, k_t optionally L2-normalised first as x / sqrt(sum x^2 + 1e-6)
 * (same page, `l2norm_rows`, `KDA_L2_EPS`) and g_t optionally clamped from
 * below, g_t <- max(g_t, lower_bound). Optionally the kernel forms g_t itself
 * from the gate input (kda_gate_mode) and takes beta_t as a probability
 * instead of a logit (`beta_is_prob`).
 *
 * Conventions shared by every entry point:
 *  - Every buffer is caller-owned DEVICE memory, except the fields whose
 *    names end in `_host`. The library allocates nothing, frees nothing and
 *    never synchronises (except the two *_status queries, which exist to
 *    wait); work is queued on the caller's stream (a cudaStream_t passed as
 *    `void *`; NULL is the legacy default stream).
 *  - Tensors are dense, row-major, in the layouts given per field. Data
 *    pointers must be 16-byte aligned (beta: 2-byte aligned for bf16,
 *    4-byte for fp32). Outputs must not alias inputs (except where stated).
 *  - Errors: every call validates its arguments on the host first and
 *    returns a status without launching anything if they are bad. A launch
 *    failure returns KDA_ERR_CUDA; kda_last_cuda_error() then gives the CUDA
 *    error code. Nothing aborts, traps or prints.
 *  - q/k L2 normalisation uses eps = 1e-6 inside the square root; states are
 *    always fp32; inputs and the output share one dtype.
 */
#ifndef KDA_H_
#define KDA_H_

/* 0.4.0: the operators around the state update added (kda_rms_norm, kda_causal_conv,
 * kda_gated_scan and their backward and single-token forms). 0.3.0: kda_chunk_args ends with `debug_flags`; kda_chunk_fwd_status,
 * kda_chunk_fwd_noalloc_status and kda_launch_count added. 0.2.0: kda_step_args and kda_token_args
 * end with `state_out` (0.1.0 had no such field). */
#define KDA_VERSION 400

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARGUMENT = 1, /* null/misaligned pointer, bad size, bad cu_seqlens ... */
    KDA_ERR_UNSUPPORTED = 2,      /* valid request this build has no kernel for */
    KDA_ERR_CUDA = 3,             /* a CUDA call or launch failed */
    KDA_ERR_TIMEOUT = 4,          /* a bounded device-side wait gave up */
    KDA_ERR_WORKSPACE = 5         /* workspace missing or smaller than required */
} kda_status;

typedef enum {
    KDA_DTYPE_F32 = 0,
    KDA_DTYPE_BF16 = 1
} kda_dtype;

/*
 * How the kernel obtains the log-decay g from the `g` input: page
 * "atlas_core/kimi_k3/kda.rs", `bounded_gate`, and page "K3/kda/ops/api.py",
 * `use_gate_in_kernel` / `safe_gate`. With x = g_in + dt_bias[h, c] and
 * rate = exp(A_log[h]), all in fp32:
 *   KDA_GATE_LOG       g = g_in, then max(g, lower_bound) if has_lower_bound
 *   KDA_GATE_SOFTPLUS  g = -rate * softplus(x)        (has_lower_bound must be 0:
 *                                                      the unbounded form has none)
 *   KDA_GATE_SAFE      g = lower_bound * sigmoid(rate * x)  (has_lower_bound must
 *                                                      be 1, lower_bound < 0)
 * A_log: [H] fp32 device, required by the two in-kernel forms. dt_bias:
 * [H, Dk] fp32 device, NULL = zeros. Both are ignored by KDA_GATE_LOG.
 */
typedef enum {
    KDA_GATE_LOG = 0,
    KDA_GATE_SOFTPLUS = 1,
    KDA_GATE_SAFE = 2
} kda_gate_mode;

/*
 * Chunkwise forward: the `chunk_kda` boundary of page "K3/kda/ops/api.py"
 * (signature and preprocessing: q/k L2 norm, sigmoid of beta, in-kernel
 * gate, lower bound, initial_state, output_final_state, chunk_size), minus
 * its backend dispatch. The result equals the token recurrence above run
 * over each sequence; internally tokens are processed chunk_size at a time.
 * The fields after `workspace_bytes` default to the plain operator when
 * zero-initialised.
 */
typedef struct {
    kda_dtype dtype;      /* dtype of q, k, v, g, beta and o */
    int B, T, H, Dk, Dv;  /* q,k,g: [B,T,H,Dk]; v,o: [B,T,H,Dv]; beta: [B,T,H] */
    const void *q, *k, *v;
    const void *g;        /* per-channel log-decay (<= 0), or the gate input (gate_mode) */
    const void *beta;     /* logits, sigmoid applied in the kernel (or see beta_is_prob) */
    void *o;              /* output [B,T,H,Dv] */
    float scale;          /* <= 0 or NaN selects 1/sqrt(Dk) */
    const float *initial_state; /* [N,H,Dk,Dv] fp32, NULL = zeros */
    float *final_state;         /* [N,H,Dk,Dv] fp32 out, NULL = not wanted; may alias initial_state */
    /* Varlen packing: when cu_seqlens != NULL, B must be 1 and the T tokens
     * hold N sequences back to back; sequence n is tokens
     * cu_seqlens[n] .. cu_seqlens[n+1]-1 (int32, device, N+1 entries,
     * cu_seqlens[0] = 0, non-decreasing, cu_seqlens[N] = T). States never
     * cross a sequence boundary. cu_seqlens_host, when given, is a host copy
     * that is validated; without it the device copy is trusted. When
     * cu_seqlens == NULL, N must equal B (each batch row is a sequence). */
    const int32_t *cu_seqlens;
    const int32_t *cu_seqlens_host;
    int N;
    int use_qk_l2norm;    /* 1: q,k <- x / sqrt(sum x^2 + 1e-6) in the kernel */
    int has_lower_bound;  /* 1: g <- max(g, lower_bound); lower_bound must be < 0 */
    float lower_bound;
    int chunk_size;       /* 0 (default, = 64), 32 or 64 tokens per chunk; the result does
                           * not depend on it (up to rounding). 32 runs on CUDA cores only */
    void *workspace;      /* device scratch, 256-byte aligned; see kda_chunk_fwd_workspace_size */
    size_t workspace_bytes;
    kda_gate_mode gate_mode;   /* KDA_GATE_LOG (0): g is the log-decay */
    const float *A_log;        /* [H] fp32, in-kernel gate forms only */
    const float *dt_bias;      /* [H,Dk] fp32 or NULL, in-kernel gate forms only */
    int beta_is_prob;          /* 1: beta is used as given (no sigmoid) */
    unsigned int debug_flags;  /* 0 in normal use; KDA_DEBUG_* bits exercise failure paths */
} kda_chunk_args;

/* debug_flags bit for tests of the bounded device waits: the tensor-core forward
 * (bf16, Dk = Dv = 128, 64-token chunks) does not issue the first input copy of
 * its first kernel, so that kernel's first wait gives up after its 2 s limit, its
 * CTAs leave cleanly and the status word reads KDA_ERR_TIMEOUT (see
 * kda_chunk_fwd_status). The outputs of such a call are undefined. Other shapes
 * ignore the bit. */
#define KDA_DEBUG_STALL_FIRST_WAIT 1u

/* Bytes of device workspace with which kda_chunk_fwd runs its fastest kernel
 * for these arguments (may be 0). Only shapes, dtype and flags are read;
 * pointers may be NULL. For bf16 with d_k = d_v = 128 this is the two-pass
 * tensor-core kernel, whose workspace holds one 65 KiB record per (chunk, head)
 * (about 1.04 bytes per input byte of q, k, g and v); a smaller workspace of at
 * least 256 bytes runs the single-pass tensor-core kernel instead (same result
 * up to rounding), and less than that returns KDA_ERR_WORKSPACE.
 * When there are few (sequence, head) pairs and the sequences are long, the size
 * also covers cutting each sequence into segments whose states are chained
 * afterwards (a few d_k x d_v fp32 states per segment and head, plus two
 * scratch copies of the v rows); this applies to the two-pass kernel and, for
 * d_k = d_v, to the token-recurrent kernel that the other shapes run, and a
 * workspace too small for it runs the unsegmented kernel (same result up to
 * rounding). */
KDA_API kda_status kda_chunk_fwd_workspace_size(const kda_chunk_args *args, size_t *bytes);

/* Queue the chunkwise forward on `stream`. Returns KDA_OK once queued.
 *
 * Device-side failure: the tensor-core kernels (bf16, Dk = Dv = 128, 64-token
 * chunks) wait on their own copies and products with a 2 s limit per wait. A wait
 * that gives up makes its CTA drain what it has in flight, free its tensor memory
 * and leave, and sets the first int32 of the workspace to 1 (it is cleared to 0 at
 * the start of every call); o and final_state are then partly written. Because
 * kda_chunk_fwd never synchronises it cannot return KDA_ERR_TIMEOUT itself: call
 * kda_chunk_fwd_status with the same arguments to read the word. Other shapes run
 * kernels without device waits. */
KDA_API kda_status kda_chunk_fwd(const kda_chunk_args *args, void *stream);

/* Outcome of the last kda_chunk_fwd queued with these arguments on `stream`:
 * waits for the stream to drain (cudaStreamSynchronize), then returns
 * KDA_ERR_TIMEOUT if a bounded device wait gave up (the status word, the first
 * int32 of args->workspace, is non-zero), KDA_OK if it is zero or the arguments
 * select a kernel without device waits, KDA_ERR_CUDA if the copy or the
 * synchronisation failed. The one entry point that synchronises; it reads 4 bytes
 * and launches nothing. */
KDA_API kda_status kda_chunk_fwd_status(const kda_chunk_args *args, void *stream);

/*
 * One recurrent decode step for N sequences at once: the recurrence above
 * applied to one token per sequence (page "atlas_core/kimi_k3/kda.rs",
 * `kda_recurrent_step`), with the state read, updated and written back IN
 * PLACE (a read-modify-write of [N,H,Dk,Dv] fp32), or written to `state_out`
 * when that is given. The out-of-place form serves callers that keep two state
 * buffers and swap them each step, so the previous state stays intact (page
 * "memra-engine tests/kda_fixture_gpu.rs", the decode with `state` / `state_alt`).
 */
typedef struct {
    kda_dtype dtype;      /* dtype of q, k, v, g, beta and o */
    int N, H, Dk, Dv;
    const void *q, *k;    /* [N,H,Dk] */
    const void *v;        /* [N,H,Dv] */
    const void *g;        /* [N,H,Dk] log-decay, or the gate input (gate_mode) */
    const void *beta;     /* [N,H] logits (or see beta_is_prob) */
    float *state;         /* [N,H,Dk,Dv] fp32, updated in place */
    void *o;              /* [N,H,Dv] out */
    float scale;          /* <= 0 or NaN selects 1/sqrt(Dk) */
    int use_qk_l2norm;
    int has_lower_bound;
    float lower_bound;
    kda_gate_mode gate_mode;   /* as in kda_chunk_args */
    const float *A_log;        /* [H] fp32 */
    const float *dt_bias;      /* [H,Dk] fp32 or NULL */
    int beta_is_prob;
    float *state_out;          /* NULL: state updated in place. Else [N,H,Dk,Dv] fp32 out, 16-byte
                                * aligned, equal to state or not overlapping it; state is then
                                * only read */
} kda_step_args;

KDA_API kda_status kda_recurrent_step(const kda_step_args *args, void *stream);

/*
 * One serving decode token for N sequences (page "atlas_core/kimi_k3/kda.rs",
 * `kda_decode_token` followed by `full_rank_output_gate`), fused in one launch:
 *   1. causal depthwise convolution + SiLU over the pre-conv projections x,
 *      channels laid out q | k | v (H*Dk, H*Dk, H*Dv): each channel's window of
 *      the last conv_kernel inputs (oldest first) shifts one slot, x enters the
 *      last slot, y = silu(sum_t conv_w[c][t] * window[c][t]); the windows are
 *      updated IN PLACE;
 *   2. the recurrent step of kda_recurrent_step on q, k, v = y (same gate,
 *      beta, scale and L2-norm options), state updated IN PLACE;
 *   3. when g_out is given, o = sigmoid(g_out) * core / sqrt(mean(core^2) + norm_eps)
 *      per head (RMSNorm without a weight); otherwise o = core.
 * Host-side validation as for kda_recurrent_step; conv_kernel in 1..8.
 */
typedef struct {
    kda_dtype dtype;      /* dtype of x, g, beta, g_out and o */
    int N, H, Dk, Dv;     /* Dk, Dv in {32, 64, 128} */
    int conv_kernel;      /* window length K, 1..8 */
    const void *x;        /* [N, H*(2*Dk+Dv)] pre-conv q | k | v */
    const float *conv_w;  /* [H*(2*Dk+Dv), K] fp32 */
    float *conv_state;    /* [N, H*(2*Dk+Dv), K] fp32, oldest input first, updated in place */
    const void *g;        /* [N,H,Dk] log-decay, or the gate input (gate_mode) */
    const void *beta;     /* [N,H] logits (or see beta_is_prob) */
    float *state;         /* [N,H,Dk,Dv] fp32, updated in place */
    const void *g_out;    /* [N,H,Dv] output-gate input, or NULL for the ungated core output */
    float norm_eps;       /* RMSNorm epsilon of the output gate (>= 0) */
    void *o;              /* [N,H,Dv] out */
    float scale;          /* <= 0 or NaN selects 1/sqrt(Dk) */
    int use_qk_l2norm;
    int has_lower_bound;
    float lower_bound;
    kda_gate_mode gate_mode;
    const float *A_log;   /* [H] fp32, in-kernel gate forms only */
    const float *dt_bias; /* [H,Dk] fp32 or NULL */
    int beta_is_prob;
    float *state_out;     /* NULL: state updated in place; else as in kda_step_args (the conv
                           * windows are always updated in place) */
} kda_token_args;

KDA_API kda_status kda_decode_token(const kda_token_args *args, void *stream);

/*
 * Gradients of the chunkwise forward (the operator above with gate_mode
 * KDA_GATE_LOG): given the output cotangent `dout` and optionally a final-state
 * cotangent, returns dq, dk, dv, dg, dbeta and the initial-state gradient. The
 * pages give no backward formulas: these are the derivatives of the token
 * recurrence of page "atlas_core/kimi_k3/kda.rs" (through the L2 norm, the clamp
 * g <- max(g, lower_bound), whose gradient is zero where the bound is taken, and
 * the sigmoid of beta), taken in one of three forms, the first that applies:
 *   - chunked, on tensor cores: bf16, Dk = Dv = 128, has_lower_bound with
 *     lower_bound >= -5. The forward is rerun in its two-pass chunk form, saving
 *     each 64-token chunk's entering state; the state cotangent is carried back
 *     over the chunks with tcgen05 products (over the forward's segments when the
 *     (sequence, head) pairs are few), and the chunk-local gradients are formed on
 *     warp-level MMAs;
 *   - micro-chunk: bf16, Dk = 32, Dv in {32, 64}, has_lower_bound with lower_bound
 *     >= -10, at least 256 (sequence, head) pairs. The 16-token micro-chunk forward
 *     saves each micro-chunk's entering state (bf16); then one warp per (sequence,
 *     head) walks its micro-chunks from the last with the state cotangent in
 *     registers, every product a warp-level MMA;
 *   - otherwise the token recurrence: a recompute of the forward stores the state
 *     every 16 tokens; a reverse sweep reruns each 16-token stretch forward from
 *     its checkpoint and walks it back, each (sequence, head) split by value
 *     columns over a cluster of Dv/32 CTAs; CUDA cores, fp32.
 * Every form gives the same gradients up to rounding. Validation as kda_chunk_fwd
 * (q, k, v, g, dout and dq, dk, dv, dg 16-byte aligned; beta and dbeta aligned to
 * their element); g is the log-decay (the in-kernel gate forms are not covered).
 */
typedef struct {
    kda_dtype dtype;            /* of q, k, v, g, beta, dout and dq, dk, dv, dg, dbeta */
    int B, T, H, Dk, Dv;        /* as kda_chunk_args */
    const void *q, *k, *v, *g, *beta;
    const void *dout;           /* [B,T,H,Dv] cotangent of o */
    float scale;                /* <= 0 or NaN selects 1/sqrt(Dk) */
    const float *initial_state; /* [N,H,Dk,Dv] or NULL (zeros) */
    const float *dfinal_state;  /* [N,H,Dk,Dv] cotangent of the final state, or NULL */
    void *dq, *dk, *dv, *dg;    /* out, layouts of q, k, v, g */
    void *dbeta;                /* out, [B,T,H] */
    float *dinitial_state;      /* out [N,H,Dk,Dv], or NULL when not wanted */
    const int32_t *cu_seqlens;  /* as kda_chunk_args */
    const int32_t *cu_seqlens_host;
    int N;
    int use_qk_l2norm;
    int has_lower_bound;
    float lower_bound;
    int beta_is_prob;           /* 1: beta is a probability (dbeta is then d/dprob) */
    void *workspace;            /* device scratch of kda_chunk_bwd_workspace_size() bytes, 16-byte aligned
                                   (256-byte aligned for the segment form) */
    size_t workspace_bytes;
} kda_chunk_bwd_args;

/* Bytes of workspace with which kda_chunk_bwd runs its fastest form for these
 * shapes: for the chunked form, the forward's records and chunk table, a 96 KB
 * record per 64-token chunk and head (the chunk's entering state, D and the
 * cotangent chain's output) and, when the (sequence, head) pairs are few, three
 * d x d fp32 maps per segment and head; for the
 * micro-chunk form, the saved bf16 states (one d_k x d_v tile per 16 tokens and
 * head, plus one slot per sequence); for the token recurrence, the state
 * checkpoints (one d_k x d_v fp32 state per 16 tokens per head), a scratch of 16
 * states per (sequence, head) and a small header, and, when there are few
 * (sequence, head) pairs of long sequences and d_k = d_v, the buffers of its
 * segment form. Each figure is at least the plain token form's. A smaller
 * workspace (but at least the plain token form's, 256-byte aligned for the other
 * forms) runs the next form that fits (same result up to rounding); less than the
 * plain token form's returns KDA_ERR_WORKSPACE. Only shapes are read. */
KDA_API kda_status kda_chunk_bwd_workspace_size(const kda_chunk_bwd_args *args, size_t *bytes);

KDA_API kda_status kda_chunk_bwd(const kda_chunk_bwd_args *args, void *stream);

/*
 * Chunkwise forward for callers that cannot allocate device memory. This entry
 * point has no counterpart in the pages; it exists for callers that run under a
 * fixed device-memory plan and may not allocate once running (an inference
 * engine that reserves its memory at start-up, a plug-in whose host application
 * owns every device buffer, a C host with no allocator at the call site), for
 * whom kda_chunk_fwd's workspace is out of reach.
 *
 * Same arguments and result as kda_chunk_fwd; `workspace` and `workspace_bytes`
 * are ignored. The scratch it needs comes from a fixed 4096-byte array in the
 * library's own device memory (one per device, held from library load until
 * process exit); requests needing more than that return KDA_ERR_WORKSPACE (none
 * do today: the chunk kernels need at most 256 bytes). Nothing is allocated or
 * freed.
 *  - The first call on a device looks up that array's device address (a
 *    cudaGetSymbolAddress with the device current); make that first call before
 *    any stream capture.
 *  - Every call on a device shares the one array, which keeps the last call's
 *    contents; the library clears what must start at zero. Calls whose work
 *    overlaps on the GPU (different streams, no ordering) race on it: order them.
 *  - The array's address is looked up on every call, so a device reset (which
 *    reloads the library's device code) does not leave a stale address behind.
 *  - The status word of the bounded device waits (see kda_chunk_fwd) lives in
 *    that array, out of the caller's reach: read it with
 *    kda_chunk_fwd_noalloc_status.
 */
KDA_API kda_status kda_chunk_fwd_noalloc(const kda_chunk_args *args, void *stream);

/* kda_chunk_fwd_status for the allocation-free entry point: synchronises
 * `stream`, then reports whether a bounded device wait of the last
 * kda_chunk_fwd_noalloc with these arguments on this device gave up
 * (KDA_ERR_TIMEOUT), or KDA_OK. Calls on other streams since then may have
 * overwritten the word. */
KDA_API kda_status kda_chunk_fwd_noalloc_status(const kda_chunk_args *args, void *stream);

/*
 * ---- The operators around the state update of a layer -----------------------
 * Shared by the entry points below:
 *  - Activations are rows of channels whose channels are contiguous; `*_stride`
 *    is the distance between rows in elements (at least the row's length; 0 means
 *    dense), so a slice of a fused projection is read in place. Outputs are dense.
 *  - Pointers need the alignment of their element only. Rows are accessed by the
 *    largest of 16, 8, 4 and 2 bytes that divides the pointers, strides and row
 *    lengths of a call's activations; 16 is the fastest.
 *  - Up to 2^28 channels (the norm: 16384) and 2^31 - 4097 rows.
 *  - Packed sequences as in kda_chunk_args: with cu_seqlens B must be 1 and
 *    cu_seqlens_host, when given, is validated; without it the device copy is
 *    trusted (it moves no access out of the buffers, whatever it holds).
 *  - An output or workspace that overlaps an input or another output is refused,
 *    except where stated.
 *  - Sums, norms, states and convolution windows are fp32. Of bf16 inputs exponentials
 *    and sigmoids come from the special-function unit, a few 2^-24 off (a decay of the
 *    scan's log form at most 7), which fp32 outputs show too; of fp32 inputs from expf.
 */

/*
 * Root-mean-square norm of `rows` rows of D channels (1 <= D <= 16384), with the
 * options that a layer needs:
 *     s = x (+ residual),  y = s / sqrt(mean(s^2) + eps) * weight * sigmoid(gate)
 * (a residual or a gate, not both).
 * The gate is the full-rank output gate of page "atlas_core/kimi_k3/kda.rs"
 * (`full_rank_output_gate`) for whole sequences. The norm is taken of the fp32 sum;
 * residual_out receives the sum in the activations' dtype.
 *
 * With `scales`, y is 8-bit e4m3 (one byte an element) for an 8-bit product: each
 * row's channels in groups of group_size have scale = max(max|y| / 448, 2^-100) --
 * with pow2_scales the next power of two -- and hold the nearest e4m3 (ties to even)
 * of the fp32 quotient y / scale, y in fp32 (a group of zeros has scale 2^-100 and
 * zeros; a NaN in a group makes its scale NaN).
 */
typedef struct {
    kda_dtype dtype;          /* of x, residual, gate, residual_out, and y without scales */
    kda_dtype weight_dtype;   /* F32, or dtype */
    long long rows;
    int heads;                /* rows that lie back to back: [tokens, heads, D] activations have
                               * rows = tokens * heads, and their strides are those between
                               * tokens (at least heads * D). 0 or 1: strides between rows */
    int D;
    const void *x;
    long long x_stride;
    const void *residual;     /* NULL: none */
    long long residual_stride;
    const void *gate;         /* NULL: none */
    long long gate_stride;
    const void *weight;       /* [D], NULL = ones */
    float eps;                /* >= 0 */
    void *y;                  /* [rows, D] out */
    void *residual_out;       /* [rows, D] out, NULL when not wanted or without a residual; may
                               * be `residual` or `x` itself (same rows) */
    float *scales;            /* [rows, ceil(D / group_size)] out: 8-bit output; NULL: y has dtype */
    int group_size;           /* channels per scale: 32, 64 or 128, 0 = the whole row */
    int pow2_scales;
} kda_rms_norm_args;

KDA_API kda_status kda_rms_norm(const kda_rms_norm_args *args, void *stream);

/*
 * Gradients of kda_rms_norm (without 8-bit output) with respect to s, the gate and
 * the weight, given dy. x is the normed sum s (the forward's residual_out where a
 * residual was added), and dx the gradient of both of its terms; dresidual, when
 * given, is the cotangent of residual_out and is added to it. The weight's gradient
 * is summed over all rows in a fixed order.
 */
typedef struct {
    kda_dtype dtype;          /* of x, dy, gate, dresidual, dx, dgate */
    kda_dtype weight_dtype;   /* of weight and dweight: F32, or dtype */
    long long rows;
    int heads, D;             /* as kda_rms_norm_args */
    const void *x;
    long long x_stride;
    const void *dy;
    long long dy_stride;
    const void *gate;
    long long gate_stride;
    const void *dresidual;    /* NULL: none */
    long long dresidual_stride;
    const void *weight;
    float eps;
    void *dx;                 /* [rows, D] out */
    void *dgate;              /* [rows, D] out; given exactly when gate is */
    void *dweight;            /* [D] out, NULL when not wanted (or without weight) */
    void *workspace;          /* device scratch, 16-byte aligned */
    size_t workspace_bytes;
} kda_rms_norm_bwd_args;

/* Bytes of workspace that kda_rms_norm_bwd needs (0 without dweight): shapes and the
 * presence of dweight are read. */
KDA_API kda_status kda_rms_norm_bwd_workspace_size(const kda_rms_norm_bwd_args *args, size_t *bytes);
KDA_API kda_status kda_rms_norm_bwd(const kda_rms_norm_bwd_args *args, void *stream);

/*
 * Causal depthwise convolution + SiLU over packed sequences: the convolution of
 * kda_decode_token (page "atlas_core/kimi_k3/kda.rs", `conv_update`) for prompts and
 * training,
 *     z[t,c] = sum_k w[c][k] in[t-K+1+k][c],  y = z sigmoid(z)
 * where each sequence's inputs follow its initial window (the layout of
 * kda_token_args.conv_state: K values a channel, oldest first; slot 0 has left the
 * reach of any input). The final window is the last K of window and inputs, so
 * kda_decode_token and kda_causal_conv_step continue from it.
 */
typedef struct {
    kda_dtype dtype;          /* of x and y */
    int B, T, C, K;           /* x, y: [B,T,C]; window length K, 1..8 */
    const void *x;
    long long x_stride;
    const float *conv_w;      /* [C, K] fp32 */
    const float *initial_state; /* [N, C, K] fp32, NULL = zeros */
    float *final_state;       /* [N, C, K] fp32 out, NULL when not wanted */
    void *y;
    const int32_t *cu_seqlens;
    const int32_t *cu_seqlens_host;
    int N;
} kda_conv_args;

KDA_API kda_status kda_causal_conv(const kda_conv_args *args, void *stream);

/* One token of N sequences: the window shifts one slot, x enters the last, and
 * y = silu(w . window). conv_state is updated IN PLACE. */
typedef struct {
    kda_dtype dtype;
    int N, C, K;
    const void *x;            /* [N, C] */
    long long x_stride;
    const float *conv_w;      /* [C, K] fp32 */
    float *conv_state;        /* [N, C, K] fp32 */
    void *y;                  /* [N, C] out */
} kda_conv_step_args;

KDA_API kda_status kda_causal_conv_step(const kda_conv_step_args *args, void *stream);

/* Gradients of kda_causal_conv given dy and, optionally, the cotangent of the final
 * windows. dconv_w is summed over all rows in a fixed order. */
typedef struct {
    kda_dtype dtype;          /* of x, dy and dx */
    int B, T, C, K;
    const void *x;
    long long x_stride;
    const void *dy;
    long long dy_stride;
    const float *conv_w;
    const float *initial_state; /* as in the forward */
    const float *dfinal_state;  /* [N, C, K] or NULL */
    void *dx;                 /* [B,T,C] out */
    float *dconv_w;           /* [C, K] out, NULL when not wanted */
    float *dinitial_state;    /* [N, C, K] out, NULL when not wanted */
    const int32_t *cu_seqlens;
    const int32_t *cu_seqlens_host;
    int N;
    void *workspace;          /* device scratch, 16-byte aligned */
    size_t workspace_bytes;
} kda_conv_bwd_args;

/* Bytes of workspace that kda_causal_conv_bwd needs (0 without dconv_w): shapes and
 * the presence of dconv_w are read. */
KDA_API kda_status kda_causal_conv_bwd_workspace_size(const kda_conv_bwd_args *args, size_t *bytes);
KDA_API kda_status kda_causal_conv_bwd(const kda_conv_bwd_args *args, void *stream);

/*
 * Gated linear recurrence: the elementwise companion of the chunkwise forward, one
 * fp32 state a channel, over packed sequences:
 *     KDA_SCAN_GATE_LOG      a = exp(g) with g clamped below by lower_bound,
 *                            h_t = a_t h_{t-1} + x_t
 *     KDA_SCAN_GATE_SIGMOID  a = sigmoid(g) (no lower bound),
 *                            h_t = a_t h_{t-1} + (1 - a_t) x_t
 * g <= 0 is expected in the log form (a decay); it is not checked. The state that
 * the recurrence carries is fp32 throughout, h is rounded as it is written.
 */
typedef enum {
    KDA_SCAN_GATE_LOG = 0,
    KDA_SCAN_GATE_SIGMOID = 1
} kda_scan_gate;

typedef struct {
    kda_dtype dtype;          /* of x, g and h */
    kda_scan_gate gate;
    int B, T, D;              /* x, g, h: [B,T,D] */
    const void *x;
    long long x_stride;
    const void *g;
    long long g_stride;
    void *h;
    const float *initial_state; /* [N, D] fp32, NULL = zeros */
    float *final_state;       /* [N, D] fp32 out, NULL when not wanted */
    const int32_t *cu_seqlens;
    const int32_t *cu_seqlens_host;
    int N;
    int has_lower_bound;
    float lower_bound;        /* < 0 */
    void *workspace;          /* device scratch, 16-byte aligned */
    size_t workspace_bytes;
} kda_scan_args;

/* Bytes of workspace that kda_gated_scan needs (0 where no sequence is cut along time).
 * Shapes, dtype and the offsets (cu_seqlens_host, and whether cu_seqlens is given) are
 * read. Calls that may overlap on the GPU, replays of captured graphs among them, need a
 * workspace each. */
KDA_API kda_status kda_gated_scan_workspace_size(const kda_scan_args *args, size_t *bytes);

/* Queue the recurrence on `stream`: one launch, or two or three where sequences are cut
 * along time to fill the GPU (results depend on the shapes alone, not on timing). */
KDA_API kda_status kda_gated_scan(const kda_scan_args *args, void *stream);

/* One token of N sequences: state <- a state + x (or (1 - a) x), h = state. */
typedef struct {
    kda_dtype dtype;
    kda_scan_gate gate;
    int N, D;
    const void *x;            /* [N, D] */
    long long x_stride;
    const void *g;
    long long g_stride;
    float *state;             /* [N, D] fp32, updated in place unless state_out is given */
    float *state_out;         /* NULL: in place. Else [N, D] fp32 out, equal to state or not
                               * overlapping it; state is then only read */
    void *h;                  /* [N, D] out */
    int has_lower_bound;
    float lower_bound;
} kda_scan_step_args;

KDA_API kda_status kda_gated_scan_step(const kda_scan_step_args *args, void *stream);

/*
 * Gradients of kda_gated_scan given dout (the cotangent of h) and, optionally, of the
 * final state. h is the forward's output: h_{t-1} is taken from it as it was rounded
 * (and from initial_state at a sequence's first row). x is read in the sigmoid form
 * only. The gradient of g passes where g >= lower_bound, as in kda_chunk_bwd.
 */
typedef struct {
    kda_dtype dtype;          /* of x, g, h, dout, dx, dg */
    kda_scan_gate gate;
    int B, T, D;
    const void *x;            /* NULL allowed in the log form */
    long long x_stride;
    const void *g;
    long long g_stride;
    const void *h;
    long long h_stride;
    const void *dout;
    long long dout_stride;
    const float *initial_state; /* as in the forward */
    const float *dfinal_state;  /* [N, D] or NULL */
    void *dx, *dg;            /* [B,T,D] out */
    float *dinitial_state;    /* [N, D] out, NULL when not wanted */
    const int32_t *cu_seqlens;
    const int32_t *cu_seqlens_host;
    int N;
    int has_lower_bound;
    float lower_bound;
    void *workspace;          /* as kda_scan_args */
    size_t workspace_bytes;
} kda_scan_bwd_args;

KDA_API kda_status kda_gated_scan_bwd_workspace_size(const kda_scan_bwd_args *args, size_t *bytes);
KDA_API kda_status kda_gated_scan_bwd(const kda_scan_bwd_args *args, void *stream);

/* Static, human-readable name of a status. */
KDA_API const char *kda_status_string(kda_status status);

/* CUDA error code (cudaError_t as int) of the last KDA_ERR_CUDA returned on
 * this host thread, 0 if none. */
KDA_API int kda_last_cuda_error(void);

/* Kernel launches the library has queued since it was loaded, over all host
 * threads and devices: a diagnostic for benchmarks, which read it before and
 * after a timed region. A launch recorded into a CUDA graph counts once, when it
 * is captured, not when the graph is replayed. */
KDA_API unsigned long long kda_launch_count(void);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH; equal to KDA_VERSION of
 * the header the library was built with. A caller built against an older header
 * passes shorter argument structs, so compare the two before calling. */
KDA_API int kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
