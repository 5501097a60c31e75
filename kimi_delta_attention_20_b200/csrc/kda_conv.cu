// Causal depthwise convolution + SiLU over packed sequences (the sequence form of the
// decode token's convolution, page "atlas_core/kimi_k3/kda.rs" `conv_update`), its backward
// pass and its single token:
//     z[t,c] = sum_i w[c,i] in[t-K+1+i, c],   y = z sigmoid(z)
// where a sequence's inputs are preceded by its initial window (K values a channel, oldest
// first, or zeros), and its final window is the last K of both.
//
// 4 bytes an element forward, 6 backward (bf16). 8192 x 6144, ragged with windows, takes 43 us a
// call (4.7 TB/s) where its bytes take 31 and its two special-function instructions an element
// 25: neither is full (59 % of that pipe, 48 % of issue), the walkers of an SM do not overlap
// them any better. 65536 x 1024 backward takes 92 us (4.4 TB/s) with 57 % of issue and 38 % of that
// pipe: latency, with 13 of its warps an SM at 126 registers. A walker slides the window
// down its piece of the rows in registers. Nothing is carried between pieces but K - 1
// rows that are read twice, so pieces are cut for full waves of walkers: sixteen an SM with
// rings of 12 KiB, since they need the arithmetic of many warps beside the bytes in flight
// (9 walkers of 24 KiB: 53 us for 8192 x 6144, 12 of 16 KiB: 43, 16 of 12 KiB: 42).
#include "kda_layer.cuh"

namespace kda {

namespace {

constexpr int kConvSlots = 148 * 16;  // walkers that run at the same time
constexpr int kMinPiece = 32;         // rows of a piece, at least
constexpr int kLB = 8, kStage = 8;     // bytes of a lane, rows of a stage
constexpr int kFwdStages = 6, kBwdStages = 3;
template <typename T, int G> using FwdRing = Ring<T, G, kLB, kStage, 1, kFwdStages>;
template <typename T, int G> using BwdRing = Ring<T, G, kLB, kStage, 2, kBwdStages>;

// The lane's weights: w[c, 0..K-1] of its channels.
template <int K, int W> __device__ __forceinline__ void load_weights(const float *w, int c, int C, float (&wr)[K][W]) {
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) wr[k][i] = c + i < C ? w[(long long)(c + i) * K + k] : 0.f;
}

// Slot k of sequence n's window (zeros where there is none).
template <int W> __device__ __forceinline__ void window_slot(const float *s0, int n, int k, int K, int c, int C, float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = s0 && c + i < C ? s0[((long long)n * C + c + i) * K + k] : 0.f;
}

// win[0..K-2]: the K - 1 inputs before `row` of sequence q.
template <typename T, int K, int W>
__device__ __forceinline__ void load_window(const T *x, long long stride, const float *s0, int row, const Seq &q, int c, int C, float (&win)[K][W]) {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        const int r = row - (K - 1) + k;
        if (r >= q.start) {
#pragma unroll
            for (int i = 0; i < W; ++i) win[k][i] = c + i < C ? to_f32(x[r * stride + c + i]) : 0.f;
        } else {
            // inputs `start - r` before the sequence's first sit that far from the window's end
            window_slot(s0, q.n, K - (q.start - r), K, c, C, win[k]);
        }
    }
}

// win <- its rotation by n: slot k becomes slot (k - n) mod K.
template <int K, int W> __device__ __forceinline__ void rotate(float (&win)[K][W], int n) {
    float t[K][W];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) t[k][i] = win[(k + n) % K][i];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) win[k][i] = t[k][i];
}

// ---------------------------------------------------------------- forward
template <typename T, int G, int K>
__global__ void __launch_bounds__(32) conv_fwd_kernel(const __grid_constant__ ConvParams p) {
    using RN = FwdRing<T, G>;
    constexpr int W = RN::W, S = kStage, ST = kFwdStages, TC = walk_channels<T, kLB>();
    extern __shared__ __align__(16) char dyn[];
    const int lane = threadIdx.x, C = p.C, R = p.span.R, units = (C + TC - 1) / TC;
    const int piece = blockIdx.x / units, c0 = (blockIdx.x - piece * units) * TC, c = c0 + lane * W;
    const int b = min(piece * p.piece, R), e = piece + 1 == p.pieces ? R : min(b + p.piece, R);
    RN ring{dyn, {walk_tensor<T>(p.x, p.x_stride, c0, C, R)}, min(TC, C - c0) * (int)sizeof(T), lane};
    ring.begin(0, b);
#pragma unroll 1
    for (int k = 0; k < ST - 1; ++k) {
        if (b + k * S < e) ring.template load<1>(k, 0, b + k * S, b, e);
        cp_async_commit();
    }
    float w[K][W];
    load_weights<K, W>(p.w, c, C, w);
    // an empty sequence hands its window through
    hand_through<W>(p.span, piece, p.pieces, lane, c, C, K, p.sT, p.s0);
    if (b >= e) return;
    Seq q = seq_of(p.span, b, lane);
    float win[K][W];  // at the s-th row of a stage slot (s + k) % K is input s + k - (K - 1)
    load_window<T, K, W>(static_cast<const T *>(p.x), p.x_stride, p.s0, b, q, c, C, win);
    T *y = static_cast<T *>(p.y) + (long long)b * C;
    int slot = 0, next = ST - 1;
#pragma unroll 1
    for (int r = b; r < e; r += S) {
        cp_async_wait_group<ST - 2>();
        __syncwarp();
        const int ahead = r + (ST - 1) * S;
        if (ahead < e) ring.template load<1>(next, 0, ahead, b, e);
        cp_async_commit();
        // row r + s with the window's oldest input in slot j
        auto one = [&](int s, int j) {
            float z[W];
            ring.get(slot, 0, s, r + s, win[(j + K - 1) % K]);
            vmul(w[0], win[j % K], z);
#pragma unroll
            for (int k = 1; k < K; ++k) vfma(w[k], win[(j + k) % K], z, z);
#pragma unroll
            for (int i = 0; i < W; ++i) z[i] *= sig<T>(z[i]);
            put_row<G>(y + (long long)s * C, c, C, lane, z);
        };
        // behind the last row of a sequence, its last K inputs in slots j, j + 1 ..
        auto close = [&](int row, int j) {
            if (p.sT) {
#pragma unroll
                for (int i = 0; i < W; ++i)
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (c + i < C) p.sT[((long long)q.n * C + c + i) * K + k] = win[(j + k) % K][i];
            }
            if (row < e) {
                q = seq_of(p.span, row, lane);
#pragma unroll
                for (int k = 0; k < K - 1; ++k) window_slot(p.s0, q.n, k + 1, K, c, C, win[(j + 1 + k) % K]);
            }
        };
        if (min(q.end, e) >= r + S) {
#pragma unroll
            for (int s = 0; s < S; ++s) one(s, s);
            if (q.end == r + S) close(r + S, S - 1);
            rotate<K, W>(win, S % K);
        } else {
            const int n = min(S, e - r);
#pragma unroll 1
            for (int s = 0; s < n; ++s) {
                one(s, 0);
                if (q.end == r + s + 1) close(r + s + 1, 0);
                rotate<K, W>(win, 1 % K);
            }
        }
        y += (long long)S * C;
        next = slot;
        slot = slot + 1 == ST ? 0 : slot + 1;
    }
}

// ---------------------------------------------------------------- backward
// dz = dy s (1 + z (1 - s)), s = sigmoid(z);  din[r] = sum_i w[i] dz[r+K-1-i] over the
// sequence's rows;  dw[i] = sum_t dz[t] in[t-K+1+i]. A walker goes on for the K - 1 rows
// behind its piece, whose dz reaches back into it, and holds the K gradients that are not
// complete yet: input r is complete at row r+K-1 or where its sequence ends. A walker's
// sums for dw leave as one slice, and a second kernel joins the slices in a fixed order.
template <typename T, int G, int K>
__global__ void __launch_bounds__(32) conv_bwd_kernel(const __grid_constant__ ConvBwdParams p) {
    using RN = BwdRing<T, G>;
    constexpr int W = RN::W, S = kStage, ST = kBwdStages, TC = walk_channels<T, kLB>();
    let_next_pass_start();
    extern __shared__ __align__(16) char dyn[];
    const int lane = threadIdx.x, C = p.C, R = p.span.R, units = (C + TC - 1) / TC;
    const int piece = blockIdx.x / units, c0 = (blockIdx.x - piece * units) * TC, c = c0 + lane * W;
    const int b = min(piece * p.piece, R), e = piece + 1 == p.pieces ? R : min(b + p.piece, R);
    const int stop = b < e ? min(e + K - 1, R) : e;  // rows that are walked
    RN ring{dyn, {walk_tensor<T>(p.x, p.x_stride, c0, C, R), walk_tensor<T>(p.dy, p.dy_stride, c0, C, R)},
            min(TC, C - c0) * (int)sizeof(T), lane};
    ring.begin(0, b);
    ring.begin(1, b);
    auto load = [&](int at, int row) {
        ring.template load<1>(at, 0, row, b, stop);
        ring.template load<1>(at, 1, row, b, stop);
    };
#pragma unroll 1
    for (int k = 0; k < ST - 1; ++k) {
        if (b + k * S < stop) load(k, b + k * S);
        cp_async_commit();
    }
    float w[K][W], dw[K][W];
    load_weights<K, W>(p.w, c, C, w);
#pragma unroll
    for (int k = 0; k < K; ++k) vset(dw[k], 0.f);
    // an empty sequence's final window is its initial one
    hand_through<W>(p.span, piece, p.pieces, lane, c, C, K, p.ds0, p.dsT);
    if (b < e) {
        Seq q = seq_of(p.span, b, lane);
        // at the s-th row t of a stage win[(s + k) % K] is input t-K+1+k, acc[(s + k) % K] its gradient so far
        float win[K][W], acc[K][W];
        load_window<T, K, W>(static_cast<const T *>(p.x), p.x_stride, p.s0, b, q, c, C, win);
#pragma unroll
        for (int k = 0; k < K; ++k) vset(acc[k], 0.f);
        T *dx = static_cast<T *>(p.dx);
        // input r of the sequence (r < start: of its window) is complete with gradient v
        auto finish = [&](int r, float (&v)[W]) {
            if (r >= e) return;
            if (r >= q.start ? r < b : (q.start < b || !p.ds0)) return;
            const int place = r - q.end + K;  // in the final window
            if (p.dsT && place >= 0) {
                float f[W];
                window_slot(p.dsT, q.n, place, K, c, C, f);
                vadd(v, f, v);
            }
            if (r >= q.start) {
                put_row<G>(dx + (long long)r * C, c, C, lane, v);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (c + i < C) p.ds0[((long long)q.n * C + c + i) * K + (r - q.start + K)] = v[i];
            }
        };
        // the oldest value of the window of a sequence that starts here is no input of any row
        auto oldest = [&]() {
            float v[W];
            vset(v, 0.f);
            finish(q.start - K, v);
        };
        if (q.start == b) oldest();
        int slot = 0, next = ST - 1;
        // one more turn than there are rows where the data ends there, for what the last sequence holds
        const int turns = stop == R ? stop + 1 : stop;
#pragma unroll 1
        for (int r = b; r < turns; r += S) {
            cp_async_wait_group<ST - 2>();
            __syncwarp();
            const int ahead = r + (ST - 1) * S;
            if (ahead < stop) load(next, ahead);
            cp_async_commit();
            // row r + s, with the oldest input in slot j; its gradient is complete after it
            auto one = [&](int s, int j, bool own) {
                float dz[W], z[W];
                ring.get(slot, 0, s, r + s, win[(j + K - 1) % K]);
                ring.get(slot, 1, s, r + s, dz);
                vmul(w[0], win[j % K], z);
#pragma unroll
                for (int k = 1; k < K; ++k) vfma(w[k], win[(j + k) % K], z, z);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float sg = sig<T>(z[i]);
                    dz[i] *= sg * fmaf(z[i], 1.f - sg, 1.f);
                }
                vmul(w[K - 1], dz, acc[(j + K - 1) % K]);  // the newest input's gradient begins here
#pragma unroll
                for (int k = 0; k + 1 < K; ++k) vfma(w[k], dz, acc[(j + k) % K], acc[(j + k) % K]);
                if (own) {
#pragma unroll
                    for (int k = 0; k < K; ++k) vfma(dz, win[(j + k) % K], dw[k], dw[k]);
                }
            };
            // plain stages: all rows the piece's and of one sequence, whose windows are out of reach
            const bool first = q.start >= b && q.start > r - K;
            if (r + S <= e && q.end > r + S && !(first && p.ds0)) {
                const int from = max(b, q.start);
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    one(s, s, true);
                    const int row = r + s - (K - 1);
                    if (s >= K - 1 || row >= from) put_row<G>(dx + (long long)row * C, c, C, lane, acc[s % K]);
                }
                rotate<K, W>(win, S % K);
                rotate<K, W>(acc, S % K);
            } else {
#pragma unroll 1
                for (int s = 0; s < S; ++s) {
                    const int t = r + s;
                    if (t >= turns) break;
                    if (t == q.end) {
                        // the sequence is over: what it still holds is complete
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) finish(t - K + 1 + k, acc[k]);
                        if (t >= e) { r = turns; break; }
                        q = seq_of(p.span, t, lane);
                        oldest();
#pragma unroll
                        for (int k = 0; k < K; ++k) vset(acc[k], 0.f);
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) window_slot(p.s0, q.n, k + 1, K, c, C, win[k]);
                    }
                    if (t >= stop) break;
                    one(s, 0, t < e);
                    finish(t - K + 1, acc[0]);
                    rotate<K, W>(win, 1 % K);
                    rotate<K, W>(acc, 1 % K);
                }
            }
            next = slot;
            slot = slot + 1 == ST ? 0 : slot + 1;
        }
    }
    if (!p.partial) return;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (c + i < C) p.partial[((long long)piece * K + k) * C + c + i] = dw[k][i];
}

// dw[c, k]: the sum of its slices [K, C].
__global__ void __launch_bounds__(1024) conv_dw_kernel(const float *partial, float *dw, int slices, int C, int K) {
    const long long cols = (long long)K * C, col = (long long)blockIdx.x * 32 + (threadIdx.x & 31);
    wait_for_last_pass();
    const float v = slice_sum(partial, slices, cols, col);
    if (threadIdx.x < 32 && col < cols) dw[col % C * K + col / C] = v;
}

// ---------------------------------------------------------------- single token
template <typename T, int K>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ ConvStepParams p) {
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const int n = (int)(i / p.C), c = (int)(i - (long long)n * p.C);
    if (n >= p.N) return;
    float win[K];
    float *s = p.state + i * K;
    const float *w = p.w + (long long)c * K;
    const float xv = to_f32(static_cast<const T *>(p.x)[n * p.x_stride + c]);
    // a window of 4 (or 8) floats is one (or two) aligned 16-byte accesses
    if (K % 4 == 0 && reinterpret_cast<uintptr_t>(p.state) % 16 == 0) {
#pragma unroll
        for (int k = 0; k < K / 4; ++k) {
            const float4 q = reinterpret_cast<const float4 *>(s)[k];
            win[4 * k] = q.x; win[4 * k + 1] = q.y; win[4 * k + 2] = q.z; win[4 * k + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) win[k] = s[k];
    }
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) win[k] = win[k + 1];
    win[K - 1] = xv;
    float z = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) z = fmaf(w[k], win[k], z);
    if (K % 4 == 0 && reinterpret_cast<uintptr_t>(p.state) % 16 == 0) {
#pragma unroll
        for (int k = 0; k < K / 4; ++k)
            reinterpret_cast<float4 *>(s)[k] = make_float4(win[4 * k], win[4 * k + 1], win[4 * k + 2], win[4 * k + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] = win[k];
    }
    static_cast<T *>(p.y)[i] = from_f32<T>(z * sig<T>(z));
}

// ---------------------------------------------------------------- host
int units_of(int C, bool bf16) {
    const int tc = bf16 ? walk_channels<__nv_bfloat16, kLB>() : walk_channels<float, kLB>();
    return (C + tc - 1) / tc;
}

// Rows of a piece: stages for one wave of walkers (a few waves where the channels alone
// make more).
int piece_rows(int rows, int C, bool bf16) {
    const int units = units_of(C, bf16), want = kConvSlots > units ? kConvSlots / units : 1;
    const int each = rows / want > kMinPiece ? (int)(((long long)rows + want - 1) / want) : kMinPiece;
    return (each + kStage - 1) / kStage * kStage;
}
int pieces_of(int rows, int piece) { return rows > piece ? (int)(((long long)rows + piece - 1) / piece) : 1; }

template <typename T, int G, int K> cudaError_t run_fwd(const ConvParams &p, cudaStream_t st) {
    return run_walk(conv_fwd_kernel<T, G, K>, p, p.pieces, units_of(p.C, sizeof(T) == 2), FwdRing<T, G>::BYTES, st);
}
template <typename T, int G, int K> cudaError_t run_bwd(const ConvBwdParams &p, cudaStream_t st) {
    const cudaError_t e = run_walk(conv_bwd_kernel<T, G, K>, p, p.pieces, units_of(p.C, sizeof(T) == 2), BwdRing<T, G>::BYTES, st);
    if (e != cudaSuccess || !p.dw) return e;
    return launch_next_pass(conv_dw_kernel, (unsigned)(((long long)p.C * K + 31) / 32), 1024, st, (const float *)p.partial, p.dw, p.pieces, p.C, K);
}
template <typename T, int K> cudaError_t run_step(const ConvStepParams &p, cudaStream_t st) {
    const long long n = (long long)p.N * p.C;
    count_launch();
    conv_step_kernel<T, K><<<(unsigned)((n + 127) / 128), 128, 0, st>>>(p);
    return cudaGetLastError();
}

// Runs F<..., K> for the window of a call.
#define KDA_CONV_K(K_, ...)                                       \
    switch (K_) {                                                 \
    case 1: return __VA_ARGS__ 1>(p, st);                         \
    case 2: return __VA_ARGS__ 2>(p, st);                         \
    case 3: return __VA_ARGS__ 3>(p, st);                         \
    case 4: return __VA_ARGS__ 4>(p, st);                         \
    case 5: return __VA_ARGS__ 5>(p, st);                         \
    case 6: return __VA_ARGS__ 6>(p, st);                         \
    case 7: return __VA_ARGS__ 7>(p, st);                         \
    case 8: return __VA_ARGS__ 8>(p, st);                         \
    }                                                             \
    return cudaErrorInvalidValue;
#define KDA_CONV_PICK(F, bf16, g)                                           \
    if (bf16 && g == 16) { KDA_CONV_K(p.K, F<__nv_bfloat16, 16, ) }         \
    if (bf16 && g == 8) { KDA_CONV_K(p.K, F<__nv_bfloat16, 8, ) }           \
    if (bf16 && g == 4) { KDA_CONV_K(p.K, F<__nv_bfloat16, 4, ) }           \
    if (bf16) { KDA_CONV_K(p.K, F<__nv_bfloat16, 2, ) }                     \
    if (g == 16) { KDA_CONV_K(p.K, F<float, 16, ) }                         \
    if (g == 8) { KDA_CONV_K(p.K, F<float, 8, ) }                           \
    KDA_CONV_K(p.K, F<float, 4, )

}  // namespace

size_t conv_bwd_workspace_bytes(int rows, int C, int K, bool bf16) {
    return sizeof(float) * (size_t)pieces_of(rows, piece_rows(rows, C, bf16)) * C * K;
}

cudaError_t launch_conv(ConvParams p, bool bf16, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4;
    p.piece = piece_rows(p.span.R, p.C, bf16);
    p.pieces = pieces_of(p.span.R, p.piece);
    RowAccess ac;
    ac.rows(p.x, p.x_stride, p.C, esz);
    ac.rows(p.y, p.C, p.C, esz);
    KDA_CONV_PICK(run_fwd, bf16, ac.g())
}

cudaError_t launch_conv_bwd(ConvBwdParams p, bool bf16, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4;
    p.piece = piece_rows(p.span.R, p.C, bf16);
    p.pieces = pieces_of(p.span.R, p.piece);
    RowAccess ac;
    ac.rows(p.x, p.x_stride, p.C, esz);
    ac.rows(p.dy, p.dy_stride, p.C, esz);
    ac.rows(p.dx, p.C, p.C, esz);
    KDA_CONV_PICK(run_bwd, bf16, ac.g())
}

cudaError_t launch_conv_step(const ConvStepParams &p, bool bf16, cudaStream_t st) {
    if (bf16) { KDA_CONV_K(p.K, run_step<__nv_bfloat16, ) }
    KDA_CONV_K(p.K, run_step<float, )
}

}  // namespace kda
