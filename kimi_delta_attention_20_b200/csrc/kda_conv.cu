// Causal depthwise convolution + SiLU over packed sequences (the sequence form of the
// decode token's convolution, page "atlas_core/kimi_k3/kda.rs" `conv_update`), its backward
// pass and its single token:
//     z[t,c] = sum_i w[c,i] in[t-K+1+i, c],   y = z sigmoid(z)
// where a sequence's inputs are preceded by its initial window (K values a channel, oldest
// first, or zeros), and its final window is the last K of both.
//
// Bound by HBM: 4 bytes an element forward, 6 backward (bf16). A warp takes S consecutive
// rows of 128 channels, four a lane, and slides the window down them in registers; the
// K - 1 rows before its own are read again (from L1 or L2: the neighbouring warp's rows).
#include "kda_layer.cuh"

namespace kda {

namespace {

constexpr int kConvWarps = 8, kConvThreads = 32 * kConvWarps;
constexpr int kConvRows = 16;  // rows of a warp

__device__ __forceinline__ float silu_(float z) { return z / (1.f + expf(-z)); }

// The sequence that row `first + at` of the map belongs to, and its first row.
template <int L>
__device__ __forceinline__ void sequence_at(const RowMap<L> &m, int row0, int at, int lane, int &seq, int &start) {
    seq = m.first_seq;
    start = m.first;
    for (int b = at & ~31; b >= 0; b -= 32) {
        const int r = b + lane;
        const unsigned hit = __ballot_sync(0xffffffffu, r <= at && m.start[r] >= 0);
        if (hit) {
            const int s = b + 31 - __clz(hit);
            seq = m.start[s];
            start = row0 + s;
            return;
        }
    }
}

// The lane's weights: w[c, 0..K-1] of its four channels.
template <bool VEC, int K>
__device__ __forceinline__ void load_weights(const float *w, int tile, int lane, int C, float (&wr)[K][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = lane_channel<VEC>(tile, lane, i);
#pragma unroll
        for (int k = 0; k < K; ++k) wr[k][i] = c < C ? w[(long long)c * K + k] : 0.f;
    }
}

// Slot k of sequence n's initial window (zeros where there is none).
template <bool VEC>
__device__ __forceinline__ void window_slot(const float *s0, int n, int k, int K, int tile, int lane, int C, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = lane_channel<VEC>(tile, lane, i);
        v[i] = s0 && c < C ? s0[((long long)n * C + c) * K + k] : 0.f;
    }
}

// win[0..K-2]: the K - 1 inputs before `row` of a sequence that starts at `start`.
template <typename T, bool VEC, int K>
__device__ __forceinline__ void load_window(const T *x, long long stride, const float *s0, int row, int seq, int start,
                                            int tile, int lane, int C, float (&win)[K][4]) {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        const int r = row - (K - 1) + k;
        if (r >= start) {
            const Raw4<T> q = load_row<T, VEC>(x + (long long)r * stride, tile, lane, C, true);
#pragma unroll
            for (int i = 0; i < 4; ++i) win[k][i] = raw_get(q, i);
        } else {
            // inputs `start - r` before the sequence's first sit that far from the window's end
            const int slot = K - (start - r);
            if (slot >= 0) window_slot<VEC>(s0, seq, slot, K, tile, lane, C, win[k]);
            else win[k][0] = win[k][1] = win[k][2] = win[k][3] = 0.f;
        }
    }
}

// ---------------------------------------------------------------- forward
template <typename T, bool VEC, int K>
__global__ void __launch_bounds__(kConvThreads) conv_fwd_kernel(const __grid_constant__ ConvParams p) {
    constexpr int S = kConvRows, L = kConvWarps * S;
    __shared__ RowMap<L> map;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles = (p.C + kTileChannels - 1) / kTileChannels, block = blockIdx.x / tiles;
    const int tile = blockIdx.x - block * tiles, row0 = block * L, wrow = row0 + warp * S, R = p.span.R, C = p.C;
    const T *x = static_cast<const T *>(p.x);

    Raw4<T> xr[S];
#pragma unroll
    for (int s = 0; s < S; ++s)
        xr[s] = load_row<T, VEC>(x + (long long)(wrow + s) * p.x_stride, tile, lane, C, wrow + s < R);
    float w[K][4];
    load_weights<VEC, K>(p.w, tile, lane, C, w);
    // an empty sequence hands its window through
    fill_rows<L>(map, p.span, row0, [&](int n) {
        if (!p.sT) return;
        const long long c0 = ((long long)n * C + tile * kTileChannels) * K, c1 = ((long long)n * C + min(C, (tile + 1) * kTileChannels)) * K;
        for (long long c = c0; c < c1; ++c) p.sT[c] = p.s0 ? p.s0[c] : 0.f;
    });
    if (wrow >= R) return;
    float win[K][4];  // win[K-1]: the row's own input
    int seq, start;
    sequence_at<L>(map, row0, warp * S, lane, seq, start);
    load_window<T, VEC, K>(x, p.x_stride, p.s0, wrow, seq, start, tile, lane, C, win);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int row = wrow + s;
        if (row < R) {
            if (s > 0 && map.start[warp * S + s] >= 0) {
                seq = map.start[warp * S + s];
#pragma unroll
                for (int k = 0; k < K - 1; ++k) window_slot<VEC>(p.s0, seq, k + 1, K, tile, lane, C, win[k]);
            }
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                win[K - 1][i] = raw_get(xr[s], i);
                float z = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) z = fmaf(w[k][i], win[k][i], z);
                y[i] = silu_(z);
            }
            store_row<T, VEC>(static_cast<T *>(p.y) + (long long)row * C, tile, lane, C, y);
            if (p.sT && map.end[warp * S + s] >= 0) {
                float *o = p.sT + (long long)map.end[warp * S + s] * C * K;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = lane_channel<VEC>(tile, lane, i);
                    if (c < C)
#pragma unroll
                        for (int k = 0; k < K; ++k) o[(long long)c * K + k] = win[k][i];
                }
            }
#pragma unroll
            for (int k = 0; k + 1 < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) win[k][i] = win[k + 1][i];
        }
    }
}

// ---------------------------------------------------------------- backward
// dz = dy s (1 + z (1 - s)), s = sigmoid(z);  din[r] = sum_i w[i] dz[r+K-1-i] over the
// sequence's rows;  dw[i] = sum_t dz[t] in[t-K+1+i]. A warp walks its S rows and the K - 1
// behind them (whose dz reaches back into its own), holding the K gradients that are not
// complete yet; input r is complete at row r+K-1 or where its sequence ends. Sums over rows
// go to one slice of dw per CTA and are joined by a second kernel in a fixed order.
template <typename T, bool VEC, int K>
__global__ void __launch_bounds__(kConvThreads) conv_bwd_kernel(const __grid_constant__ ConvBwdParams p) {
    constexpr int S = kConvRows, L = kConvWarps * S;
    __shared__ RowMap<L> map;
    __shared__ float red[kConvWarps][kTileChannels];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles = (p.C + kTileChannels - 1) / kTileChannels, block = blockIdx.x / tiles;
    const int tile = blockIdx.x - block * tiles, row0 = block * L, wrow = row0 + warp * S, R = p.span.R, C = p.C;
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);

    float w[K][4], dw[K][4];
    load_weights<VEC, K>(p.w, tile, lane, C, w);
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k][0] = dw[k][1] = dw[k][2] = dw[k][3] = 0.f;
    // an empty sequence's final window is its initial one
    fill_rows<L>(map, p.span, row0, [&](int n) {
        if (!p.ds0) return;
        const long long c0 = ((long long)n * C + tile * kTileChannels) * K, c1 = ((long long)n * C + min(C, (tile + 1) * kTileChannels)) * K;
        for (long long c = c0; c < c1; ++c) p.ds0[c] = p.dsT ? p.dsT[c] : 0.f;
    });
    if (wrow < R) {
        int seq, start;
        sequence_at<L>(map, row0, warp * S, lane, seq, start);
        float win[K][4], acc[K][4];  // acc[j]: the gradient of input t-K+1+j, so far
        load_window<T, VEC, K>(x, p.x_stride, p.s0, wrow, seq, start, tile, lane, C, win);
#pragma unroll
        for (int k = 0; k < K; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
        int end = p.span.cu ? min(max(p.span.cu[seq + 1], 0), R) : min((seq + 1) * p.span.T, R);
        // input r of the sequence (r < start: its window) is complete with gradient v
        auto finish = [&](int r, float (&v)[4]) {
            if (r >= wrow + S) return;
            if (r >= start ? r < wrow : (start < wrow || !p.ds0 || r < start - K)) return;
            const int slot = r - end + K;  // place in the final window
            if (p.dsT && slot >= 0) {
                float f[4];
                window_slot<VEC>(p.dsT, seq, slot, K, tile, lane, C, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += f[i];
            }
            if (r >= start) {
                store_row<T, VEC>(static_cast<T *>(p.dx) + (long long)r * C, tile, lane, C, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = lane_channel<VEC>(tile, lane, i);
                    if (c < C) p.ds0[((long long)seq * C + c) * K + (r - start + K)] = v[i];
                }
            }
        };
        // the oldest value of the first window of a sequence that starts here is no input of any row
        auto oldest = [&]() {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            finish(start - K, v);
        };
        if (start == wrow) oldest();
        int t = wrow;
        const int stop = min(wrow + S + K - 1, R);
#pragma unroll 1
        for (; t < stop; ++t) {
            if (t == end) {
                // the sequence is over: what it still holds is complete
#pragma unroll
                for (int k = 0; k < K - 1; ++k) finish(t - K + 1 + k, acc[k]);
                if (t >= wrow + S) break;
                seq = map.start[t - row0];
                if (seq < 0) break;  // offsets that do not cover the rows
                start = t;
                end = p.span.cu ? min(max(p.span.cu[seq + 1], 0), R) : min((seq + 1) * p.span.T, R);
                oldest();
#pragma unroll
                for (int k = 0; k < K; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
#pragma unroll
                for (int k = 0; k < K - 1; ++k) window_slot<VEC>(p.s0, seq, k + 1, K, tile, lane, C, win[k]);
            }
            const Raw4<T> xr = load_row<T, VEC>(x + (long long)t * p.x_stride, tile, lane, C, true);
            const Raw4<T> dr = load_row<T, VEC>(dy + (long long)t * p.dy_stride, tile, lane, C, true);
            const bool own = t < wrow + S;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                win[K - 1][i] = raw_get(xr, i);
                float z = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) z = fmaf(w[k][i], win[k][i], z);
                const float sg = 1.f / (1.f + expf(-z));
                const float dz = raw_get(dr, i) * sg * fmaf(z, 1.f - sg, 1.f);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    acc[k][i] = fmaf(w[k][i], dz, acc[k][i]);
                    if (own) dw[k][i] = fmaf(dz, win[k][i], dw[k][i]);
                }
            }
            finish(t - K + 1, acc[0]);
#pragma unroll
            for (int k = 0; k + 1 < K; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) { acc[k][i] = acc[k + 1][i]; win[k][i] = win[k + 1][i]; }
            acc[K - 1][0] = acc[K - 1][1] = acc[K - 1][2] = acc[K - 1][3] = 0.f;
        }
        // the last row of all: nothing follows
        if (t == R && t == end && t < wrow + S + K - 1)
#pragma unroll
            for (int k = 0; k < K - 1; ++k) finish(t - K + 1 + k, acc[k]);
    }
    if (!p.partial) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][lane_channel<VEC>(0, lane, i)] = dw[k][i];
        __syncthreads();
        const int c = threadIdx.x;
        if (c < kTileChannels && tile * kTileChannels + c < C) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < kConvWarps; ++j) s += red[j][c];
            p.partial[((long long)block * K + k) * C + tile * kTileChannels + c] = s;
        }
    }
}

// dw[c, k]: the sum of its slices. One warp column of 32 channels, the slices shared out
// over the CTA's warps and joined in a fixed order.
__global__ void __launch_bounds__(256) conv_dw_kernel(const float *partial, float *dw, int slices, int C, int K) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
    float s = 0.f;
    if (c < C)
        for (int j = warp; j < slices; j += 8) s += partial[((long long)j * K + k) * C + c];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < C) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) v += red[j][lane];
        dw[(long long)c * K + k] = v;
    }
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
    static_cast<T *>(p.y)[i] = from_f32<T>(silu_(z));
}

// ---------------------------------------------------------------- host
bool vec_ok(const void *p, long long stride, size_t esz) {
    return !p || (reinterpret_cast<uintptr_t>(p) % (4 * esz) == 0 && stride % 4 == 0);
}

// Blocks of rows, and CTAs: one for each block and channel tile.
long long conv_blocks(int rows) {
    const int L = kConvWarps * kConvRows;
    return rows > L ? (rows + L - 1) / L : 1;
}
long long conv_ctas(int rows, int C) { return conv_blocks(rows) * ((C + kTileChannels - 1) / kTileChannels); }

template <typename T, bool VEC, int K> cudaError_t run_fwd(const ConvParams &p, cudaStream_t st) {
    count_launch();
    conv_fwd_kernel<T, VEC, K><<<(unsigned)conv_ctas(p.span.R, p.C), kConvThreads, 0, st>>>(p);
    return cudaGetLastError();
}
template <typename T, bool VEC, int K> cudaError_t run_bwd(const ConvBwdParams &p, cudaStream_t st) {
    count_launch();
    conv_bwd_kernel<T, VEC, K><<<(unsigned)conv_ctas(p.span.R, p.C), kConvThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.dw) return e;
    count_launch();
    conv_dw_kernel<<<dim3((p.C + 31) / 32, K), 256, 0, st>>>(p.partial, p.dw, (int)conv_blocks(p.span.R), p.C, K);
    return cudaGetLastError();
}
template <typename T, bool VEC, int K> cudaError_t run_step(const ConvStepParams &p, cudaStream_t st) {
    const long long n = (long long)p.N * p.C;
    count_launch();
    conv_step_kernel<T, K><<<(unsigned)((n + 127) / 128), 128, 0, st>>>(p);
    return cudaGetLastError();
}

// Runs F<T, VEC, K> for the type, layout and window of a call.
#define KDA_CONV_K(F, T, V, p, st)                                                                     \
    switch (p.K) {                                                                                     \
    case 1: return F<T, V, 1>(p, st); case 2: return F<T, V, 2>(p, st); case 3: return F<T, V, 3>(p, st); \
    case 4: return F<T, V, 4>(p, st); case 5: return F<T, V, 5>(p, st); case 6: return F<T, V, 6>(p, st); \
    case 7: return F<T, V, 7>(p, st); case 8: return F<T, V, 8>(p, st);                                \
    }                                                                                                  \
    return cudaErrorInvalidValue;
#define KDA_CONV_PICK(F, p, bf16, vec, st)                                                             \
    if (bf16) { if (vec) { KDA_CONV_K(F, __nv_bfloat16, true, p, st) } else { KDA_CONV_K(F, __nv_bfloat16, false, p, st) } } \
    if (vec) { KDA_CONV_K(F, float, true, p, st) } else { KDA_CONV_K(F, float, false, p, st) }

}  // namespace

size_t conv_bwd_workspace_bytes(int rows, int C, int K) {
    return sizeof(float) * (size_t)conv_blocks(rows) * C * K;
}

cudaError_t launch_conv(const ConvParams &p, bool bf16, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4;
    const bool vec = p.C % 4 == 0 && vec_ok(p.x, p.x_stride, esz) && vec_ok(p.y, p.C, esz);
    if (conv_ctas(p.span.R, p.C) > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    KDA_CONV_PICK(run_fwd, p, bf16, vec, st)
}

cudaError_t launch_conv_bwd(const ConvBwdParams &p, bool bf16, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4;
    const bool vec = p.C % 4 == 0 && vec_ok(p.x, p.x_stride, esz) && vec_ok(p.dy, p.dy_stride, esz) && vec_ok(p.dx, p.C, esz);
    if (conv_ctas(p.span.R, p.C) > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    KDA_CONV_PICK(run_bwd, p, bf16, vec, st)
}

cudaError_t launch_conv_step(const ConvStepParams &p, bool bf16, cudaStream_t st) {
    if (bf16) { KDA_CONV_K(run_step, __nv_bfloat16, true, p, st) }
    KDA_CONV_K(run_step, float, true, p, st)
}

}  // namespace kda
