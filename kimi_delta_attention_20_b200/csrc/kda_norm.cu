// Root-mean-square norm of rows, as a layer uses it: with the residual's addition, with
// the sigmoid output gate (page "atlas_core/kimi_k3/kda.rs", `full_rank_output_gate`), with
// the output in 8 bits, and the backward pass:
//     s = x (+ residual),  r = 1 / sqrt(mean s^2 + eps),  y = s r w sigmoid(gate)
//     8 bits: per group of channels scale = max |y| / 448 (at least 2^-100; the next power
//     of two on request) and e4m3(y / scale)
//     with u = dy w sigmoid(gate): dx = r (u - s r^2 mean(u s)) + dresidual,
//     dgate = dy s r w sigmoid'(gate),  dw = sum over rows of dy s r sigmoid(gate)
//
// Bound by HBM: every tensor passes once, the row stays in registers between the sum of
// squares and the output. A row belongs to TPR threads (part of a warp for heads, up to a
// CTA for layers), each with NU runs of eight channels. The sum x + residual is rounded
// to its type for `residual_out` alone: the norm is taken of the fp32 sum.
#include <cuda_fp8.h>

#include "kda_layer.cuh"

namespace kda {

namespace {

constexpr int kRun = 8;          // channels of a run
constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100: keeps y / scale finite

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Eight neighbouring channels from column c on; beyond D they read as zero. VEC: the row
// is 16-byte aligned and D a multiple of eight.
template <typename T, bool VEC>
__device__ __forceinline__ void load_run(const T *row, int c, int D, float (&v)[kRun]) {
    if (VEC) {
        if (c >= D) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) v[i] = 0.f;
        } else if (sizeof(T) == 2) {
            const uint4 q = *reinterpret_cast<const uint4 *>(row + c);
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        } else {
            const float4 a = reinterpret_cast<const float4 *>(row + c)[0], b = reinterpret_cast<const float4 *>(row + c)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) v[i] = c + i < D ? to_f32(row[c + i]) : 0.f;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_run(T *row, int c, int D, const float (&v)[kRun]) {
    if (VEC) {
        if (c >= D) return;
        if (sizeof(T) == 2) {
            *reinterpret_cast<uint4 *>(row + c) =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        } else {
            reinterpret_cast<float4 *>(row + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(row + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i)
        if (c + i < D) row[c + i] = from_f32<T>(v[i]);
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

template <bool VEC> __device__ __forceinline__ void store_e4m3(uint8_t *row, int c, int D, const float (&v)[kRun]) {
    if (c >= D) return;
    const uint32_t a = e4m3_pair(v[0], v[1]) | e4m3_pair(v[2], v[3]) << 16, b = e4m3_pair(v[4], v[5]) | e4m3_pair(v[6], v[7]) << 16;
    if (VEC) {
        *reinterpret_cast<uint2 *>(row + c) = make_uint2(a, b);
        return;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i)
        if (c + i < D) row[c + i] = (uint8_t)((i < 4 ? a >> 8 * i : b >> 8 * (i - 4)) & 0xffu);
}

// The channels' weights, of either type; 1 without weights.
template <typename T, bool VEC>
__device__ __forceinline__ void load_weight(const void *w, int f32, int c, int D, float (&v)[kRun]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < kRun; ++i) v[i] = 1.f;
    } else if (f32) {
        load_run<float, VEC>(static_cast<const float *>(w), c, D, v);
    } else {
        load_run<T, VEC>(static_cast<const T *>(w), c, D, v);
    }
}

// A sum (maximum) over the TPR threads of a row; the result in all of them. red: one
// float per warp of the CTA where rows span warps, free to be written.
template <int TPR, bool MAX> __device__ __forceinline__ float row_reduce(float v, float *red) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? max_nan(v, u) : v + u;
    }
    if (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        const float *own = red + threadIdx.x / TPR * (TPR / 32);  // this row's warps
        v = own[0];
#pragma unroll
        for (int w = 1; w < TPR / 32; ++w) v = MAX ? max_nan(v, own[w]) : v + own[w];
    }
    return v;
}

template <int TPR> constexpr int norm_threads() { return TPR > 128 ? TPR : 128; }
// Floats that row_reduce needs.
template <int TPR> constexpr int norm_red() { return TPR > 32 ? norm_threads<TPR>() / 32 : 1; }

// ---------------------------------------------------------------- forward
template <typename T, bool VEC, int TPR, int NU>
__global__ void __launch_bounds__(norm_threads<TPR>()) norm_fwd_kernel(const __grid_constant__ NormParams p) {
    constexpr int ROWS = norm_threads<TPR>() / TPR;
    __shared__ float red[2][norm_red<TPR>()];
    const int t = threadIdx.x % TPR, D = p.D;
    const long long row = (long long)blockIdx.x * ROWS + threadIdx.x / TPR;
    const bool ok = row < p.rows;  // threads without a row take part in the reductions
    const long long r = ok ? row : 0;
    const T *x = static_cast<const T *>(p.x) + r * p.x_stride;

    float s[NU][kRun], ss = 0.f;
#pragma unroll
    for (int u = 0; u < NU; ++u) load_run<T, VEC>(x, (u * TPR + t) * kRun, D, s[u]);
    if (p.residual) {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            float q[kRun];
            load_run<T, VEC>(static_cast<const T *>(p.residual) + r * p.residual_stride, (u * TPR + t) * kRun, D, q);
#pragma unroll
            for (int i = 0; i < kRun; ++i) s[u][i] += q[i];
        }
    }
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < kRun; ++i) ss = fmaf(s[u][i], s[u][i], ss);
    if (p.residual_out && ok)
#pragma unroll
        for (int u = 0; u < NU; ++u) store_run<T, VEC>(static_cast<T *>(p.residual_out) + row * D, (u * TPR + t) * kRun, D, s[u]);
    ss = row_reduce<TPR, false>(ss, red[0]);
    const float inv = 1.f / sqrtf(ss / D + p.eps);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int c = (u * TPR + t) * kRun;
        float w[kRun];
        load_weight<T, VEC>(p.weight, p.weight_f32, c, D, w);
#pragma unroll
        for (int i = 0; i < kRun; ++i) s[u][i] = s[u][i] * inv * w[i];
        if (p.gate) {
            float q[kRun];
            load_run<T, VEC>(static_cast<const T *>(p.gate) + r * p.gate_stride, c, D, q);
#pragma unroll
            for (int i = 0; i < kRun; ++i) s[u][i] /= 1.f + expf(-q[i]);
        }
    }
    if (!p.scales) {
        if (ok)
#pragma unroll
            for (int u = 0; u < NU; ++u) store_run<T, VEC>(static_cast<T *>(p.y) + row * D, (u * TPR + t) * kRun, D, s[u]);
        return;
    }
    float top[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        top[u] = 0.f;
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if ((u * TPR + t) * kRun + i < D) top[u] = max_nan(top[u], fabsf(s[u][i]));
    }
    const bool whole = p.group >= D;
    if (whole) {
#pragma unroll
        for (int u = 1; u < NU; ++u) top[0] = max_nan(top[0], top[u]);
        top[0] = row_reduce<TPR, true>(top[0], red[1]);
#pragma unroll
        for (int u = 1; u < NU; ++u) top[u] = top[0];
    } else {
        // groups of 32, 64 or 128 channels are 4, 8 or 16 neighbouring threads, which lie in one warp
#pragma unroll
        for (int u = 0; u < NU; ++u)
            for (int o = p.group / kRun / 2; o > 0; o >>= 1) top[u] = max_nan(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
    }
    const int groups = whole ? 1 : (D + p.group - 1) / p.group;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int c = (u * TPR + t) * kRun;
        float scale = max_nan(top[u] / kE4m3Max, kScaleFloor);
        if (p.pow2) {
            // the next power of two: the exponent, one more unless the mantissa is zero
            const uint32_t b = __float_as_uint(scale);
            if ((b & 0x7f800000u) != 0x7f800000u) scale = __uint_as_float((b + 0x007fffffu) & 0x7f800000u);
        }
        const float to = 1.f / scale;
        float q[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) q[i] = s[u][i] * to;
        if (ok) {
            store_e4m3<VEC>(static_cast<uint8_t *>(p.y) + row * D, c, D, q);
            if (c < D && c % (whole ? (1 << 30) : p.group) == 0) p.scales[row * groups + (whole ? 0 : c / p.group)] = scale;
        }
    }
}

// ---------------------------------------------------------------- backward
// CTAs walk rows; a thread's channels stay the same, so the weights and the sums for dw
// stay in registers and leave once, as one slice of dw per CTA.
template <typename T, bool VEC, int TPR, int NU>
__global__ void __launch_bounds__(norm_threads<TPR>()) norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
    constexpr int NT = norm_threads<TPR>(), ROWS = NT / TPR;
    __shared__ float red[2][2][norm_red<TPR>()];
    __shared__ float slice[ROWS > 1 ? ROWS * TPR * kRun : 1];
    const int t = threadIdx.x % TPR, lr = threadIdx.x / TPR, D = p.D;
    float w[NU][kRun], dw[NU][kRun];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        load_weight<T, VEC>(p.weight, p.weight_f32, (u * TPR + t) * kRun, D, w[u]);
#pragma unroll
        for (int i = 0; i < kRun; ++i) dw[u][i] = 0.f;
    }
    int flip = 0;
    for (long long base = (long long)blockIdx.x * ROWS; base < p.rows; base += (long long)gridDim.x * ROWS, flip ^= 1) {
        const long long row = base + lr;
        const bool ok = row < p.rows;
        const long long r = ok ? row : 0;
        float s[NU][kRun], d[NU][kRun], g[NU][kRun], ss = 0.f, us = 0.f;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c = (u * TPR + t) * kRun;
            load_run<T, VEC>(static_cast<const T *>(p.x) + r * p.x_stride, c, D, s[u]);
            load_run<T, VEC>(static_cast<const T *>(p.dy) + r * p.dy_stride, c, D, d[u]);
            if (p.gate) load_run<T, VEC>(static_cast<const T *>(p.gate) + r * p.gate_stride, c, D, g[u]);
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                const float sg = p.gate ? 1.f / (1.f + expf(-g[u][i])) : 1.f;
                g[u][i] = sg;
                ss = fmaf(s[u][i], s[u][i], ss);
                us = fmaf(d[u][i] * sg * w[u][i], s[u][i], us);
            }
#pragma unroll
        for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            us += __shfl_xor_sync(0xffffffffu, us, o);
        }
        if (TPR > 32) {
            // two buffers in turn: one barrier a row
            const int warp = threadIdx.x >> 5, own = lr * (TPR / 32);
            if ((threadIdx.x & 31) == 0) { red[flip][0][warp] = ss; red[flip][1][warp] = us; }
            __syncthreads();
            ss = red[flip][0][own];
            us = red[flip][1][own];
#pragma unroll
            for (int v = 1; v < TPR / 32; ++v) { ss += red[flip][0][own + v]; us += red[flip][1][own + v]; }
        }
        const float inv = 1.f / sqrtf(ss / D + p.eps), k = us / D * inv * inv;
        if (!ok) continue;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int c = (u * TPR + t) * kRun;
            float o[kRun], q[kRun];
            if (p.dresidual) load_run<T, VEC>(static_cast<const T *>(p.dresidual) + row * p.dresidual_stride, c, D, q);
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                const float n = s[u][i] * inv, e = d[u][i] * g[u][i];
                dw[u][i] = fmaf(e, n, dw[u][i]);
                o[i] = inv * (e * w[u][i] - s[u][i] * k) + (p.dresidual ? q[i] : 0.f);
                d[u][i] = e * n * w[u][i] * (1.f - g[u][i]);
            }
            store_run<T, VEC>(static_cast<T *>(p.dx) + row * D, c, D, o);
            if (p.gate) store_run<T, VEC>(static_cast<T *>(p.dgate) + row * D, c, D, d[u]);
        }
    }
    if (!p.partial) return;
    float *out = p.partial + (long long)blockIdx.x * D;
    if (ROWS > 1) {
        // NU is 1: the rows of the CTA are joined in their order
#pragma unroll
        for (int i = 0; i < kRun; ++i) slice[(lr * TPR + t) * kRun + i] = dw[0][i];
        __syncthreads();
        for (int c = threadIdx.x; c < TPR * kRun && c < D; c += NT) {
            float v = 0.f;
            for (int j = 0; j < ROWS; ++j) v += slice[j * TPR * kRun + c];
            out[c] = v;
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int c = (u * TPR + t) * kRun;
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            if (c + i < D) out[c + i] = dw[u][i];
    }
}

// dw: the sum of its slices, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(256) norm_dw_kernel(const float *partial, void *dw, int f32, int slices, int D) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < D)
        for (int j = warp; j < slices; j += 8) s += partial[(long long)j * D + c];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < D) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) v += red[j][lane];
        if (f32) static_cast<float *>(dw)[c] = v;
        else static_cast<T *>(dw)[c] = from_f32<T>(v);
    }
}

// ---------------------------------------------------------------- host
bool vec_ok(const void *p, long long stride, size_t esz) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * (long long)esz % 16 == 0);
}

// Threads per row and runs per thread: the row's runs of eight channels, one to a thread up
// to 512 threads.
struct NormShape { int tpr, nu; };
NormShape norm_shape(int D) {
    const int runs = (D + kRun - 1) / kRun;
    int tpr = 4;
    while (tpr < runs && tpr < 512) tpr *= 2;
    return {tpr, runs <= tpr ? 1 : runs <= 2 * tpr ? 2 : 4};
}

int norm_rows_per_cta(int tpr) { return tpr >= 128 ? 1 : 128 / tpr; }

// CTAs of the backward: each walks its share of the rows.
int norm_bwd_ctas(long long rows, int D) {
    const NormShape s = norm_shape(D);
    const long long need = (rows + norm_rows_per_cta(s.tpr) - 1) / norm_rows_per_cta(s.tpr);
    const long long most = 148LL * (s.tpr > 256 ? 2 : s.tpr > 128 ? 4 : 8);
    return (int)(need < most ? need : most);
}

template <typename T, bool VEC, int TPR, int NU> struct Fwd {
    static cudaError_t run(const NormParams &p, cudaStream_t st) {
        const long long ctas = (p.rows + norm_rows_per_cta(TPR) - 1) / norm_rows_per_cta(TPR);
        if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        count_launch();
        norm_fwd_kernel<T, VEC, TPR, NU><<<(unsigned)ctas, norm_threads<TPR>(), 0, st>>>(p);
        return cudaGetLastError();
    }
};
template <typename T, bool VEC, int TPR, int NU> struct Bwd {
    static cudaError_t run(const NormBwdParams &p, cudaStream_t st) {
        const int ctas = norm_bwd_ctas(p.rows, p.D);
        count_launch();
        norm_bwd_kernel<T, VEC, TPR, NU><<<ctas, norm_threads<TPR>(), 0, st>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || !p.dweight) return e;
        count_launch();
        norm_dw_kernel<T><<<(p.D + 31) / 32, 256, 0, st>>>(p.partial, p.dweight, p.weight_f32, ctas, p.D);
        return cudaGetLastError();
    }
};

template <template <typename, bool, int, int> class F, typename T, bool VEC, typename P>
cudaError_t pick(const P &p, cudaStream_t st) {
    const NormShape s = norm_shape(p.D);
    switch (s.tpr) {
    case 4: return F<T, VEC, 4, 1>::run(p, st);
    case 8: return F<T, VEC, 8, 1>::run(p, st);
    case 16: return F<T, VEC, 16, 1>::run(p, st);
    case 32: return F<T, VEC, 32, 1>::run(p, st);
    case 64: return F<T, VEC, 64, 1>::run(p, st);
    case 128: return F<T, VEC, 128, 1>::run(p, st);
    case 256: return F<T, VEC, 256, 1>::run(p, st);
    }
    if (s.nu == 1) return F<T, VEC, 512, 1>::run(p, st);
    if (s.nu == 2) return F<T, VEC, 512, 2>::run(p, st);
    return F<T, VEC, 512, 4>::run(p, st);
}

}  // namespace

size_t rms_norm_bwd_workspace_bytes(long long rows, int D, bool, bool weight) {
    return weight ? sizeof(float) * (size_t)norm_bwd_ctas(rows, D) * D : 0;
}

cudaError_t launch_rms_norm(const NormParams &p, bool bf16, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4, wsz = p.weight_f32 ? 4 : esz;
    const bool vec = p.D % kRun == 0 && vec_ok(p.x, p.x_stride, esz) && vec_ok(p.residual, p.residual_stride, esz) &&
                     vec_ok(p.gate, p.gate_stride, esz) && vec_ok(p.weight, p.D, wsz) && vec_ok(p.y, p.D, 2) &&
                     vec_ok(p.residual_out, p.D, esz);
    if (bf16) return vec ? pick<Fwd, __nv_bfloat16, true>(p, st) : pick<Fwd, __nv_bfloat16, false>(p, st);
    return vec ? pick<Fwd, float, true>(p, st) : pick<Fwd, float, false>(p, st);
}

cudaError_t launch_rms_norm_bwd(const NormBwdParams &p, bool bf16, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4, wsz = p.weight_f32 ? 4 : esz;
    const bool vec = p.D % kRun == 0 && vec_ok(p.x, p.x_stride, esz) && vec_ok(p.dy, p.dy_stride, esz) &&
                     vec_ok(p.gate, p.gate_stride, esz) && vec_ok(p.dresidual, p.dresidual_stride, esz) &&
                     vec_ok(p.weight, p.D, wsz) && vec_ok(p.dx, p.D, esz) && vec_ok(p.dgate, p.D, esz);
    if (bf16) return vec ? pick<Bwd, __nv_bfloat16, true>(p, st) : pick<Bwd, __nv_bfloat16, false>(p, st);
    return vec ? pick<Bwd, float, true>(p, st) : pick<Bwd, float, false>(p, st);
}

}  // namespace kda
