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
// squares and the output (786432 x 128 gated 105 us a call, 5.8 TB/s; 16384 x 4096 with residual
// to 8 bits 92 us, 5.1 TB/s, where conversions and the quotient's rounding take issue too, 61 %
// of the slots). A row belongs to TPR threads (part of a warp for heads, up to a CTA for
// layers), each with NU runs of eight channels. The sum x + residual is rounded to its type for
// `residual_out` alone: the norm is taken of the fp32 sum.
#pragma once

#include <cuda_fp8.h>

#include "kda_layer.cuh"

namespace kda {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100: keeps y / scale finite

// A thread reaches its channels by accesses of G bytes, P channels each: access q holds
// channels (q TPR + t) P and on, so that neighbouring threads touch neighbouring bytes for
// every G (16 where all rows are aligned to it, else 4, or 2 for odd bf16 rows).
template <typename T, int G> constexpr int access_channels() { return G / (int)sizeof(T); }

template <int G> struct Bits {  // an access as stored
    uint32_t w[G < 4 ? 1 : G / 4];
};
template <typename T, int G> __device__ __forceinline__ Bits<G> fetch(const T *row, int c, bool ok) {
    Bits<G> q;
    if constexpr (G == 16) reinterpret_cast<uint4 &>(q) = ok ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0u, 0u, 0u, 0u);
    else if constexpr (G == 4) q.w[0] = ok ? *reinterpret_cast<const uint32_t *>(row + c) : 0u;
    else q.w[0] = ok ? (uint32_t)*reinterpret_cast<const unsigned short *>(row + c) : 0u;
    return q;
}
template <typename T, int G> __device__ __forceinline__ void widen(const Bits<G> &q, float *v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < G / 4; ++i) v[i] = __uint_as_float(q.w[i]);
    } else if constexpr (G == 2) {
        v[0] = __uint_as_float(q.w[0] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < G / 4; ++i) {
            v[2 * i] = __uint_as_float(q.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(q.w[i] & 0xffff0000u);
        }
    }
}
template <typename T, int G> __device__ __forceinline__ void load_access(const T *row, int c, int D, float *v) {
    widen<T, G>(fetch<T, G>(row, c, c < D), v);
}
template <typename T, int G> __device__ __forceinline__ void store_access(T *row, int c, int D, const float *v) {
    constexpr int P = access_channels<T, G>();
    if (c >= D) return;
    if constexpr (G == 16 && sizeof(T) == 2)
        *reinterpret_cast<uint4 *>(row + c) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    else if constexpr (G == 16)
        *reinterpret_cast<float4 *>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
    else if constexpr (P == 2)
        *reinterpret_cast<uint32_t *>(row + c) = pack_bf16(v[0], v[1]);
    else
        row[c] = from_f32<T>(v[0]);
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
template <int P, bool VEC> __device__ __forceinline__ void store_e4m3(uint8_t *row, int c, int D, const float *v) {
    if (c >= D) return;
    if constexpr (VEC && P == 8) {
        *reinterpret_cast<uint2 *>(row + c) = make_uint2(e4m3_pair(v[0], v[1]) | e4m3_pair(v[2], v[3]) << 16, e4m3_pair(v[4], v[5]) | e4m3_pair(v[6], v[7]) << 16);
    } else if constexpr (VEC && P == 4) {
        *reinterpret_cast<uint32_t *>(row + c) = e4m3_pair(v[0], v[1]) | e4m3_pair(v[2], v[3]) << 16;
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) row[c + i] = (uint8_t)(e4m3_pair(v[i], 0.f) & 0xffu);
    }
}

// The channels' weights, of either type; 1 without weights.
template <typename T, int G> __device__ __forceinline__ void load_weight(const void *w, int f32, int c, int D, float *v) {
    constexpr int P = access_channels<T, G>();
    if (!w) {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = 1.f;
    } else if (!f32) {
        load_access<T, G>(static_cast<const T *>(w), c, D, v);
    } else if constexpr (G == 16) {
#pragma unroll
        for (int i = 0; i < P; i += 4) load_access<float, 16>(static_cast<const float *>(w), c + i, D, v + i);
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = c + i < D ? static_cast<const float *>(w)[c + i] : 0.f;
    }
}

template <int TPR> constexpr int norm_threads() { return TPR > 128 ? TPR : 128; }
// Floats that a reduction over rows that span warps needs.
template <int TPR> constexpr int norm_red() { return TPR > 32 ? norm_threads<TPR>() / 32 : 1; }

// Sums (maxima) of N values over the TPR threads of a row; the results in all of them. red:
// free to be written.
template <int TPR, bool MAX, int N, int M> __device__ __forceinline__ void row_reduce(float (&v)[N], float (&red)[N][M]) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float u = __shfl_xor_sync(0xffffffffu, v[n], o);
            v[n] = MAX ? max_nan(v[n], u) : v[n] + u;
        }
    if constexpr (TPR > 32) {
        const int own = threadIdx.x / TPR * (TPR / 32);  // this row's warps
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) red[n][threadIdx.x >> 5] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = red[n][own];
#pragma unroll
            for (int w = 1; w < TPR / 32; ++w) v[n] = MAX ? max_nan(v[n], red[n][own + w]) : v[n] + red[n][own + w];
        }
    }
}

// The scale of a group whose largest magnitude is `top`.
__device__ __forceinline__ float group_scale(float top, int pow2) {
    float scale = max_nan(top / kE4m3Max, kScaleFloor);
    if (pow2) {
        // the next power of two: the exponent, one more unless the mantissa is zero
        const uint32_t b = __float_as_uint(scale);
        if ((b & 0x7f800000u) != 0x7f800000u) scale = __uint_as_float((b + 0x007fffffu) & 0x7f800000u);
    }
    return scale;
}

// A row's accesses of a thread, as stored; zeros without the row.
template <typename T, int G, int TPR, int NA>
__device__ __forceinline__ void fetch_row(const NormRows &rows, long long row, bool ok, int t, int D, Bits<G> (&q)[NA]) {
    constexpr int P = access_channels<T, G>();
    long long at = row * rows.stride;
    if (rows.heads > 1) {  // 32-bit row numbers, see the entry points
        const unsigned token = (unsigned)row / (unsigned)rows.heads;
        at = token * rows.stride + (long long)((unsigned)row - token * rows.heads) * D;
    }
    const T *r = static_cast<const T *>(rows.at) + at;
#pragma unroll
    for (int i = 0; i < NA; ++i) q[i] = fetch<T, G>(r, (i * TPR + t) * P, ok && (i * TPR + t) * P < D);
}

// CTAs walk rows; a thread's channels stay the same. The next row's accesses are under way
// while a row is worked on, so that memory is kept busy whatever the row's barriers and
// reductions take. Registers of a thread, and so CTAs an SM:
constexpr int norm_regs(bool backward, int nu) { return backward ? (nu == 1 ? 96 : 168) : (nu == 1 ? 64 : nu == 2 ? 80 : 128); }
constexpr int norm_resident(bool backward, int tpr, int nu) {
    const int threads = tpr > 128 ? tpr : 128, n = 65536 / (norm_regs(backward, nu) * threads);
    return n > 0 ? n : 1;
}

// ---------------------------------------------------------------- host
// Threads per row and runs of eight channels per thread. Where rows fill the GPU, several
// runs a thread from 257 channels on: more bytes in flight and fewer barriers. Four in the
// forward of bf16 rows with 16-byte accesses (16384 x 4096 to 8 bits: 85 us, 89 with two),
// two elsewhere, where four take too many registers (16384 x 1023: 52 us with two, 74 with
// four). Few rows are spread over as many threads as they have runs, which shortens each.
struct NormShape { int tpr, nu; };
inline NormShape norm_shape(int D, int nu) {
    const int runs = (D + 7) / 8;
    int tpr = 4;
    while (tpr * nu < runs && tpr < 512) tpr *= 2;
    while (tpr * nu < runs) nu *= 2;
    return {tpr, nu};
}
constexpr int fwd_runs(bool bf16, int g) { return bf16 && g == 16 ? 4 : 2; }
inline NormShape fwd_shape(long long rows, int D, bool bf16, int g) { return norm_shape(D, rows >= 592 && D > 256 ? fwd_runs(bf16, g) : 1); }
inline NormShape bwd_shape(long long rows, int D) { return norm_shape(D, rows >= 592 && D > 256 ? 2 : 1); }

inline int rows_per_cta(int tpr) { return tpr >= 128 ? 1 : 128 / tpr; }

// CTAs: as many as run at a time, each walking its share of the rows.
inline int norm_ctas(long long rows, NormShape s, bool backward) {
    const long long need = (rows + rows_per_cta(s.tpr) - 1) / rows_per_cta(s.tpr), most = 148LL * norm_resident(backward, s.tpr, s.nu);
    return (int)(need < most ? need : most);
}

// The access that the forward's inputs and the sum allow.
inline RowAccess norm_access(const NormParams &p, bool bf16) {
    const size_t esz = bf16 ? 2 : 4;
    RowAccess ac;
    for (const NormRows *r : {&p.x, &p.residual, &p.gate}) ac.rows(r->at, r->stride, p.D, esz);
    ac.rows(p.weight, p.D, p.D, p.weight_f32 ? 4 : esz);
    ac.rows(p.residual_out, p.D, p.D, esz);
    return ac;
}

// Runs F<T, G, threads per row, runs per thread>::run; NU: the runs that `s` has where it
// has more than one (rows of over 4096 NU channels take what they need).
template <template <typename, int, int, int> class F, int NU, typename T, int G, typename P>
cudaError_t pick_shape(const P &p, NormShape s, cudaStream_t st) {
    if (s.nu == 1) {
        switch (s.tpr) {
        case 4: return F<T, G, 4, 1>::run(p, st);
        case 8: return F<T, G, 8, 1>::run(p, st);
        case 16: return F<T, G, 16, 1>::run(p, st);
        case 32: return F<T, G, 32, 1>::run(p, st);
        case 64: return F<T, G, 64, 1>::run(p, st);
        case 128: return F<T, G, 128, 1>::run(p, st);
        case 256: return F<T, G, 256, 1>::run(p, st);
        }
        return F<T, G, 512, 1>::run(p, st);
    }
    if (s.tpr < 512) {
        switch (s.tpr) {
        case 16: if constexpr (NU == 4) return F<T, G, 16, NU>::run(p, st); break;
        case 32: return F<T, G, 32, NU>::run(p, st);
        case 64: return F<T, G, 64, NU>::run(p, st);
        case 128: return F<T, G, 128, NU>::run(p, st);
        case 256: return F<T, G, 256, NU>::run(p, st);
        }
    }
    return s.nu == 2 ? F<T, G, 512, 2>::run(p, st) : F<T, G, 512, 4>::run(p, st);
}

template <template <typename, int, int, int> class F, bool BACKWARD, typename P>
cudaError_t pick(const P &p, bool bf16, int g, cudaStream_t st) {
    g = g >= 16 ? 16 : g >= 4 || !bf16 ? 4 : 2;
    const NormShape s = BACKWARD ? bwd_shape(p.rows, p.D) : fwd_shape(p.rows, p.D, bf16, g);
    if (bf16) {
        if (g == 16) return pick_shape<F, BACKWARD ? 2 : fwd_runs(true, 16), __nv_bfloat16, 16>(p, s, st);
        if (g == 4) return pick_shape<F, 2, __nv_bfloat16, 4>(p, s, st);
        return pick_shape<F, 2, __nv_bfloat16, 2>(p, s, st);
    }
    if (g == 16) return pick_shape<F, 2, float, 16>(p, s, st);
    return pick_shape<F, 2, float, 4>(p, s, st);
}

}  // namespace

}  // namespace kda
