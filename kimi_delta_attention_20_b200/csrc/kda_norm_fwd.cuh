// The forward kernel of the RMS norm (see kda_norm.cuh), for the two files that hold its
// instances: rows in the activations' type, and in 8 bits.
#pragma once

#include "kda_norm.cuh"

namespace kda {

namespace {

// ---------------------------------------------------------------- forward
enum : int { kPlain = 0, kResidual = 1, kGate = 2 };

template <typename T, int G, int TPR, int NU, int MODE, bool QUANT>
__global__ void __launch_bounds__(norm_threads<TPR>(), norm_resident(false, TPR, NU)) norm_fwd_kernel(const __grid_constant__ NormParams p) {
    constexpr int NT = norm_threads<TPR>(), ROWS = NT / TPR, P = access_channels<T, G>(), NA = 8 * NU / P;
    __shared__ float red[2][2][1][norm_red<TPR>()];
    const int t = threadIdx.x % TPR, lr = threadIdx.x / TPR, D = p.D;
    const float per = 1.f / D;
    const NormRows &other = MODE == kResidual ? p.residual : p.gate;
    const long long step = (long long)gridDim.x * ROWS;
    long long row = (long long)blockIdx.x * ROWS + lr;
    Bits<G> bx[NA], bo[NA];
    fetch_row<T, G, TPR, NA>(p.x, row, row < p.rows, t, D, bx);
    if (MODE != kPlain) fetch_row<T, G, TPR, NA>(other, row, row < p.rows, t, D, bo);
    int flip = 0;  // two buffers in turn: one barrier a reduction
    for (long long base = row - lr; base < p.rows; base += step, row += step, flip ^= 1) {
        const bool ok = row < p.rows;  // threads without a row take part in the reductions
        float s[8 * NU], ss[1] = {0.f};
        Bits<G> cur[NA];
#pragma unroll
        for (int q = 0; q < NA; ++q) {
            widen<T, G>(bx[q], s + q * P);
            cur[q] = bo[q];
        }
        fetch_row<T, G, TPR, NA>(p.x, row + step, row + step < p.rows, t, D, bx);
        if (MODE != kPlain) fetch_row<T, G, TPR, NA>(other, row + step, row + step < p.rows, t, D, bo);
        if (MODE == kResidual)
#pragma unroll
            for (int q = 0; q < NA; ++q) {
                float v[P];
                widen<T, G>(cur[q], v);
#pragma unroll
                for (int i = 0; i < P; ++i) s[q * P + i] += v[i];
            }
        float odd = 0.f;
#pragma unroll
        for (int i = 0; i < 8 * NU; i += 2) {
            ss[0] = fmaf(s[i], s[i], ss[0]);
            odd = fmaf(s[i + 1], s[i + 1], odd);
        }
        ss[0] += odd;
        if (MODE == kResidual && p.residual_out && ok)
#pragma unroll
            for (int q = 0; q < NA; ++q) store_access<T, G>(static_cast<T *>(p.residual_out) + row * D, (q * TPR + t) * P, D, s + q * P);
        row_reduce<TPR, false>(ss, red[flip][0]);
        const float inv = 1.f / sqrtf(fmaf(ss[0], per, p.eps));
#pragma unroll
        for (int q = 0; q < NA; ++q) {
            float w[P], v[P];
            load_weight<T, G>(p.weight, p.weight_f32, (q * TPR + t) * P, D, w);
            if (MODE == kGate) widen<T, G>(cur[q], v);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                s[q * P + i] *= inv * w[i];
                if (MODE == kGate) s[q * P + i] *= sig<T>(v[i]);
            }
        }
        if constexpr (!QUANT) {
            if (ok)
#pragma unroll
                for (int q = 0; q < NA; ++q) store_access<T, G>(static_cast<T *>(p.y) + row * D, (q * TPR + t) * P, D, s + q * P);
        } else {
            const bool whole = p.group >= D;
            const int groups = whole ? 1 : (D + p.group - 1) / p.group;
            float top[NA];
#pragma unroll
            for (int q = 0; q < NA; ++q) {
                top[q] = 0.f;
                // channels beyond D hold 0, or NaN where the row's norm is NaN: they have no part
                if ((q * TPR + t) * P < D)
#pragma unroll
                    for (int i = 0; i < P; ++i) top[q] = max_nan(top[q], fabsf(s[q * P + i]));
            }
            // the largest magnitude of each access's group, in all its threads
            if (whole) {
                float all[1] = {top[0]};
#pragma unroll
                for (int q = 1; q < NA; ++q) all[0] = max_nan(all[0], top[q]);
                row_reduce<TPR, true>(all, red[flip][1]);
#pragma unroll
                for (int q = 0; q < NA; ++q) top[q] = all[0];
            } else if constexpr (G == 16) {
                // 32, 64 or 128 channels are 4 to 32 neighbouring threads of one warp
#pragma unroll
                for (int q = 0; q < NA; ++q)
                    for (int o = p.group / P / 2; o > 0; o >>= 1) top[q] = max_nan(top[q], __shfl_xor_sync(0xffffffffu, top[q], o));
            } else {
                // rows of any alignment: by way of shared memory, where magnitudes compare as integers (NaN above all)
                constexpr int MOST = (8 * NU * TPR + 31) / 32;
                __shared__ int gm[ROWS][MOST];
                __syncthreads();
                for (int i = threadIdx.x; i < ROWS * MOST; i += NT) (&gm[0][0])[i] = 0;
                __syncthreads();
#pragma unroll
                for (int q = 0; q < NA; ++q)
                    if ((q * TPR + t) * P < D) atomicMax(&gm[lr][(q * TPR + t) * P / p.group], __float_as_int(top[q]) & 0x7fffffff);
                __syncthreads();
#pragma unroll
                for (int q = 0; q < NA; ++q)
                    if ((q * TPR + t) * P < D) top[q] = __int_as_float(gm[lr][(q * TPR + t) * P / p.group]);
            }
            if (ok)
#pragma unroll
                for (int q = 0; q < NA; ++q) {
                    const int c = (q * TPR + t) * P;
                    // s / scale as a division would round it: the product with the reciprocal is up to two
                    // steps off, which would show next to a border of e4m3, and its remainder says by how
                    // much. An infinite scale leaves no remainder to take: 0, or NaN of an infinity.
                    const float scale = group_scale(top[q], p.pow2), to = 1.f / scale, by = scale < INFINITY ? scale : 0.f;
                    float v[P];
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        v[i] = s[q * P + i] * to;
                        v[i] = fmaf(fmaf(-v[i], by, s[q * P + i]), to, v[i]);
                    }
                    store_e4m3<P, G == 16>(static_cast<uint8_t *>(p.y) + row * D, c, D, v);
                    if (whole ? c == 0 : c < D && c % p.group == 0) p.scales[row * groups + (whole ? 0 : c / p.group)] = scale;
                }
        }
    }
}

}  // namespace

}  // namespace kda
