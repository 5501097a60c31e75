// Gradients of the RMS norm (see kda_norm.cuh).
#include "kda_norm.cuh"

namespace kda {

namespace {

// The gate's sigmoid p and c = 1 - p, both as exact as their own size allows: 1 - p by
// subtraction would lose an open gate's gradient, all of it from a gate of 17 on. With the
// exponential infinite or beyond the reciprocal's range p is 0, and c some number up to 1.
template <typename T> __device__ __forceinline__ void gate_both(float g, float &p, float &c) {
    const float e = sizeof(T) == 2 ? ex2_fast(-kLog2e * g) : expf(-g);
    p = sizeof(T) == 2 ? rcp_fast(1.f + e) : 1.f / (1.f + e);
    c = fminf(e * p, 1.f);  // 1 of the NaN of inf x 0
}
// The same in one register: the smaller of p and c with the gate's sign, and both of that.
template <typename T> __device__ __forceinline__ float gate_small(float g) {
    const float e = sizeof(T) == 2 ? ex2_fast(-kLog2e * fabsf(g)) : expf(-fabsf(g));
    return copysignf(sizeof(T) == 2 ? e * rcp_fast(1.f + e) : e / (1.f + e), g);
}
__device__ __forceinline__ void gate_both_of(float small, float &p, float &c) {
    const float q = fabsf(small), r = 1.f - q;
    p = signbit(small) ? q : r;
    c = signbit(small) ? r : q;
}

// ---------------------------------------------------------------- backward
// The weights and the sums for dw stay in registers and leave once, as one slice of dw per CTA.
template <typename T, int G, int TPR, int NU, bool GATE>
__global__ void __launch_bounds__(norm_threads<TPR>(), norm_resident(true, TPR, NU)) norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
    constexpr int NT = norm_threads<TPR>(), ROWS = NT / TPR, P = access_channels<T, G>(), NA = 8 * NU / P;
    // Between the row's sums and its output p and c stay in a register each; in one where 512
    // threads with several runs have 128 registers each (4096 x 8192 fp32: 130 us, 139 with two).
    constexpr bool SMALL = TPR == 512 && NU > 1;
    let_next_pass_start();
    __shared__ float red[2][2][norm_red<TPR>()];
    __shared__ float slice[ROWS > 1 ? ROWS * TPR * 8 * NU : 1];
    const int t = threadIdx.x % TPR, lr = threadIdx.x / TPR, D = p.D;
    const float per = 1.f / D;
    float w[8 * NU], dw[8 * NU];
#pragma unroll
    for (int q = 0; q < NA; ++q) load_weight<T, G>(p.weight, p.weight_f32, (q * TPR + t) * P, D, w + q * P);
#pragma unroll
    for (int i = 0; i < 8 * NU; ++i) dw[i] = 0.f;
    const long long step = (long long)gridDim.x * ROWS;
    long long row = (long long)blockIdx.x * ROWS + lr;
    // the third tensor: the gate, or the cotangent of the sum
    const NormRows &third = GATE ? p.gate : p.dresidual;
    Bits<G> bx[NA], bd[NA], bt[NA];
    auto fetch_all = [&](long long r) {
        const bool ok = r < p.rows;
        fetch_row<T, G, TPR, NA>(p.x, r, ok, t, D, bx);
        fetch_row<T, G, TPR, NA>(p.dy, r, ok, t, D, bd);
        fetch_row<T, G, TPR, NA>(third, r, ok && third.at, t, D, bt);
    };
    fetch_all(row);
    int flip = 0;  // two buffers in turn: one barrier a row
    for (long long base = row - lr; base < p.rows; base += step, row += step, flip ^= 1) {
        const bool ok = row < p.rows;
        float s[8 * NU], d[8 * NU], g[GATE ? 8 * NU : 1], shut[GATE && !SMALL ? 8 * NU : 1], sum[2] = {0.f, 0.f};
        Bits<G> cur[NA];
#pragma unroll
        for (int q = 0; q < NA; ++q) {
            widen<T, G>(bx[q], s + q * P);
            widen<T, G>(bd[q], d + q * P);
            if (GATE) widen<T, G>(bt[q], g + (GATE ? q * P : 0));
            else cur[q] = bt[q];
        }
        fetch_all(row + step);
#pragma unroll
        for (int i = 0; i < 8 * NU; ++i) {
            float u = d[i] * w[i];
            if (GATE) {
                if constexpr (SMALL) {
                    float open, rest;
                    g[i] = gate_small<T>(g[i]);
                    gate_both_of(g[i], open, rest);
                    u *= open;
                } else {
                    gate_both<T>(g[i], g[i], shut[i]);
                    u *= g[i];
                }
            }
            sum[0] = fmaf(s[i], s[i], sum[0]);
            sum[1] = fmaf(u, s[i], sum[1]);
        }
        row_reduce<TPR, false>(sum, red[flip]);
        const float inv = 1.f / sqrtf(fmaf(sum[0], per, p.eps)), k = sum[1] * per * inv * inv;
        if (!ok) continue;
#pragma unroll
        for (int q = 0; q < NA; ++q) {
            const int c = (q * TPR + t) * P;
            float o[P], v[P];
            if (!GATE) widen<T, G>(cur[q], v);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int j = q * P + i;
                const float n = s[j] * inv;
                float e = d[j], rest = 0.f;
                if constexpr (GATE && SMALL) {
                    float open;
                    gate_both_of(g[j], open, rest);
                    e *= open;
                } else if constexpr (GATE) {
                    e *= g[j];
                    rest = shut[j];
                }
                dw[j] = fmaf(e, n, dw[j]);
                o[i] = inv * fmaf(-s[j], k, e * w[j]);
                if (!GATE) o[i] += v[i];
                if (GATE) v[i] = e * n * w[j] * rest;
            }
            store_access<T, G>(static_cast<T *>(p.dx) + row * D, c, D, o);
            if (GATE) store_access<T, G>(static_cast<T *>(p.dgate) + row * D, c, D, v);
        }
    }
    if (!p.partial) return;
    float *out = p.partial + (long long)blockIdx.x * D;
    if constexpr (ROWS > 1) {
        // the rows of the CTA are joined in their order
#pragma unroll
        for (int q = 0; q < NA; ++q)
#pragma unroll
            for (int i = 0; i < P; ++i) slice[(lr * 8 * NU) * TPR + (q * TPR + t) * P + i] = dw[q * P + i];
        __syncthreads();
        for (int c = threadIdx.x; c < TPR * 8 * NU && c < D; c += NT) {
            float v = 0.f;
            for (int j = 0; j < ROWS; ++j) v += slice[j * TPR * 8 * NU + c];
            out[c] = v;
        }
    } else {
#pragma unroll
        for (int q = 0; q < NA; ++q)
#pragma unroll
            for (int i = 0; i < P; ++i)
                if ((q * TPR + t) * P + i < D) out[(q * TPR + t) * P + i] = dw[q * P + i];
    }
}

// dw: the sum of its slices.
template <typename T> __global__ void __launch_bounds__(1024) norm_dw_kernel(const float *partial, void *dw, int f32, int slices, int D) {
    const int c = blockIdx.x * 32 + (threadIdx.x & 31);
    wait_for_last_pass();
    const float v = slice_sum(partial, slices, D, c);
    if (threadIdx.x >= 32 || c >= D) return;
    if (f32) static_cast<float *>(dw)[c] = v;
    else static_cast<T *>(dw)[c] = from_f32<T>(v);
}

template <typename T, int G, int TPR, int NU> struct Bwd {
    static cudaError_t run(const NormBwdParams &p, cudaStream_t st) {
        const int ctas = norm_ctas(p.rows, {TPR, NU}, true);
        count_launch();
        if (p.gate.at) norm_bwd_kernel<T, G, TPR, NU, true><<<ctas, norm_threads<TPR>(), 0, st>>>(p);
        else norm_bwd_kernel<T, G, TPR, NU, false><<<ctas, norm_threads<TPR>(), 0, st>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || !p.dweight) return e;
        return launch_next_pass(norm_dw_kernel<T>, (p.D + 31) / 32, 1024, st, (const float *)p.partial, p.dweight, p.weight_f32, ctas, p.D);
    }
};

}  // namespace

size_t rms_norm_bwd_workspace_bytes(long long rows, int D, bool weight) {
    return weight ? sizeof(float) * (size_t)norm_ctas(rows, bwd_shape(rows, D), true) * D : 0;
}

cudaError_t launch_rms_norm_bwd(const NormBwdParams &p, bool bf16, cudaStream_t st) {
    const size_t esz = bf16 ? 2 : 4, wsz = p.weight_f32 ? 4 : esz;
    RowAccess ac;
    for (const NormRows *r : {&p.x, &p.dy, &p.gate, &p.dresidual}) ac.rows(r->at, r->stride, p.D, esz);
    ac.rows(p.weight, p.D, p.D, wsz);
    ac.rows(p.dx, p.D, p.D, esz);
    ac.rows(p.dgate, p.D, p.D, esz);
    return pick<Bwd, true>(p, bf16, ac.g(), st);
}

}  // namespace kda
