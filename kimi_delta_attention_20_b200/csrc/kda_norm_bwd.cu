// Gradients of the RMS norm (see kda_norm.cuh).
#include "kda_norm.cuh"

namespace kda {

namespace {

// ---------------------------------------------------------------- backward
// The weights and the sums for dw stay in registers and leave once, as one slice of dw per CTA.
template <typename T, int G, int TPR, int NU, bool GATE>
__global__ void __launch_bounds__(norm_threads<TPR>(), norm_resident(true, TPR, NU)) norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
    constexpr int NT = norm_threads<TPR>(), ROWS = NT / TPR, P = access_channels<T, G>(), NA = 8 * NU / P;
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
        float s[8 * NU], d[8 * NU], g[GATE ? 8 * NU : 1], sum[2] = {0.f, 0.f};
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
                g[i] = sig<T>(g[i]);
                u *= g[i];
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
                const float n = s[j] * inv, e = GATE ? d[j] * g[j] : d[j];
                dw[j] = fmaf(e, n, dw[j]);
                o[i] = inv * fmaf(-s[j], k, e * w[j]);
                if (!GATE) o[i] += v[i];
                if (GATE) v[i] = e * n * w[j] * (1.f - g[j]);
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
