// RMS norm, rows in 8 bits (e4m3) with their scales.
#include "kda_norm_fwd.cuh"

namespace kda {

namespace {

template <typename T, int G, int TPR, int NU> struct Fwd {
    template <int MODE> static cudaError_t launch(const NormParams &p, cudaStream_t st) {
        count_launch();
        norm_fwd_kernel<T, G, TPR, NU, MODE, true><<<norm_ctas(p.rows, {TPR, NU}, false), norm_threads<TPR>(), 0, st>>>(p);
        return cudaGetLastError();
    }
    static cudaError_t run(const NormParams &p, cudaStream_t st) {
        return p.residual.at ? launch<kResidual>(p, st) : p.gate.at ? launch<kGate>(p, st) : launch<kPlain>(p, st);
    }
};

}  // namespace

cudaError_t launch_rms_norm_quant(const NormParams &p, bool bf16, int g, cudaStream_t st) {
    // the 8-bit row is written by half (bf16) or a quarter of an access
    if (reinterpret_cast<uintptr_t>(p.y) % 8 && g > 4) g = 4;
    return pick<Fwd, false>(p, bf16, g, st);
}

}  // namespace kda
