// RMS norm, rows in the activations' type.
#include "kda_norm_fwd.cuh"

namespace kda {

namespace {

template <typename T, int G, int TPR, int NU> struct Fwd {
    template <int MODE> static cudaError_t launch(const NormParams &p, cudaStream_t st) {
        count_launch();
        norm_fwd_kernel<T, G, TPR, NU, MODE, false><<<norm_ctas(p.rows, {TPR, NU}, false), norm_threads<TPR>(), 0, st>>>(p);
        return cudaGetLastError();
    }
    static cudaError_t run(const NormParams &p, cudaStream_t st) {
        return p.residual.at ? launch<kResidual>(p, st) : p.gate.at ? launch<kGate>(p, st) : launch<kPlain>(p, st);
    }
};

}  // namespace

cudaError_t launch_rms_norm(const NormParams &p, bool bf16, cudaStream_t st) {
    RowAccess ac = norm_access(p, bf16);
    if (p.scales) return launch_rms_norm_quant(p, bf16, ac.g(), st);
    ac.rows(p.y, p.D, p.D, bf16 ? 2 : 4);
    return pick<Fwd, false>(p, bf16, ac.g(), st);
}

}  // namespace kda
