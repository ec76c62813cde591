// The per-irrep norm and gated residual on rows stored as f64.
#include "norm_kernels.cuh"

namespace cgtp {

cudaError_t launch_norm_forward_f64(const NormTable& tab, const NormForward& a, int vector,
                                    cudaStream_t s) {
    return launch_norm<double>(tab, a, vector, s);
}
cudaError_t launch_norm_backward_f64(const NormTable& tab, const NormBackward& a, int vector,
                                     cudaStream_t s) {
    return launch_norm<double>(tab, a, vector, s);
}

}  // namespace cgtp
