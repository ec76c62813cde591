// The per-irrep norm and gated residual on rows stored as f16.
#include "norm_kernels.cuh"

namespace cgtp {

cudaError_t launch_norm_forward_f16(const NormTable& tab, const NormForward& a, int vector,
                                    cudaStream_t s) {
    return launch_norm<__half>(tab, a, vector, s);
}
cudaError_t launch_norm_backward_f16(const NormTable& tab, const NormBackward& a, int vector,
                                     cudaStream_t s) {
    return launch_norm<__half>(tab, a, vector, s);
}

}  // namespace cgtp
