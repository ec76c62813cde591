// The per-irrep norm and gated residual on rows stored as f32.
#include "norm_kernels.cuh"

namespace cgtp {

cudaError_t launch_norm_forward_f32(const NormTable& tab, const NormForward& a, bool vectors,
                                   cudaStream_t s) {
    return forward<float>(tab, a, vectors, s);
}
cudaError_t launch_norm_backward_f32(const NormTable& tab, const NormBackward& a, bool vectors,
                                    cudaStream_t s) {
    return backward<float>(tab, a, vectors, s);
}

}  // namespace cgtp
