// The per-irrep norm and gated residual on rows stored as bf16.
#include "norm_kernels.cuh"

namespace cgtp {

cudaError_t launch_norm_forward_bf16(const NormTable& tab, const NormForward& a, bool vectors,
                                   cudaStream_t s) {
    return forward<__nv_bfloat16>(tab, a, vectors, s);
}
cudaError_t launch_norm_backward_bf16(const NormTable& tab, const NormBackward& a, bool vectors,
                                    cudaStream_t s) {
    return backward<__nv_bfloat16>(tab, a, vectors, s);
}

}  // namespace cgtp
