// k3_dx_act.cu -- the dX GEMM's large-tile kernels (k3_dx.cuh) with the factor
// act'(z) of a z kept in 8 bits and an added gradient in the epilogue.
#include "k3_dx.cuh"

namespace qlora {

cudaError_t launch_gemm_dx_act(const void* dY, const int8_t* Wq, const float* sw, int M, int N, int K,
                               const DxEpilogue& ep, int* status, cudaStream_t s, int mode) {
    return launch_gemm_dx_tiles<true>(dY, Wq, sw, M, N, K, ep, status, s, mode);
}

}  // namespace qlora
