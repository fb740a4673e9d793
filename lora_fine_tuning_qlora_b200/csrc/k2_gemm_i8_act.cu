// k2_gemm_i8_act.cu -- the forward int8 GEMM's large-tile kernels
// (k2_gemm_i8.cuh) with activation, residual and 8-bit checkpoint in the
// epilogue.
#include "k2_gemm_i8.cuh"

namespace qlora {

cudaError_t launch_gemm_i8_fwd_act(Act act, const int8_t* Xq, const int8_t* Wq, int M, int N, int K,
                                   const FwdEpilogue& ep, int* status, cudaStream_t s, bool w4) {
    return launch_gemm_i8_fwd_tiles<true>(act, Xq, Wq, M, N, K, ep, status, s, w4);
}

}  // namespace qlora
