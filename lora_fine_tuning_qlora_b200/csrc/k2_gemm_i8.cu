// k2_gemm_i8.cu -- dispatch of the forward int8 GEMM and its large-tile
// kernels with the plain epilogue (k2_gemm_i8.cuh).
#include "k2_gemm_i8.cuh"

namespace qlora {

cudaError_t launch_gemm_i8_fwd(Act act, const int8_t* Xq, const int8_t* Wq, int M, int N, int K,
                               const FwdEpilogue& ep, int* status, cudaStream_t s, bool w4) {
    if (small_m_applies(M, N, ep.r, K, ep.ex)) return launch_gemm_i8_fwd_small(act, Xq, Wq, M, N, K, ep, status, s, w4);
    if (ep.ex && !w4 && gemm_fwd_pair_act_applies(act, M, N, K, ep.r))
        return launch_gemm_i8_fwd_pair_act(Xq, Wq, M, N, K, ep, status, s);
    if (gemm_fwd_pair_applies(act, M, N, K, ep.r))
        return launch_gemm_i8_fwd_pair(Xq, Wq, M, N, K, ep, status, s, w4);
    if (ep.ex) return launch_gemm_i8_fwd_act(act, Xq, Wq, M, N, K, ep, status, s, w4);
    return launch_gemm_i8_fwd_tiles<false>(act, Xq, Wq, M, N, K, ep, status, s, w4);
}

}  // namespace qlora
