// k3_dx.cu -- dispatch of the dX GEMM and its kernels with the plain epilogue
// (k3_dx.cuh).
#include "k3_dx.cuh"

namespace qlora {

cudaError_t launch_gemm_dx(Act act, const void* dY, const int8_t* Wq, const float* sw, int M,
                           int N, int K, const DxEpilogue& ep, int* status, cudaStream_t s, bool w4) {
    const bool tc = act == kBF16 && (N % 8) == 0 && (!ep.ol.par || (K % 16) == 0);
    const int mode = ep.ol.par ? 2 : (w4 ? 1 : 0);
    if (!tc)
        return ep.ex ? launch_gemm_dx_simt_act(act, dY, Wq, sw, M, N, K, ep, s, w4)
                     : launch_gemm_dx_simt(act, dY, Wq, sw, M, N, K, ep, s, mode);
    if (mode != 2 && !ep.bias && small_m_applies(M, K, ep.r, N, ep.ex))
        return launch_gemm_dx_small(dY, Wq, sw, M, N, K, ep, status, s, w4);
    if (gemm_dx_pair_applies(M, N, K, ep.r))
        return launch_gemm_dx_pair(dY, Wq, sw, M, N, K, ep, status, s, w4);
    return ep.ex ? launch_gemm_dx_act(dY, Wq, sw, M, N, K, ep, status, s, mode)
                 : launch_gemm_dx_tiles<false>(dY, Wq, sw, M, N, K, ep, status, s, mode);
}

}  // namespace qlora
