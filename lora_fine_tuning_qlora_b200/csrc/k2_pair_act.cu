// k2_pair_act.cu -- the forward of the CTA-pair GEMM with activation, residual
// and 8-bit checkpoint (pair_act.cuh).
#include "pair_act.cuh"

namespace qlora {

// Outputs whose rows start at 16-byte boundaries.
bool gemm_fwd_pair_act_applies(Act act, int M, int N, int K, int r) {
    return N % 8 == 0 && gemm_fwd_pair_applies(act, M, N, K, r);
}

cudaError_t launch_gemm_i8_fwd_pair_act(const int8_t* Xq, const int8_t* Wq, int M, int N, int K,
                                        const FwdEpilogue& ep, int* status, cudaStream_t s) {
    PairActArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    a.r = ep.r;
    a.c = ep.c;
    a.rowf = ep.xA;
    a.nsl = 1;
    a.colf = ep.B;
    a.cs_j = N;
    a.cs_n = 1;
    a.sx = ep.sx;
    a.sw = ep.sw;
    a.bias = ep.bias;
    a.act = ep.act;
    a.add = ep.res != nullptr;
    a.zq = ep.zq;
    a.ztma = ep.zq && N % 16 == 0;
    a.zs_out = ep.zs;
    CUtensorMap ta, tb, to, tr, tz;
    if (!make_tmap_2d(&ta, Xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, M, K, K, kTM, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tmap_2d(&tb, Wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, N, K, K, kTN / 2, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !pair_act_maps(a, ep.Y, ep.res, ep.zq, &to, &tr, &tz))
        return cudaErrorInvalidValue;
    // epilogue warps: sixteen where the tables leave shared memory for four
    // operand stages beside their pieces
    if (ep.r <= 4) return launch_pair_act<4, true, 16>(ta, tb, to, tr, tz, a, status, s);
    if (ep.r <= 8) return launch_pair_act<8, true, 16>(ta, tb, to, tr, tz, a, status, s);
    return launch_pair_act<16, true, 8>(ta, tb, to, tr, tz, a, status, s);
}

}  // namespace qlora
