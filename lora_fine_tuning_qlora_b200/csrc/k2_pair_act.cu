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
    // Short contractions are bound by the epilogue, long ones by the operand
    // ring: sixteen epilogue warps over four stages up to K = 2048, else eight
    // over five (us, 8192 x K x 8192 rank 4, GELU(tanh) + residual + checkpoint:
    // K 1024: 165 against 199; 2816: 203 against 194; 4096: 254 against 237).
    // Rank 16's tables leave no room for sixteen.
    const bool wide = K <= 2048;
    if (ep.r <= 4)
        return wide ? launch_pair_act<4, true, 16>(ta, tb, to, tr, tz, a, status, s)
                    : launch_pair_act<4, true, 8>(ta, tb, to, tr, tz, a, status, s);
    if (ep.r <= 8)
        return wide ? launch_pair_act<8, true, 16>(ta, tb, to, tr, tz, a, status, s)
                    : launch_pair_act<8, true, 8>(ta, tb, to, tr, tz, a, status, s);
    return launch_pair_act<16, true, 8>(ta, tb, to, tr, tz, a, status, s);
}

}  // namespace qlora
