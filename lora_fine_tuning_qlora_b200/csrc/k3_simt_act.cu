// k3_simt_act.cu -- dX = (dY (Wq sw)^T + c G A^T) * act'(z) + add on CUDA cores,
// for fp32 activations and for rows of dY that the Tensor Memory Accelerator
// cannot describe (N not a multiple of 8): small layers and classifier heads.
//
// A CTA of 256 threads computes 16 TM x 64 outputs, TM x 4 per thread (rows ty,
// ty + 16, ..; four neighbouring columns), over 32 contraction steps at a time
// through two shared-memory buffers: the next step's dY values and codes are
// loaded into registers before the current step's products, so a step costs
// no memory latency (one buffer with the loads between two barriers: 34 us at
// 64 x 784 x 128 in the backward, 13 CTAs on 8 steps of 16).  Fp32 products
// and sums; for bf16 activations the kernel is rounded to bf16 first, as on
// the tensor cores, so that dX follows one rule whatever N % 8 is.  Few tiles
// share their contraction over a cluster of S CTAs (along x), whose partial
// tiles the first adds in rank order through distributed shared memory.
#include "dx_common.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "act_epilogue.cuh"

namespace qlora {

namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;
constexpr int kStep = 32;

template <typename T, bool W4, int TM>
__global__ void __launch_bounds__(kThreads) k3_simt_act_kernel(const T* __restrict__ dY,
                                                               const uint8_t* __restrict__ Wq,
                                                               const float* __restrict__ sw, int M, int N, int K,
                                                               int S, DxEpilogue ep) {
    constexpr int kRows = 16 * TM;
    constexpr int kPerD = kRows * kStep / kThreads;
    __shared__ __align__(16) float sW[2][kStep][kCols];
    __shared__ float sD[2][kStep][kRows + 1];
    static_assert(sizeof(sD) >= kRows * 65 * sizeof(float), "c G rows of the tile");
    float(*sG)[65] = reinterpret_cast<float(*)[65]>(&sD[0][0][0]);  // after the products
    pdl_wait();
    pdl_trigger();  // after the wait: see launch_rank_x_q
    const int tid = threadIdx.x;
    const int tx = tid % 16, ty = tid / 16;
    const int split = static_cast<int>(blockIdx.x) % S;
    const int m0 = blockIdx.y * kRows, k0 = static_cast<int>(blockIdx.x) / S * kCols;
    const int steps = (N + kStep - 1) / kStep;
    const int nbeg = steps * split / S * kStep, nend = min(N, steps * (split + 1) / S * kStep);
    // a thread's part of a step: kPerD values of dY (consecutive threads along
    // n), eight codes of one contraction row
    const int wn = tid / 8, wk = (tid % 8) * 8;
    float dreg[kPerD];
    uint2 wreg;
    float wscale;
    auto fetch = [&](int n0) {
#pragma unroll
        for (int i = 0; i < kPerD; ++i) {
            const int e = tid + i * kThreads;
            const int m = m0 + e / kStep, n = n0 + e % kStep;
            dreg[i] = (m < M && n < nend) ? ActIO<T>::to_f(dY[static_cast<size_t>(m) * N + n]) : 0.f;
        }
        const int n = n0 + wn;
        wreg = make_uint2(0u, 0u);
        wscale = 0.f;
        if (n < nend && k0 + wk < K) {  // K is a multiple of 16
            wscale = __ldg(sw + n);
            if constexpr (W4)
                wreg.x = __ldg(reinterpret_cast<const uint32_t*>(Wq + (static_cast<size_t>(n) * K + k0 + wk) / 2));
            else
                wreg = __ldg(reinterpret_cast<const uint2*>(Wq + static_cast<size_t>(n) * K + k0 + wk));
        }
    };
    auto put = [&](int b) {
#pragma unroll
        for (int i = 0; i < kPerD; ++i) {
            const int e = tid + i * kThreads;
            sD[b][e % kStep][e / kStep] = dreg[i];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            int code;
            if constexpr (W4) code = static_cast<int>(wreg.x << (28 - 4 * e)) >> 28;
            else code = static_cast<int8_t>((e < 4 ? wreg.x : wreg.y) >> (8 * (e & 3)));
            float w = __fmul_rn(static_cast<float>(code), wscale);
            if constexpr (sizeof(T) == 2) w = __bfloat162float(__float2bfloat16_rn(w));
            sW[b][wn][wk + e] = w;
        }
    };
    float acc[TM][4] = {};
    fetch(nbeg);
    put(0);
    __syncthreads();
    int b = 0;
    for (int n0 = nbeg; n0 < nend; n0 += kStep, b ^= 1) {
        const bool more = n0 + kStep < nend;
        if (more) fetch(n0 + kStep);
#pragma unroll 8
        for (int n = 0; n < kStep; ++n) {
            const float4 w = *reinterpret_cast<const float4*>(&sW[b][n][4 * tx]);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const float d = sD[b][n][ty + 16 * i];
                acc[i][0] = fmaf(d, w.x, acc[i][0]);
                acc[i][1] = fmaf(d, w.y, acc[i][1]);
                acc[i][2] = fmaf(d, w.z, acc[i][2]);
                acc[i][3] = fmaf(d, w.w, acc[i][3]);
            }
        }
        if (more) put(b ^ 1);
        __syncthreads();
    }
    if (S > 1) {
        // partial tiles [kRows][kCols] in the buffers that the products are done with
        float* part = &sW[0][0][0];
        static_assert(sizeof(sW) >= kRows * kCols * sizeof(float), "partial tile");
#pragma unroll
        for (int i = 0; i < TM; ++i)
            *reinterpret_cast<float4*>(part + (ty + 16 * i) * kCols + 4 * tx) =
                make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        cluster_arrive();
        cluster_wait();
        if (split == 0) {
            for (int q = 1; q < S; ++q) {
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const uint32_t at = dsmem_addr(part + (ty + 16 * i) * kCols + 4 * tx, static_cast<uint32_t>(q));
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][e] += __uint_as_float(dsmem_ld_u32(at + 4u * e));
                }
            }
        }
        cluster_arrive();  // the partial tiles may go
        cluster_wait();
        if (split != 0) return;
    }
    for (int i = tid; i < kRows * ep.r; i += kThreads) {
        const int mm = i / ep.r, j = i - mm * ep.r;
        sG[mm][j] = m0 + mm < M ? ep.c * g_row(ep, M, m0 + mm, j) : 0.f;
    }
    __syncthreads();
    const int k = k0 + 4 * tx;
    if (k >= K) return;
    T* dX = static_cast<T*>(ep.dX);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int mm = ty + 16 * i, m = m0 + mm;
        if (m >= M) continue;
        for (int j = 0; j < ep.r; ++j) {
            const float g = sG[mm][j];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(g, a_at(ep, k + e, j), acc[i][e]);
        }
        const size_t at = static_cast<size_t>(m) * K + k;
        if (ep.act != kActNone) {
            const float s = __ldg(ep.zs + static_cast<size_t>(k / kCkptBlock) * M + m);
            const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(ep.zq + at));
            float z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = static_cast<float>(static_cast<int8_t>(q >> (8 * e))) * s;
            slope_apply<T>(ep.act, z, acc[i]);
        }
        const T* add = static_cast<const T*>(ep.add);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (add) acc[i][e] += ActIO<T>::to_f(add[at + e]);
            dX[at + e] = ActIO<T>::from_f(acc[i][e]);
        }
    }
}

template <typename T, bool W4>
cudaError_t run(const T* dY, const uint8_t* Wq, const float* sw, int M, int N, int K, const DxEpilogue& ep,
                cudaStream_t s) {
    // 64-row tiles where they fill the machine, else 32, and the contraction
    // split while that leaves SMs idle and a CTA at least two steps
    const int across = (K + kCols - 1) / kCols;
    if (static_cast<long long>((M + 63) / 64) * across >= 2 * sm_count())
        return launch_k(k3_simt_act_kernel<T, W4, 4>, dim3(across, (M + 63) / 64), dim3(kThreads), 0, s, 1, dY, Wq, sw,
                        M, N, K, 1, ep);
    const int down = (M + 31) / 32, steps = (N + kStep - 1) / kStep;
    int S = 1;
    while (S < 8 && 2 * S * across * down <= sm_count() && 4 * S <= steps) S *= 2;
    return launch_kx(k3_simt_act_kernel<T, W4, 2>, dim3(across * S, down), dim3(kThreads), 0, s, S, dY, Wq, sw, M, N, K,
                     S, ep);
}

}  // namespace

cudaError_t launch_gemm_dx_simt_act(Act act, const void* dY, const int8_t* Wq, const float* sw, int M, int N, int K,
                                    const DxEpilogue& ep, cudaStream_t s, bool w4) {
    const uint8_t* w = reinterpret_cast<const uint8_t*>(Wq);
    if (act == kBF16) {
        const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(dY);
        return w4 ? run<__nv_bfloat16, true>(dy, w, sw, M, N, K, ep, s)
                  : run<__nv_bfloat16, false>(dy, w, sw, M, N, K, ep, s);
    }
    const float* dy = static_cast<const float*>(dY);
    return w4 ? run<float, true>(dy, w, sw, M, N, K, ep, s) : run<float, false>(dy, w, sw, M, N, K, ep, s);
}

}  // namespace qlora
