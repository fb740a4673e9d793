// k1_act.cu -- the input quantizer of qlora_forward_act: Xq, sx and xA = X A as
// in k1_quantize.cu (codes and scales are the same bits; the fp32 sums of xA
// are grouped differently), in two forms for the sizes where the kernels there
// leave the machine idle:
//
//   split  few rows: a row is spread over a cluster of S CTAs, each 256
//          threads with one 16-byte chunk (or more) of it; the row's maximum
//          and the partial sums meet in distributed shared memory.  Bound by
//          latency (two block reductions and two cluster barriers): 1 x 2048 3.8
//          us, 16 x 16384 5.2 us (one CTA that walked all 16 rows: 85 us).
//   rows   many bf16 rows of at most 4096: each warp holds R whole rows in
//          registers, so that the maximum and the sums need no other warp
//          and no barrier, and the factor A is read from shared memory once
//          per R rows.  HBM: 2 + 1 bytes per element; what bounds it is the
//          instruction count per element (unpack, maximum, multiply, convert,
//          pack, r / 2 paired FMAs, 2 / R shared loads for rank 4): 16384 x
//          4096 rank 4 in 47 us, 4.3 TB/s.
#include "internal.h"
#include "ptx.cuh"

namespace qlora {

namespace {

constexpr int kSplitThreads = 256;
constexpr int kMaxS = 8;
constexpr int kRowsThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        bf16x8_to_f(__ldg(reinterpret_cast<const uint4*>(p)), v);
    } else {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p));
        const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// acc[j] += sum_e v[e] A[k + e, j]
template <int RP>
__device__ __forceinline__ void fma_rows(const float* __restrict__ A, int k, int r, bool vec, const float (&v)[8],
                                         float (&acc)[RP]) {
    const float* a = A + static_cast<size_t>(k) * r;
    if (vec) {  // r == RP, 16-byte aligned rows
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int j4 = 0; j4 < RP / 4; ++j4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(a) + e * (RP / 4) + j4);
                acc[4 * j4 + 0] = fmaf(v[e], f.x, acc[4 * j4 + 0]);
                acc[4 * j4 + 1] = fmaf(v[e], f.y, acc[4 * j4 + 1]);
                acc[4 * j4 + 2] = fmaf(v[e], f.z, acc[4 * j4 + 2]);
                acc[4 * j4 + 3] = fmaf(v[e], f.w, acc[4 * j4 + 3]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < RP; ++j) {
            if (j >= r) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[j] = fmaf(v[e], __ldg(a + e * r + j), acc[j]);
        }
    }
}

// One row per cluster: CTA s of S takes chunks [s n / S, (s + 1) n / S).
template <typename T, int RP>
__global__ void __launch_bounds__(kSplitThreads) k1_split_kernel(const T* __restrict__ X, const float* __restrict__ A,
                                                                 int K, int r, bool vec, int8_t* __restrict__ Xq,
                                                                 float* __restrict__ sx, float* __restrict__ xA) {
    constexpr int kWarps = kSplitThreads / 32;
    __shared__ uint32_t wmax[kWarps];
    __shared__ uint32_t smax[kMaxS];
    __shared__ float wsum[kWarps][RP];
    __shared__ float ssum[kMaxS][RP];
    const int t = threadIdx.x, warp = t / 32, lane = t % 32;
    const int m = blockIdx.x;
    const int S = gridDim.y, s = blockIdx.y;
    const int nch = K / 8;
    const int c0 = static_cast<int>(static_cast<long long>(nch) * s / S);
    const int c1 = static_cast<int>(static_cast<long long>(nch) * (s + 1) / S);
    pdl_trigger();
    cluster_arrive_relaxed();  // every CTA of the row runs before another writes to it
    pdl_wait();
    const T* xr = X + static_cast<size_t>(m) * K;
    float v0[8] = {};  // the first chunk stays in registers; longer slices are read again
    if (c0 + t < c1) load8(xr + static_cast<size_t>(c0 + t) * 8, v0);
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(v0[e]));
    for (int c = c0 + t + kSplitThreads; c < c1; c += kSplitThreads) {
        float v[8];
        load8(xr + static_cast<size_t>(c) * 8, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(v[e]));
    }
    const uint32_t wm = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));  // amax >= 0 or NaN (above all)
    if (lane == 0) wmax[warp] = wm;
    // x . A needs no maximum: its loads go out before the barriers
    float acc[RP];
#pragma unroll
    for (int j = 0; j < RP; ++j) acc[j] = 0.f;
    if (c0 + t < c1) fma_rows<RP>(A, (c0 + t) * 8, r, vec, v0, acc);
    for (int c = c0 + t + kSplitThreads; c < c1; c += kSplitThreads) {
        float v[8];
        load8(xr + static_cast<size_t>(c) * 8, v);
        fma_rows<RP>(A, c * 8, r, vec, v, acc);
    }
    {
        const float x = xreduce<RP, false>(acc);
        if ((lane & (32 / RP - 1)) == 0) wsum[warp][xreduce_index<RP>(lane)] = x;
    }
    __syncthreads();
    cluster_wait();
    if (t < S) {  // this CTA's maximum to every CTA
        uint32_t top = wmax[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = max(top, wmax[w]);
        dsmem_st(dsmem_addr(&smax[s], static_cast<uint32_t>(t)), __uint_as_float(top));
    }
    if (t >= 32 && t < 32 + RP) {  // its sums to the first
        float sum = wsum[0][t - 32];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) sum += wsum[w][t - 32];
        dsmem_st(dsmem_addr(&ssum[s][t - 32], 0), sum);
    }
    cluster_arrive();
    cluster_wait();
    uint32_t top = 0;
    for (int q = 0; q < S; ++q) top = max(top, smax[q]);
    amax = __uint_as_float(top);
    const float inv = amax > 0.f ? __fdiv_rn(127.0f, amax) : 0.f;
    int8_t* qr = Xq + static_cast<size_t>(m) * K;
    if (c0 + t < c1) *reinterpret_cast<uint2*>(qr + static_cast<size_t>(c0 + t) * 8) = codes8(v0, inv);
    for (int c = c0 + t + kSplitThreads; c < c1; c += kSplitThreads) {
        float v[8];
        load8(xr + static_cast<size_t>(c) * 8, v);
        *reinterpret_cast<uint2*>(qr + static_cast<size_t>(c) * 8) = codes8(v, inv);
    }
    if (s == 0) {
        if (t == 0) sx[m] = __fdiv_rn(amax, 127.0f);
        if (t < r) {
            float sum = ssum[0][t];
            for (int q = 1; q < S; ++q) sum += ssum[q][t];
            xA[static_cast<size_t>(m) * r + t] = sum;
        }
    }
}

// R whole rows per warp: chunk i of a lane is chunk lane + 32 i of the row.
// A warp's next R rows arrive by one bulk copy in its own part of shared
// memory while it computes the current ones from registers (loading straight
// into registers, with no copy ahead, ran 62 us at 16384 x 4096).
// A in shared memory as [pair p of a chunk's 8 rows][j / 2][chunk] of
// (A[2p, j], A[2p+1, j], A[2p, j+1], A[2p+1, j+1]), so that neighbouring lanes
// read neighbouring 16 bytes and a paired FMA takes two rows of A.
// FULL: rows of exactly 256 NCH elements.
template <int NCH, int RP, int R, bool FULL>
__global__ void __launch_bounds__(kRowsThreads) k1_rows_kernel(const __nv_bfloat16* __restrict__ X,
                                                               const float* __restrict__ A, int M, int K, int r,
                                                               int8_t* __restrict__ Xq, float* __restrict__ sx,
                                                               float* __restrict__ xA, int* status) {
    constexpr int kWarps = kRowsThreads / 32;
    extern __shared__ float4 sA[];  // [4][RP / 2][nch], then the warps' rows, then their barriers
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int nch = K / 8;
    const uint32_t row_bytes = static_cast<uint32_t>(K) * 2u;
    uint8_t* rows = reinterpret_cast<uint8_t*>(sA + 4 * (RP / 2) * nch) + warp * R * row_bytes;
    uint64_t* bar = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sA + 4 * (RP / 2) * nch) +
                                                kWarps * R * row_bytes) + warp;
    pdl_trigger();
    if (lane == 0) mbar_init(bar, 1);
    fence_mbar_init();
    __syncwarp();
    pdl_wait();
    const int groups = (M + R - 1) / R;
    const int step = gridDim.x * kWarps;
    auto fetch = [&](int g) {  // the group's rows into this warp's buffer
        if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(min(R, M - g * R)) * row_bytes;
            mbar_arrive_expect_tx(bar, bytes);
            bulk_load(rows, X + static_cast<size_t>(g) * R * K, bytes, bar);
        }
    };
    uint4 x[R][NCH];
    int g = blockIdx.x * kWarps + warp;
    if (g < groups) fetch(g);
    uint32_t phase = 0;
    // A, while the first rows are in flight
    for (int i = threadIdx.x; i < nch * 4 * (RP / 2); i += kRowsThreads) {
        const int c = i % nch, pj = i / nch;
        const int p = pj / (RP / 2), j = 2 * (pj % (RP / 2));
        const float* a0 = A + static_cast<size_t>(8 * c + 2 * p) * r;
        const float* a1 = a0 + r;
        sA[i] = make_float4(j < r ? __ldg(a0 + j) : 0.f, j < r ? __ldg(a1 + j) : 0.f,
                            j + 1 < r ? __ldg(a0 + j + 1) : 0.f, j + 1 < r ? __ldg(a1 + j + 1) : 0.f);
    }
    __syncthreads();
    const ulonglong2* sA2 = reinterpret_cast<const ulonglong2*>(sA);
    for (; g < groups; g += step) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar, phase, status))) break;
        phase ^= 1u;
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const uint4* p = reinterpret_cast<const uint4*>(rows + q * row_bytes);
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int c = lane + 32 * i;
                x[q][i] = (g * R + q < M && (FULL || c < nch)) ? p[c] : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        float inv[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const uint32_t w[4] = {x[q][i].x, x[q][i].y, x[q][i].z, x[q][i].w};
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    m2 = __hmax2_nan(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[h])));
            }
            const float top = max_nan(__low2float(m2), __high2float(m2));
            const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            inv[q] = amax > 0.f ? __fdiv_rn(127.0f, amax) : 0.f;
            if (lane == 0 && g * R + q < M) sx[g * R + q] = __fdiv_rn(amax, 127.0f);
        }
        // The next copy overwrites the rows that the loads above read: the loads
        // must be complete, not only issued (behind other warps' loads they can
        // wait longer than a copy from L2 takes), which the proxy fence orders.
        fence_proxy_async_smem();
        __syncwarp();
        if (g + step < groups) fetch(g + step);
        unsigned long long acc[R][RP];  // even and odd k apart
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int j = 0; j < RP; ++j) acc[q][j] = 0ull;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = lane + 32 * i;
            const bool in = FULL || c < nch;
            float f[R][8];
#pragma unroll
            for (int q = 0; q < R; ++q) {
                bf16x8_to_f(x[q][i], f[q]);
                const int m = g * R + q;
                if (in && m < M) *reinterpret_cast<uint2*>(Xq + static_cast<size_t>(m) * K + c * 8) = codes8(f[q], inv[q]);
            }
            const int cs = in ? c : 0;  // outside the row x is zero
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                unsigned long long x2[R];
#pragma unroll
                for (int q = 0; q < R; ++q) x2[q] = pk2(f[q][2 * p], f[q][2 * p + 1]);
#pragma unroll
                for (int j2 = 0; j2 < RP / 2; ++j2) {
                    const ulonglong2 a = sA2[(p * (RP / 2) + j2) * (FULL ? 32 * NCH : nch) + cs];
#pragma unroll
                    for (int q = 0; q < R; ++q) {
                        fma2(acc[q][2 * j2], x2[q], a.x);
                        fma2(acc[q][2 * j2 + 1], x2[q], a.y);
                    }
                }
            }
        }
        constexpr int V = R * RP;
        float v[V];
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int j = 0; j < RP; ++j) {
                float lo, hi;
                unpk2(acc[q][j], lo, hi);
                v[q * RP + j] = lo + hi;
            }
        const float s = xreduce<V, false>(v);
        if ((lane & (32 / V - 1)) == 0) {
            const int idx = xreduce_index<V>(lane);
            const int m = g * R + idx / RP, j = idx % RP;
            if (m < M && j < r) xA[static_cast<size_t>(m) * r + j] = s;
        }
    }
}

template <typename T, int RP>
cudaError_t launch_split(const T* X, const float* A, int M, int K, int r, int8_t* Xq, float* sx, float* xA,
                         cudaStream_t s) {
    // CTAs per row: one chunk a thread where that stays within two waves
    const int nch = K / 8;
    int S = 1;
    while (S < kMaxS && S * kSplitThreads < nch && 2 * S * M <= 2 * sm_count()) S *= 2;
    const bool vec = r == RP && (reinterpret_cast<uintptr_t>(A) & 15) == 0;
    return launch_k(k1_split_kernel<T, RP>, dim3(M, S), dim3(kSplitThreads), 0, s, S, X, A, K, r, vec, Xq, sx, xA);
}

template <int NCH, int RP, int R>
cudaError_t launch_rows(const __nv_bfloat16* X, const float* A, int M, int K, int r, int8_t* Xq, float* sx, float* xA,
                        int per_sm, int* status, cudaStream_t s) {
    constexpr int kWarps = kRowsThreads / 32;
    auto kern = K == 256 * NCH ? k1_rows_kernel<NCH, RP, R, true> : k1_rows_kernel<NCH, RP, R, false>;
    const int smem = K / 8 * 4 * (RP / 2) * 16 + kWarps * R * K * 2 + kWarps * 8;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    const int groups = (M + R - 1) / R;
    const int ctas = (groups + kWarps - 1) / kWarps;
    const int cap = per_sm * sm_count();
    return launch_k(kern, dim3(ctas < cap ? ctas : cap), dim3(kRowsThreads), smem, s, 1, X, A, M, K, r, Xq, sx, xA,
                    status);
}

}  // namespace

cudaError_t launch_quantize_rows_act(Act act, const void* X, const float* A, int M, int K, int r, int8_t* Xq,
                                     float* sx, float* xA, int* status, cudaStream_t s) {
    const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(X);
    if (M <= sm_count() && r <= 16) {
        if (act == kBF16) {
            if (r <= 4) return launch_split<__nv_bfloat16, 4>(xb, A, M, K, r, Xq, sx, xA, s);
            if (r <= 8) return launch_split<__nv_bfloat16, 8>(xb, A, M, K, r, Xq, sx, xA, s);
            return launch_split<__nv_bfloat16, 16>(xb, A, M, K, r, Xq, sx, xA, s);
        }
        const float* xf = static_cast<const float*>(X);
        if (r <= 4) return launch_split<float, 4>(xf, A, M, K, r, Xq, sx, xA, s);
        if (r <= 8) return launch_split<float, 8>(xf, A, M, K, r, Xq, sx, xA, s);
        return launch_split<float, 16>(xf, A, M, K, r, Xq, sx, xA, s);
    }
    // us against the kernels there: 16384 x 4096 47 / 68, 16384 x 2048 29 / 46,
    // 8192 x 4096 31 / 39, but 4096 x 2048 15 / 12: from 2^24 elements.  Two
    // CTAs per SM where A and the rows fit twice.
    if (static_cast<long long>(M) * K < (1LL << 24))
        return launch_quantize_rows(act, X, A, M, K, r, Xq, sx, xA, status, s);
    if (act == kBF16 && r <= 4 && K <= 4096) {
        if (K <= 1024) return launch_rows<4, 4, 2>(xb, A, M, K, r, Xq, sx, xA, 2, status, s);
        if (K <= 2048) return launch_rows<8, 4, 2>(xb, A, M, K, r, Xq, sx, xA, 2, status, s);
        return launch_rows<16, 4, 2>(xb, A, M, K, r, Xq, sx, xA, 1, status, s);
    }
    if (act == kBF16 && r <= 8 && K <= 4096) {
        if (K <= 1024) return launch_rows<4, 8, 2>(xb, A, M, K, r, Xq, sx, xA, 2, status, s);
        if (K <= 2048) return launch_rows<8, 8, 1>(xb, A, M, K, r, Xq, sx, xA, 2, status, s);
        return launch_rows<16, 8, 1>(xb, A, M, K, r, Xq, sx, xA, 1, status, s);
    }
    return launch_quantize_rows(act, X, A, M, K, r, Xq, sx, xA, status, s);
}

}  // namespace qlora
