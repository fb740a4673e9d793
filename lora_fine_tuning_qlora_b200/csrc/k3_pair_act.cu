// k3_pair_act.cu -- dX of large layers from the kernel de-quantized once into a
// workspace: a pass that writes Wd = bf16(Wq sw), then the CTA-pair GEMM
// dY Wd with the rank-r term, act'(z) and the added gradient in its epilogue
// (pair_act.cuh).
//
// ("How to fine-tune the 4-bit model?" thread: de-quantize, then the matrix
// unit.)  The kernels that de-quantize in shared memory convert the whole
// kernel once per 256 rows of dY, and that conversion, not the tensor cores,
// sets their pace; for many rows one pass over the kernel (3 bytes per weight,
// most of it in L2) is cheaper.
#include "pair_act.cuh"

namespace qlora {

namespace {

constexpr int kDqThreads = 256;

// 16 codes (int8) or 32 (packed int4) a thread and step; the same rounding as
// in the kernels that de-quantize in shared memory: to bf16, since the products
// take both operands in one 16-bit type and dY needs the range of bf16.  A second
// bf16 term of the kernel would double the products, which bound these layers.
template <bool W4>
__global__ void __launch_bounds__(kDqThreads) dequantize_kernel(const uint8_t* __restrict__ Wq,
                                                                const float* __restrict__ sw, int N, int K,
                                                                uint4* __restrict__ Wd) {
    pdl_trigger();
    pdl_wait();
    constexpr int kCodes = W4 ? 32 : 16;
    const int per_row = K / kCodes;
    const size_t items = static_cast<size_t>(N) * per_row;
    for (size_t i = blockIdx.x * static_cast<size_t>(kDqThreads) + threadIdx.x; i < items;
         i += static_cast<size_t>(gridDim.x) * kDqThreads) {
        const float scale = __ldg(sw + i / per_row);
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(Wq) + i);
        uint4 part[2] = {raw, raw};
        if constexpr (W4) unpack_int4x32(raw, part[0], part[1]);
#pragma unroll
        for (int h = 0; h < (W4 ? 2 : 1); ++h) {
            uint32_t o[8];
            dequant16(part[h], scale, o);
            uint4* dst = Wd + i * (kCodes / 8) + 2 * h;
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

}  // namespace

// Where the extra pass pays, in us against the kernels that de-quantize in
// shared memory (graph replays, SILU and an added gradient): K 4096, N 4096: 512
// rows 44 / 51, 1024 46 / 47, 4096 126 / 145, 8192 227 / 260; K 16384, N 2048:
// 512 rows 61 / 55, 1024 88 / 100, 8192 492 / 653; K 2304, N 768: 2048 rows 20 /
// 23.  So from 1024 rows, from 512 for kernels of up to 2^24 weights, and for
// grids of at least 20 tiles (12 tiles: 18.9 / 18.3).
constexpr int kDenseMinM = 1024, kDenseMinMSmall = 512;
constexpr size_t kDenseSmall = size_t{1} << 24;
constexpr int kDenseMinTiles = 20;

size_t dx_dense_bytes(Act act, int M, int N, int K, int r) {
    const size_t weights = static_cast<size_t>(N) * K;
    if (act != kBF16 || N % 8 != 0 || r > 16) return 0;
    if (M < (weights <= kDenseSmall ? kDenseMinMSmall : kDenseMinM)) return 0;
    const long long tiles = static_cast<long long>((M + 2 * kTM - 1) / (2 * kTM)) * ((K + kTN - 1) / kTN);
    return tiles >= kDenseMinTiles ? weights * 2 : 0;
}

cudaError_t launch_dequantize(const void* Wq, const float* sw, int N, int K, bool w4, void* Wd, cudaStream_t s) {
    const size_t items = static_cast<size_t>(N) * (K / (w4 ? 32 : 16));
    const size_t want = (items + kDqThreads - 1) / kDqThreads;
    const size_t cap = 8 * static_cast<size_t>(sm_count());
    const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
    auto run = [&](auto kern) {
        return launch_k(kern, grid, dim3(kDqThreads), 0, s, 1, static_cast<const uint8_t*>(Wq), sw, N, K,
                        static_cast<uint4*>(Wd));
    };
    return w4 ? run(dequantize_kernel<true>) : run(dequantize_kernel<false>);
}

cudaError_t launch_gemm_dx_dense(const void* dY, const void* Wd, int M, int N, int K, const DxEpilogue& ep,
                                 int* status, cudaStream_t s) {
    PairActArgs a{};
    a.M = M;
    a.N = K;
    a.K = N;
    a.r = ep.r;
    a.c = ep.c;
    a.rowf = ep.Gp;
    a.nsl = ep.ncb;
    a.colf = ep.A;
    a.cs_j = 1;
    a.cs_n = ep.r;
    a.act = ep.act;
    a.add = ep.add != nullptr;
    a.ztma = ep.act != kActNone;
    a.zs_in = ep.zs;
    CUtensorMap ta, tb, to, tadd, tz;
    if (!make_tmap_2d(&ta, dY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, N, static_cast<uint64_t>(N) * 2, kTM, 64,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tmap_2d(&tb, Wd, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, N, K, static_cast<uint64_t>(K) * 2, 64, 64,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
        !pair_act_maps(a, ep.dX, ep.add, ep.zq, &to, &tadd, &tz))
        return cudaErrorInvalidValue;
    if (ep.r <= 4) return launch_pair_act<4, false, 8>(ta, tb, to, tadd, tz, a, status, s);
    if (ep.r <= 8) return launch_pair_act<8, false, 8>(ta, tb, to, tadd, tz, a, status, s);
    return launch_pair_act<16, false, 8>(ta, tb, to, tadd, tz, a, status, s);
}

}  // namespace qlora
