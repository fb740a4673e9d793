// ckpt.cu -- activations kept in 8 bits between the forward and the backward
// pass, and read back: blocks of 32 consecutive columns of a row share the
// scale amax / 127 (act_epilogue.cuh has the reading, which the GEMM epilogues
// share); rows quantized with one scale each (the forward's input codes) are
// read back by the same call.
//
// Both are bound by HBM: a bf16 element costs 2 + 1 + 1/8 bytes either way.
// One thread takes one block (16 columns when reading back): its bytes are
// whole 32-byte sectors, so a warp needs no exchange between threads and no
// shared memory, and the block's maximum stays in registers.  A warp covers 8
// rows x 4 pieces: runs of 256 bytes per row, and the 8 rows' scales, which
// lie side by side, make one sector.
#include "internal.h"
#include "ptx.cuh"
#include "act_epilogue.cuh"

namespace qlora {

namespace {

constexpr int kCkThreads = 128;
constexpr int kCkRows = 8, kCkPieces = 4;  // of a warp's step

// The (row, piece) pairs of a thread: warps step through the 8 x 4 groups of
// the matrix, along the rows first.  A pair may lie outside the matrix.
struct Pieces {
    size_t group, step, groups;
    int across;
    __device__ __forceinline__ Pieces(int rows, int pieces) {
        across = (pieces + kCkPieces - 1) / kCkPieces;
        groups = static_cast<size_t>((rows + kCkRows - 1) / kCkRows) * across;
        group = blockIdx.x * static_cast<size_t>(kCkThreads / 32) + threadIdx.x / 32;
        step = static_cast<size_t>(gridDim.x) * (kCkThreads / 32);
    }
    __device__ __forceinline__ bool next(int& row, int& piece) {
        if (group >= groups) return false;
        const int lane = threadIdx.x & 31;
        const int g = static_cast<int>(group / across);
        row = g * kCkRows + lane / kCkPieces;
        piece = static_cast<int>(group - static_cast<size_t>(g) * across) * kCkPieces + lane % kCkPieces;
        group += step;
        return true;
    }
};

template <typename T>
__global__ void __launch_bounds__(kCkThreads) ckpt_save_kernel(const T* __restrict__ X, int rows, int cols, int nb,
                                                               bool vec, int8_t* __restrict__ q,
                                                               float* __restrict__ scales) {
    pdl_trigger();
    pdl_wait();
    Pieces it(rows, nb);
    for (int row, b; it.next(row, b);) {
        if (row >= rows || b >= nb) continue;
        RowPiece<T, kCkptBlock> p;
        p.load(X, row, true, b * kCkptBlock, cols, vec);
        float v[kCkptBlock];
#pragma unroll
        for (int e = 0; e < kCkptBlock; ++e) v[e] = 0.f;
        p.add_to(v);
        ckpt_store(v, q, scales, row, rows, b * kCkptBlock, cols);
    }
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) ckpt_load_kernel(const int8_t* __restrict__ q,
                                                               const float* __restrict__ scales, int rows, int cols,
                                                               int nc, int block, bool vec, T* __restrict__ X) {
    pdl_trigger();
    pdl_wait();
    Pieces it(rows, nc);  // 16 columns each
    for (int row, c16; it.next(row, c16);) {
        if (row >= rows || c16 >= nc) continue;
        const int n = c16 * 16;
        const float scale = __ldg(scales + (block ? static_cast<size_t>(n / kCkptBlock) * rows : 0) + row);
        const int8_t* src = q + static_cast<size_t>(row) * cols + n;
        T* dst = X + static_cast<size_t>(row) * cols + n;
        if (vec) {  // cols % 16 == 0
            float v[16];
            ckpt_values16(__ldg(reinterpret_cast<const uint4*>(src)), scale, v);
            constexpr int kPer = 16 / static_cast<int>(sizeof(T));
#pragma unroll
            for (int c = 0; c < 16 / kPer; ++c) {
                T o[kPer];
#pragma unroll
                for (int e = 0; e < kPer; ++e) o[e] = ActIO<T>::from_f(v[c * kPer + e]);
                reinterpret_cast<uint4*>(dst)[c] = *reinterpret_cast<const uint4*>(o);
            }
        } else {
            for (int e = 0; e < 16 && n + e < cols; ++e)
                dst[e] = ActIO<T>::from_f(static_cast<float>(src[e]) * scale);
        }
    }
}

int ck_grid(int rows, int pieces) {
    const size_t warps = static_cast<size_t>((rows + kCkRows - 1) / kCkRows) * ((pieces + kCkPieces - 1) / kCkPieces);
    const size_t b = (warps + kCkThreads / 32 - 1) / (kCkThreads / 32);
    const size_t cap = 16 * static_cast<size_t>(sm_count());
    return static_cast<int>(b < 1 ? 1 : (b > cap ? cap : b));
}

}  // namespace

cudaError_t launch_ckpt_save(Act act, const void* T, int rows, int cols, int8_t* q, float* scales, cudaStream_t s) {
    const int nb = (cols + kCkptBlock - 1) / kCkptBlock;
    const int grid = ck_grid(rows, nb);
    const bool vec = cols % (act == kBF16 ? 8 : 4) == 0;
    if (act == kBF16)
        return launch_k(ckpt_save_kernel<__nv_bfloat16>, dim3(grid), dim3(kCkThreads), 0, s, 1,
                        static_cast<const __nv_bfloat16*>(T), rows, cols, nb, vec, q, scales);
    return launch_k(ckpt_save_kernel<float>, dim3(grid), dim3(kCkThreads), 0, s, 1, static_cast<const float*>(T), rows,
                    cols, nb, vec, q, scales);
}

cudaError_t launch_ckpt_load(Act act, const int8_t* q, const float* scales, int rows, int cols, int block, void* T,
                             cudaStream_t s) {
    const int nc = (cols + 15) / 16;
    const int grid = ck_grid(rows, nc);
    const bool vec = cols % 16 == 0;
    if (act == kBF16)
        return launch_k(ckpt_load_kernel<__nv_bfloat16>, dim3(grid), dim3(kCkThreads), 0, s, 1, q, scales, rows, cols,
                        nc, block, vec, static_cast<__nv_bfloat16*>(T));
    return launch_k(ckpt_load_kernel<float>, dim3(grid), dim3(kCkThreads), 0, s, 1, q, scales, rows, cols, nc, block,
                    vec, static_cast<float*>(T));
}

}  // namespace qlora
