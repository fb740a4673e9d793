// ckpt.cu -- activations kept in 8 bits between the forward and the backward
// pass, and read back: blocks of 32 consecutive columns of a row share the
// scale amax / 127 (act_epilogue.cuh has the reading, which the GEMM epilogues
// share); rows quantized with one scale each (the forward's input codes) are
// read back by the same call.
//
// Both are bound by HBM: a bf16 element costs 2 + 1 + 1/8 bytes either way.
// A lane takes 16 columns (reading back: 8) of 8 consecutive rows: neighbouring
// lanes touch neighbouring bytes, several rows' loads are in flight together,
// two lanes make a block (a shuffle finds its maximum), and the 8 rows' scales
// of a block lie side by side in one sector.  At 16384 x 4096 a lane that
// owned a whole block of one row read back in 44 us, against 33 us now.
#include "internal.h"
#include "ptx.cuh"
#include "act_epilogue.cuh"

namespace qlora {

namespace {

constexpr int kCkThreads = 128;
constexpr int kCkRows = 8;  // rows of a lane's step

// The steps of a thread: `chunks` 8-column chunks across, groups of 8 rows
// down.  A warp's lanes lie along the columns (lanes_c of them, a power of
// two of at least 4) and, for narrow matrices, over further row groups.
struct Steps {
    size_t at, step, total;
    int across, lanes_c, shift, lane;
    __device__ __forceinline__ Steps(int rows, int chunks, int lanes_log2) {
        shift = lanes_log2;
        lanes_c = 1 << lanes_log2;
        lane = threadIdx.x & 31;
        across = (chunks + lanes_c - 1) >> lanes_log2;
        const int down = (rows + kCkRows * (32 >> lanes_log2) - 1) / (kCkRows * (32 >> lanes_log2));
        total = static_cast<size_t>(down) * across;
        at = blockIdx.x * static_cast<size_t>(kCkThreads / 32) + threadIdx.x / 32;
        step = static_cast<size_t>(gridDim.x) * (kCkThreads / 32);
    }
    __device__ __forceinline__ bool next(int& row0, int& chunk) {
        if (at >= total) return false;
        const size_t g = at / across;
        row0 = static_cast<int>(g * (32 >> shift) + (lane >> shift)) * kCkRows;
        chunk = static_cast<int>(at - g * across) * lanes_c + (lane & (lanes_c - 1));
        at += step;
        return true;
    }
};

// E columns (8 or 16) a lane and row; columns a multiple of E.  With 16, two
// lanes make a block: half the divisions and shuffles per element (42 us with
// 8 at 16384 x 4096).
template <typename T, int E>
__global__ void __launch_bounds__(kCkThreads) ckpt_save_kernel(const T* __restrict__ X, int rows, int cols, int lanes,
                                                               int8_t* __restrict__ q, float* __restrict__ scales) {
    constexpr int kSub = kCkRows / 2;              // rows whose loads are in flight together
    constexpr int kShare = kCkptBlock / E;         // lanes of a block
    pdl_trigger();
    pdl_wait();
    const int chunks = cols / E;
    Steps it(rows, chunks, lanes);
    for (int row0, c; it.next(row0, c);) {
        const bool in = c < chunks;
        float* sc = scales + static_cast<size_t>(c / kShare) * rows + row0;
#pragma unroll
        for (int u0 = 0; u0 < kCkRows; u0 += kSub) {
            RowPiece<T, E> raw[kSub];
#pragma unroll
            for (int u = 0; u < kSub; ++u)
                raw[u].load(X, row0 + u0 + u, in && row0 + u0 + u < rows, c * E, cols, true);
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                float f[E];
#pragma unroll
                for (int e = 0; e < E; ++e) f[e] = 0.f;
                raw[u].add_to(f);
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) top = max(top, abs_bits(f[e]));
#pragma unroll
                for (int o = 1; o < kShare; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                float inv, scale;
                ckpt_scale(top, inv, scale);
                const int row = row0 + u0 + u;
                if (in && row < rows) {
                    int8_t* dst = q + static_cast<size_t>(row) * cols + c * E;
                    uint2 w[E / 8];
#pragma unroll
                    for (int h = 0; h < E / 8; ++h) {
                        float g[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) g[e] = f[8 * h + e];
                        w[h] = codes8(g, inv);
                    }
                    if constexpr (E == 16) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0].x, w[0].y, w[E / 8 - 1].x, w[E / 8 - 1].y);
                    else *reinterpret_cast<uint2*>(dst) = w[0];
                    if (c % kShare == 0) sc[u0 + u] = scale;
                }
            }
        }
    }
}

// Columns a multiple of 8.  block 32, or 0: one scale per row.
template <typename T>
__global__ void __launch_bounds__(kCkThreads) ckpt_load_kernel(const int8_t* __restrict__ q,
                                                               const float* __restrict__ scales, int rows, int cols,
                                                               int lanes, int block, T* __restrict__ X) {
    pdl_trigger();
    pdl_wait();
    const int chunks = cols / 8;
    Steps it(rows, chunks, lanes);
    for (int row0, c; it.next(row0, c);) {
        if (c >= chunks) continue;
        uint2 raw[kCkRows];
        float s[kCkRows];
        const float* sc = scales + (block ? static_cast<size_t>(c / 4) * rows : 0) + row0;
#pragma unroll
        for (int u = 0; u < kCkRows; ++u) {
            const bool in = row0 + u < rows;
            raw[u] = in ? __ldg(reinterpret_cast<const uint2*>(q + static_cast<size_t>(row0 + u) * cols + c * 8))
                        : make_uint2(0u, 0u);
            s[u] = in ? __ldg(sc + u) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kCkRows; ++u) {
            if (row0 + u >= rows) break;
            float v[16];
            ckpt_values16(make_uint4(raw[u].x, raw[u].y, 0u, 0u), s[u], v);
            uint4* dst = reinterpret_cast<uint4*>(X + static_cast<size_t>(row0 + u) * cols + c * 8);
            if constexpr (sizeof(T) == 2) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                    w[k] = *reinterpret_cast<const uint32_t*>(&h);
                }
                dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    dst[k] = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]),
                                        __float_as_uint(v[4 * k + 2]), __float_as_uint(v[4 * k + 3]));
            }
        }
    }
}

// Any column count: a warp takes blocks of 32 columns, a lane each, of kCkRows
// consecutive rows, element by element.
template <typename T>
__global__ void __launch_bounds__(kCkThreads) ckpt_save_any_kernel(const T* __restrict__ X, int rows, int cols, int nb,
                                                                   int8_t* __restrict__ q, float* __restrict__ scales) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const size_t total = static_cast<size_t>((rows + kCkRows - 1) / kCkRows) * nb;
    for (size_t w = blockIdx.x * static_cast<size_t>(kCkThreads / 32) + threadIdx.x / 32; w < total;
         w += static_cast<size_t>(gridDim.x) * (kCkThreads / 32)) {
        const int g = static_cast<int>(w / nb), b = static_cast<int>(w - static_cast<size_t>(g) * nb);
        const int row0 = g * kCkRows, col = b * kCkptBlock + lane;
        float v[kCkRows];
#pragma unroll
        for (int u = 0; u < kCkRows; ++u)
            v[u] = col < cols && row0 + u < rows ? ActIO<T>::to_f(X[static_cast<size_t>(row0 + u) * cols + col]) : 0.f;
#pragma unroll
        for (int u = 0; u < kCkRows; ++u) {
            float inv, scale;
            ckpt_scale(__reduce_max_sync(0xffffffffu, abs_bits(v[u])), inv, scale);
            if (row0 + u >= rows) break;
            if (col < cols) q[static_cast<size_t>(row0 + u) * cols + col] = static_cast<int8_t>(quant_code(v[u], inv));
            if (lane == 0) scales[static_cast<size_t>(b) * rows + row0 + u] = scale;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kCkThreads) ckpt_load_any_kernel(const int8_t* __restrict__ q,
                                                                   const float* __restrict__ scales, int rows, int cols,
                                                                   int nb, int block, T* __restrict__ X) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const size_t total = static_cast<size_t>((rows + kCkRows - 1) / kCkRows) * nb;
    for (size_t w = blockIdx.x * static_cast<size_t>(kCkThreads / 32) + threadIdx.x / 32; w < total;
         w += static_cast<size_t>(gridDim.x) * (kCkThreads / 32)) {
        const int g = static_cast<int>(w / nb), b = static_cast<int>(w - static_cast<size_t>(g) * nb);
        const int row0 = g * kCkRows, col = b * kCkptBlock + lane;
        if (col >= cols) continue;
        float v[kCkRows];
#pragma unroll
        for (int u = 0; u < kCkRows; ++u) {
            const int row = row0 + u < rows ? row0 + u : rows - 1;
            v[u] = static_cast<float>(q[static_cast<size_t>(row) * cols + col]) *
                   __ldg(scales + (block ? static_cast<size_t>(b) * rows : 0) + row);
        }
#pragma unroll
        for (int u = 0; u < kCkRows; ++u)
            if (row0 + u < rows) X[static_cast<size_t>(row0 + u) * cols + col] = ActIO<T>::from_f(v[u]);
    }
}

// log2 of the lanes along the columns, at least a whole block's
int ck_lanes(int chunks) {
    int l = 2;
    while (l < 5 && (1 << l) < chunks) ++l;
    return l;
}

dim3 ck_grid(size_t warps) {
    const size_t b = (warps + kCkThreads / 32 - 1) / (kCkThreads / 32);
    const size_t cap = 16 * static_cast<size_t>(sm_count());
    return dim3(static_cast<unsigned>(b < 1 ? 1 : (b > cap ? cap : b)));
}

size_t ck_warps(int rows, int chunks, int lanes) {
    const size_t down = (static_cast<size_t>(rows) + kCkRows * (32 >> lanes) - 1) / (kCkRows * (32 >> lanes));
    return down * ((chunks + (1 << lanes) - 1) >> lanes);
}

template <typename T>
cudaError_t save_t(const T* X, int rows, int cols, int8_t* q, float* scales, cudaStream_t s) {
    if (cols % 8 == 0) {
        const int chunks = cols % 16 == 0 ? cols / 16 : cols / 8;
        const int lanes = ck_lanes(chunks);
        auto kern = cols % 16 == 0 ? ckpt_save_kernel<T, 16> : ckpt_save_kernel<T, 8>;
        return launch_k(kern, ck_grid(ck_warps(rows, chunks, lanes)), dim3(kCkThreads), 0, s, 1, X, rows, cols, lanes,
                        q, scales);
    }
    const int nb = (cols + kCkptBlock - 1) / kCkptBlock;
    return launch_k(ckpt_save_any_kernel<T>, ck_grid(static_cast<size_t>((rows + kCkRows - 1) / kCkRows) * nb),
                    dim3(kCkThreads), 0, s, 1, X, rows, cols, nb, q, scales);
}

template <typename T>
cudaError_t load_t(const int8_t* q, const float* scales, int rows, int cols, int block, T* X, cudaStream_t s) {
    if (cols % 8 == 0) {
        const int lanes = ck_lanes(cols / 8);
        return launch_k(ckpt_load_kernel<T>, ck_grid(ck_warps(rows, cols / 8, lanes)), dim3(kCkThreads), 0, s, 1, q,
                        scales, rows, cols, lanes, block, X);
    }
    const int nb = (cols + kCkptBlock - 1) / kCkptBlock;
    return launch_k(ckpt_load_any_kernel<T>, ck_grid(static_cast<size_t>((rows + kCkRows - 1) / kCkRows) * nb),
                    dim3(kCkThreads), 0, s, 1, q, scales, rows, cols, nb, block, X);
}

}  // namespace

cudaError_t launch_ckpt_save(Act act, const void* T, int rows, int cols, int8_t* q, float* scales, cudaStream_t s) {
    return act == kBF16 ? save_t(static_cast<const __nv_bfloat16*>(T), rows, cols, q, scales, s)
                        : save_t(static_cast<const float*>(T), rows, cols, q, scales, s);
}

cudaError_t launch_ckpt_load(Act act, const int8_t* q, const float* scales, int rows, int cols, int block, void* T,
                             cudaStream_t s) {
    return act == kBF16 ? load_t(q, scales, rows, cols, block, static_cast<__nv_bfloat16*>(T), s)
                        : load_t(q, scales, rows, cols, block, static_cast<float*>(T), s);
}

}  // namespace qlora
