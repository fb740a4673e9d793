// tma_epilogue.cuh -- the warp-private shared-memory pieces of a GEMM epilogue
// whose rows move by TMA: 32 rows x 32 columns, as bf16 (64-byte rows, 64-byte
// swizzle) or as 8-bit codes (32-byte rows, 32-byte swizzle).  A bf16 piece
// receives what the epilogue adds (the residual, or a gradient) while the
// piece before is computed, each lane turns its row's values into outputs in
// place, and one bulk store writes the piece.  Against per-lane 16-byte
// accesses to 32 different rows, the loads hold no registers and the rows
// move in whole sectors with one instruction (forward at 16384 x 4096 x 4096
// with a residual: 246 -> 209 us with a ReLU).
#pragma once

#include "act_epilogue.cuh"
#include "ptx.cuh"

namespace qlora {

constexpr int kPieceCols = 32;
constexpr int kPieceBytes = 32 * kPieceCols * 2;
constexpr int kCodePieceBytes = 32 * kPieceCols;
static_assert(kPieceCols == kCkptBlock, "one checkpoint block per piece row");

// 16-byte chunk ch (0 .. 3) of row r of a bf16 piece.  The eight rows of a
// shared-memory phase fall on eight different 16-byte bank groups.
__device__ __forceinline__ uint4* piece_chunk(uint8_t* piece, int r, int ch) {
    return reinterpret_cast<uint4*>(piece + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
}

// 16-byte chunk ch (0, 1) of row r of a code piece.
__device__ __forceinline__ uint4* code_chunk(uint8_t* piece, int r, int ch) {
    return reinterpret_cast<uint4*>(piece + r * 32 + ((ch ^ ((r >> 2) & 1)) << 4));
}

// y += the row's values
__device__ __forceinline__ void piece_add(uint8_t* piece, int r, float (&y)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 u = *piece_chunk(piece, r, i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            y[8 * i + 2 * k] += __uint_as_float(w[k] << 16);
            y[8 * i + 2 * k + 1] += __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
}

// the row's outputs, rounded to bf16
__device__ __forceinline__ void piece_put(uint8_t* piece, int r, const float (&y)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(y[8 * i + 2 * k], y[8 * i + 2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *piece_chunk(piece, r, i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Persistent GEMMs: tile t of an mt x nt grid of tiles, in groups of
// kRasterRows tile rows walked down first, so that the tiles in flight at a
// time cover a near-square region and share operand tiles in L2.
constexpr int kRasterRows = 8;
__device__ __forceinline__ void raster_tile(int t, int mt, int nt, int& m, int& n) {
    const int per = kRasterRows * nt;
    const int g = t / per, rest = t - g * per;
    const int rows = min(kRasterRows, mt - g * kRasterRows);
    n = rest / rows;
    m = g * kRasterRows + rest - n * rows;
}

}  // namespace qlora
