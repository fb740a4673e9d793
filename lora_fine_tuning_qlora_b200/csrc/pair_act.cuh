// pair_act.cuh -- a persistent GEMM on CTA pairs whose both operands arrive by
// TMA, with the layer's activation epilogues:
//
//   forward  Z = (Xq Wq^T) sx sw + bias + (c xA) B     int8 operands
//            Y = act(Z) + res, Z kept in 8 bits
//   dX       (dY Wd + (c G) A^T) * act'(z) + add       bf16 operands, Wd the
//            kernel de-quantized to bf16 beforehand, z read from 8 bits
//
// ("Introduce QLoRA-like technique", Results, and "Parameter-efficient
// fine-tuning of GPT-2 with LoRA", "LoRA equation", for the two products.)
// A cluster of two CTAs computes a 256 x 256 tile: CTA r loads rows
// [128 r, 128 r + 128) of the left operand and columns [128 r, 128 r + 128) of
// the right one, 128 bytes of the contraction per stage, and holds its 128
// rows x 256 columns of the accumulator in TMEM, twice, so that a tile's
// epilogue runs under the next tile's products.
//
// What bounds it: the tensor cores, once the epilogue of a tile takes less
// than its products.  The epilogue is bound by instruction latency (forward at
// 4096 x 2048 x 16384 with GELU(tanh) and checkpoint, W = 16: 0.47 instructions
// per scheduler and cycle, the conversion / exponential pipe 26% busy, ALU 31%,
// tensor 42%), so it runs on many warps (W, two or four per scheduler), takes
// its rank-r sums in paired fp32 instructions, and fetches the next tile's row
// and column factors while the current one is computed.  Forward, 16384 x 4096 x 4096 bf16 rank 4,
// GELU(tanh) + residual + checkpoint: 289 us with four epilogue warps, 237 with
// eight (the forward's launch rule has W).  With SILU + residual 204 us, 2.7
// PTOP/s; dX of that size 400 us, 1.37 PFLOP/s, the rate at which plain bf16
// products run under the power cap.
//
// Warps per CTA: 0 TMA producer; 1 TMEM owner and, in CTA 0, MMA issuer; then
// W epilogue warps, W / 4 per TMEM lane quarter, each with its own columns.
// Barriers as in the other pair kernels; every wait is bounded.  The pieces'
// barriers belong to one warp each, so one epilogue warp can give up alone: it
// then skips its tiles but still counts at the named barriers of all of them,
// which have no limit of their own.
#pragma once

#include "dx_common.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "act_epilogue.cuh"
#include "tile_epilogue.cuh"
#include "tma_epilogue.cuh"

namespace qlora {

namespace {

constexpr int kTM = 128;               // rows per CTA (256 per pair)
constexpr int kTN = 256;               // columns per tile (128 of the right operand per CTA)
constexpr int kPairSmemLimit = 232448;

struct PairActArgs {
    int M, N, K;          // output rows, output columns, contraction
    int r;
    float c;
    const float* rowf;    // [M, r] (forward xA) or nsl slices of it (dX, G)
    int nsl;
    const float* colf;    // column factor: element (j, n) at colf[j * cs_j + n * cs_n]
    size_t cs_j, cs_n;
    const float* sx;      // forward: row scale
    const float* sw;      // forward: column scale
    const float* bias;    // forward: [N] or null
    int act;
    int add;              // whether tmAdd is read
    int8_t* zq;           // forward: codes of Z (rows not a multiple of 16 bytes), or null
    int ztma;             // forward: codes of Z go out by tmZ; dX: codes of z come in by tmZ
    float* zs_out;        // forward: scales of Z, or null
    const float* zs_in;   // dX: scales of z
};

template <int RP, bool FWD, int W>
struct PairActCfg {
    static constexpr int kStageBytes = 2 * kTM * 128;     // 128 bytes of contraction of both operands
    static constexpr int kCodeBufs = FWD ? 1 : 2;
    static constexpr int kWarpBytes = 2 * kPieceBytes + kCodeBufs * kCodePieceBytes;
    static constexpr int kTabFloats = kTN * (RP + (FWD ? 2 : 0));
    static constexpr int kFixed = W * kWarpBytes + kTabFloats * 4 + 512 + 1024;
    static constexpr int kFit = (kPairSmemLimit - kFixed) / kStageBytes;
    static constexpr int STAGES = kFit > 6 ? 6 : kFit;
    static_assert(STAGES >= 4, "shared memory budget");
    static constexpr int kPieceOff = STAGES * kStageBytes;
    static constexpr int kCodeOff = kPieceOff + W * 2 * kPieceBytes;
    static constexpr int kTabOff = kPieceOff + W * kWarpBytes;
    static constexpr int kBarOff = kTabOff + kTabFloats * 4;
    static constexpr int kTotal = kBarOff + 512 + 1024;
    static_assert((2 * STAGES + 4 + 2 * W) * 8 + 4 <= 512, "barrier area");
    static constexpr int kThreads = 32 * (2 + W);
    static constexpr int kCols = kTN / (W / 4);           // columns of a tile per epilogue warp
};

template <int RP, bool FWD, int W>
__global__ void __launch_bounds__(PairActCfg<RP, FWD, W>::kThreads, 1)
    pair_act_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmAdd,
                    const __grid_constant__ CUtensorMap tmZ, PairActArgs a, int* status) {
    using C = PairActCfg<RP, FWD, W>;
    constexpr int S = C::STAGES;
    constexpr int kET = 32 * W;                     // epilogue threads
    constexpr int kKS = FWD ? 128 : 64;             // contraction elements per stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // [S] (CTA 0)
    uint64_t* empty = full + S;                                       // [S]
    uint64_t* tfull = empty + S;                                      // [2]
    uint64_t* tempty = tfull + 2;                                     // [2] (CTA 0)
    uint64_t* pbars = tempty + 2;                                     // [W][2] a warp's pieces landed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pbars + 2 * W);
    // column factors of a tile, two columns' values of one j side by side:
    // element (j, col) at [col / 2][j][col % 2]; then sw and bias (forward)
    float* sF = reinterpret_cast<float*>(smem + C::kTabOff);
    float* sSw = sF + kTN * RP;
    float* sBias = sSw + kTN;

    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const int pair = static_cast<int>(blockIdx.x) / 2;
    const int npairs = static_cast<int>(gridDim.x) / 2;
    const int M = a.M, N = a.N;
    const int num_mt = (M + 2 * kTM - 1) / (2 * kTM);
    const int num_nt = (N + kTN - 1) / kTN;
    const int tiles = num_mt * num_nt;
    const int nkb = (a.K + kKS - 1) / kKS;
    // this CTA's first row and the first column of tile t
    auto tile_at = [&](int t, int& m0, int& n0) {
        raster_tile(t, num_mt, num_nt, m0, n0);
        m0 = m0 * 2 * kTM + static_cast<int>(rank) * kTM;
        n0 *= kTN;
    };
    if constexpr (FWD) pdl_trigger();

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * W);
        }
        for (int i = 0; i < 2 * W; ++i) mbar_init(&pbars[i], 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // neither CTA signals the other's barriers before both have initialised them
    cluster_arrive();
    cluster_wait();
    pdl_wait();  // nothing above touched global memory
    if constexpr (!FWD) pdl_trigger();  // after the wait: see launch_rank_x_q

    if (warp == 0) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmB);
            const uint32_t full0 = dsmem_addr(full, 0);  // CTA 0's full[0]
            int g = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += npairs) {
                int m0, n0;
                tile_at(t, m0, n0);
                n0 += static_cast<int>(rank) * (kTN / 2);
                for (int kb = 0; kb < nkb; ++kb, ++g) {
                    const int s = g % S;
                    if (g >= S && !mbar_wait(&empty[s], ((g / S) - 1) & 1, status)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sa = smem + s * C::kStageBytes;
                    uint8_t* sb = sa + kTM * 128;
                    const uint32_t fb = full0 + 8u * static_cast<uint32_t>(s);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStageBytes);
                    tma_load_2d_pair(sa, &tmA, fb, kb * kKS, m0);
                    if constexpr (FWD) {
                        tma_load_2d_pair(sb, &tmB, fb, kb * kKS, n0);
                    } else {
                        // 64 contraction rows x two blocks of 64 columns (MN-major)
                        tma_load_2d_pair(sb, &tmB, fb, n0, kb * kKS);
                        tma_load_2d_pair(sb + 8192, &tmB, fb, n0 + 64, kb * kKS);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer (CTA 0)
        if (rank == 0 && lane == 0) {
            int g = 0, i = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += npairs, ++i) {
                const int ab = i & 1;
                const int use = i >> 1;
                if (use > 0 && !mbar_wait(&tempty[ab], (use - 1) & 1, status)) break;
                tc_fence_after();
                const uint32_t dacc = tmem + ab * kTN;
                for (int kb = 0; kb < nkb; ++kb, ++g) {
                    const int s = g % S;
                    if (!mbar_wait(&full[s], (g / S) & 1, status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ab_ = smem_u32(smem + s * C::kStageBytes);
                    const uint32_t bb = ab_ + kTM * 128;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t ad = smem_desc(ab_ + kk * 32, 16, 1024, kLayoutSw128);
                        const uint32_t acc = (kb != 0 || kk != 0) ? 1u : 0u;
                        if constexpr (FWD) {
                            const uint64_t bd = smem_desc(bb + kk * 32, 16, 1024, kLayoutSw128);
                            mma_i8_pair(dacc, ad, bd, idesc_i8(2 * kTM, kTN), acc);
                        } else {
                            const uint64_t bd = smem_desc(bb + kk * 2048, 8192, 1024, kLayoutSw128);
                            mma_bf16_pair(dacc, ad, bd, idesc_bf16(2 * kTM, kTN, false, true), acc);
                        }
                    }
                    mma_commit_pair(&empty[s], 0x3);
                }
                if (ok) mma_commit_pair(&tfull[ab], 0x3);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue
        const int ew = warp - 2;
        const int q = warp & 3;                  // TMEM lane quarter of this warp
        const int cw = (ew >> 2) * C::kCols;     // this warp's first column of a tile
        const int et = threadIdx.x - 64;
        const uint32_t tempty0 = dsmem_addr(tempty, 0);
        uint8_t* pieces = smem + C::kPieceOff + ew * 2 * kPieceBytes;
        uint8_t* codes = smem + C::kCodeOff + ew * C::kCodeBufs * kCodePieceBytes;
        uint64_t* pbar = pbars + 2 * ew;
        const bool zin = !FWD && a.ztma;                  // codes of z come in
        const bool zout = FWD && a.zs_out != nullptr;     // Z goes out in 8 bits
        const bool loads = a.add || zin;
        const uint32_t load_bytes = (a.add ? kPieceBytes : 0) + (zin ? kCodePieceBytes : 0);

        // Pieces are numbered over all of the warp's tiles; piece i uses
        // buffers i % 2.  Their loads are issued a piece ahead.
        int piece = 0, issued = 0;
        auto load_piece = [&](int row, int n) {
            if (lane == 0) {
                const int b = issued & 1;
                mbar_arrive_expect_tx(&pbar[b], load_bytes);
                if (a.add) tma_load_2d(pieces + b * kPieceBytes, &tmAdd, &pbar[b], n, row);
                if (zin) tma_load_2d(codes + (b % C::kCodeBufs) * kCodePieceBytes, &tmZ, &pbar[b], n, row);
            }
            ++issued;
        };
        float zs_next = 0.f;  // dX: scale of the next piece's block of this lane's row
        auto fetch_piece = [&](int t, int m0, int n) {
            (void)t;
            const int row = m0 + q * 32 + lane;
            if (zin) zs_next = row < M ? __ldg(a.zs_in + static_cast<size_t>(n / kCkptBlock) * M + row) : 0.f;
            if (loads) load_piece(m0 + q * 32, n);
        };
        // the first piece of this warp from tile t on
        auto fetch_tile = [&](int t) {
            for (; t < tiles; t += npairs) {
                int m0, n0;
                tile_at(t, m0, n0);
                if (n0 + cw < N) {
                    fetch_piece(t, m0, n0 + cw);
                    return;
                }
            }
        };
        // a tile's row and column factors, loaded a tile ahead
        constexpr int kPer = kTN * RP / kET;
        constexpr int kVec = (2 * kTN + kET - 1) / kET;
        float ft[kPer], fv[kVec], fsx = 0.f, frow[RP];
        auto fetch_factors = [&](int t) {
            if (t >= tiles) return;
            int m0, n0;
            tile_at(t, m0, n0);
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int e = et + u * kET;
                const int j = FWD ? e / kTN : e % RP, n = n0 + (FWD ? e % kTN : e / RP);
                ft[u] = (n < N && j < a.r) ? __ldg(a.colf + j * a.cs_j + n * a.cs_n) : 0.f;
            }
            if constexpr (FWD) {
#pragma unroll
                for (int u = 0; u < kVec; ++u) {
                    const int e = et + u * kET;
                    const int n = n0 + e % kTN;
                    const float* src = e < kTN ? a.sw : a.bias;
                    fv[u] = (n < N && src) ? __ldg(src + n) : 0.f;
                }
            }
            const int row = m0 + q * 32 + lane;
            const bool row_ok = row < M;
            if constexpr (FWD) fsx = row_ok ? __ldg(a.sx + row) : 0.f;
            const size_t slice = static_cast<size_t>(M) * a.r;
#pragma unroll
            for (int j = 0; j < RP; ++j)
                frow[j] = !(row_ok && j < a.r) ? 0.f
                          : FWD               ? __ldg(a.rowf + static_cast<size_t>(row) * a.r + j)
                                              : sum_slices(a.rowf + static_cast<size_t>(row) * a.r + j, slice, a.nsl);
        };
        fetch_factors(pair);
        fetch_tile(pair);
        bool ok = true;  // false once a wait of this warp gave up
        int i = 0;
        for (int t = pair; t < tiles; t += npairs, ++i) {
            const int ab = i & 1;
            const int use = i >> 1;
            int m0, n0;
            tile_at(t, m0, n0);
            const int row0 = m0 + q * 32;
            const int row = row0 + lane;
            const bool row_ok = row < M;
            named_bar_sync(1, kET);  // the last tile's tables are read
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int e = et + u * kET;
                const int j = FWD ? e / kTN : e % RP, col = FWD ? e % kTN : e / RP;
                sF[(col >> 1) * 2 * RP + 2 * j + (col & 1)] = ft[u];
            }
            if constexpr (FWD) {
#pragma unroll
                for (int u = 0; u < kVec; ++u)
                    if (et + u * kET < 2 * kTN) sSw[et + u * kET] = fv[u];
            }
            named_bar_sync(1, kET);
            unsigned long long rf[RP];  // (c row factor), twice
#pragma unroll
            for (int j = 0; j < RP; ++j) rf[j] = pk2(frow[j] * a.c, frow[j] * a.c);
            const unsigned long long sx2 = pk2(fsx, fsx);
            fetch_factors(t + npairs);
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&tfull[ab], use & 1, status));
            if (!ok) continue;  // the other warps may still meet at the next tile's named barriers
            tc_fence_after();
            const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + ab * kTN;
            bool given_back = false;
            auto give_back = [&] {  // the accumulator is read: the MMAs may have it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(&tempty[ab]);
                    else mbar_arrive_remote_cta(tempty0 + 8u * static_cast<uint32_t>(ab));
                }
                given_back = true;
            };
#pragma unroll 1
            for (int col = cw; col < cw + C::kCols && n0 + col < N; col += kPieceCols, ++piece) {
                uint8_t* pc = pieces + (piece & 1) * kPieceBytes;
                const bool last = col + kPieceCols >= cw + C::kCols || n0 + col + kPieceCols >= N;
                // the buffers that this step or the next piece's loads write have
                // been read by the stores before
                if (lane == 0) {
                    if (loads || zout) bulk_wait_read<0>();
                    else bulk_wait_read<1>();
                }
                __syncwarp();
                const float zscale = zs_next;
                if (!last) fetch_piece(t, m0, n0 + col + kPieceCols);
                else fetch_tile(t + npairs);
                uint32_t v0[kEpiCols], v1[kEpiCols];
                tmem_ld16(tbase + col, v0);
                tmem_ld16(tbase + col + kEpiCols, v1);
                if (loads) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&pbar[piece & 1], (piece >> 1) & 1, status));
                    if (!ok) {
                        tmem_ld_wait();
                        break;
                    }
                }
                tmem_ld_wait();
                if (last) give_back();
                float y[32];
#pragma unroll
                for (int p = 0; p < 16; ++p) {  // two columns at a time
                    const uint32_t u0 = p < 8 ? v0[2 * p] : v1[2 * p - 16];
                    const uint32_t u1 = p < 8 ? v0[2 * p + 1] : v1[2 * p - 15];
                    unsigned long long z2;
                    if constexpr (FWD) {
                        unsigned long long f2;
                        asm("mul.rn.f32x2 %0, %1, %2;"
                            : "=l"(f2)
                            : "l"(pk2(static_cast<float>(static_cast<int32_t>(u0)),
                                      static_cast<float>(static_cast<int32_t>(u1)))),
                              "l"(sx2));
                        z2 = *reinterpret_cast<const unsigned long long*>(sBias + col + 2 * p);
                        fma2(z2, f2, *reinterpret_cast<const unsigned long long*>(sSw + col + 2 * p));
                    } else {
                        z2 = pk2(__uint_as_float(u0), __uint_as_float(u1));
                    }
                    const ulonglong2* f = reinterpret_cast<const ulonglong2*>(sF + (col / 2 + p) * 2 * RP);
#pragma unroll
                    for (int j2 = 0; j2 < RP / 2; ++j2) {
                        const ulonglong2 b = f[j2];
                        fma2(z2, rf[2 * j2], b.x);
                        fma2(z2, rf[2 * j2 + 1], b.y);
                    }
                    unpk2(z2, y[2 * p], y[2 * p + 1]);
                }
                if constexpr (FWD) {
                    if (zout) {
                        if (a.ztma) {
                            uint32_t w[kCkptBlock / 4];
                            const float scale = ckpt_codes(y, w);
                            if (row_ok) a.zs_out[static_cast<size_t>((n0 + col) / kCkptBlock) * M + row] = scale;
                            *code_chunk(codes, lane, 0) = make_uint4(w[0], w[1], w[2], w[3]);
                            *code_chunk(codes, lane, 1) = make_uint4(w[4], w[5], w[6], w[7]);
                        } else if (row_ok) {
                            ckpt_store(y, a.zq, a.zs_out, row, M, n0 + col, N);
                        }
                    }
                    act_apply<__nv_bfloat16>(a.act, y);
                } else if (zin) {
                    uint8_t* zc = codes + (piece % C::kCodeBufs) * kCodePieceBytes;
                    float z[32];
                    ckpt_values16(*code_chunk(zc, lane, 0), zscale, *reinterpret_cast<float(*)[16]>(z));
                    ckpt_values16(*code_chunk(zc, lane, 1), zscale, *reinterpret_cast<float(*)[16]>(z + 16));
                    slope_apply<__nv_bfloat16>(a.act, z, y);
                }
                if (a.add) piece_add(pc, lane, y);
                piece_put(pc, lane, y);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (row0 < M) {
                        tma_store_2d(&tmOut, pc, n0 + col, row0);
                        if (zout && a.ztma) tma_store_2d(&tmZ, codes, n0 + col, row0);
                    }
                    bulk_commit();
                }
            }
            if (!ok) continue;
            if (!given_back) give_back();
        }
        // after a give-up: this warp's loads still in flight
        for (; loads && piece < issued; ++piece) mbar_wait(&pbar[piece & 1], (piece >> 1) & 1, status);
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // both CTAs are done with the pair's TMEM and with each other's barriers
    cluster_arrive();
    cluster_wait();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// Maps of the epilogue's rows: bf16 pieces of out and add, code pieces of z.
inline bool pair_act_maps(const PairActArgs& a, const void* out, const void* add, const void* zq, CUtensorMap* to,
                          CUtensorMap* ta, CUtensorMap* tz) {
    const uint64_t pitch = static_cast<uint64_t>(a.N) * 2;
    if (!make_tmap_2d(to, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.M, a.N, pitch, 32, kPieceCols,
                      CU_TENSOR_MAP_SWIZZLE_64B))
        return false;
    *ta = *to;  // unused maps are copies of a valid one
    *tz = *to;
    if (add && !make_tmap_2d(ta, add, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.M, a.N, pitch, 32, kPieceCols,
                             CU_TENSOR_MAP_SWIZZLE_64B))
        return false;
    return !a.ztma || make_tmap_2d(tz, zq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.M, a.N, a.N, 32, kPieceCols,
                                   CU_TENSOR_MAP_SWIZZLE_32B);
}

template <int RP, bool FWD, int W>
cudaError_t launch_pair_act(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& to,
                            const CUtensorMap& tadd, const CUtensorMap& tz, const PairActArgs& a, int* status,
                            cudaStream_t s) {
    using C = PairActCfg<RP, FWD, W>;
    auto kern = pair_act_kernel<RP, FWD, W>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kTotal);
    if (e != cudaSuccess) return e;
    const int tiles = ((a.M + 2 * kTM - 1) / (2 * kTM)) * ((a.N + kTN - 1) / kTN);
    const int pairs = tiles < sm_count() / 2 ? tiles : sm_count() / 2;
    if (FWD)
        return launch_kx(kern, dim3(2 * pairs), dim3(C::kThreads), C::kTotal, s, 2, ta, tb, to, tadd, tz, a, status);
    // dX: at the greatest priority, so that a rank pass on another stream
    // takes only the SMs its pairs leave
    return launch_kx_urgent(kern, dim3(2 * pairs), dim3(C::kThreads), C::kTotal, s, 2, ta, tb, to, tadd, tz, a,
                            status);
}

}  // namespace

}  // namespace qlora
