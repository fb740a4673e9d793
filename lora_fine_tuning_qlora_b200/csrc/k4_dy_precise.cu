// k4_dy_precise.cu -- the dY pass of the backward from 8-bit checkpoints (bf16
// activations, ranks up to 32), with the fp32 factors at fp32 precision:
//
//   Gp[b][m,j] = sum_{n in block b} dY[m,n] B[j,n]      (G slices)
//   dB[j,n]    = c sum_m xA[m,j] dY[m,n]
//   dbias[n]   = sum_m dY[m,n]
//
// ("How to fine-tune the 4-bit model?" thread: the adapter's products drive the
// gradient; "Parameter-efficient fine-tuning of GPT-2 with LoRA", "LoRA
// equation", for the shapes.)  The structure is k4_rank_tc.cu's: a CTA owns 128
// columns of dY and a run of 128-row tiles, each tile arrives once by TMA and
// is read two ways by tcgen05.mma.kind::f16 (K-major for G, MN-major for the
// column sums), and the columns' partial sums meet over a cluster of up to 8
// CTAs in rank order.  Two things differ:
//   * The factors enter as three bf16 terms (v = hi + mid + lo, 24 bits; every
//     product with a bf16 dY is exact in fp32), ceil4(r) table rows apart, so
//     that rank 4 with its ones row (dbias) fills one 16-wide MMA.
//   * The column sums leave TMEM every kDrain tiles, from two accumulators in
//     turn, and are added in fp32 by the operand warps: the tensor cores' fp32
//     accumulation truncates, which over the 256 products of 4096 rows shrank
//     dB by 4.4e-6 of itself; chains of 32 leave 4.7e-7 at 16384 rows.
// HBM-bound: 16384 x 4096 at rank 4 reads 134 MB in 33 us, 4.1 TB/s (two terms,
// 16 columns apart: 46 us).
//
// Warps: 0 TMA producer, 1 TMEM owner + MMA issuer, 2..5 operand tables and
// epilogues (warp w owns TMEM lane quarter w % 4).
#include "internal.h"
#include "ptx.cuh"

namespace qlora {

namespace {

constexpr int kTileRows = 128;
constexpr int kTileCols = 128;
constexpr int kBoxCols = 64;                         // one 128-byte swizzle row of bf16
constexpr uint32_t kBoxBytes = kTileRows * kBoxCols * 2;
constexpr uint32_t kTileBytes = 2 * kBoxBytes;
constexpr int kWorkers = 4;
constexpr int kThreads = 64 + 32 * kWorkers;
constexpr int kMaxCluster = 8;
constexpr uint32_t kTabSbo = (kTileCols / 8) * 128;  // 8-row group stride of a 128-wide table
constexpr int kMaxBulkR = 8;                         // rank limit of the bulk-copied xA rows
constexpr int kTerms = 3;
constexpr int kDrain = 4;                            // tiles per column accumulator

struct DyArgs {
    const float* V;      // xA [M, r]
    const float* B;      // [r, C]
    float* Gp;           // slices out [ceil(C/128)][M, r]
    float* dB;           // [r, C]
    float* dbias;        // [C] or nullptr
    int M, C, r;
    int tiles_per_cta;   // 128-row tiles per CTA
    float c;
    int vbulk;           // r % 4 == 0, r <= kMaxBulkR, V 16-byte aligned: V's tile rows arrive by bulk copy
};

// Shared-memory and TMEM layout for rank r (same on host and device).
struct DyLayout {
    int RP, NG, NV, JP;
    uint32_t vtab, bcat, recv, bar, vraw, vslot, drain, total;
    uint32_t tmem_cols, g_col;
    __host__ __device__ DyLayout(int r, bool vbulk) {
        RP = (r + 3) / 4 * 4;
        NG = (kTerms * RP + 15) / 16 * 16;
        NV = (kTerms * RP + 1 + 15) / 16 * 16;
        JP = r + 1;
        vtab = 2 * kTileBytes;
        bcat = vtab + 2 * static_cast<uint32_t>(NV) * 256;
        recv = bcat + static_cast<uint32_t>(NG) * 256;
        bar = recv + (((kTileCols + kMaxCluster) * JP * 4 + 15) / 16) * 16;
        vraw = bar + 192;  // [2][128 rows][r] fp32 with vbulk
        vslot = vbulk ? static_cast<uint32_t>(kTileRows * r * 4) : 0u;
        drain = vraw + 2 * vslot;  // [128][JP]
        total = drain + static_cast<uint32_t>(kTileCols * JP * 4);
        g_col = static_cast<uint32_t>(2 * NV);  // behind the two column accumulators
        tmem_cols = 32;
        while (tmem_cols < static_cast<uint32_t>(2 * NV + 2 * NG)) tmem_cols <<= 1;
    }
};

// Byte offset of element (row, k) of a K-major bf16 operand table that is 128
// elements long in K, no swizzle: 8-row x 16-byte core matrices, K-adjacent
// ones 128 B apart (leading byte offset), 8-row groups 2048 B apart (stride
// byte offset).
__device__ __forceinline__ uint32_t ktab_off(int row, int k) {
    return static_cast<uint32_t>((row >> 3) * kTabSbo + (k >> 3) * 128 + (row & 7) * 16 + (k & 7) * 2);
}

// The bf16 terms of v: each the nearest bf16 of what the ones before leave.
__device__ __forceinline__ void split_terms(float v, __nv_bfloat16 (&t)[kTerms]) {
#pragma unroll
    for (int i = 0; i < kTerms; ++i) {
        t[i] = __float2bfloat16_rn(v);
        v -= __bfloat162float(t[i]);
    }
}

// Term i of v into row `row` + i * RP.
__device__ __forceinline__ void put_split(uint8_t* tab, int row, int RP, int k, float v) {
    __nv_bfloat16 t[kTerms];
    split_terms(v, t);
#pragma unroll
    for (int i = 0; i < kTerms; ++i) *reinterpret_cast<__nv_bfloat16*>(tab + ktab_off(row + i * RP, k)) = t[i];
}

// sink(j, sum) for the r sums of the terms' accumulators, RP TMEM columns apart.
template <typename Sink>
__device__ __forceinline__ void read_sums(uint32_t base, int RP, int r, Sink sink) {
    for (int c0 = 0; c0 < r; c0 += 4) {
        uint32_t v[kTerms][4];
#pragma unroll
        for (int i = 0; i < kTerms; ++i) tmem_ld4(base + i * RP + c0, v[i]);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c0 + e < r)
                sink(c0 + e, __uint_as_float(v[0][e]) + (__uint_as_float(v[1][e]) + __uint_as_float(v[2][e])));
    }
}

__global__ void __launch_bounds__(kThreads) k4_dy_precise_kernel(const __grid_constant__ CUtensorMap tmT,
                                                                 int t3d, DyArgs a, int* status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const DyLayout L(a.r, a.vbulk != 0);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bar);
    uint64_t* full = bars;        // [2] tile landed
    uint64_t* vready = bars + 2;  // [2] Vcat table written
    uint64_t* empty = bars + 4;   // [2] tile and table consumed by the MMAs
    uint64_t* gfull = bars + 6;   // [2] G accumulator ready
    uint64_t* gempty = bars + 8;  // [2] G accumulator read out
    uint64_t* vfull = bars + 10;   // [2] vbulk: the tile's V rows landed
    uint64_t* dgroup = bars + 12;  // [2] a group's column sums are complete
    uint64_t* dempty = bars + 14;  // [2] and have been read
    uint64_t* rbar = bars + 16;    // every CTA of the cluster delivered this CTA's column slice
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 17);
    float* drained = reinterpret_cast<float*>(smem + L.drain);  // the columns' sums so far
    // recv[q][c][j]: partial of CTA q for column cbeg + c of this CTA's slice
    float* recv = reinterpret_cast<float*>(smem + L.recv);

    uint32_t CL;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(CL));
    const uint32_t crank = cluster_ctarank();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int cb = blockIdx.x;
    const int col0 = cb * kTileCols;
    const int mtiles = (a.M + kTileRows - 1) / kTileRows;
    const int t0 = blockIdx.y * a.tiles_per_cta;
    const int t1 = min(mtiles, t0 + a.tiles_per_cta);
    const int nt = t1 > t0 ? t1 - t0 : 0;
    // the 128 columns are split over the cluster: CTA q sums columns [q*per, q*per + per)
    const int per = (kTileCols + static_cast<int>(CL) - 1) / static_cast<int>(CL);
    const int cbeg = static_cast<int>(crank) * per;
    const int cend = min(kTileCols, cbeg + per);
    pdl_trigger();

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&vready[s], kWorkers);
            mbar_init(&empty[s], 1);
            mbar_init(&gfull[s], 1);
            mbar_init(&gempty[s], kWorkers);
            mbar_init(&vfull[s], 1);
            mbar_init(&dgroup[s], 1);
            mbar_init(&dempty[s], kWorkers);
        }
        mbar_init(rbar, static_cast<uint32_t>(CL * (cend > cbeg ? cend - cbeg : 1)));
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, L.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // no CTA of the cluster arrives on another's barrier before all are initialised
    cluster_arrive_relaxed();
    pdl_wait();  // nothing above read global memory

    if (warp == 0) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&tmT);
            for (int i = 0; i < nt; ++i) {
                const int s = i & 1;
                if (i >= 2 && !mbar_wait(&empty[s], ((i >> 1) - 1) & 1, status)) break;
                uint8_t* dst = smem + s * kTileBytes;
                const int m0 = (t0 + i) * kTileRows;
                // with vbulk, the tile's rows of V (16-byte multiples: r % 4 == 0) first, on a
                // barrier of their own, so the V table is written while the tile is in flight
                if (a.vbulk) {
                    const uint32_t vbytes = static_cast<uint32_t>(min(kTileRows, a.M - m0) * a.r * 4);
                    mbar_arrive_expect_tx(&vfull[s], vbytes);
                    bulk_load(smem + L.vraw + s * L.vslot, a.V + static_cast<size_t>(m0) * a.r, vbytes, &vfull[s]);
                }
                mbar_arrive_expect_tx(&full[s], kTileBytes);
                if (t3d) {  // both 64-column blocks in one box
                    tma_load_3d(dst, &tmT, &full[s], 0, m0, col0 / kBoxCols);
                } else {
                    tma_load_2d(dst, &tmT, &full[s], col0, m0);
                    tma_load_2d(dst + kBoxBytes, &tmT, &full[s], col0 + kBoxCols, m0);
                }
            }
        }
        __syncwarp();
        cluster_wait();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t tiles = smem_u32(smem);
            const uint32_t vt = smem_u32(smem + L.vtab);
            const uint32_t bt = smem_u32(smem + L.bcat);
            const uint32_t id_g = idesc_bf16(128, L.NG, false, false);
            const uint32_t id_d = idesc_bf16(128, L.NV, true, false);
            for (int i = 0; i < nt; ++i) {
                const int s = i & 1;
                if (!mbar_wait(&full[s], (i >> 1) & 1, status) || !mbar_wait(&vready[s], (i >> 1) & 1, status)) break;
                tc_fence_after();
                const uint32_t tb = tiles + s * kTileBytes;
                // G rows of this tile: T (K-major) x Bcat
                if (i >= 2 && !mbar_wait(&gempty[s], ((i >> 1) - 1) & 1, status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kTileCols / 16; ++kk) {
                    const uint64_t ad = smem_desc(tb + (kk >> 2) * kBoxBytes + (kk & 3) * 32, 16, 1024, kLayoutSw128);
                    const uint64_t bd = smem_desc(bt + kk * 256, 128, kTabSbo, kLayoutNone);
                    mma_bf16(tmem + L.g_col + s * L.NG, ad, bd, id_g, kk > 0 ? 1u : 0u);
                }
                mma_commit(&gfull[s]);
                // column sums: T^T (MN-major, the two blocks 64 columns apart) x Vcat
                const int grp = i / kDrain;
                const uint32_t dcol = (grp & 1) * L.NV;
                const bool fresh = i % kDrain == 0;
                if (fresh && grp >= 2 && !mbar_wait(&dempty[grp & 1], ((grp >> 1) - 1) & 1, status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kTileRows / 16; ++kk) {
                    const uint64_t ad = smem_desc(tb + kk * 2048, kBoxBytes, 1024, kLayoutSw128);
                    const uint64_t bd = smem_desc(vt + s * L.NV * 256 + kk * 256, 128, kTabSbo, kLayoutNone);
                    mma_bf16(tmem + dcol, ad, bd, id_d, (!fresh || kk > 0) ? 1u : 0u);
                }
                if (i % kDrain == kDrain - 1 || i == nt - 1) mma_commit(&dgroup[grp & 1]);
                mma_commit(&empty[s]);
            }
        }
        __syncwarp();
        cluster_wait();
    } else {
        // ------------------------------------------------------ tables, epilogues
        const int wq = warp & 3;
        const int rr = wq * 32 + lane;  // tile row for the tables; column for the readback
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        bool ok = true;
        {
            // Bcat[t RP + j][n] = term t of B[j, col0 + n], eight loads in flight
            // per round (from clamped addresses, zeroed outside B after them,
            // so that no select waits on a single load)
            uint8_t* bt = smem + L.bcat;
            const int n = col0 + rr;
            const int nc = n < a.C ? n : a.C - 1;
            for (int j0 = 0; j0 < L.RP; j0 += 8) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int jc = j0 + e < a.r ? j0 + e : a.r - 1;
                    v[e] = __ldg(a.B + static_cast<size_t>(jc) * a.C + nc);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j0 + e < L.RP) put_split(bt, j0 + e, L.RP, rr, (j0 + e < a.r && n < a.C) ? v[e] : 0.f);
            }
        }
        auto g_epilogue = [&](int i) {
            const int b = i & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(&gfull[b], (i >> 1) & 1, status));
            if (!ok) return;
            tc_fence_after();
            const int m = (t0 + i) * kTileRows + rr;
            const uint32_t base = tmem + lane_base + L.g_col + b * L.NG;
            float* g = a.Gp + (static_cast<size_t>(cb) * a.M + m) * a.r;
            read_sums(base, L.RP, a.r, [&](int j, float sum) {
                if (m < a.M) g[j] = sum;
            });
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&gempty[b]);
        };
        // adds group g's column sums to this column's running ones
        auto drain_group = [&](int g) {
            ok = __all_sync(0xffffffffu, mbar_wait(&dgroup[g & 1], (g >> 1) & 1, status));
            if (!ok) return;
            tc_fence_after();
            const uint32_t base = tmem + lane_base + (g & 1) * L.NV;
            float* row = drained + rr * L.JP;
            read_sums(base, L.RP, a.r, [&](int j, float sum) { row[j] = g == 0 ? sum : row[j] + sum; });
            uint32_t ones[4];
            tmem_ld4(base + kTerms * L.RP, ones);
            tmem_ld_wait();
            row[a.r] = g == 0 ? __uint_as_float(ones[0]) : row[a.r] + __uint_as_float(ones[0]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dempty[g & 1]);
        };
        {
            const int tw = threadIdx.x - 64;  // 0 .. 127
            if (a.vbulk) {
                // the parts of both V tables that no tile changes: zero rows
                // beyond r in the terms' parts, and the ones block
                // (a ones row, then zeros; the tile's rows past M are zero, so
                // their ones add nothing), as 16-byte chunks of 8 tile rows
                const int nconst = L.NV - kTerms * a.r;
                for (int idx = tw; idx < 2 * nconst * 16; idx += 32 * kWorkers) {
                    const int b = idx / (nconst * 16), rem = idx % (nconst * 16);
                    const int jj = rem / 16, kg = rem % 16;
                    const int pad = L.RP - a.r;  // zero rows of one term
                    const int j = jj < kTerms * pad ? jj / pad * L.RP + a.r + jj % pad : kTerms * L.RP + jj - kTerms * pad;
                    const uint32_t w = j == kTerms * L.RP ? 0x3F803F80u : 0u;  // bf16 1.0 pairs
                    *reinterpret_cast<uint4*>(smem + L.vtab + b * L.NV * 256 + ktab_off(j, 8 * kg)) =
                        make_uint4(w, w, w, w);
                }
            }
            for (int i = 0; i < nt && ok; ++i) {
                const int s = i & 1;
                const int m = (t0 + i) * kTileRows + rr;
                ok = __all_sync(0xffffffffu,
                                i < 2 || mbar_wait(&empty[s], ((i >> 1) - 1) & 1, status));
                if (!ok) break;
                uint8_t* vt = smem + L.vtab + s * L.NV * 256;
                const bool mok = m < a.M;
                if (a.vbulk) {
                    // the tile's V rows have landed: chunk (j, kg) of the head and
                    // remainder tables from rows 8 kg .. 8 kg + 7
                    ok = __all_sync(0xffffffffu, mbar_wait(&vfull[s], (i >> 1) & 1, status));
                    if (!ok) break;
                    const float* vr = reinterpret_cast<const float*>(smem + L.vraw + s * L.vslot);
                    const int mt0 = (t0 + i) * kTileRows;
                    for (int idx = tw; idx < a.r * 16; idx += 32 * kWorkers) {
                        const int kg = idx / a.r, j = idx % a.r;
                        uint32_t w[kTerms][4];
#pragma unroll
                        for (int e2 = 0; e2 < 4; ++e2) {
                            float v2[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int row = 8 * kg + 2 * e2 + h;
                                v2[h] = mt0 + row < a.M ? vr[row * a.r + j] : 0.f;
                            }
                            __nv_bfloat16 t0[kTerms], t1[kTerms];
                            split_terms(v2[0], t0);
                            split_terms(v2[1], t1);
#pragma unroll
                            for (int i2 = 0; i2 < kTerms; ++i2)
                                w[i2][e2] = static_cast<uint32_t>(__bfloat16_as_ushort(t0[i2])) |
                                            (static_cast<uint32_t>(__bfloat16_as_ushort(t1[i2])) << 16);
                        }
#pragma unroll
                        for (int i2 = 0; i2 < kTerms; ++i2)
                            *reinterpret_cast<uint4*>(vt + ktab_off(i2 * L.RP + j, 8 * kg)) =
                                make_uint4(w[i2][0], w[i2][1], w[i2][2], w[i2][3]);
                    }
                } else {
                for (int j0 = 0; j0 < L.RP; j0 += 8) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = mok && j0 + e < a.r ? __ldg(a.V + static_cast<size_t>(m) * a.r + j0 + e) : 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (j0 + e < L.RP) put_split(vt, j0 + e, L.RP, rr, v[e]);
                }
                {
                    const __nv_bfloat16 one = __float2bfloat16_rn(mok ? 1.f : 0.f);
                    const __nv_bfloat16 zero = __float2bfloat16_rn(0.f);
                    *reinterpret_cast<__nv_bfloat16*>(vt + ktab_off(kTerms * L.RP, rr)) = one;
                    for (int j = kTerms * L.RP + 1; j < L.NV; ++j)
                        *reinterpret_cast<__nv_bfloat16*>(vt + ktab_off(j, rr)) = zero;
                }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&vready[s]);
                if (i >= 1) g_epilogue(i - 1);
                if (ok && i >= kDrain && i % kDrain == 0) drain_group(i / kDrain - 1);
            }
            if (ok && nt >= 1) g_epilogue(nt - 1);
            if (ok && nt >= 1) drain_group((nt - 1) / kDrain);
            // this CTA's partial of column rr goes to the CTA that owns the column
            cluster_wait();  // every CTA of the cluster has initialised its barriers
            const int owner = rr / per;
            const uint32_t dst = dsmem_addr(recv + (static_cast<int>(crank) * per + rr - owner * per) * L.JP,
                                            static_cast<uint32_t>(owner));
            const bool sums = ok && nt > 0;
            for (int j = 0; j < L.JP; ++j) dsmem_st(dst + 4 * j, sums ? drained[rr * L.JP + j] : 0.f);
            mbar_arrive_remote(dsmem_addr(rbar, static_cast<uint32_t>(owner)));
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L.tmem_cols);
    }
    // this CTA's slice of the columns: the CL partials added in rank order.
    // Once every CTA's partials have arrived nothing reads or writes this
    // CTA's shared memory from outside, so it may exit without a cluster
    // barrier.
    const int width = cend - cbeg;
    if (width > 0 && mbar_wait_cluster(rbar, 0, status)) {
        for (int idx = threadIdx.x; idx < L.JP * width; idx += kThreads) {
            const int j = idx / width, cc = idx % width;  // consecutive threads: consecutive columns of dB [r, C]
            const int col = col0 + cbeg + cc;
            if (col >= a.C || (j == a.r && a.dbias == nullptr)) continue;
            float sum = 0.f;
            for (int q = 0; q < static_cast<int>(CL); ++q) sum += recv[(q * per + cc) * L.JP + j];
            if (j < a.r) a.dB[static_cast<size_t>(j) * a.C + col] = a.c * sum;
            else a.dbias[col] = sum;
        }
    }
}

}  // namespace

cudaError_t launch_dy_precise(const void* dY, const float* B, const float* xA, int M, int N, int r, float c, float* Gp,
                              float* dB, float* dbias, int* status, cudaStream_t s) {
    DyArgs a{};
    a.V = xA;
    a.B = B;
    a.Gp = Gp;
    a.dB = dB;
    a.dbias = dbias;
    a.M = M;
    a.C = N;
    a.r = r;
    a.c = c;
    // dY as [row][64-column block][64] when its rows split into whole blocks
    // (one box per tile), else one 2-D box per 64-column block
    CUtensorMap tm;
    const int t3d = (N % kBoxCols) == 0 ? 1 : 0;
    if (!(t3d ? make_tmap_3d_blocks(&tm, dY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, N, kBoxCols, kTileRows, 2)
              : make_tmap_2d(&tm, dY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, N, static_cast<uint64_t>(N) * 2, kTileRows,
                             kBoxCols, CU_TENSOR_MAP_SWIZZLE_128B)))
        return cudaErrorInvalidValue;
    a.vbulk = r % 4 == 0 && r <= kMaxBulkR && (reinterpret_cast<uintptr_t>(xA) & 15) == 0;
    const DyLayout L(r, a.vbulk != 0);
    if (r > kMaxPreciseR) return cudaErrorInvalidValue;
    const size_t smem = L.total + 1024;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(k4_dy_precise_kernel), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    // rows split over a cluster of CTAs, every CTA at least one tile; CTAs too
    // large for two per SM take clusters of at most 4
    const int mtiles = (M + kTileRows - 1) / kTileRows;
    const int max_cl = smem > 110 * 1024 ? 4 : kMaxCluster;
    a.tiles_per_cta = (mtiles + max_cl - 1) / max_cl;
    const int want = (rank_pass_rows() + kTileRows - 1) / kTileRows;  // a caller's minimum rows per CTA
    if (want > a.tiles_per_cta) a.tiles_per_cta = want;
    const int cl = (mtiles + a.tiles_per_cta - 1) / a.tiles_per_cta;
    return launch_k(k4_dy_precise_kernel, dim3((N + kTileCols - 1) / kTileCols, cl), dim3(kThreads), smem, s, cl, tm, t3d,
                    a, status);
}

}  // namespace qlora
