// k4_rank_q.cu -- the LoRA gradient of A from an input that the forward kept
// as its row codes (Xq [M,K] int8, sx [M]):
//
//   dA[k,j] = c sum_m (Xq[m,k] sx[m]) G[m,j] = c sum_m Xq[m,k] V[m,j],
//   V[m,j]  = sx[m] G[m,j]
//
// ("Parameter-efficient fine-tuning of GPT-2 with LoRA", "LoRA equation", for
// the product; the kept codes are those of the forward's input quantizer.)
// The row scale moves to the skinny factor, so the wide operand stays the
// codes as they lie in memory and the sum runs on tcgen05.mma.kind::i8 with
// exact int32 accumulation: V is written as four signed 8-bit digits of a
// fixed-point value per column,
//   V[m,j] 2^p_j = d0 + 2^8 d1 + 2^16 d2 + 2^24 d3,  |V 2^p| <= 2^30,
// p_j from the column's largest magnitude, so a digit's sums over the rows
// are integers and dA is the same bits whatever the order or the split (the
// only roundings: V to 31 bits below its column's maximum, and the result).
//
// Bound by reading the codes once: M K bytes, half of a bf16 input.  The
// codes need no conversion on the way: a TMA box of 128 rows x 128 columns
// (128-byte swizzle) is the MN-major A operand (M = 128 columns, K = 32 rows
// per MMA) as it lands.  The digits of a 128-row tile are prepared once, by two
// small kernels (V with its columns' maxima; the digits), in the K-major table
// layout the MMA reads, so every CTA only copies 512 ceil4(r) bytes of them
// beside each 16 KB tile.  16384 x 4096 codes at rank 4: 19 us, 3.5 TB/s (the
// bf16 input's pass: 28.7 us alone).
//
// Rows are split over a cluster of CL <= 8 CTAs per 128-column block, whose
// partial sums meet in the shared memory of the CTA that owns the column, as
// int64.  Warps: 0 producer, 1 TMEM owner and MMA issuer, 2..5 read-out.
//
// Up to 128 rows (one tile) there are no such kernels: warps 2..5 of every CTA
// make the tile's table themselves, two launches less.
#include "internal.h"
#include "ptx.cuh"
#include "tile_epilogue.cuh"

namespace qlora {

namespace {

constexpr int kRows = 128;                        // rows of a tile (contraction)
constexpr int kCols = 128;                        // columns of a tile: one swizzle row of codes
constexpr uint32_t kTileBytes = kRows * kCols;
constexpr uint32_t kSbo = (kRows / 16) * 128;     // 8-row group stride of a digit table
constexpr int kThreads = 32 * 6;
constexpr int kMaxCl = 8;
constexpr int kMaxTilesPerCta = 1023;             // 1023 * 128 * 128 * 128 < 2^31
constexpr int kMaxStages = 8;
constexpr int kPrepThreads = 256;
constexpr int kPrepCtas = 64;                     // of the scaling pass, at most

__host__ __device__ constexpr int ceil4(int r) { return (r + 3) / 4 * 4; }

// digits buffer: int p[64] (the columns' exponents), then the tables [tile][4 ceil4(r)][128]
constexpr uint32_t kExpBytes = 256;
constexpr int kExpNaN = -0x40000000;  // the column holds an infinity or a NaN

// Byte offset of digit row n (= digit * ceil4(r) + j) of tile row k.
__device__ __forceinline__ uint32_t digit_off(int n, int k) {
    return static_cast<uint32_t>((n >> 3) * kSbo + (k >> 4) * 128 + (n & 7) * 16 + (k & 15));
}

// The exponent p of a column whose largest magnitude has the bits `top`: top <
// 2^(E - 126) for its biased exponent E, so V 2^(156 - E) < 2^30.
__device__ __forceinline__ int column_exponent(uint32_t top) {
    const int E = static_cast<int>(top >> 23);
    return top >= 0x7F800000u ? kExpNaN : (top == 0u ? 0 : 156 - (E > 0 ? E : 1));
}

// The four digits of v 2^p, lowest first.
__device__ __forceinline__ void make_digits(float v, int p, int (&d)[4]) {
    // v 2^p in two exact steps (-98 <= p <= 155)
    const int h = p / 2;
    int t = __float2int_rn(v * __int_as_float((h + 127) << 23) * __int_as_float((p - h + 127) << 23));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        d[i] = i < 3 ? static_cast<int>(static_cast<int8_t>(t & 0xFF)) : t;
        t = (t - d[i]) >> 8;
    }
}

// V = sx G [M, r] and, per CTA, its columns' largest magnitudes part[CTA][64].
// A thread takes a row, so that a warp reduction per column replaces the
// shared-memory atomics of its 32 rows (with those, and both sweeps on one
// cluster of eight CTAs, the digits of 11416 rows at rank 8 took 38 us).
__global__ void __launch_bounds__(kPrepThreads) k4_q_scale_kernel(const float* __restrict__ G, int nsl,
                                                                  const float* __restrict__ sx, int M, int r,
                                                                  float* __restrict__ V, uint32_t* __restrict__ part) {
    __shared__ uint32_t top[64];
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_trigger();
    if (tid < 64) top[tid] = 0u;
    __syncthreads();
    pdl_wait();
    const size_t slice = static_cast<size_t>(M) * r;
    for (int m0 = blockIdx.x * kPrepThreads; m0 < M; m0 += gridDim.x * kPrepThreads) {
        const int m = m0 + tid;
        const float s = m < M ? __ldg(sx + m) : 0.f;
        const size_t at = static_cast<size_t>(m < M ? m : 0) * r;
        for (int j = 0; j < r; ++j) {
            const float g = nsl == 1 ? __ldg(G + at + j) : sum_slices(G + at + j, slice, nsl);
            const float v = m < M ? g * s : 0.f;
            if (m < M) V[at + j] = v;
            const uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu);
            if (lane == 0) atomicMax(&top[j], t);
        }
    }
    __syncthreads();
    if (tid < 64) part[blockIdx.x * 64 + tid] = top[tid];
}

// The columns' exponents from the `ctas` partial maxima, and the digit tables.
__global__ void __launch_bounds__(kPrepThreads) k4_q_digits_kernel(const float* __restrict__ V,
                                                                   const uint32_t* __restrict__ part, int ctas, int M,
                                                                   int r, uint8_t* __restrict__ digits) {
    __shared__ int pexp[64];
    const int tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    if (tid < 64) {
        uint32_t t = 0;
        for (int q = 0; q < ctas; ++q) t = max(t, __ldg(part + q * 64 + tid));
        pexp[tid] = column_exponent(t);
        if (blockIdx.x == 0) reinterpret_cast<int*>(digits)[tid] = pexp[tid];
    }
    __syncthreads();
    // one word (four rows) of each of the four digits an item; the items of
    // all tiles are fewer than 2^25
    const uint32_t RP = static_cast<uint32_t>(ceil4(r));
    const uint32_t items = static_cast<uint32_t>((M + kRows - 1) / kRows) * RP * (kRows / 4);
    for (uint32_t i = blockIdx.x * kPrepThreads + tid; i < items; i += gridDim.x * kPrepThreads) {
        const uint32_t rest = i / RP;
        const int j = static_cast<int>(i - rest * RP);
        const int g = static_cast<int>(rest % (kRows / 4));
        const uint32_t tile = rest / (kRows / 4);
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        const int p = j < r ? pexp[j] : kExpNaN;
        if (p != kExpNaN) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t m = tile * kRows + 4 * g + e;
                if (m >= static_cast<uint32_t>(M)) continue;
                int dg[4];
                make_digits(__ldg(V + static_cast<size_t>(m) * r + j), p, dg);
#pragma unroll
                for (int d = 0; d < 4; ++d) w[d] |= (static_cast<uint32_t>(dg[d]) & 0xFFu) << (8 * e);
            }
        }
        uint8_t* tab = digits + kExpBytes + static_cast<size_t>(tile) * (4 * RP * kRows);
#pragma unroll
        for (int d = 0; d < 4; ++d)
            *reinterpret_cast<uint32_t*>(tab + digit_off(d * static_cast<int>(RP) + j, 4 * g)) = w[d];
    }
}

struct RankQArgs {
    const uint8_t* digits;  // null: one tile, whose digits the kernel makes itself from
    const float* G;         // the nsl slices of G and sx
    int nsl;
    const float* sx;
    float* dA;
    int M, K, r;
    int tiles_per_cta;
    int stages;
    int early;              // wait for the predecessor at the end
    float c;
};

struct RqLayout {
    int RP, NV;
    uint32_t stage, recv, bar, total, tmem_cols;
    __host__ __device__ RqLayout(int r, int stages) {
        RP = ceil4(r);
        NV = 4 * RP;
        stage = kTileBytes + static_cast<uint32_t>(NV) * kRows;
        recv = static_cast<uint32_t>(stages) * stage;
        bar = recv + static_cast<uint32_t>((kCols + kMaxCl) * r * 8);
        total = bar + (2 * kMaxStages + 4) * 8;  // full, empty, dfull, rbar, vready, TMEM address
        tmem_cols = 32;
        while (tmem_cols < static_cast<uint32_t>(NV)) tmem_cols <<= 1;
    }
};

// sum_slices past L1: a kernel that has not waited for its predecessor must not
// meet a line that the SM read before G was written.
__device__ __forceinline__ float sum_slices_l2(const float* p, size_t stride, int n) {
    float s = __ldcg(p);
#pragma unroll 8
    for (int b = 1; b < n; ++b) s += __ldcg(p + b * stride);
    return s;
}

__global__ void __launch_bounds__(kThreads) k4_rank_q_kernel(const __grid_constant__ CUtensorMap tmX, RankQArgs a,
                                                             int* status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int S = a.stages;
    const RqLayout L(a.r, S);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.bar);
    uint64_t* empty = full + kMaxStages;
    uint64_t* dfull = empty + kMaxStages;
    uint64_t* rbar = dfull + 1;
    uint64_t* vready = rbar + 1;  // without a digits buffer: the table is written
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(vready + 1);
    __shared__ uint32_t s_top[64];
    __shared__ int s_exp[64];
    const bool own = a.digits == nullptr;
    // recv[q][c][j]: the sums of CTA q for column cbeg + c of this CTA's slice
    long long* recv = reinterpret_cast<long long*>(smem + L.recv);
    uint32_t CL;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(CL));
    const uint32_t crank = cluster_ctarank();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int col0 = blockIdx.x * kCols;
    const int mtiles = (a.M + kRows - 1) / kRows;
    const int t0 = blockIdx.y * a.tiles_per_cta;
    const int nt = max(0, min(mtiles, t0 + a.tiles_per_cta) - t0);
    const int per = (kCols + static_cast<int>(CL) - 1) / static_cast<int>(CL);
    const int cbeg = static_cast<int>(crank) * per;
    const int cend = min(kCols, cbeg + per);
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(dfull, 1);
        mbar_init(vready, 4);
        mbar_init(rbar, static_cast<uint32_t>(static_cast<int>(CL) * max(1, cend - cbeg)));
        fence_mbar_init();
    }
    if (threadIdx.x < 64) s_top[threadIdx.x] = 0u;
    if (warp == 1) {
        tmem_alloc(tmem_slot, L.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    cluster_arrive_relaxed();  // no CTA arrives on another's barrier before it is initialised
    if (!a.early) pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&tmX);
            const uint32_t tab = static_cast<uint32_t>(L.NV) * kRows;
            const uint8_t* src = own ? nullptr : a.digits + kExpBytes;
            for (int i = 0; i < nt; ++i) {
                const int s = i % S;
                if (i >= S && !mbar_wait(&empty[s], ((i / S) - 1) & 1, status)) break;
                uint8_t* st = smem + s * L.stage;
                mbar_arrive_expect_tx(&full[s], own ? kTileBytes : L.stage);
                tma_load_2d(st, &tmX, &full[s], col0, (t0 + i) * kRows);
                if (!own) bulk_load(st + kTileBytes, src + static_cast<size_t>(t0 + i) * tab, tab, &full[s]);
            }
        }
        __syncwarp();
        cluster_wait();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t id = idesc_i8_at(kCols, L.NV);
            bool ok = true;
            for (int i = 0; i < nt; ++i) {
                const int s = i % S;
                if (!mbar_wait(&full[s], (i / S) & 1, status) || (own && !mbar_wait(vready, 0, status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t xb = smem_u32(smem + s * L.stage);
                const uint32_t vb = xb + kTileBytes;
#pragma unroll
                for (int kk = 0; kk < kRows / 32; ++kk) {
                    // 32 rows: four 8-row swizzle groups of the tile, two 16-byte
                    // core matrices of the digit table
                    const uint64_t ad = smem_desc(xb + kk * 4096, kTileBytes, 1024, kLayoutSw128);
                    const uint64_t bd = smem_desc(vb + kk * 256, 128, kSbo, kLayoutNone);
                    mma_i8(tmem, ad, bd, id, (i > 0 || kk > 0) ? 1u : 0u);
                }
                mma_commit(&empty[s]);
            }
            if (ok) mma_commit(dfull);
        }
        __syncwarp();
        cluster_wait();
    } else {
        if (own) {
            // the one tile's table (stage 0): thread = row
            const int m = threadIdx.x - 64;
            const size_t n = static_cast<size_t>(a.M) * a.r;
            const float sxm = m < a.M ? __ldcg(a.sx + m) : 0.f;
            float* sV = reinterpret_cast<float*>(smem + L.stage);  // [r][128], in the ring's idle second stage
            for (int j0 = 0; j0 < a.r; j0 += 4) {
                float v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    v[u] = 0.f;
                    if (m < a.M && j0 + u < a.r)
                        v[u] = sum_slices_l2(a.G + static_cast<size_t>(m) * a.r + j0 + u, n, a.nsl) * sxm;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (j0 + u >= a.r) break;
                    sV[(j0 + u) * kRows + m] = v[u];
                    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v[u]) & 0x7FFFFFFFu);
                    if (lane == 0) atomicMax(&s_top[j0 + u], top);
                }
            }
            named_bar_sync(1, 128);
            if (m < 64) s_exp[m] = column_exponent(s_top[m]);
            named_bar_sync(1, 128);
            uint8_t* tab = smem + kTileBytes;
            for (int j = 0; j < L.RP; ++j) {
                int d[4] = {0, 0, 0, 0};
                if (j < a.r && s_exp[j] != kExpNaN) make_digits(sV[j * kRows + m], s_exp[j], d);
#pragma unroll
                for (int i = 0; i < 4; ++i) tab[digit_off(i * L.RP + j, m)] = static_cast<uint8_t>(d[i]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(vready);
        }
        cluster_wait();  // every CTA of the cluster has initialised its barriers
        const int wq = warp & 3;
        const int rr = wq * 32 + lane;  // column of the block
        const int owner = rr / per;
        const uint32_t dst =
            dsmem_addr(recv + static_cast<size_t>(static_cast<int>(crank) * per + rr - owner * per) * a.r,
                       static_cast<uint32_t>(owner));
        bool ok = nt > 0;
        if (nt > 0) ok = __all_sync(0xffffffffu, mbar_wait(dfull, 0, status));
        tc_fence_after();
        const uint32_t base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        for (int j0 = 0; j0 < L.RP; j0 += 4) {
            long long sum[4] = {0, 0, 0, 0};
            if (ok) {
                uint32_t d[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld4(base + i * L.RP + j0, d[i]);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[e] = static_cast<long long>(static_cast<int>(d[0][e])) +
                             static_cast<long long>(static_cast<int>(d[1][e])) * 256 +
                             static_cast<long long>(static_cast<int>(d[2][e])) * 65536 +
                             static_cast<long long>(static_cast<int>(d[3][e])) * 16777216;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j0 + e < a.r) dsmem_st_i64(dst + 8u * static_cast<uint32_t>(j0 + e), sum[e]);
        }
        tc_fence_before();
        mbar_arrive_remote(dsmem_addr(rbar, static_cast<uint32_t>(owner)));
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L.tmem_cols);
    }
    // this CTA's slice of the columns; once every partial has arrived nothing
    // touches this CTA's shared memory from outside
    const int width = cend - cbeg;
    if (width > 0 && mbar_wait_cluster(rbar, 0, status)) {
        for (int idx = threadIdx.x; idx < width * a.r; idx += kThreads) {
            const int cc = idx / a.r, j = idx - cc * a.r;
            const int col = col0 + cbeg + cc;
            if (col >= a.K) continue;
            long long sum = 0;
            for (int q = 0; q < static_cast<int>(CL); ++q)
                sum += recv[static_cast<size_t>(q * per + cc) * a.r + j];
            const int p = own ? s_exp[j] : __ldcg(reinterpret_cast<const int*>(a.digits) + j);
            const double v = p == kExpNaN ? __longlong_as_double(0x7FF8000000000000LL)
                                          : scalbn(static_cast<double>(sum), -p) * static_cast<double>(a.c);
            a.dA[static_cast<size_t>(col) * a.r + j] = static_cast<float>(v);
        }
    }
    if (a.early) pdl_wait();
}

}  // namespace

// The exponents and tables; behind them the partial maxima and V.
static size_t digit_table_bytes(int M, int r) {
    return kExpBytes + static_cast<size_t>((M + kRows - 1) / kRows) * 4 * ceil4(r) * kRows;
}

size_t rank_q_digit_bytes(int M, int r) {
    return digit_table_bytes(M, r) + kPrepCtas * 64 * 4 + static_cast<size_t>(M) * r * 4;
}

// `early`: the launch right before is a dX kernel that starts its dependents
// only after its own pdl_wait(), so that everything before it, G and the
// digits with it, is complete when this kernel starts.  It needs nothing of
// that dX kernel: it runs beside it, on the SMs it leaves, and waits for it at
// its end, so that whoever waits for this kernel has waited for both.
cudaError_t launch_rank_x_q(const int8_t* Xq, const float* sx, const float* G, int nsl, int M, int K, int r,
                            float c, void* digits, float* dA, int* status, cudaStream_t s, RankQPart part_of,
                            bool early) {
    if (M > kRankQMaxRows) return cudaErrorInvalidValue;
    const bool own = M <= kRows;
    cudaError_t e = cudaSuccess;
    if (!own && part_of != RankQPart::kSum) {
        uint8_t* buf = static_cast<uint8_t*>(digits);
        uint32_t* part = reinterpret_cast<uint32_t*>(buf + digit_table_bytes(M, r));
        float* V = reinterpret_cast<float*>(part + kPrepCtas * 64);
        const int want = (M + kPrepThreads - 1) / kPrepThreads;
        const int ctas = want < kPrepCtas ? want : kPrepCtas;
        e = launch_k(k4_q_scale_kernel, dim3(ctas), dim3(kPrepThreads), 0, s, 1, G, nsl, sx, M, r, V, part);
        if (e != cudaSuccess) return e;
        const size_t items = static_cast<size_t>((M + kRows - 1) / kRows) * ceil4(r) * (kRows / 4);
        const size_t blocks = (items + kPrepThreads - 1) / kPrepThreads, cap = 2 * static_cast<size_t>(sm_count());
        e = launch_k(k4_q_digits_kernel, dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(kPrepThreads), 0,
                     s, 1, static_cast<const float*>(V), static_cast<const uint32_t*>(part), ctas, M, r, buf);
        if (e != cudaSuccess) return e;
    }
    if (part_of == RankQPart::kDigits) return cudaSuccess;
    CUtensorMap tm;
    if (!make_tmap_2d(&tm, Xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, M, K, K, kRows, kCols, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    RankQArgs a{};
    a.digits = own ? nullptr : static_cast<const uint8_t*>(digits);
    a.G = G;
    a.nsl = nsl;
    a.sx = sx;
    a.dA = dA;
    a.M = M;
    a.K = K;
    a.r = r;
    a.c = c;
    a.early = early;
    const int mtiles = (M + kRows - 1) / kRows;
    a.tiles_per_cta = (mtiles + kMaxCl - 1) / kMaxCl;
    const int want = (rank_pass_rows() + kRows - 1) / kRows;  // a caller's minimum rows per CTA
    if (want > a.tiles_per_cta) a.tiles_per_cta = want;
    if (a.tiles_per_cta > kMaxTilesPerCta) a.tiles_per_cta = kMaxTilesPerCta;
    const int cl = (mtiles + a.tiles_per_cta - 1) / a.tiles_per_cta;
    // two CTAs per SM: about 100 KB each
    const RqLayout one(r, 1);
    int S = static_cast<int>((104 * 1024 - (one.total - one.recv)) / static_cast<double>(one.stage));
    S = S < 2 ? 2 : (S > kMaxStages ? kMaxStages : S);
    a.stages = S;
    const RqLayout L(r, S);
    const size_t smem = L.total + 1024;
    e = ensure_smem_attr(reinterpret_cast<const void*>(k4_rank_q_kernel), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_k(k4_rank_q_kernel, dim3((K + kCols - 1) / kCols, cl), dim3(kThreads), smem, s, cl, tm, a, status);
}

}  // namespace qlora
