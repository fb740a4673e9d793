// act_epilogue.cuh -- the activation, residual and 8-bit checkpoint pieces of
// the GEMM epilogues (forward: Y = act(Z) + R, Z kept in 8 bits; dX: the
// accumulated gradient times act'(z) of a kept z, plus an added gradient).
//
// Activations, with s(x) = 1 / (1 + exp(-x)):
//   relu       max(z, 0)                       z > 0
//   gelu       z P(z), P the normal CDF        P + z exp(-z^2/2) / sqrt(2 pi)
//   gelu_tanh  z s(2u), u = k (z + a z^3)      s + z s (1 - s) 2 u'
//   silu       z s(z)                          s (1 + z (1 - s))
// (k = sqrt(2/pi), a = 0.044715; z s(2u) is 0.5 z (1 + tanh u)).  The logistic
// form keeps the relative accuracy of the small negative tail that 1 + tanh
// would cancel away, with one base-2 exponential and one reciprocal per
// element.  For bf16 activations the normal CDF uses the rational approximation
// 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical Functions (|error of
// erf| <= 1.5e-7; the CDF evaluated in fp32 is off by up to 2.6e-7 on [-1, 1],
// 2^-13 of a step of bf16 but several of fp32): branch-free, and its exp(-x^2)
// is the density that the derivative needs.  For fp32 activations P keeps fp32
// accuracy, in the tail too (normal_cdf_f32).
//
// An 8-bit checkpoint holds blocks of 32 consecutive columns of a row:
// scale = amax / 127, code = rne(v * (127 / amax)), fp32 operations rounded
// once each.  32 columns are one epilogue step of a thread that owns a row,
// so the block's maximum needs no exchange between threads; the scales lie
// [block][row], so that the 32 rows of a warp write neighbouring words.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace qlora {

enum ActFn { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

constexpr int kCkptBlock = 32;
// blocks whose abs-max is below this are stored as zeros (127 / amax would
// leave fp32's range below 3.8e-37; 2^-100 keeps every product normal)
constexpr float kCkptTiny = 7.888609052210118e-31f;

__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhK = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

__device__ __forceinline__ float logistic(float x) { return rcp_approx(1.f + ex2_approx(-kLog2e * x)); }

// P(z) and e = exp(-z^2 / 2) to fp32 accuracy, without a branch: for |z| <= 1 the
// odd series 1/2 + z q(z^2); beyond, P(-|z|) = exp(-z^2/2) t r(t), t = 1 / (1 +
// 0.45 |z|).  q and r are minimax fits in the relative error (7e-10 and 3.2e-8,
// up to |z| = 13.5), made for this file by reweighted least squares.  exp(-z^2/2)
// is corrected by what z^2 loses to its rounding.  In all P is off by at most 7
// 2^-24 of itself (found over 2.4 million points of [-12, 12]).  4096 x 1024 x
// 1024 in fp32 with GELU and residual, quantizer included: 65 us (59 with 7.1.26,
// 72 with normcdff and expf).
__device__ __forceinline__ float normal_cdf_f32(float z, float& e) {
    const float x = fminf(fabsf(z), 16.f);  // exp(-128) is 0 already
    const float x2 = x * x;
    e = expf(-0.5f * x2);
    e = fmaf(e, -0.5f * fmaf(x, x, -x2), e);
    float q = fmaf(-7.654314e-06f, x2, 1.1348666e-04f);
    q = fmaf(q, x2, -1.1863302e-03f);
    q = fmaf(q, x2, 9.973324e-03f);
    q = fmaf(q, x2, -6.649036e-02f);
    q = fmaf(q, x2, 3.989423e-01f);
    const float t = rcp_approx(fmaf(0.45f, x, 1.f));
    float r = fmaf(-0.070279345f, t, 0.268677f);
    r = fmaf(r, t, -0.35148543f);
    r = fmaf(r, t, 0.109136745f);
    r = fmaf(r, t, 0.036813885f);
    r = fmaf(r, t, 0.1485123f);
    r = fmaf(r, t, 0.17906073f);
    r = fmaf(r, t, 0.17954089f);
    const float tail = r * t * e;
    const float outer = z < 0.f ? tail : 1.f - tail;
    return x <= 1.f ? fmaf(z, q, 0.5f) : outer;
}

// P(z) and e = exp(-z^2 / 2); FULL: to fp32 accuracy
template <bool FULL>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    if constexpr (FULL) return normal_cdf_f32(z, e);
    const float x = fabsf(z) * 0.7071067811865476f;
    const float t = rcp_approx(fmaf(0.3275911f, x, 1.f));
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    e = ex2_approx(z * z * (-0.5f * kLog2e));
    const float tail = 0.5f * p * t * e;  // P(-|z|)
    return z < 0.f ? tail : 1.f - tail;
}

// 2u of gelu_tanh; the cubic's z^2 is capped where s(2u) is 0 or 1 already,
// so that no product overflows against a zero
__device__ __forceinline__ float tanh_arg2(float z, float& z2) {
    z2 = fminf(z * z, 1e6f);
    return (2.f * kTanhK) * z * fmaf(kTanhA, z2, 1.f);
}

template <int F, bool FULL>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (F == kActRelu) return z > 0.f ? z : (z != z ? z : 0.f);
    if constexpr (F == kActGelu) {
        float e;
        return z * normal_cdf<FULL>(z, e);
    }
    if constexpr (F == kActGeluTanh) {
        float z2;
        return z * logistic(tanh_arg2(z, z2));
    }
    if constexpr (F == kActSilu) return z * logistic(z);
    return z;
}

template <int F, bool FULL>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (F == kActRelu) return z > 0.f ? 1.f : (z != z ? z : 0.f);
    if constexpr (F == kActGelu) {
        float e;
        const float p = normal_cdf<FULL>(z, e);
        return fmaf(z * 0.3989422804014327f, e, p);
    }
    if constexpr (F == kActGeluTanh) {
        float z2;
        const float s = logistic(tanh_arg2(z, z2));
        const float du2 = (2.f * kTanhK) * fmaf(3.f * kTanhA, z2, 1.f);
        return fmaf(z * s * (1.f - s), du2, s);
    }
    if constexpr (F == kActSilu) {
        const float s = logistic(z);
        return s * fmaf(z, 1.f - s, 1.f);
    }
    return 1.f;
}

// y[e] = act(y[e]); one uniform branch for the whole step.  T: the activations' type
template <typename T, int N>
__device__ __forceinline__ void act_apply(int act, float (&y)[N]) {
#define QL_ACT_CASE(F)                                       \
    case F:                                                  \
        _Pragma("unroll") for (int e = 0; e < N; ++e) y[e] = act_value<F, sizeof(T) == 4>(y[e]); \
        break;
    switch (act) {
        QL_ACT_CASE(kActRelu)
        QL_ACT_CASE(kActGelu)
        QL_ACT_CASE(kActGeluTanh)
        QL_ACT_CASE(kActSilu)
        default: break;
    }
#undef QL_ACT_CASE
}

// y[e] *= act'(z[e])
template <typename T, int N>
__device__ __forceinline__ void slope_apply(int act, const float (&z)[N], float (&y)[N]) {
#define QL_ACT_CASE(F)                                       \
    case F:                                                  \
        _Pragma("unroll") for (int e = 0; e < N; ++e) y[e] *= act_slope<F, sizeof(T) == 4>(z[e]); \
        break;
    switch (act) {
        QL_ACT_CASE(kActRelu)
        QL_ACT_CASE(kActGelu)
        QL_ACT_CASE(kActGeluTanh)
        QL_ACT_CASE(kActSilu)
        default: break;
    }
#undef QL_ACT_CASE
}

// |v| as bits: ordered like the magnitudes, infinities above every finite
// value and NaN above those, so one integer maximum carries both
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The block's scale and 127 / amax from the largest abs_bits.  A block that
// holds an infinity or a NaN reads back as NaN: a gradient that meets it says so.
__device__ __forceinline__ void ckpt_scale(uint32_t top, float& inv, float& scale) {
    const float amax = __uint_as_float(top);
    inv = 0.f;
    scale = 0.f;
    if (top >= 0x7F800000u) {
        scale = __uint_as_float(0x7FC00000u);
    } else if (amax >= kCkptTiny) {
        inv = __fdiv_rn(127.0f, amax);
        scale = __fdiv_rn(amax, 127.0f);
    }
}

// Codes and scale of one block.
__device__ __forceinline__ float ckpt_codes(const float (&z)[kCkptBlock], uint32_t (&w)[kCkptBlock / 4]) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < kCkptBlock; ++e) top = max(top, abs_bits(z[e]));
    float inv, scale;
    ckpt_scale(top, inv, scale);
#pragma unroll
    for (int i = 0; i < kCkptBlock / 8; ++i) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = z[8 * i + e];
        const uint2 c = codes8(f, inv);
        w[2 * i] = c.x;
        w[2 * i + 1] = c.y;
    }
    return scale;
}

// Stores the codes of one block (columns n .. n + 31 of row `row`) and its
// scale.  Columns >= N hold zeros and are not written.
__device__ __forceinline__ void ckpt_store(const float (&z)[kCkptBlock], int8_t* __restrict__ zq,
                                           float* __restrict__ zs, int row, int M, int n, int N) {
    uint32_t w[kCkptBlock / 4];
    zs[static_cast<size_t>(n / kCkptBlock) * M + row] = ckpt_codes(z, w);
    int8_t* dst = zq + static_cast<size_t>(row) * N + n;
    if (N % 16 == 0) {  // whole 16-byte chunks lie inside the row or outside it
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (n + 16 * i < N)
                reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < kCkptBlock; ++e)
            if (n + e < N) dst[e] = static_cast<int8_t>(w[e >> 2] >> (8 * (e & 3)));
    }
}

// 16 codes (one 16-byte chunk) times a scale
__device__ __forceinline__ void ckpt_values16(const uint4 c, float scale, float (&v)[16]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        // byte + 128 under 2^23's exponent, less 2^23 + 128: the code, exactly
        const float q = __uint_as_float(__byte_perm(w[e >> 2] ^ 0x80808080u, 0x4B000000u, 0x7540 + (e & 3))) - 8388736.0f;
        v[e] = q * scale;
    }
}

// E consecutive elements of a row of an activation-typed matrix, held as
// loaded (columns n .. n + E - 1; `vec`: rows start at 16-byte boundaries
// and hold whole 16-byte chunks).  Plain loads: the matrix may be the
// output's own buffer, each element of which is read before it is written.
template <typename T, int E>
struct RowPiece {
    static constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    static constexpr int kChunks = E / kPer;
    uint4 raw[kChunks];

    __device__ __forceinline__ void load(const T* base, int row, bool row_ok, int n, int N, bool vec) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (!row_ok) return;
        const T* p = base + static_cast<size_t>(row) * N + n;
        if (vec) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                if (n + i * kPer < N) raw[i] = *(reinterpret_cast<const uint4*>(p) + i);
        } else {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    const int c = i * kPer + e;
                    if (n + c >= N) continue;
                    if constexpr (sizeof(T) == 2)
                        w[e >> 1] |= static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(p + c)) << (16 * (e & 1));
                    else
                        w[e] = *reinterpret_cast<const uint32_t*>(p + c);
                }
                raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }

    __device__ __forceinline__ void add_to(float (&y)[E]) const {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if constexpr (sizeof(T) == 2) {
                    y[i * 8 + 2 * u] += __uint_as_float(w[u] << 16);
                    y[i * 8 + 2 * u + 1] += __uint_as_float(w[u] & 0xFFFF0000u);
                } else {
                    y[i * 4 + u] += __uint_as_float(w[u]);
                }
            }
        }
    }
};

// What the EX form of the dX epilogue reads for 16 columns of a row: the codes
// of z with their block's scale, and the added gradient.
template <typename T>
struct DxPiece {
    uint4 codes;
    float scale;
    RowPiece<T, 16> add;

    __device__ __forceinline__ void load(const DxEpilogue& ep, int M, int K, int row, bool row_ok, int k,
                                         bool vec) {
        codes = make_uint4(0u, 0u, 0u, 0u);
        scale = 0.f;
        if (ep.act != kActNone && row_ok && k < K) {  // K is a multiple of 16
            codes = __ldg(reinterpret_cast<const uint4*>(ep.zq + static_cast<size_t>(row) * K + k));
            scale = __ldg(ep.zs + static_cast<size_t>(k / kCkptBlock) * M + row);
        }
        if (ep.add) add.load(static_cast<const T*>(ep.add), row, row_ok && k < K, k, K, vec);
    }

    __device__ __forceinline__ void apply(const DxEpilogue& ep, float (&y)[16]) const {
        if (ep.act != kActNone) {
            float z[16];
            ckpt_values16(codes, scale, z);
            slope_apply<T>(ep.act, z, y);
        }
        if (ep.add) add.add_to(y);
    }
};

}  // namespace qlora
