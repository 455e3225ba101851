// ffn.hpp -- the gated feed-forward block, the BitLinear gradients and the W8A8 product:
// activation helpers and launch declarations.
#pragma once

#include "bitlinear.h"
#include "common.hpp"

namespace bitlinear {

// exp(-x) for |x| <= 128, within 4 * 2^-24 relative (x >= -88: finite): the exponent x log2(e) as a
// rounded product and its remainder, the hardware's 2^h (within one unit) and a first-order factor.
__device__ __forceinline__ float exp_neg(float x) {
    constexpr float L = 1.44269504088896341f, L_LO = 1.92596299112661746e-8f, LN2 = 0.69314718055994531f;
    const float h = x * -L;
    const float r = __builtin_fmaf(x, -L_LO, __builtin_fmaf(x, -L, -h));
    const float e = __builtin_amdgcn_exp2f(h);
    return __builtin_fmaf(e, r * LN2, e);
}

// The larger of g and a bound; NaN for NaN (fmaxf would give the bound).
__device__ __forceinline__ float at_least(float g, float bound) { return __builtin_elementwise_maximum(g, bound); }

// a(g) of the gated block, in fp32.  SiLU: g / (1 + exp(-g)), by the hardware's reciprocal and one
// correction of it; below -88 it stays at its value there, -5.3e-37.  Both sides of the quotient are taken
// 2^-8 times: the hardware's reciprocal of more than 2^126 is zero, and exp(88) is 2^127.  (The reciprocal
// is corrected, not the quotient, whose remainder is NaN where g is infinite.  14 instructions; the
// library's exp and an IEEE division took 40, a third of the epilogue of a short GEMM.)
// GELU: the BitMLP's.  Squared ReLU: one rounding.
template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    if constexpr (ACT == BITLINEAR_ACT_SILU) {
        constexpr float S = 0x1p-8f;
        const float v = at_least(g, -88.0f), d = __builtin_fmaf(exp_neg(fminf(v, 128.0f)), S, S);
        const float r = __builtin_amdgcn_rcpf(d);
        return v * S * __builtin_fmaf(__builtin_fmaf(-r, d, 1.0f), r, r);
    } else if constexpr (ACT == BITLINEAR_ACT_GELU) {
        return gelu_f32(g);
    } else {
        const float r = at_least(g, 0.0f);
        return r * r;
    }
}

// a(g) and a'(g) for the gradients, to a few fp32 roundings.
//   SiLU: with e = exp(-|g|), s(|g|) = 1 / (1 + e) and s(-|g|) = e / (1 + e), so neither
//     logistic value is formed as a difference (the reciprocal is the hardware's, within one unit); a = g s(g),
//     a' = s(g) + g s(g) s(-g).
//   GELU: a = g Phi(g), a' = Phi(g) + g phi(g) in fp64 (Phi from the erfc polynomial of the
//     forward pass, whose tail below g = -8 is off relative to itself but below 1e-14).
//   Squared ReLU: a = r^2, a' = 2 r.
// At an infinite g the limits (GELU: a(-inf) is NaN, as in the forward pass): a factor g beside one that has
// underflowed is bounded where the product has long been zero.  NaN stays NaN.
template <int ACT>
__device__ __forceinline__ void act_grad(float g, float& a, float& slope) {
    if constexpr (ACT == BITLINEAR_ACT_SILU) {
        const float e = exp_neg(fminf(fabsf(g), 128.0f)), t = __builtin_amdgcn_rcpf(1.0f + e), p = e * t;
        const float s = g >= 0.0f ? t : p, sc = g >= 0.0f ? p : t;
        const float low = at_least(g, -128.0f), v = __builtin_elementwise_minimum(low, 128.0f);
        a = low * s;
        slope = s + v * s * sc;
    } else if constexpr (ACT == BITLINEAR_ACT_GELU) {
        const double v = (double)g, y = fabs(v) * 0.70710678118654752440, d = 2.0 + y;
        double r = __builtin_amdgcn_rcp(d);
        r = fma(r, fma(-d, r, 1.0), r);
        r = fma(r, fma(-d, r, 1.0), r);
        const double t = fmax(fma(r, gelu_poly::kS2, gelu_poly::kO), -1.0);
        double c = gelu_poly::kC[16];
#pragma unroll
        for (int i = 15; i >= 0; --i) c = fma(c, t, gelu_poly::kC[i]);
        const double ex = exp(-0.5 * v * v), q = 0.5 * ex * c;
        const double cdf = v < 0.0 ? q : 1.0 - q;
        a = (float)(v * cdf);
        const double b = y > 64.0 ? 0.0 : v;                    // exp(-v^2 / 2) is zero long before
        slope = (float)(cdf + b * ex * 0.39894228040143267794);
    } else {
        const float r = at_least(g, 0.0f);
        a = r * r;
        slope = 2.0f * r;
    }
}

// Reductions over the 64 lanes, the same in every lane: exchanges inside rows of 16 lanes by DPP (pairs,
// quads, halves, rows), then the four rows' values.  The maximum is of non-negative values.
template <int CTRL>
__device__ __forceinline__ int row_exchange(int v) { return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true); }

__device__ __forceinline__ float wave_max_pos(float f) {
    auto larger = [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); };
    int v = __float_as_int(f);
    v = larger(v, row_exchange<0xB1>(v));       // quad_perm [1, 0, 3, 2]
    v = larger(v, row_exchange<0x4E>(v));       // quad_perm [2, 3, 0, 1]
    v = larger(v, row_exchange<0x141>(v));      // row_half_mirror
    v = larger(v, row_exchange<0x140>(v));      // row_mirror
    return __int_as_float(larger(larger(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
                                 larger(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48))));
}

__device__ __forceinline__ int wave_sum_rows(int v) {
    v += row_exchange<0xB1>(v);
    v += row_exchange<0x4E>(v);
    v += row_exchange<0x141>(v);
    v += row_exchange<0x140>(v);
    return __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) + __builtin_amdgcn_readlane(v, 32) +
           __builtin_amdgcn_readlane(v, 48);
}

// 16 bytes at p, whatever its alignment.  DWORDS: from the aligned dwords that hold them (five, or four
// when p is aligned: no dword is read that holds none of the bytes), for operands that lie off a dword's
// boundary: there a load of 16 bytes takes several times as long.
template <bool DWORDS = false>
__device__ __forceinline__ u32x4 load_16(const uint8_t* __restrict__ p) {
    u32x4 v;
    if constexpr (!DWORDS) {
        __builtin_memcpy(&v, p, 16);
        return v;
    } else {
        const uint32_t off = (uint32_t)(uintptr_t)p & 3u;
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p - off);
        __builtin_memcpy(&v, __builtin_assume_aligned(q, 4), 16);
        const uint32_t last = q[off ? 4 : 3];
        return u32x4{__builtin_amdgcn_alignbyte(v.y, v.x, off), __builtin_amdgcn_alignbyte(v.z, v.y, off),
                     __builtin_amdgcn_alignbyte(v.w, v.z, off), __builtin_amdgcn_alignbyte(last, v.w, off)};
    }
}

// 16 bytes at p + i (i a multiple of 16) of a row of `row` bytes, zeros past its end; no alignment is
// assumed.  What is left of a row at its end comes as the row's last 16 bytes, shifted down by `n`.
template <bool DWORDS = false>
__device__ __forceinline__ u32x4 row_16(const uint8_t* __restrict__ p, int64_t i, int64_t row) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (i + 16 <= row) {
        v = load_16<DWORDS>(p + i);
    } else if (i < row) {
        if (row >= 16) {
            const u32x4 t = load_16<DWORDS>(p + row - 16);
            const int n = 16 - (int)(row & 15);
            const u32x4 a = n & 8 ? u32x4{t.z, t.w, 0u, 0u} : t;
            const u32x4 b = n & 4 ? u32x4{a.y, a.z, a.w, 0u} : a;
            v = u32x4{__builtin_amdgcn_alignbyte(b.y, b.x, n & 3), __builtin_amdgcn_alignbyte(b.z, b.y, n & 3),
                      __builtin_amdgcn_alignbyte(b.w, b.z, n & 3), __builtin_amdgcn_alignbyte(0u, b.w, n & 3)};
        } else {
            for (int j = 0; j < 16; ++j)
                if (i + j < row) v[j >> 2] |= (uint32_t)p[i + j] << (8 * (j & 3));
        }
    }
    return v;
}

struct GatedArgs {
    const int8_t* xq;
    const float* beta;
    int64_t M, K, F;
    const uint8_t *wg, *wu;        // packed [F, K/4]
    const float *ag, *au;          // alpha [1]
    const float *bg, *bu;          // bias [F] or null
    int act;                       // bitlinear_activation
    float* h;                      // [M, F]
    float *g, *u;                  // [M, F] or both null
};

hipError_t launch_gated(const GatedArgs& a, hipStream_t s);
// One token with x quantized in the same launch (a.xq and a.beta are written, not read).
bool gated_gemv_supports(const GatedArgs& a, const float* x);
hipError_t launch_gated_gemv(const GatedArgs& a, const float* x, int8_t* xq, float* beta, hipStream_t s);

struct I8Args {
    const int8_t* xq;
    const float* beta;
    int64_t M, K, N;
    const int8_t* wq;              // [N, K]
    const float* gamma;            // [N]
    const float* bias;             // [N] or null
    float* y;
    int32_t* acc;                  // [M, N] or null
};

// Largest K for which |acc| <= 127 * 127 * K fits int32.
constexpr int64_t I8_MAX_K = 133144;
hipError_t launch_forward_i8(const I8Args& a, hipStream_t s);

// Gradients of one or two (gate and up) ternary projections of the same x_q.
struct BackwardArgs {
    const float* dy;               // one projection: dy [M, N]; gated: dh [M, N]
    const float *g, *u;            // gated: saved [M, N]; one projection: null
    int act;
    int64_t M, K, N;               // N: rows of each weight matrix
    const int8_t* xq;
    const float* beta;
    const uint8_t *w0, *w1;        // packed [N, K/4]; w1 null for one projection
    const float *al0, *al1;        // alpha [1]
    float* dx;                     // [M, K] or null
    float *dw0, *dw1;              // [N, K] or null
    float *db0, *db1;              // [N] or null
    void* ws;
};
// Largest M and N: 512 bytes of a panel for each row of the sum, two projections, within 2^31 bytes.
constexpr int64_t BACKWARD_MAX_ROWS = (int64_t)1 << 21;
size_t backward_workspace(int64_t M, int64_t K, int64_t N, bool gated);
hipError_t launch_backward(const BackwardArgs& a, hipStream_t s);

}  // namespace bitlinear
