// fp8.hip -- e4m3 quantizers with a scale for each block of 128, and the e4m3 x e4m3 product with
// those scales, gfx950.
//
// What is computed: scale = fp32(absmax / 448), code = e4m3(clip(fp32(v / scale), +-448)) for blocks of
// 1 x 128 (activations) and 128 x 128 (weights); and
//     y[m, n] = sum_b (xs[b, m] ws[n / 128, b]) sum_{k in b} x_q[m, k] W_q[n, k]  (+ bias[n]).
#include "experts.hpp"

namespace bitlinear {

// Four values as e4m3 bytes (rounded to nearest, ties to even).
__device__ __forceinline__ uint32_t e4m3_4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}
__device__ __forceinline__ float e4m3_quotient(float v, float scale) {
    return scale > 0.0f ? fminf(fmaxf(v / scale, -448.0f), 448.0f) : 0.0f;
}

// Four floats at p + i of a row that ends at n, zeros past it.
template <bool WHOLE>
__device__ __forceinline__ float4 row_4(const float* __restrict__ p, int64_t i, int64_t n) {
    if constexpr (WHOLE) {
        return i < n ? *reinterpret_cast<const float4*>(p + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    } else {
        return make_float4(i < n ? p[i] : 0.0f, i + 1 < n ? p[i + 1] : 0.0f, i + 2 < n ? p[i + 2] : 0.0f,
                           i + 3 < n ? p[i + 3] : 0.0f);
    }
}
// The four bytes of v to p + i of a row that ends at n.
template <bool WHOLE>
__device__ __forceinline__ void put_4(uint8_t* __restrict__ p, int64_t i, int64_t n, uint32_t v) {
    if constexpr (WHOLE) {
        if (i < n) *reinterpret_cast<uint32_t*>(p + i) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < n) p[i + e] = (uint8_t)(v >> (8 * e));
    }
}
__device__ __forceinline__ float abs_max_4(float4 v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// ---- activations ----------------------------------------------------------------------------
// Half a wave takes a block of one token, four values a lane; the eight halves of a workgroup take `tm`
// tokens (a power of two) of 8 / tm neighbouring blocks, so that their scales are written together.
// WHOLE: rows of x and x_q are read and written four at a time (K % 4 == 0 and aligned).
template <bool WHOLE>
__global__ __launch_bounds__(256) void k_quantize_act_fp8(const float* __restrict__ x, int64_t M, int64_t K,
                                                          uint8_t* __restrict__ xq, float* __restrict__ xs, int tm_log) {
    const int half = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t m = ((int64_t)blockIdx.x << tm_log) + (half & ((1 << tm_log) - 1));
    const int64_t b = ((int64_t)blockIdx.y << (3 - tm_log)) + (half >> tm_log);
    if (m >= M || b * 128 >= K) return;
    const float4 v = row_4<WHOLE>(x + m * K, b * 128 + 4 * lane, K);
    float top = abs_max_4(v);
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor(top, s, 32));
    const float scale = top / 448.0f;
    put_4<WHOLE>(xq + m * K, b * 128 + 4 * lane, K,
                 e4m3_4(e4m3_quotient(v.x, scale), e4m3_quotient(v.y, scale), e4m3_quotient(v.z, scale), e4m3_quotient(v.w, scale)));
    if (lane == 0) xs[b * M + m] = scale;
}

hipError_t launch_quantize_act_fp8(const float* x, int64_t M, int64_t K, uint8_t* xq, float* xs, hipStream_t s) {
    const int tm_log = M >= 8 ? 3 : M >= 4 ? 2 : M >= 2 ? 1 : 0;
    const int64_t nb = (K + 127) / 128;
    const dim3 grid((unsigned)((M + (1 << tm_log) - 1) >> tm_log), (unsigned)((nb + (8 >> tm_log) - 1) >> (3 - tm_log)));
    const bool whole = K % 4 == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)xq % 4 == 0;
    if (whole) hipLaunchKernelGGL((k_quantize_act_fp8<true>), grid, dim3(256), 0, s, x, M, K, xq, xs, tm_log);
    else hipLaunchKernelGGL((k_quantize_act_fp8<false>), grid, dim3(256), 0, s, x, M, K, xq, xs, tm_log);
    return hipGetLastError();
}

// ---- weights --------------------------------------------------------------------------------
// A workgroup takes a block of 128 x 128: 16 times eight rows of 32 lanes, kept in registers between the
// maximum and the codes.
template <bool WHOLE>
__global__ __launch_bounds__(256) void k_quantize_weights_fp8(const float* __restrict__ W, int64_t N, int64_t K,
                                                              uint8_t* __restrict__ wq, float* __restrict__ ws) {
    __shared__ float red[4];
    const int tid = threadIdx.x, r = tid >> 5;
    const int64_t n0 = (int64_t)blockIdx.y * 128, k = (int64_t)blockIdx.x * 128 + 4 * (tid & 31);
    float4 v[16];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t n = n0 + 8 * i + r;
        v[i] = n < N ? row_4<WHOLE>(W + n * K, k, K) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, abs_max_4(v[i]));
    top = wave_max_f32(top);
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float scale = top / 448.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t n = n0 + 8 * i + r;
        if (n < N)
            put_4<WHOLE>(wq + n * K, k, K, e4m3_4(e4m3_quotient(v[i].x, scale), e4m3_quotient(v[i].y, scale),
                                                  e4m3_quotient(v[i].z, scale), e4m3_quotient(v[i].w, scale)));
    }
    if (tid == 0) ws[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = scale;
}

hipError_t launch_quantize_weights_fp8(const float* W, int64_t N, int64_t K, uint8_t* wq, float* ws, hipStream_t s) {
    const bool whole = K % 4 == 0 && (uintptr_t)W % 16 == 0 && (uintptr_t)wq % 4 == 0;
    // a grid dimension holds 65535 blocks of rows (y): more rows in several launches
    const int64_t nb = (K + 127) / 128, step = (int64_t)65535 * 128;
    for (int64_t n0 = 0; n0 < N; n0 += step) {
        const int64_t n = N - n0 < step ? N - n0 : step;
        const dim3 grid((unsigned)nb, (unsigned)((n + 127) / 128));
        const float* w = W + n0 * K;
        uint8_t* q = wq + n0 * K;
        float* sc = ws + n0 / 128 * nb;
        if (whole) hipLaunchKernelGGL((k_quantize_weights_fp8<true>), grid, dim3(256), 0, s, w, n, K, q, sc);
        else hipLaunchKernelGGL((k_quantize_weights_fp8<false>), grid, dim3(256), 0, s, w, n, K, q, sc);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// ---- product --------------------------------------------------------------------------------
// One output a thread, block after block.
__global__ __launch_bounds__(256) void k_fp8_plain(Fp8Args a) {
    const int64_t n = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63), m = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6);
    if (n >= a.N || m >= a.M) return;
    const int64_t nb = (a.K + 127) / 128;
    const uint8_t *x = a.xq + m * a.K, *w = a.wq + n * a.K;
    float sum = 0.0f;
    for (int64_t b = 0; b < nb; ++b) {
        const int64_t end = (b + 1) * 128 < a.K ? (b + 1) * 128 : a.K;
        float part = 0.0f;
        for (int64_t k = b * 128; k < end; ++k)
            part += __builtin_amdgcn_cvt_f32_fp8((int)x[k], 0) * __builtin_amdgcn_cvt_f32_fp8((int)w[k], 0);
        sum += part * (a.xs[b * a.M + m] * a.ws[n / 128 * nb + b]);
    }
    a.y[m * a.N + n] = a.bias ? sum + a.bias[n] : sum;
}

hipError_t launch_forward_fp8(const Fp8Args& a, hipStream_t s) {
    const int64_t step = (int64_t)65535 * 4;
    for (int64_t m0 = 0; m0 < a.M; m0 += step) {
        if (m0) return hipErrorInvalidValue;
        hipLaunchKernelGGL(k_fp8_plain, dim3((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 3) / 4)), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace bitlinear
