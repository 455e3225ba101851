// backward.hip -- gradients of ternary projections, straight through the quantizers, gfx950.
//
// What is computed, for each projection p with incoming gradient d_p [M, N]:
//     dx[m, k]    = sum_p alpha_p sum_n d_p[m, n] W_p[n, k]
//     dW_p[n, k]  = sum_m d_p[m, n] (beta[m] / 127) x_q[m, k]
//     dbias_p[n]  = sum_m d_p[m, n]
// One projection: d = dy.  The gated block h = a(g) u: d_gate = dh u a'(g), d_up = dh a(g).
#include "ffn.hpp"

namespace bitlinear {

// d [M, P N] fp32 from dh, g, u (gated, P = 2: gate columns, then up columns).
template <int ACT>
__global__ __launch_bounds__(256) void k_gated_slopes(BackwardArgs a, float* __restrict__ d) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.M * a.N) return;
    const int64_t m = i / a.N, n = i % a.N;
    float v, slope;
    act_grad<ACT>(a.g[i], v, slope);
    const float dh = a.dy[i];
    d[m * 2 * a.N + n] = dh * a.u[i] * slope;
    d[m * 2 * a.N + a.N + n] = dh * v;
}

// 16 x 16 outputs per workgroup, one per thread, 16 steps of the sum through LDS at a time.
// DX: rows m, columns k, the sum over P N gradient columns; else rows over P N, columns k, the
// sum over m.
template <bool DX>
__global__ __launch_bounds__(256) void k_backward_simple(BackwardArgs a, const float* __restrict__ d, int P) {
    __shared__ float As[16][17], Bs[16][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t NT = P * a.N, rowb = a.K >> 2;
    const int64_t R = DX ? a.M : NT, L = DX ? NT : a.M;
    const int64_t ctiles = (a.K + 15) / 16;
    const int64_t r0 = (int64_t)blockIdx.x / ctiles * 16, c0 = (int64_t)blockIdx.x % ctiles * 16;
    float acc = 0.0f;
    for (int64_t l0 = 0; l0 < L; l0 += 16) {
        // As[row][l], Bs[l][column]
        if constexpr (DX) {
            const int64_t r = r0 + ty, l = l0 + tx;
            As[ty][tx] = r < R && l < L ? d[r * NT + l] * (l < a.N ? a.al0[0] : a.al1[0]) : 0.0f;
            const int64_t lb = l0 + ty, c = c0 + tx;
            float w = 0.0f;
            if (lb < L && c < a.K) {
                const uint8_t* p = lb < a.N ? a.w0 + lb * rowb : a.w1 + (lb - a.N) * rowb;
                w = (float)((int)((p[c >> 2] >> (2 * (c & 3))) & 3) - 1);
            }
            Bs[ty][tx] = w;
        } else {
            const int64_t l = l0 + ty, r = r0 + tx;
            As[tx][ty] = r < R && l < L ? d[l * NT + r] * (a.beta[l] / 127.0f) : 0.0f;
            const int64_t c = c0 + tx;
            Bs[ty][tx] = l < L && c < a.K ? (float)a.xq[l * a.K + c] : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) acc = fmaf(As[ty][i], Bs[i][tx], acc);
        __syncthreads();
    }
    const int64_t r = r0 + ty, c = c0 + tx;
    if (r >= R || c >= a.K) return;
    if constexpr (DX) a.dx[r * a.K + c] = acc;
    else if (r < a.N) a.dw0[r * a.K + c] = acc;
    else a.dw1[(r - a.N) * a.K + c] = acc;
}

// Column sums, one thread per column.
__global__ __launch_bounds__(256) void k_bias_simple(BackwardArgs a, const float* __restrict__ d, int P) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, NT = P * a.N;
    if (n >= NT) return;
    float* out = n < a.N ? a.db0 : a.db1;
    if (!out) return;
    double s = 0.0;
    for (int64_t m = 0; m < a.M; ++m) s += (double)d[m * NT + n];
    out[n < a.N ? n : n - a.N] = (float)s;
}

size_t backward_workspace(int64_t M, int64_t K, int64_t N, bool gated) {
    (void)K;
    return gated ? (size_t)M * (size_t)N * 8 : 16;
}

hipError_t launch_backward(const BackwardArgs& a, hipStream_t s) {
    const int P = a.g ? 2 : 1;
    const float* d = a.dy;
    if (a.g) {
        float* dst = static_cast<float*>(a.ws);
        const dim3 grid((unsigned)((a.M * a.N + 255) / 256));
        switch (a.act) {
            case BITLINEAR_ACT_GELU: hipLaunchKernelGGL(k_gated_slopes<BITLINEAR_ACT_GELU>, grid, dim3(256), 0, s, a, dst); break;
            case BITLINEAR_ACT_SILU: hipLaunchKernelGGL(k_gated_slopes<BITLINEAR_ACT_SILU>, grid, dim3(256), 0, s, a, dst); break;
            default: hipLaunchKernelGGL(k_gated_slopes<BITLINEAR_ACT_RELU2>, grid, dim3(256), 0, s, a, dst);
        }
        d = dst;
    }
    const int64_t ct = (a.K + 15) / 16;
    if (a.dx) hipLaunchKernelGGL(k_backward_simple<true>, dim3((unsigned)((a.M + 15) / 16 * ct)), dim3(256), 0, s, a, d, P);
    if (a.dw0)
        hipLaunchKernelGGL(k_backward_simple<false>, dim3((unsigned)((P * a.N + 15) / 16 * ct)), dim3(256), 0, s, a, d, P);
    if (a.db0 || a.db1) hipLaunchKernelGGL(k_bias_simple, dim3((unsigned)((P * a.N + 255) / 256)), dim3(256), 0, s, a, d, P);
    return hipGetLastError();
}

}  // namespace bitlinear
