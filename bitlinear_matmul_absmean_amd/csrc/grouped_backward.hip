// grouped_backward.hip -- gradients of the ternary BitLinears grouped by expert and of the gated block, gfx950.
//
// What is computed, row m of group e reading token r, for one projection or two (gate and up):
//     dx[m, k]    = sum_p alpha_p,e sum_n d_p[m, n] W_p,e[n, k]
//     dW_p,e[n, k] = sum_{m in e} d_p[m, n] (beta[r] / 127) x_q[r, k],   dbias_p,e[n] = sum_{m in e} d_p[m, n]
// with d = dy, or dg = dh u a'(g) and du = dh a(g), which a first kernel leaves in the workspace.
#include "experts.hpp"
#include "ffn.hpp"

namespace bitlinear {

size_t grouped_backward_workspace(int64_t M, int64_t K, int64_t N, int64_t E, bool gated) {
    return 256 + (gated ? (size_t)M * N * 8 : 0);
}

bool grouped_backward_fits(int64_t M, int64_t K, int64_t N, int64_t E) {
    // dW: tiles of 128 x 128 at least, of 512 threads, two projections
    return grid_fits(E * ((N + 127) / 128) * ((K + 127) / 128) * 2, 512) && grid_fits((M / 64 + E) * ((K + 127) / 128), 512);
}

// dg and du, one element a thread.
template <int ACT>
__global__ __launch_bounds__(256) void k_gate_gradients(const float* __restrict__ dh, const float* __restrict__ g,
                                                        const float* __restrict__ u, int64_t n, float* __restrict__ dg,
                                                        float* __restrict__ du) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float a, slope;
        act_grad<ACT>(g[i], a, slope);
        dg[i] = dh[i] * u[i] * slope;
        du[i] = dh[i] * a;
    }
}

__device__ __forceinline__ float weight(const uint8_t* w, int64_t k) { return (float)(int)((w[k >> 2] >> (2 * (k & 3))) & 3) - 1.0f; }

struct Products {
    GroupedBackwardArgs a;
    const float *d0, *d1;
};

__global__ __launch_bounds__(256) void k_grouped_dx_plain(Products p) {
    const GroupedBackwardArgs& a = p.a;
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
    if (k >= a.K) return;
    int64_t e = -1;
    for (int64_t i = 0; i < a.E; ++i) {
        const Group g = group_rows(a.offsets, i, a.M);
        if (m >= g.lo && m < g.hi) e = i;
    }
    if (e < 0) return;
    float sum = 0.0f;
    for (int q = 0; q < (a.w1 ? 2 : 1); ++q) {
        const float* d = (q ? p.d1 : p.d0) + m * a.N;
        const uint8_t* w = (q ? a.w1 : a.w0) + e * a.N * (a.K / 4);
        const float alpha = (q ? a.al1 : a.al0)[e];
        for (int64_t n = 0; n < a.N; ++n) sum += d[n] * alpha * weight(w + n * (a.K / 4), k);
    }
    a.dx[m * a.K + k] = sum;
}

__global__ __launch_bounds__(256) void k_grouped_dw_plain(Products p) {
    const GroupedBackwardArgs& a = p.a;
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x, n = blockIdx.y, e = blockIdx.z >> 1;
    const int q = blockIdx.z & 1;
    float* dw = q ? a.dw1 : a.dw0;
    if (k >= a.K || !dw) return;
    const float* d = q ? p.d1 : p.d0;
    const Group g = group_rows(a.offsets, e, a.M);
    float sum = 0.0f;
    for (int64_t m = g.lo; m < g.hi; ++m) {
        const int64_t r = row_token(a.rows, m, a.T);
        if (r >= 0) sum += d[m * a.N + n] * (a.beta[r] / 127.0f) * (float)a.xq[r * a.K + k];
    }
    dw[(e * a.N + n) * a.K + k] = sum;
}

__global__ __launch_bounds__(256) void k_grouped_db_plain(Products p) {
    const GroupedBackwardArgs& a = p.a;
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, e = blockIdx.y;
    float* db = blockIdx.z ? a.db1 : a.db0;
    if (n >= a.N || !db) return;
    const float* d = blockIdx.z ? p.d1 : p.d0;
    const Group g = group_rows(a.offsets, e, a.M);
    double sum = 0.0;
    for (int64_t m = g.lo; m < g.hi; ++m) sum += (double)d[m * a.N + n];
    db[e * a.N + n] = (float)sum;
}

hipError_t launch_grouped_backward(const GroupedBackwardArgs& a, hipStream_t s) {
    Products p{a, a.dy, nullptr};
    if (a.w1 && a.M > 0) {
        float* dg = reinterpret_cast<float*>(a.ws);
        float* du = dg + a.M * a.N;
        const int64_t n = a.M * a.N, wgs = (n + 255) / 256;
        const dim3 grid((unsigned)(wgs < 16384 ? wgs : 16384));
        if (a.act == BITLINEAR_ACT_SILU) hipLaunchKernelGGL(k_gate_gradients<BITLINEAR_ACT_SILU>, grid, dim3(256), 0, s, a.dy, a.g, a.u, n, dg, du);
        else if (a.act == BITLINEAR_ACT_GELU) hipLaunchKernelGGL(k_gate_gradients<BITLINEAR_ACT_GELU>, grid, dim3(256), 0, s, a.dy, a.g, a.u, n, dg, du);
        else hipLaunchKernelGGL(k_gate_gradients<BITLINEAR_ACT_RELU2>, grid, dim3(256), 0, s, a.dy, a.g, a.u, n, dg, du);
        p.d0 = dg;
        p.d1 = du;
    }
    const unsigned kx = (unsigned)((a.K + 255) / 256), two = a.w1 ? 2 : 1;
    if (a.dx && a.M > 0) hipLaunchKernelGGL(k_grouped_dx_plain, dim3(kx, (unsigned)a.M), dim3(256), 0, s, p);
    if (a.dw0) hipLaunchKernelGGL(k_grouped_dw_plain, dim3(kx, (unsigned)a.N, (unsigned)a.E * 2), dim3(256), 0, s, p);
    if (a.db0 || a.db1) hipLaunchKernelGGL(k_grouped_db_plain, dim3((unsigned)((a.N + 255) / 256), (unsigned)a.E, two), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace bitlinear
