// grouped.hip -- ternary BitLinears grouped by expert, one projection or a gated block, gfx950.
//
// What is computed: rows sorted by expert, row m of group e reading token r = rows[m]:
//     acc[m, n] = sum_k x_q[r, k] W_e[n, k]                                   (int32, exact)
//     y[m, n]   = fp32(acc) * fp32(alpha_e beta[r] / 127)  (+ bias_e[n])
// and for the gated block h = a(gate) up of two such projections.
#include "experts.hpp"
#include "ffn.hpp"

namespace bitlinear {

// One output a thread.
__global__ __launch_bounds__(256) void k_grouped_plain(GroupedArgs a) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
    if (n >= a.N) return;
    int64_t e = -1;
    for (int64_t i = 0; i < a.E; ++i) {
        const Group g = group_rows(a.offsets, i, a.M);
        if (m >= g.lo && m < g.hi) e = i;
    }
    if (e < 0) return;
    const int64_t r = row_token(a.rows, m, a.T), rowb = a.K / 4;
    const float beta = r < 0 ? 0.0f : a.beta[r];
    float v[2];
    for (int p = 0; p < (a.w1 ? 2 : 1); ++p) {
        const uint8_t* w = (p ? a.w1 : a.w0) + (e * a.N + n) * rowb;
        const float* bias = p ? a.b1 : a.b0;
        int acc = 0;
        if (r >= 0)
            for (int64_t k = 0; k < a.K; ++k) acc += (int)a.xq[r * a.K + k] * (int)(((w[k / 4] >> (2 * (k % 4))) & 3) - 1);
        v[p] = (float)acc * dequant_scale((p ? a.al1 : a.al0)[e], beta);
        if (bias) v[p] = v[p] + bias[e * a.N + n];
    }
    const int64_t at = m * a.N + n;
    if (!a.w1) {
        a.y[at] = v[0];
        return;
    }
    if (a.g) {
        a.g[at] = v[0];
        a.u[at] = v[1];
    }
    a.y[at] = (a.act == BITLINEAR_ACT_SILU   ? act_value<BITLINEAR_ACT_SILU>(v[0])
               : a.act == BITLINEAR_ACT_GELU ? act_value<BITLINEAR_ACT_GELU>(v[0])
                                             : act_value<BITLINEAR_ACT_RELU2>(v[0])) * v[1];
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_grouped_plain, dim3((unsigned)((a.N + 255) / 256), (unsigned)a.M), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace bitlinear
