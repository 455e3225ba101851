// gated.hip -- the gated feed-forward block's two ternary projections, its activation and the
// product, in one kernel, gfx950.
//
// What is computed: with x_q, beta the absmax codes of x, for both projections p in {gate, up}
//     acc_p[m, n] = sum_k x_q[m, k] W_p[n, k]                                (int32, exact)
//     p[m, n]     = fp32(acc_p) * fp32(alpha_p beta[m] / 127)  (+ bias_p[n])
//     h[m, n]     = a(gate[m, n]) * up[m, n]                                 (one fp32 rounding)
// so that gate and up equal two BitLinear forwards bit for bit.
#include "ffn.hpp"

namespace bitlinear {

// One wave per output column n, lanes over packed bytes; any K % 4 == 0, any alignment.
template <int ACT>
__global__ __launch_bounds__(256) void k_gated_generic(GatedArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= a.F) return;
    const int64_t K = a.K, rowb = K >> 2;
    for (int64_t m = 0; m < a.M; ++m) {
        int sg = 0, su = 0;
        for (int64_t b = lane; b < rowb; b += 64) {
            const uint32_t cg = a.wg[n * rowb + b], cu = a.wu[n * rowb + b];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = a.xq[m * K + 4 * b + i];
                sg += ((int)((cg >> (2 * i)) & 3u) - 1) * x;
                su += ((int)((cu >> (2 * i)) & 3u) - 1) * x;
            }
        }
        sg = wave_sum_i32(sg);
        su = wave_sum_i32(su);
        if (lane == 0) {
            const float g = dequant(sg, dequant_scale(a.ag[0], a.beta[m]), a.bg, n);
            const float u = dequant(su, dequant_scale(a.au[0], a.beta[m]), a.bu, n);
            a.h[m * a.F + n] = act_value<ACT>(g) * u;
            if (a.g) {
                a.g[m * a.F + n] = g;
                a.u[m * a.F + n] = u;
            }
        }
    }
}

template <int ACT>
static hipError_t launch_gated_act(const GatedArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((k_gated_generic<ACT>), dim3((unsigned)((a.F + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_gated(const GatedArgs& a, hipStream_t s) {
    switch (a.act) {
        case BITLINEAR_ACT_GELU: return launch_gated_act<BITLINEAR_ACT_GELU>(a, s);
        case BITLINEAR_ACT_SILU: return launch_gated_act<BITLINEAR_ACT_SILU>(a, s);
        default: return launch_gated_act<BITLINEAR_ACT_RELU2>(a, s);
    }
}

}  // namespace bitlinear
