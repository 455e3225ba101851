// i8.hip -- int8 x int8 matmul with a scale for each token and each output channel (W8A8), gfx950.
//
// What is computed: acc[m, n] = sum_k x_q[m, k] W_q[n, k]  (int32, exact),
//     y[m, n] = (fp32(acc) * fp32(beta[m] / 127)) * fp32(gamma[n] / 127)  (+ bias[n]),
// every step one fp32 rounding.
#include "ffn.hpp"

namespace bitlinear {

// Scale of a token or a channel: fp32(s / 127), an IEEE division.
__device__ __forceinline__ float i8_scale(float s) { return s / 127.0f; }

__device__ __forceinline__ float i8_dequant(int acc, float bs, float gs, const float* __restrict__ bias, int64_t n) {
    float v = (float)acc * bs * gs;
    if (bias) v = v + bias[n];
    return v;
}

// One wave per output column, lanes over k; any K, any alignment.
__global__ __launch_bounds__(256) void k_i8_generic(I8Args a) {
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= a.N) return;
    for (int64_t m = 0; m < a.M; ++m) {
        int s = 0;
        for (int64_t k = lane; k < a.K; k += 64) s += (int)a.xq[m * a.K + k] * (int)a.wq[n * a.K + k];
        s = wave_sum_i32(s);
        if (lane == 0) {
            a.y[m * a.N + n] = i8_dequant(s, i8_scale(a.beta[m]), i8_scale(a.gamma[n]), a.bias, n);
            if (a.acc) a.acc[m * a.N + n] = s;
        }
    }
}

hipError_t launch_forward_i8(const I8Args& a, hipStream_t s) {
    hipLaunchKernelGGL(k_i8_generic, dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace bitlinear
