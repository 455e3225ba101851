// backward.hip -- gradients of ternary projections, straight through the quantizers, gfx950.
//
// What is computed, for each projection p with incoming gradient d_p [M, N]:
//     dx[m, k]    = sum_p alpha_p sum_n d_p[m, n] W_p[n, k]
//     dW_p[n, k]  = sum_m d_p[m, n] (beta[m] / 127) x_q[m, k]
//     dbias_p[n]  = sum_m d_p[m, n]
// One projection: d = dy.  The gated block h = a(g) u: d_gate = dh u a'(g), d_up = dh a(g).
//
// Both products pair an fp32 gradient with a small integer (a ternary weight, an int8 code) that
// fp16 holds exactly.  So each gradient row (a token's for dx, a channel's for dW) is scaled by a
// power of two that brings its largest element to [2^14, 2^15), and every element is split into
// hi + lo, two fp16 numbers: hi is the element rounded to 11 bits, lo the exact remainder rounded
// to 11 bits, together at least 22 bits (2^-40 of the row's largest where lo is subnormal).  Two
// f16 MFMA products into one fp32 accumulator then give the product to fp32 accuracy at half the
// f16 matrix rate, several times the rate of fp32 products.
//
// Steps, each a launch over the whole problem:
//   1. k_grad_max: the largest |d alpha| of every token and |d beta / 127| of every channel;
//   2. k_grad_split: d once more, scaled and split, written token-major (dx) and channel-major (dW);
//   3. k_weights_t, k_codes_t: the integer operands in fp16 with the sum's index contiguous;
//   4. k_split_gemm (and k_split_sum where a sum is cut into parts) for dx and for dW;
//   5. k_bias_sum.
#include <limits.h>

#include "ffn.hpp"

namespace bitlinear {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Exponent s of the power of two that scales a row whose largest element is mx to [2^14, 2^15);
// clamped so that 2^s and 2^-s are normal numbers.
__device__ __forceinline__ int scale_exponent(float mx) {
    if (mx == 0.0f) return 0;
    const int s = 15 - __builtin_amdgcn_frexp_expf(mx);
    return s > 126 ? 126 : s < -126 ? -126 : s;
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// d of element (m, n): one projection d[0] = dy; gated d[0] = dh u a'(g), d[1] = dh a(g).
// ACT 0: one projection.
template <int ACT>
__device__ __forceinline__ void grad_at(const BackwardArgs& a, int64_t i, float (&d)[2]) {
    const float dy = a.dy[i];
    if constexpr (ACT == 0) {
        d[0] = dy;
    } else {
        float v, slope;
        act_grad<ACT>(a.g[i], v, slope);
        d[0] = dy * a.u[i] * slope;
        d[1] = dy * v;
    }
}

struct GradPlan {
    int64_t Np, Mp, Lx;            // N and M rounded up to 64, P Np
    uint32_t *rmax, *cmax;         // bits of the largest |d alpha| [M], |d beta / 127| [P N]
    double* bias_part;             // [ceil(M / 64)][P N]
    _Float16 *xh, *xl;             // dx: split gradients [M, Lx]
    _Float16 *wh, *wl;             // dW: split gradients [P N, Mp]
    _Float16 *wt, *ct;             // W_hat^T [K, Lx], x_q^T [K, Mp]
    float* part;                   // partial sums of a product cut into parts
    int parts_x, parts_w;
    size_t bytes;
};

constexpr int SG_BM = 128, SG_BN = 256, SG_BK = 32, SG_SLOTS = 512;

// Parts to cut a sum of length L into: the fewest rounds of workgroups over the 512 slots per part,
// counting each part's share of the sum; parts of at least 512 terms, at most 8.
static int sum_parts(int64_t I, int64_t J, int64_t L) {
    const int64_t tiles = ((I + SG_BM - 1) / SG_BM) * ((J + SG_BN - 1) / SG_BN);
    int best = 1;
    double cost = 1e30;
    for (int s = 1; s <= 8 && (s == 1 || L / s >= 512); ++s) {
        const double c = (double)((tiles * s + SG_SLOTS - 1) / SG_SLOTS) / s * (1.0 + 0.03 * (s > 1 ? s : 0));
        if (c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

static GradPlan grad_plan(int64_t M, int64_t K, int64_t N, bool gated, void* ws) {
    GradPlan p{};
    const int64_t P = gated ? 2 : 1;
    p.Np = (N + 63) / 64 * 64;
    p.Mp = (M + 63) / 64 * 64;
    p.Lx = P * p.Np;
    p.parts_x = sum_parts(M, K, p.Lx);
    p.parts_w = sum_parts(P * N, K, p.Mp);
    uint8_t* base = static_cast<uint8_t*>(ws);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t* q = base + off;
        off += (bytes + 255) / 256 * 256;
        return q;
    };
    p.rmax = reinterpret_cast<uint32_t*>(take((size_t)(M + P * N) * 4));
    p.cmax = p.rmax + M;
    p.bias_part = reinterpret_cast<double*>(take((size_t)(p.Mp / 64) * P * N * 8));
    p.xh = reinterpret_cast<_Float16*>(take((size_t)M * p.Lx * 2));
    p.xl = reinterpret_cast<_Float16*>(take((size_t)M * p.Lx * 2));
    p.wh = reinterpret_cast<_Float16*>(take((size_t)P * N * p.Mp * 2));
    p.wl = reinterpret_cast<_Float16*>(take((size_t)P * N * p.Mp * 2));
    p.wt = reinterpret_cast<_Float16*>(take((size_t)K * p.Lx * 2));
    p.ct = reinterpret_cast<_Float16*>(take((size_t)K * p.Mp * 2));
    const size_t px = p.parts_x > 1 ? (size_t)p.parts_x * M * K * 4 : 0;
    const size_t pw = p.parts_w > 1 ? (size_t)p.parts_w * P * N * K * 4 : 0;
    p.part = reinterpret_cast<float*>(take(px > pw ? px : pw));
    p.bytes = off;
    return p;
}

size_t backward_workspace(int64_t M, int64_t K, int64_t N, bool gated) { return grad_plan(M, K, N, gated, nullptr).bytes; }

__global__ __launch_bounds__(256) void k_zero(uint32_t* __restrict__ p, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0u;
}

// Largest elements.  A workgroup takes 64 tokens x 256 columns, a wave 16 of the tokens, a lane four
// columns 64 apart (whole lines whatever the alignment).  Non-negative floats compare as their
// bits, and maxima do not depend on order, so integer atomics give the same result every time.
template <int ACT>
__global__ __launch_bounds__(256) void k_grad_max(BackwardArgs a, GradPlan p, int ctiles) {
    constexpr int P = ACT == 0 ? 1 : 2;
    __shared__ float cm[4][P][256];
    __shared__ double cs[4][P][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)(blockIdx.x % ctiles) * 256, m0 = (int64_t)(blockIdx.x / ctiles) * 64;
    const float al[2] = {a.al0[0], ACT == 0 ? 0.0f : a.al1[0]};
    const bool bias = a.db0 || a.db1;
    float cmx[P][4];
    double sum[P][4];
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            cmx[q][c] = 0.0f;
            sum[q][c] = 0.0;
        }
    for (int t = 0; t < 16; ++t) {
        const int64_t m = m0 + 16 * wave + t;
        if (m >= a.M) break;
        const float bs = a.beta[m] / 127.0f;
        float rm = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int64_t n = n0 + 64 * c + lane;
            if (n < a.N) {
                float d[2];
                grad_at<ACT>(a, m * a.N + n, d);
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    rm = fmaxf(rm, fabsf(d[q] * al[q]));
                    cmx[q][c] = fmaxf(cmx[q][c], fabsf(d[q] * bs));
                    if (bias) sum[q][c] += (double)d[q];
                }
            }
        }
        rm = wave_max_f32(rm);
        if (lane == 0) atomicMax(&p.rmax[m], __float_as_uint(rm));
    }
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            cm[wave][q][64 * c + lane] = cmx[q][c];
            cs[wave][q][64 * c + lane] = sum[q][c];
        }
    __syncthreads();
    const int64_t n = n0 + threadIdx.x;
    if (n >= a.N) return;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        float v = 0.0f;
        double s = 0.0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            v = fmaxf(v, cm[w][q][threadIdx.x]);
            s += cs[w][q][threadIdx.x];
        }
        atomicMax(&p.cmax[q * a.N + n], __float_as_uint(v));
        if (bias) p.bias_part[(m0 / 64) * P * a.N + q * a.N + n] = s;
    }
}

__device__ __forceinline__ uint32_t split_f16(float v) {
    const _Float16 hi = (_Float16)v;
    const _Float16 lo = (_Float16)(v - (float)hi);
    return (uint32_t)__builtin_bit_cast(uint16_t, hi) | (uint32_t)__builtin_bit_cast(uint16_t, lo) << 16;
}

// Scaled and split gradients, 64 tokens x 64 columns per workgroup: token-major as they are read,
// channel-major through LDS.  Padded columns and tokens are written as zeros.
template <int ACT>
__global__ __launch_bounds__(256) void k_grad_split(BackwardArgs a, GradPlan p, int ctiles) {
    constexpr int P = ACT == 0 ? 1 : 2;
    __shared__ uint32_t tile[P][64][65];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)(blockIdx.x % ctiles) * 64, m0 = (int64_t)(blockIdx.x / ctiles) * 64;
    const int64_t n = n0 + lane;
    const float al[2] = {a.al0[0], ACT == 0 ? 0.0f : a.al1[0]};
    float cscale[P];
#pragma unroll
    for (int q = 0; q < P; ++q) cscale[q] = n < a.N ? pow2f(scale_exponent(__uint_as_float(p.cmax[q * a.N + n]))) : 0.0f;
    for (int t = 0; t < 16; ++t) {
        const int64_t m = m0 + 16 * wave + t;
        float d[2] = {0.0f, 0.0f}, bs = 0.0f, rscale = 0.0f;
        if (m < a.M) {
            bs = a.beta[m] / 127.0f;
            rscale = pow2f(scale_exponent(__uint_as_float(p.rmax[m])));
            if (n < a.N) grad_at<ACT>(a, m * a.N + n, d);
        }
#pragma unroll
        for (int q = 0; q < P; ++q) {
            if (a.dx && m < a.M) {
                const uint32_t v = split_f16(d[q] * al[q] * rscale);
                reinterpret_cast<uint16_t*>(p.xh)[m * p.Lx + q * p.Np + n] = (uint16_t)v;
                reinterpret_cast<uint16_t*>(p.xl)[m * p.Lx + q * p.Np + n] = (uint16_t)(v >> 16);
            }
            tile[q][lane][16 * wave + t] = split_f16(d[q] * bs * cscale[q]);
        }
    }
    if (!a.dw0) return;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < P; ++q)
        for (int r = wave; r < 64; r += 4) {
            if (n0 + r >= a.N) break;
            const uint32_t v = tile[q][r][lane];
            const int64_t o = (q * a.N + n0 + r) * p.Mp + m0 + lane;
            reinterpret_cast<uint16_t*>(p.wh)[o] = (uint16_t)v;
            reinterpret_cast<uint16_t*>(p.wl)[o] = (uint16_t)(v >> 16);
        }
}

// W_hat^T in fp16, [K, Lx]: 64 weight rows x 64 columns k per workgroup.  Codes 0, 1, 2 become -1, 0, 1.
__global__ __launch_bounds__(256) void k_weights_t(BackwardArgs a, GradPlan p, int ktiles) {
    __shared__ uint8_t tile[64][20];
    const int64_t k0 = (int64_t)(blockIdx.x % ktiles) * 64, l0 = (int64_t)(blockIdx.x / ktiles) * 64;
    const int q = l0 >= p.Np;
    const int64_t n0 = l0 - q * p.Np, rowb = a.K >> 2;
    const uint8_t* w = q ? a.w1 : a.w0;
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
        const int r = i >> 4, b = i & 15;
        const int64_t n = n0 + r, kb = (k0 >> 2) + b;
        tile[r][b] = n < a.N && kb < rowb ? w[n * rowb + kb] : (uint8_t)0x55;
    }
    __syncthreads();
    const int r = threadIdx.x & 63;
    for (int j = threadIdx.x >> 6; j < 64; j += 4) {
        if (k0 + j >= a.K) break;
        const int c = (tile[r][j >> 2] >> (2 * (j & 3))) & 3;
        p.wt[(k0 + j) * p.Lx + l0 + r] = (_Float16)(float)(c - 1);
    }
}

// x_q^T in fp16, [K, Mp]: 64 tokens x 64 columns per workgroup.
__global__ __launch_bounds__(256) void k_codes_t(BackwardArgs a, GradPlan p, int ktiles) {
    __shared__ int8_t tile[64][68];
    const int64_t k0 = (int64_t)(blockIdx.x % ktiles) * 64, m0 = (int64_t)(blockIdx.x / ktiles) * 64;
    const int lane = threadIdx.x & 63;
    for (int r = threadIdx.x >> 6; r < 64; r += 4)
        tile[r][lane] = m0 + r < a.M && k0 + lane < a.K ? a.xq[(m0 + r) * a.K + k0 + lane] : (int8_t)0;
    __syncthreads();
    for (int j = threadIdx.x >> 6; j < 64; j += 4) {
        if (k0 + j >= a.K) break;
        p.ct[(k0 + j) * p.Mp + m0 + lane] = (_Float16)(float)tile[lane][j];
    }
}

struct SplitArgs {
    const _Float16 *ah, *al;       // [I, L] hi and lo planes
    const _Float16* b;             // [J, L]
    const uint32_t* amax;          // [I] bits of the rows' largest elements
    int64_t I, J, L;               // L a multiple of 64
    float *c0, *c1;                // rows below I0 go to c0 [I0, J], the others to c1
    int64_t I0;
    float* part;                   // parts > 1: [parts][I][J] unscaled sums
    int parts, tiles_i, tiles_j;
};

// C[i, j] = 2^-s_i sum_l (hi[i, l] + lo[i, l]) b[j, l].  A workgroup of four waves computes 128 x 256
// outputs, a wave 64 x 128 of them in 32 x 32 blocks (128 accumulator registers), in steps of 32 l.
// Both LDS stages (32 KiB each: 128 rows of hi, of lo, 256 rows of b, 64 bytes a row) are filled by
// loads that go past the registers; a stage is loaded while the other is multiplied.  Unit u (16
// bytes) of row r lies at slot u ^ ((r / 2) % 4) of its row, so that eight consecutive lanes of an
// operand read (eight rows, one unit) meet eight different bank groups.
__global__ __launch_bounds__(256, 2) void k_split_gemm(SplitArgs a) {
    __shared__ i32x4 st0[2048];
    __shared__ i32x4 st1[2048];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // consecutive workgroups go to the eight XCDs in turn: give each XCD a contiguous run of tiles,
    // four rows of tiles at a time, so that its L2 holds the panels its workgroups share
    const int T = a.parts * a.tiles_i * a.tiles_j;
    const int xcd = blockIdx.x & 7, per = T >> 3, rem = T & 7;
    int t = xcd * per + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
    const int part = t / (a.tiles_i * a.tiles_j);
    t -= part * a.tiles_i * a.tiles_j;
    const int grp = t / (4 * a.tiles_j), gi = a.tiles_i - 4 * grp < 4 ? a.tiles_i - 4 * grp : 4;
    t -= grp * 4 * a.tiles_j;
    const int64_t i0 = (int64_t)(4 * grp + t % gi) * SG_BM, j0 = (int64_t)(t / gi) * SG_BN;
    const int KS = (int)(a.L / SG_BK);
    const int ks0 = (int)((int64_t)KS * part / a.parts), ks1 = (int)((int64_t)KS * (part + 1) / a.parts);

    // loads: instruction q of a wave fills 64 slots (16 rows); rows past the end repeat the last one
    const int lrow = lane >> 2, unit = (lane & 3) ^ ((lane >> 3) & 3);
    const uint32_t ldb = (uint32_t)(a.L * 2);
    const int64_t rows_i = a.I - i0 < SG_BM ? a.I - i0 : SG_BM, rows_j = a.J - j0 < SG_BN ? a.J - j0 : SG_BN;
    const __amdgpu_buffer_rsrc_t rh = raw_buffer(a.ah + i0 * a.L, (uint32_t)rows_i * ldb);
    const __amdgpu_buffer_rsrc_t rl = raw_buffer(a.al + i0 * a.L, (uint32_t)rows_i * ldb);
    const __amdgpu_buffer_rsrc_t rb = raw_buffer(a.b + j0 * a.L, (uint32_t)rows_j * ldb);
    uint32_t ao[2], bo[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int r = 16 * (2 * wave + q) + lrow;
        ao[q] = (uint32_t)(r < rows_i ? r : (int)rows_i - 1) * ldb + 16u * unit;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = 16 * (4 * wave + q) + lrow;
        bo[q] = (uint32_t)(r < rows_j ? r : (int)rows_j - 1) * ldb + 16u * unit;
    }
    auto fetch = [&](i32x4* st, int ks) {
        const uint32_t so = (uint32_t)ks * (SG_BK * 2);
#pragma unroll
        for (int q = 0; q < 2; ++q) load_lds16(rh, ao[q], so, st + 64 * (2 * wave + q));
#pragma unroll
        for (int q = 0; q < 2; ++q) load_lds16(rl, ao[q], so, st + 512 + 64 * (2 * wave + q));
#pragma unroll
        for (int q = 0; q < 4; ++q) load_lds16(rb, bo[q], so, st + 1024 + 64 * (4 * wave + q));
        __builtin_amdgcn_sched_barrier(0);         // issued here, not where their data is needed
    };

    f32x16 acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
    const int wi = wave & 1, wj = wave >> 1, lr = lane & 31, lg = lane >> 5;
    const int sw = (lr >> 1) & 3;
    auto multiply = [&](const i32x4* st) {
        f16x8 fh[2][2], fl[2][2], fb[2][4];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int s = (2 * kk + lg) ^ sw;
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[kk][j] = __builtin_bit_cast(f16x8, st[1024 + (128 * wj + 32 * j + lr) * 4 + s]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fh[kk][i] = __builtin_bit_cast(f16x8, st[(64 * wi + 32 * i + lr) * 4 + s]);
                fl[kk][i] = __builtin_bit_cast(f16x8, st[512 + (64 * wi + 32 * i + lr) * 4 + s]);
            }
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fh[kk][i], fb[kk][j], acc[i][j], 0, 0, 0);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fl[kk][i], fb[kk][j], acc[i][j], 0, 0, 0);
                }
    };
    // every load into a stage has landed, for every wave, and every read of the other stage is over
    auto turn = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0070);        // vmcnt(0) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    int ks = ks0;
    if (ks < ks1) fetch(st0, ks);
    for (; ks + 2 <= ks1; ks += 2) {
        turn();
        fetch(st1, ks + 1);
        multiply(st0);
        turn();
        if (ks + 2 < ks1) fetch(st0, ks + 2);
        multiply(st1);
    }
    if (ks < ks1) {
        turn();
        multiply(st0);
    }

    // accumulator r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4 of the block, column l % 32
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int64_t row = i0 + 64 * wi + 32 * i + 8 * (r / 4) + 4 * lg + r % 4;
            if (row >= a.I) continue;
            float* out;
            float inv = 1.0f;
            if (a.parts > 1) {
                out = a.part + ((int64_t)part * a.I + row) * a.J;
            } else {
                inv = pow2f(-scale_exponent(__uint_as_float(a.amax[row])));
                out = row < a.I0 ? a.c0 + row * a.J : a.c1 + (row - a.I0) * a.J;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t col = j0 + 128 * wj + 32 * j + lr;
                if (col < a.J) out[col] = acc[i][j][r] * inv;
            }
        }
}

// The parts of a sum added in their order, scaled back.
__global__ __launch_bounds__(256) void k_split_sum(SplitArgs a) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x, n = a.I * a.J;
    if (e >= n) return;
    const int64_t row = e / a.J;
    float s = 0.0f;
    for (int q = 0; q < a.parts; ++q) s += a.part[q * n + e];
    s *= pow2f(-scale_exponent(__uint_as_float(a.amax[row])));
    if (row < a.I0) a.c0[e] = s;
    else a.c1[e - a.I0 * a.J] = s;
}

static hipError_t launch_split(SplitArgs a, hipStream_t s) {
    a.tiles_i = (int)((a.I + SG_BM - 1) / SG_BM);
    a.tiles_j = (int)((a.J + SG_BN - 1) / SG_BN);
    const int64_t grid = (int64_t)a.parts * a.tiles_i * a.tiles_j;
    hipLaunchKernelGGL(k_split_gemm, dim3((unsigned)grid), dim3(256), 0, s, a);
    if (a.parts > 1) hipLaunchKernelGGL(k_split_sum, dim3((unsigned)((a.I * a.J + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

// Column sums from the 64-token partial sums, in token order.
__global__ __launch_bounds__(256) void k_bias_sum(BackwardArgs a, GradPlan p, int P) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, NT = P * a.N;
    if (n >= NT) return;
    float* out = n < a.N ? a.db0 : a.db1;
    if (!out) return;
    double s = 0.0;
    for (int64_t t = 0; t < p.Mp / 64; ++t) s += p.bias_part[t * NT + n];
    out[n < a.N ? n : n - a.N] = (float)s;
}

template <int ACT>
static hipError_t launch_grads(const BackwardArgs& a, hipStream_t s) {
    constexpr int P = ACT == 0 ? 1 : 2;
    const GradPlan p = grad_plan(a.M, a.K, a.N, P == 2, a.ws);
    auto blocks = [](int64_t n) { return dim3((unsigned)n); };
    const int64_t nmax = a.M + P * a.N;
    hipLaunchKernelGGL(k_zero, blocks((nmax + 255) / 256), dim3(256), 0, s, p.rmax, nmax);
    const int64_t mt = p.Mp / 64, ct256 = (a.N + 255) / 256, ct64 = p.Np / 64, kt = (a.K + 63) / 64;
    hipLaunchKernelGGL(k_grad_max<ACT>, blocks(mt * ct256), dim3(256), 0, s, a, p, (int)ct256);
    if (a.dx || a.dw0) hipLaunchKernelGGL(k_grad_split<ACT>, blocks(mt * ct64), dim3(256), 0, s, a, p, (int)ct64);
    if (a.dx) {
        hipLaunchKernelGGL(k_weights_t, blocks(p.Lx / 64 * kt), dim3(256), 0, s, a, p, (int)kt);
        const hipError_t e = launch_split(SplitArgs{p.xh, p.xl, p.wt, p.rmax, a.M, a.K, p.Lx, a.dx, nullptr, a.M, p.part,
                                                    p.parts_x, 0, 0}, s);
        if (e != hipSuccess) return e;
    }
    if (a.dw0) {
        hipLaunchKernelGGL(k_codes_t, blocks(mt * kt), dim3(256), 0, s, a, p, (int)kt);
        const hipError_t e = launch_split(SplitArgs{p.wh, p.wl, p.ct, p.cmax, P * a.N, a.K, p.Mp, a.dw0, a.dw1, a.N, p.part,
                                                    p.parts_w, 0, 0}, s);
        if (e != hipSuccess) return e;
    }
    if (a.db0 || a.db1) hipLaunchKernelGGL(k_bias_sum, blocks((P * a.N + 255) / 256), dim3(256), 0, s, a, p, P);
    return hipGetLastError();
}

hipError_t launch_backward(const BackwardArgs& a, hipStream_t s) {
    if (!a.g) return launch_grads<0>(a, s);
    switch (a.act) {
        case BITLINEAR_ACT_GELU: return launch_grads<BITLINEAR_ACT_GELU>(a, s);
        case BITLINEAR_ACT_SILU: return launch_grads<BITLINEAR_ACT_SILU>(a, s);
        default: return launch_grads<BITLINEAR_ACT_RELU2>(a, s);
    }
}

}  // namespace bitlinear
