// gated.hip -- the gated feed-forward block's two ternary projections, its activation and the
// product, in one kernel, gfx950.
//
// What is computed: with x_q, beta the absmax codes of x, for both projections p in {gate, up}
//     acc_p[m, n] = sum_k x_q[m, k] W_p[n, k]                                (int32, exact)
//     p[m, n]     = fp32(acc_p) * fp32(alpha_p beta[m] / 127)  (+ bias_p[n])
//     h[m, n]     = a(gate[m, n]) * up[m, n]                                 (one fp32 rounding)
// so that gate and up equal two BitLinear forwards bit for bit.
//
// Every kernel gives the same lanes a gate row and the up row of the same column, so that the
// product is formed where the sums end.  Three kernels:
//   * one token in aligned rows: k_gated_gemv, which also quantizes x, on v_dot4_i32_i8;
//   * up to 32 tokens, and more where a GEMM would have few tiles (64 of 64 tokens x 128 columns):
//     k_gated_dec, the weight streams on the 16x16x64 int8 MFMA;
//   * else: k_gated_gemm, LDS tiles on the 32x32x32 int8 MFMA;
// the last two also in a form for any K % 4 == 0 and any alignment.
#include <type_traits>

#include "ffn.hpp"

namespace bitlinear {

// Element `at` of column n: g and u from their sums and scales, the activation and the product.
template <int ACT>
__device__ __forceinline__ void gated_store(const GatedArgs& a, int64_t at, int sg, int su, float scale_g, float scale_u, float bg,
                                            float bu) {
    float g = (float)sg * scale_g, u = (float)su * scale_u;
    if (a.bg) g = g + bg;
    if (a.bu) u = u + bu;
    a.h[at] = act_value<ACT>(g) * u;
    if (a.g) {
        a.g[at] = g;
        a.u[at] = u;
    }
}

// The same with the activation chosen at run time, for the kernels with few elements a lane.
__device__ __forceinline__ void gated_store(const GatedArgs& a, int64_t at, int64_t n, int sg, int su, float scale_g,
                                            float scale_u) {
    const float bg = a.bg ? a.bg[n] : 0.0f, bu = a.bu ? a.bu[n] : 0.0f;
    if (a.act == BITLINEAR_ACT_SILU) gated_store<BITLINEAR_ACT_SILU>(a, at, sg, su, scale_g, scale_u, bg, bu);
    else if (a.act == BITLINEAR_ACT_GELU) gated_store<BITLINEAR_ACT_GELU>(a, at, sg, su, scale_g, scale_u, bg, bu);
    else gated_store<BITLINEAR_ACT_RELU2>(a, at, sg, su, scale_g, scale_u, bg, bu);
}

// ---- one token ------------------------------------------------------------------------------
// A workgroup of eight waves quantizes x for itself (absmax, codes, their sum) while its first weight
// rows are on their way; a wave then takes `pairs` gate and up rows, R of each at a time.  A lane's
// load is 64 codes of a row (16 bytes); the matching x_q lies in LDS transposed 4 x 4 in each group
// of 16, so that a masked dword of codes meets its four fields' x_q in v_dot4 (chunk_sum).
// CPL: chunks of 64 weights per lane and row.
// Bound: the weight stream on large layers (K = 8192, F = 28672: 23.0 us, 5.1 TB/s), a launch and one round
// of loads on small ones (K = 4096, F = 11008: 8.0 us, 2.8 TB/s, six pairs of rows a wave; two BitLinear
// calls and a product would take 11).
constexpr int GV_WAVES = 8;

template <int CPL, int R>
__global__ __launch_bounds__(64 * GV_WAVES) void k_gated_gemv(GatedArgs a, const float* __restrict__ x, int8_t* __restrict__ xq_out,
                                                              float* __restrict__ beta_out, int pairs) {
    constexpr int NT = 64 * GV_WAVES, FPT = CPL * 1024 / NT;        // float4s of x per thread, at most
    __shared__ u32x4 xs[CPL * 256];                                 // unit (chunk / 64, group of 16, lane)
    __shared__ float red_f[GV_WAVES];
    __shared__ int red_i[GV_WAVES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t K = a.K, rowb = K >> 2;
    const int C = (int)(K >> 6), k4 = (int)(K >> 2);
    const int64_t rb = ((int64_t)blockIdx.x * GV_WAVES + wave) * pairs;
    const int64_t re = rb + pairs < a.F ? rb + pairs : a.F;         // may be <= rb: no rows
    float4 xv[FPT];
#pragma unroll
    for (int i = 0; i < FPT; ++i) xv[i] = reinterpret_cast<const float4*>(x)[tid + NT * i < k4 ? tid + NT * i : 0];
    // rows past the wave's range re-read its last row (not written); chunks past the row re-read
    // chunk 0, whose x_q there is zero
    u32x4 wg[R][CPL], wu[R][CPL];
    auto load = [&](int64_t r0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = r0 + r < re ? r0 + r : re > 0 ? re - 1 : 0;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const int c = lane + 64 * j < C ? lane + 64 * j : 0;
                wg[r][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.wg + row * rowb + 16 * c));
                wu[r][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.wu + row * rowb + 16 * c));
            }
        }
    };
    load(rb);
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < FPT; ++i) mx = fmaxf(mx, fmaxf(fmaxf(fabsf(xv[i].x), fabsf(xv[i].y)), fmaxf(fabsf(xv[i].z), fabsf(xv[i].w))));
    mx = wave_max_pos(mx);
    if (lane == 0) red_f[wave] = mx;
    __syncthreads();
    mx = red_f[0];
#pragma unroll
    for (int w = 1; w < GV_WAVES; ++w) mx = fmaxf(mx, red_f[w]);
    const float beta = mx + 1e-8f;
    uint8_t* xb = reinterpret_cast<uint8_t*>(xs);
    int sum = 0;
#pragma unroll
    for (int i = 0; i < FPT; ++i) {
        const int f = tid + NT * i, c = f >> 4, q = (f >> 2) & 3, jj = f & 3;
        const float v[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
        uint32_t d = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float t = fminf(fmaxf(rintf(v[e] * 127.0f / beta), -127.0f), 127.0f);
            const int code = f < k4 ? (int)t : 0;
            sum += code;
            d |= (uint32_t)(uint8_t)code << (8 * e);
            xb[((((c >> 6) * 4 + q) << 6) + (c & 63)) * 16 + 4 * e + jj] = (uint8_t)code;
        }
        if (blockIdx.x == 0 && f < k4) {
            for (int e = 0; e < 4; ++e) xq_out[4 * f + e] = (int8_t)(d >> (8 * e));
        }
    }
    if (blockIdx.x == 0 && tid == 0) beta_out[0] = beta;
    sum = wave_sum_rows(sum);
    if (lane == 0) red_i[wave] = sum;
    __syncthreads();
    int xsum = 0;
#pragma unroll
    for (int w = 0; w < GV_WAVES; ++w) xsum += red_i[w];
    const float scale_g = dequant_scale(a.ag[0], beta), scale_u = dequant_scale(a.au[0], beta);
    for (int64_t r0 = rb; r0 < re; r0 += R) {
        int sg[R], su[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sg[r] = su[r] = 0;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                sg[r] += chunk_sum(wg[r][j], xs + j * 256 + lane, 64, 0);
                su[r] += chunk_sum(wu[r][j], xs + j * 256 + lane, 64, 0);
            }
        }
        if (r0 + R < re) load(r0 + R);
        int mg = 0, mu = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int tg = wave_sum_rows(sg[r]), tu = wave_sum_rows(su[r]);
            if (lane == r) {
                mg = tg;
                mu = tu;
            }
        }
        if (lane < R && r0 + lane < re) gated_store(a, r0 + lane, r0 + lane, mg - xsum, mu - xsum, scale_g, scale_u);
    }
}

template <int CPL, int R>
static hipError_t launch_gated_gemv_r(const GatedArgs& a, const float* x, int8_t* xq, float* beta, int64_t pairs, hipStream_t s) {
    const int64_t waves = (a.F + pairs - 1) / pairs;
    hipLaunchKernelGGL((k_gated_gemv<CPL, R>), dim3((unsigned)((waves + GV_WAVES - 1) / GV_WAVES)), dim3(64 * GV_WAVES), 0, s, a, x,
                       xq, beta, (int)pairs);
    return hipGetLastError();
}

// About 2048 waves: 256 workgroups, since every one of them quantizes x.  Rows of one chunk a lane: all of
// a wave's rows at once if they are at most six (K = 4096, F = 11008, six pairs a wave: 8.0 against 8.4 us
// in steps of four; K = 2048, F = 8192, four: 5.3 against 6.7 us with room for six).  Longer rows: two pairs
// of two chunks, one of more (K = 8192, F = 28672: 23.6 against 24.1 us with three; K = 16384, F = 4096: 11.2
// against 12.0 with two).
template <int CPL>
static hipError_t launch_gated_gemv_cpl(const GatedArgs& a, const float* x, int8_t* xq, float* beta, hipStream_t s) {
    const int64_t pairs = (a.F + 2047) / 2048;
    if constexpr (CPL > 1) {
        return launch_gated_gemv_r<CPL, CPL == 2 ? 2 : 1>(a, x, xq, beta, pairs, s);
    } else {
        if (pairs <= 2) return launch_gated_gemv_r<1, 2>(a, x, xq, beta, pairs, s);
        if (pairs <= 4 || pairs > 6) return launch_gated_gemv_r<1, 4>(a, x, xq, beta, pairs, s);
        return launch_gated_gemv_r<1, 6>(a, x, xq, beta, pairs, s);
    }
}

bool gated_gemv_supports(const GatedArgs& a, const float* x) {
    return a.M == 1 && a.K % 64 == 0 && a.K <= 16384 && (uintptr_t)x % 16 == 0 && (uintptr_t)a.wg % 16 == 0 &&
           (uintptr_t)a.wu % 16 == 0;
}

hipError_t launch_gated_gemv(const GatedArgs& a, const float* x, int8_t* xq, float* beta, hipStream_t s) {
    switch ((a.K / 64 + 63) / 64) {
        case 1: return launch_gated_gemv_cpl<1>(a, x, xq, beta, s);
        case 2: return launch_gated_gemv_cpl<2>(a, x, xq, beta, s);
        case 3: return launch_gated_gemv_cpl<3>(a, x, xq, beta, s);
        default: return launch_gated_gemv_cpl<4>(a, x, xq, beta, s);
    }
}

// ---- few tokens or few tiles ----------------------------------------------------------------
// A workgroup of eight waves computes 16 MT tokens x 16 RB columns of both projections; wave w takes
// the steps of 256 k w, w + 8, ..., and the partial tiles are added at the end (integers: exact in
// any order).  In MFMA q of a step lane group g (lanes 16 g ..) holds weights 64 g + 16 q ..
// 64 g + 16 q + 15, dword q of the lane's 16 bytes of codes, expanded in weight order to signed bytes.
// Aligned rows (16-byte aligned tensors, K % 64 == 0): operands come through a wave's own LDS image, filled by loads that go
// past the registers; a step's image is read into registers, the next step's loads are started into
// it, and the MFMAs run while they are in flight.  Token T's 16-byte unit u of a step lies at position
// u ^ (T % 16) of its sixteen.  Otherwise operands are read straight into registers.
// Bound: beside the weights every workgroup reads its tokens' x_q, as many bytes at 16 tokens and 16 columns
// as twice the weights (from L2), and loads reach a compute unit at about 28 bytes a cycle: M = 16, K = 8192,
// F = 28672: 38 us with quantize_act (117 MB of codes from HBM, 235 MB of x_q from L2), 29 at two tokens.
// Workgroups that stay and keep x_q in registers measured 35 us there, but 16 against 12.8 us at K = 4096,
// F = 11008, and are not kept.
// 16x16x64 lane layout: A/B lane l holds row/column l % 16, k = 16 (l / 16) + j; accumulator r of
// lane l is row 4 (l / 16) + r, column l % 16.
constexpr int GD_WAVES = 8;

template <bool ALIGNED, int MT, int RB>
__global__ __launch_bounds__(64 * GD_WAVES) void k_gated_dec(GatedArgs a, int slices) {
    constexpr int IMG = (4 * MT + 2 * RB) * 64;                     // 16-byte units of a wave's image
    constexpr int TILES = 2 * RB * MT * 64;                         // of a wave's partial tiles
    constexpr int PER = ALIGNED && IMG > TILES ? IMG : TILES;
    __shared__ i32x4 lds[GD_WAVES * PER];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t K = a.K, rowb = K >> 2;
    const int64_t m0 = (int64_t)(blockIdx.x % slices) * (16 * MT), n0 = (int64_t)(blockIdx.x / slices) * (16 * RB);
    const int rows_m = (int)(a.M - m0 < 16 * MT ? a.M - m0 : 16 * MT), rows_n = (int)(a.F - n0 < 16 * RB ? a.F - n0 : 16 * RB);
    const int8_t* x0 = a.xq + m0 * K;
    const uint8_t *g0 = a.wg + n0 * rowb, *u0 = a.wu + n0 * rowb;
    const int steps = (int)((K + 255) / 256);
    const int lr = lane & 15, lg = lane >> 4;
    i32x4 acc[2 * RB][MT];
#pragma unroll
    for (int r = 0; r < 2 * RB; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[r][t] = i32x4{0, 0, 0, 0};
    // rows 0 .. RB - 1 of w: gate blocks, RB .. 2 RB - 1: up blocks
    auto multiply = [&](const i32x4 (&xv)[MT][4], const u32x4 (&w)[2 * RB]) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int r = 0; r < 2 * RB; ++r) {
                const i32x4 b = expand_signed_in_order(w[r][q]);
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xv[t][q], b, acc[r][t], 0, 0, 0);
            }
    };
    // step s with its operands read straight into registers
    auto direct = [&](int s) {
        const int64_t k = (int64_t)s * 256 + 64 * lg;
        i32x4 xv[MT][4];
        u32x4 w[2 * RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int64_t row = (int64_t)min(16 * r + lr, rows_n - 1) * rowb;
            w[r] = row_16(g0 + row, k >> 2, rowb);
            w[RB + r] = row_16(u0 + row, k >> 2, rowb);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                xv[t][q] = (i32x4)row_16(reinterpret_cast<const uint8_t*>(x0) + (int64_t)min(16 * t + lr, rows_m - 1) * K, k + 16 * q, K);
        multiply(xv, w);
    };
    if constexpr (ALIGNED) {
        const int whole = (int)(K / 256);                           // a last part step is read directly
        i32x4* img = lds + wave * IMG;
        const __amdgpu_buffer_rsrc_t rx = raw_buffer(x0, (uint32_t)rows_m * (uint32_t)K);
        const __amdgpu_buffer_rsrc_t rg = raw_buffer(g0, (uint32_t)rows_n * (uint32_t)rowb);
        const __amdgpu_buffer_rsrc_t ru = raw_buffer(u0, (uint32_t)rows_n * (uint32_t)rowb);
        // load i of x: tokens 4 i .. 4 i + 3, sixteen lanes each; load r of a matrix: lane (lr, lg) reads
        // 64 codes of row 16 r + lr.  Rows past the end repeat the last one; groups of four tokens past it
        // are not loaded (what they hold reaches only outputs that are not written).
        uint32_t xo[4 * MT], wo[RB];
#pragma unroll
        for (int i = 0; i < 4 * MT; ++i)
            xo[i] = (uint32_t)min(4 * i + lg, rows_m - 1) * (uint32_t)K + 16u * (uint32_t)(lr ^ ((4 * i + lg) & 15));
#pragma unroll
        for (int r = 0; r < RB; ++r) wo[r] = (uint32_t)min(16 * r + lr, rows_n - 1) * (uint32_t)rowb + 16u * (uint32_t)lg;
        auto fetch = [&](int s) {
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                load_lds16(rg, wo[r], (uint32_t)s * 64u, img + 64 * (4 * MT + r));
                load_lds16(ru, wo[r], (uint32_t)s * 64u, img + 64 * (4 * MT + RB + r));
            }
#pragma unroll
            for (int i = 0; i < 4 * MT; ++i)
                if (4 * i < rows_m) load_lds16(rx, xo[i], (uint32_t)s * 256u, img + 64 * i);
        };
        if (wave < whole) fetch(wave);
        for (int s = wave; s < whole; s += GD_WAVES) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0x0F70);                     // vmcnt(0): the image is whole
            __builtin_amdgcn_sched_barrier(0);
            i32x4 xv[MT][4];
            u32x4 w[2 * RB];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) xv[t][q] = img[(16 * t + lr) * 16 + ((4 * lg + q) ^ lr)];
#pragma unroll
            for (int r = 0; r < 2 * RB; ++r) w[r] = (u32x4)img[64 * (4 * MT + r) + lane];
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xC07F);                     // lgkmcnt(0): every read of it is over
            __builtin_amdgcn_sched_barrier(0);
            if (s + GD_WAVES < whole) fetch(s + GD_WAVES);
            multiply(xv, w);
        }
        if (whole < steps && whole % GD_WAVES == wave) direct(whole);
    } else {
        struct Part {
            i32x4 x[MT][4];
            u32x4 w[2 * RB];
        };
        auto load = [&](int s) {
            const int64_t k = (int64_t)s * 256 + 64 * lg;
            Part f;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int64_t row = (int64_t)min(16 * r + lr, rows_n - 1) * rowb + (k >> 2);
                f.w[r] = load_16(g0 + row);
                f.w[RB + r] = load_16(u0 + row);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    f.x[t][q] = (i32x4)load_16(reinterpret_cast<const uint8_t*>(x0) + (int64_t)min(16 * t + lr, rows_m - 1) * K + k + 16 * q);
            return f;
        };
        // whole steps, the next one's loads under way; the last part step goes to the next wave in turn
        const int whole = (int)(K / 256);
        if (wave < whole) {
            Part f = load(wave);
            for (int s = wave; s < whole; s += GD_WAVES) {
                const Part next = load(min(s + GD_WAVES, whole - 1));
                multiply(f.x, f.w);
                f = next;
            }
        }
        if (whole < steps && whole % GD_WAVES == wave) direct(whole);
    }
    __syncthreads();                                                // every wave is done with its image
#pragma unroll
    for (int r = 0; r < 2 * RB; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) lds[(wave * 2 * RB * MT + r * MT + t) * 64 + lane] = acc[r][t];
    __syncthreads();
    const float ag = a.ag[0], au = a.au[0];
    // element e = (block, token block, lane, i): i-th accumulator
    for (int e = tid; e < RB * MT * 256; e += 64 * GD_WAVES) {
        const int l = e & 63, i = (e >> 6) & 3, tile = e >> 8, r = tile / MT, t = tile % MT;
        const int n = 16 * r + (l & 15), m = 16 * t + 4 * (l >> 4) + i;
        if (n >= rows_n || m >= rows_m) continue;
        int sg = 0, su = 0;
#pragma unroll
        for (int w = 0; w < GD_WAVES; ++w) {
            const int* p = reinterpret_cast<const int*>(lds + (w * 2 * RB * MT + tile) * 64 + l);
            sg += p[i];
            su += p[i + RB * MT * 256];
        }
        const float beta = a.beta[m0 + m];
        gated_store(a, (m0 + m) * a.F + n0 + n, n0 + n, sg, su, dequant_scale(ag, beta), dequant_scale(au, beta));
    }
}

template <bool ALIGNED, int MT, int RB>
static hipError_t launch_gated_dec_rb(const GatedArgs& a, hipStream_t s) {
    const int64_t slices = (a.M + 16 * MT - 1) / (16 * MT), blocks = (a.F + 16 * RB - 1) / (16 * RB);
    hipLaunchKernelGGL((k_gated_dec<ALIGNED, MT, RB>), dim3((unsigned)(slices * blocks)), dim3(64 * GD_WAVES), 0, s, a, (int)slices);
    return hipGetLastError();
}

// One block of 16 columns a workgroup; two where 48 or 64 tokens leave room for one workgroup per compute
// unit only and there would be more than 256 (K = 11008, F = 4096: M = 64 (256 workgroups) 20.3 against
// 25.8 us with two blocks, M = 128 (512) 34.7 against 27.7; K = 4096, F = 11008, M = 16 (688) 12.2 against
// 13.2; M = 32 15.0 against 18.6 us).
template <bool ALIGNED, int MT>
static hipError_t launch_gated_dec_mt(const GatedArgs& a, hipStream_t s) {
    if constexpr (MT >= 3)
        if ((a.M + 16 * MT - 1) / (16 * MT) * ((a.F + 15) / 16) > 256) return launch_gated_dec_rb<ALIGNED, MT, 2>(a, s);
    return launch_gated_dec_rb<ALIGNED, MT, 1>(a, s);
}

template <bool ALIGNED>
static hipError_t launch_gated_dec(const GatedArgs& a, hipStream_t s) {
    const int64_t tiles = (a.M + 15) / 16;
    return tiles == 1   ? launch_gated_dec_mt<ALIGNED, 1>(a, s)
           : tiles == 2 ? launch_gated_dec_mt<ALIGNED, 2>(a, s)
           : tiles == 3 ? launch_gated_dec_mt<ALIGNED, 3>(a, s)
                        : launch_gated_dec_mt<ALIGNED, 4>(a, s);
}

// ---- many tiles -----------------------------------------------------------------------------
// A workgroup of four waves computes 32 FM tokens x 128 columns of both projections, a wave all the
// tokens x 32 columns of each: FM 32-token operands against one gate and one up operand, so that the
// expansion of a weight operand (17 instructions) serves FM MFMAs.  Steps of 128 k, three LDS stages
// (4 FM + 8 KiB each: 32 FM token rows of 128 bytes, 256 weight rows of 32 bytes) filled two steps
// ahead by loads that go past the registers (aligned rows: 16-byte aligned tensors, K % 64 == 0), or two filled through
// registers.  Unit u of token row r lies at slot u ^ ((r / 2) % 8), unit u of weight row r at slot
// u ^ ((r / 8) % 2), so that an operand read spreads over all banks.
// Bound: power.  M = 2048, K = 4096, F = 11008: 181 us, 2.04 POPS (a library's plain int8 product of 8192^3:
// 2.04); the matrix cores are busy 47% of the cycles and the clock is down at 2.0 GHz.
// In the two MFMAs of k 64 h .. 64 h + 63 (h = 0, 1) a lane group holds 32 codes, eight bytes of a
// weight row: the lane's unit h, of which group lg uses dwords 2 lg and 2 lg + 1.
constexpr int GG_BF = 128, GG_BK = 128;

template <int ACT, bool ALIGNED, int FM>
__global__ __launch_bounds__(256, 2) void k_gated_gemm(GatedArgs a, int tiles_m, int tiles_f) {
    constexpr int GG_BM = 32 * FM, OB = GG_BM * 8, UNITS = OB + 2 * GG_BF * 2;
    __shared__ i32x4 st0[UNITS];
    __shared__ i32x4 st1[UNITS];
    __shared__ i32x4 st2[ALIGNED ? UNITS : 1];
    __shared__ __align__(16) float scale[2][GG_BM];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // a contiguous run of tiles for each XCD, four rows of tiles at a time
    const int T = tiles_m * tiles_f, xcd = blockIdx.x & 7, per = T >> 3, rem = T & 7;
    int t = xcd * per + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
    const int grp = t / (4 * tiles_f), gm = tiles_m - 4 * grp < 4 ? tiles_m - 4 * grp : 4;
    t -= grp * 4 * tiles_f;
    const int64_t m0 = (int64_t)(4 * grp + t % gm) * GG_BM, n0 = (int64_t)(t / gm) * GG_BF;
    const int64_t K = a.K, rowb = K >> 2;
    const int rows_m = (int)(a.M - m0 < GG_BM ? a.M - m0 : GG_BM), rows_n = (int)(a.F - n0 < GG_BF ? a.F - n0 : GG_BF);
    const uint8_t* x0 = reinterpret_cast<const uint8_t*>(a.xq) + m0 * K;
    const uint8_t *g0 = a.wg + n0 * rowb, *u0 = a.wu + n0 * rowb;
    if (tid < GG_BM) {
        const float beta = a.beta[m0 + (tid < rows_m ? tid : 0)];
        scale[0][tid] = dequant_scale(a.ag[0], beta);
        scale[1][tid] = dequant_scale(a.au[0], beta);
    }

    i32x16 acc[FM][2];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = i32x16{};
    const int lr = lane & 31, lg = lane >> 5, sw = (lr >> 1) & 7, sb = (lr >> 3) & 1;
    auto multiply = [&](const i32x4* st, int halves) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h >= halves) break;
            // weight rows of a stage: 128 gate rows, then 128 up rows
            uint2 w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                w[j] = reinterpret_cast<const uint2*>(st + OB + (128 * j + 32 * wave + lr) * 2 + (h ^ sb))[lg];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                i32x4 fa[FM], fb[2];
                const int u = 4 * h + 2 * lg + kk;
#pragma unroll
                for (int i = 0; i < FM; ++i) fa[i] = st[(32 * i + lr) * 8 + (u ^ sw)];
#pragma unroll
                for (int j = 0; j < 2; ++j) fb[j] = expand_signed_in_order(kk ? w[j].y : w[j].x);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
            }
        }
    };
    // load block q of x: token rows 8 q .. 8 q + 7 (wave w takes FM w .. FM w + FM - 1); of a matrix: rows
    // 32 q .. 32 q + 31 (wave w takes q = w of both)
    const int wrow = 32 * wave + (lane >> 1), wunit = (lane & 1) ^ ((wrow >> 3) & 1);
    auto xrow = [&](int q) { return 8 * (FM * wave + q) + (lane >> 3); };
    auto xunit = [&](int q) { return (lane & 7) ^ ((xrow(q) >> 1) & 7); };
    if constexpr (ALIGNED) {
        const __amdgpu_buffer_rsrc_t rx = raw_buffer(x0, (uint32_t)rows_m * (uint32_t)K);
        const __amdgpu_buffer_rsrc_t rg = raw_buffer(g0, (uint32_t)rows_n * (uint32_t)rowb);
        const __amdgpu_buffer_rsrc_t ru = raw_buffer(u0, (uint32_t)rows_n * (uint32_t)rowb);
        uint32_t xo[FM];
#pragma unroll
        for (int q = 0; q < FM; ++q) xo[q] = (uint32_t)min(xrow(q), rows_m - 1) * (uint32_t)K + 16u * xunit(q);
        const uint32_t wo = (uint32_t)min(wrow, rows_n - 1) * (uint32_t)rowb + 16u * wunit;
        const int steps = (int)(K / GG_BK), last = steps - 1;
        auto fetch = [&](i32x4* st, int s) {
            s = s < last ? s : last;
#pragma unroll
            for (int q = 0; q < FM; ++q) load_lds16(rx, xo[q], (uint32_t)s * GG_BK, st + 64 * (FM * wave + q));
            load_lds16(rg, wo, (uint32_t)s * (GG_BK / 4), st + OB + 64 * wave);
            load_lds16(ru, wo, (uint32_t)s * (GG_BK / 4), st + OB + 256 + 64 * wave);
            __builtin_amdgcn_sched_barrier(0);
        };
        // the stage to be read has landed, for every wave, and every read of the stage to be filled is
        // over; loads past the last step repeat it and are not read
        auto turn = [&]() {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0x0070 | (FM + 2));          // vmcnt(the next stage's loads) lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        };
        int s = 0;
        if (steps > 0) {
            fetch(st0, 0);
            fetch(st1, 1);
        }
        for (; s + 3 <= steps; s += 3) {
            turn();
            fetch(st2, s + 2);
            multiply(st0, 2);
            turn();
            fetch(st0, s + 3);
            multiply(st1, 2);
            turn();
            fetch(st1, s + 4);
            multiply(st2, 2);
        }
        if (s < steps) {
            turn();
            multiply(st0, 2);
        }
        __builtin_amdgcn_s_waitcnt(0x0070);                         // nothing is in flight into the stages any more
        __builtin_amdgcn_s_barrier();
        if (s + 1 < steps) multiply(st1, 2);
        if (K % GG_BK) {
            // the last 64 k through st0, which nobody reads any more
            const int64_t k = (int64_t)steps * GG_BK;
#pragma unroll
            for (int j = 0; j < (FM + 1) / 2; ++j) {
                const int r = (tid >> 2) + 64 * j, u = tid & 3;
                if (r >= GG_BM) break;
                st0[r * 8 + (u ^ ((r >> 1) & 7))] = *reinterpret_cast<const i32x4*>(x0 + (int64_t)min(r, rows_m - 1) * K + k + 16 * u);
            }
            const uint8_t* w = tid < 128 ? g0 : u0;
            st0[OB + tid * 2 + ((tid >> 3) & 1)] = *reinterpret_cast<const i32x4*>(w + (int64_t)min(tid & 127, rows_n - 1) * rowb + (k >> 2));
            __syncthreads();
            multiply(st0, 1);
        }
    } else {
        struct Regs {
            u32x4 v[FM + 2];
        };
        const int64_t wr = (int64_t)min(wrow, rows_n - 1) * rowb;
        auto load = [&](int s) {
            const int64_t k = (int64_t)s * GG_BK;
            Regs r;
#pragma unroll
            for (int q = 0; q < FM; ++q) r.v[q] = load_16(x0 + (int64_t)min(xrow(q), rows_m - 1) * K + k + 16 * xunit(q));
            r.v[FM] = load_16(g0 + wr + (k >> 2) + 16 * wunit);
            r.v[FM + 1] = load_16(u0 + wr + (k >> 2) + 16 * wunit);
            return r;
        };
        auto put = [&](i32x4* st, const Regs& r) {
#pragma unroll
            for (int q = 0; q < FM; ++q) st[64 * (FM * wave + q) + lane] = (i32x4)r.v[q];
            st[OB + 64 * wave + lane] = (i32x4)r.v[FM];
            st[OB + 256 + 64 * wave + lane] = (i32x4)r.v[FM + 1];
        };
        // The last part step first (sums of integers are exact in any order), through st0, while the first
        // whole steps' loads are under way; then whole steps in st1 and st0 in turn, loaded three ahead.
        const int whole = (int)(K / GG_BK), last = whole - 1;
        Regs r0, r1;
        if (whole > 0) {
            r0 = load(0);
            r1 = load(min(1, last));
        }
        if (K % GG_BK) {
            const int64_t k = (int64_t)whole * GG_BK;
            Regs r;
#pragma unroll
            for (int q = 0; q < FM; ++q) r.v[q] = row_16(x0 + (int64_t)min(xrow(q), rows_m - 1) * K, k + 16 * xunit(q), K);
            r.v[FM] = row_16(g0 + wr, (k >> 2) + 16 * wunit, rowb);
            r.v[FM + 1] = row_16(u0 + wr, (k >> 2) + 16 * wunit, rowb);
            put(st0, r);
            __syncthreads();
            multiply(st0, 2);
        } else {
            __syncthreads();                                        // the tokens' scales
        }
        for (int s = 0; s < whole; s += 2) {
            put(st1, r0);                                           // its last readers are past the barrier before this one
            r0 = load(min(s + 2, last));
            __syncthreads();
            multiply(st1, 2);
            if (s + 1 >= whole) break;
            put(st0, r1);
            r1 = load(min(s + 3, last));
            __syncthreads();
            multiply(st0, 2);
        }
    }
    // accumulator r of lane l: token 8 (r / 4) + 4 (l / 32) + r % 4 of the block, column l % 32
    const int n = 32 * wave + lr;
    if (n >= rows_n) return;
    const float bg = a.bg ? a.bg[n0 + n] : 0.0f, bu = a.bu ? a.bu[n0 + n] : 0.0f;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int m = 32 * i + 8 * q + 4 * lg;
            const float4 g4 = *reinterpret_cast<const float4*>(&scale[0][m]), u4 = *reinterpret_cast<const float4*>(&scale[1][m]);
            const float gs[4] = {g4.x, g4.y, g4.z, g4.w}, us[4] = {u4.x, u4.y, u4.z, u4.w};
            const int64_t at = (m0 + m) * a.F + n0 + n;
            float g[4], u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g[e] = (float)acc[i][0][4 * q + e] * gs[e];
                u[e] = (float)acc[i][1][4 * q + e] * us[e];
                if (a.bg) g[e] = g[e] + bg;
                if (a.bu) u[e] = u[e] + bu;
            }
            float v[4];
            if constexpr (ACT == BITLINEAR_ACT_GELU) {
                const float4 v4 = gelu4_f32(make_float4(g[0], g[1], g[2], g[3]));
                v[0] = v4.x, v[1] = v4.y, v[2] = v4.z, v[3] = v4.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = act_value<ACT>(g[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e < rows_m) a.h[at + e * a.F] = v[e] * u[e];
            if (a.g) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m + e < rows_m) {
                        a.g[at + e * a.F] = g[e];
                        a.u[at + e * a.F] = u[e];
                    }
            }
        }
}

template <int ACT, bool ALIGNED, int FM>
static hipError_t launch_gated_gemm_fm(const GatedArgs& a, hipStream_t s) {
    const int64_t tm = (a.M + 32 * FM - 1) / (32 * FM), tf = (a.F + GG_BF - 1) / GG_BF;
    hipLaunchKernelGGL((k_gated_gemm<ACT, ALIGNED, FM>), dim3((unsigned)(tm * tf)), dim3(256), 0, s, a, (int)tm, (int)tf);
    return hipGetLastError();
}

// Tiles of 32 tokens while they all run at once, of 64 while those of 128 would not fill the 512 workgroup
// slots well: K = 4096, F = 11008, M = 64 (172 tiles of 32) 21.6 against 26.0 us, M = 128 (344) 30.4 against
// 27.0 with 64-token tiles and 39.4 with 128, M = 512 (344 of 128) 58.6 against 61.3 with 128, M = 1024 (688)
// 106.6 against 97.8; K = 8192, F = 28672, M = 256 (448) 131 against 113 us.
template <bool ALIGNED>
static hipError_t launch_gated_gemm(const GatedArgs& a, hipStream_t s) {
    const int64_t tf = (a.F + GG_BF - 1) / GG_BF;
    const int fm = (a.M + 31) / 32 * tf <= 256 ? 1 : (a.M + 127) / 128 * tf <= 384 ? 2 : 4;
    auto run = [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        return fm == 1 ? launch_gated_gemm_fm<ACT, ALIGNED, 1>(a, s)
               : fm == 2 ? launch_gated_gemm_fm<ACT, ALIGNED, 2>(a, s)
                         : launch_gated_gemm_fm<ACT, ALIGNED, 4>(a, s);
    };
    switch (a.act) {
        case BITLINEAR_ACT_SILU: return run(std::integral_constant<int, BITLINEAR_ACT_SILU>());
        case BITLINEAR_ACT_GELU: return run(std::integral_constant<int, BITLINEAR_ACT_GELU>());
        default: return run(std::integral_constant<int, BITLINEAR_ACT_RELU2>());
    }
}

// The streaming kernel up to 32 tokens, and beyond while the GEMM has at most 64 tiles of 64 x 128, too
// few to fill the chip: K = 4096, F = 11008: M = 32 15.2 against 21.3 us, M = 64 (86 tiles) 26.3 against
// 21.6, M = 128 38.2 against 27.0; K = 11008, F = 4096: M = 128 (64 tiles) 27.9 against 56.6, M = 512 (256)
// 86.9 against 61.4; K = 1024, F = 2816: M = 64 (22) 7.2 against 9.4, M = 256 (88) 16.4 against 10.0 us.
hipError_t launch_gated(const GatedArgs& a, hipStream_t s) {
    const bool aligned = a.K % 64 == 0 && (uintptr_t)a.xq % 16 == 0 && (uintptr_t)a.wg % 16 == 0 && (uintptr_t)a.wu % 16 == 0;
    if (a.M <= 32 || (a.M + 63) / 64 * ((a.F + GG_BF - 1) / GG_BF) <= 64)
        return aligned ? launch_gated_dec<true>(a, s) : launch_gated_dec<false>(a, s);
    return aligned ? launch_gated_gemm<true>(a, s) : launch_gated_gemm<false>(a, s);
}

}  // namespace bitlinear
