// i8.hip -- int8 x int8 matmul with a scale for each token and each output channel (W8A8), gfx950.
//
// What is computed: acc[m, n] = sum_k x_q[m, k] W_q[n, k]  (int32, exact),
//     y[m, n] = (fp32(acc) * fp32(beta[m] / 127)) * fp32(gamma[n] / 127)  (+ bias[n]),
// every step one fp32 rounding.
//
// Three kernels by the number of tokens, each in a form for aligned rows (16-byte aligned tensors,
// K % 16 == 0) and one for any K and alignment, the last two also in one for rows off dword boundaries
// (K = 4098, N = 4096, 48 tokens: 13.5 us against 30.3 without):
//   * one token: k_i8_gemv, the weight stream against x_q in LDS, on v_dot4_i32_i8;
//   * few tokens: k_i8_dec, the weight stream on the 16x16x64 int8 MFMA, the waves of a workgroup
//     taking turns along K;
//   * many: k_i8_gemm, LDS tiles on the 32x32x32 int8 MFMA.
#include "ffn.hpp"

namespace bitlinear {

// Scale of a token or a channel: fp32(s / 127), an IEEE division.
__device__ __forceinline__ float i8_scale(float s) { return s / 127.0f; }

// Output `at` (m N + n) from its sum, with the token's and the channel's scale and the bias.
__device__ __forceinline__ void i8_store(const I8Args& a, int64_t at, int acc, float bs, float gs, float bias) {
    float v = (float)acc * bs * gs;
    if (a.bias) v = v + bias;
    a.y[at] = v;
    if (a.acc) a.acc[at] = acc;
}

template <bool DWORDS = false>
__device__ __forceinline__ i32x4 row_16(const int8_t* __restrict__ p, int64_t i, int64_t row) {
    return (i32x4)row_16<DWORDS>(reinterpret_cast<const uint8_t*>(p), i, row);
}
template <bool DWORDS = false>
__device__ __forceinline__ i32x4 load_16(const int8_t* __restrict__ p) {
    return (i32x4)load_16<DWORDS>(reinterpret_cast<const uint8_t*>(p));
}

// How the rows lie: 16-byte aligned (and K % 16 == 0), on dwords, or anywhere.
constexpr int ROWS_16 = 16, ROWS_4 = 4, ROWS_1 = 1;

// ---- one token ------------------------------------------------------------------------------
// A wave takes R weight rows, 1 KiB of each at a time, so that R loads of 16 bytes a lane are in
// flight while the last ones meet x_q, which lies in LDS as it is, in whole units of 16 (zeros up to the
// next KiB); what is left of K goes to lane 0.
// Bound: the weight stream (K = 4096, N = 32000: 25 us, 5.2 TB/s from HBM).
template <bool ALIGNED, int R>
__global__ __launch_bounds__(256) void k_i8_gemv(I8Args a) {
    extern __shared__ i32x4 xs[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t K = a.K, r0 = ((int64_t)blockIdx.x * 4 + wave) * R;
    const int chunks = (int)((K + 1023) / 1024);
    const int8_t* w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = a.wq + (r0 + r < a.N ? r0 + r : a.N - 1) * K;
    auto load = [&](i32x4 (&v)[R], int c) {
        const int64_t k = (int64_t)c * 1024 + 16 * lane;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // past the last whole unit x_q is zero: any bytes will do, the row's first (rows of fewer than
            // 16 have no whole unit, and are not read here)
            const int8_t* p = w[r] + (k + 16 <= K ? k : 0);
            if constexpr (ALIGNED) v[r] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(p));
            else if (K >= 16) v[r] = load_16(p);
            else v[r] = i32x4{0, 0, 0, 0};
        }
    };
    i32x4 v0[R], v1[R];
    load(v0, 0);
    for (int i = tid; i < chunks * 64; i += 256)
        xs[i] = (int64_t)i * 16 + 16 <= K ? load_16(a.xq + (int64_t)i * 16) : i32x4{0, 0, 0, 0};
    __syncthreads();
    int s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = 0;
    auto dot = [&](const i32x4 (&v)[R], int c) {
        const i32x4 x = xs[c * 64 + lane];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[r] = dot4((uint32_t)v[r][j], (uint32_t)x[j], s[r]);
    };
    for (int c = 0; c < chunks; c += 2) {
        if (c + 1 < chunks) load(v1, c + 1);
        dot(v0, c);
        if (c + 1 >= chunks) break;
        if (c + 2 < chunks) load(v0, c + 2);
        dot(v1, c + 1);
    }
    if (!ALIGNED && K % 16 && lane == 0) {
        const int64_t k = K / 16 * 16;
        const i32x4 x = row_16(a.xq, k, K);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const i32x4 v = row_16(w[r], k, K);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[r] = dot4((uint32_t)v[j], (uint32_t)x[j], s[r]);
        }
    }
    int mine = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int t = wave_sum_rows(s[r]);
        if (lane == r) mine = t;
    }
    const int64_t n = r0 + lane;
    if (lane < R && n < a.N) i8_store(a, n, mine, i8_scale(a.beta[0]), i8_scale(a.gamma[n]), a.bias ? a.bias[n] : 0.0f);
}

template <bool ALIGNED>
static hipError_t launch_i8_gemv(const I8Args& a, hipStream_t s) {
    constexpr int R = 4;
    const size_t lds = (size_t)((a.K + 1023) / 1024) * 1024;
    return launch_with_lds(k_i8_gemv<ALIGNED, R>, dim3((unsigned)((a.N + 4 * R - 1) / (4 * R))), dim3(256), lds, s, a);
}

// Position of 16-byte unit u (0..3) in the four slots of row r of an LDS tile of 64-byte rows: the
// lanes of an operand read (16 rows or more, one unit each) then meet 16 different groups of banks.
__device__ __forceinline__ int unit_swizzle(int r) { return ((r >> 2) & 3) ^ (((r >> 1) & 1) << 1); }

// ---- few tokens -----------------------------------------------------------------------------
// A workgroup of eight waves computes 16 MT tokens x 16 RB channels; wave w takes the steps of 64 k
// w, w + 8, ..., and the eight partial tiles are added at the end (integers: exact in any order).
// Aligned rows: each wave has a ring of D LDS images of a step (16-row blocks of 64 bytes a row), filled
// by loads that go past the registers, D - 1 steps ahead; no wave waits for another.
// Any K and alignment: operands straight into registers in the MFMA's layout.
// Bound: the weight stream at 16 tokens (K = N = 8192: 14.9 us, 4.5 TB/s); beyond, every workgroup's own
// reading of x_q, 100 MB from L2 beside 67 of weights at 48 tokens (19 us).  Steps of 128 k in pairs for
// whole lines measured 6 to 15% slower.
// 16x16x64 lane layout: A/B lane l holds row/column l % 16, k = 16 (l / 16) + j; accumulator r of
// lane l is row 4 (l / 16) + r, column l % 16.
constexpr int I8_WAVES = 8;

template <int ROWS, int MT, int RB>
__global__ __launch_bounds__(64 * I8_WAVES) void k_i8_dec(I8Args a, int slices) {
    constexpr bool ALIGNED = ROWS == ROWS_16, DWORDS = ROWS == ROWS_1;
    constexpr int IMG = (RB + MT) * 64;
    constexpr int D = 3;                                           // images of a ring
    __shared__ i32x4 st0[I8_WAVES * IMG];
    __shared__ i32x4 st1[ALIGNED ? I8_WAVES * IMG : 1];
    __shared__ i32x4 st2[ALIGNED ? I8_WAVES * IMG : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t K = a.K;
    const int64_t m0 = (int64_t)(blockIdx.x % slices) * (16 * MT), n0 = (int64_t)(blockIdx.x / slices) * (16 * RB);
    const int rows_m = (int)(a.M - m0 < 16 * MT ? a.M - m0 : 16 * MT), rows_n = (int)(a.N - n0 < 16 * RB ? a.N - n0 : 16 * RB);
    const int8_t* x0 = a.xq + m0 * K;
    const int8_t* w0 = a.wq + n0 * K;
    const int steps = (int)((K + 63) / 64);
    const int lr = lane & 15, lg = lane >> 4;
    i32x4 acc[RB][MT];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[r][t] = i32x4{0, 0, 0, 0};
    auto multiply = [&](const i32x4 (&x)[MT], const i32x4 (&w)[RB]) {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[t], w[r], acc[r][t], 0, 0, 0);
    };
    if constexpr (ALIGNED) {
        // lane l of a load fills slot l: row l / 4; rows past the end repeat the last one, and offsets
        // past the buffers (the end of the last step when K % 64 != 0) are not read from memory
        const int row = lane >> 2, unit = (lane & 3) ^ unit_swizzle(row);
        const __amdgpu_buffer_rsrc_t rx = raw_buffer(x0, (uint32_t)rows_m * (uint32_t)K);
        const __amdgpu_buffer_rsrc_t rw = raw_buffer(w0, (uint32_t)rows_n * (uint32_t)K);
        uint32_t xo[MT], wo[RB];
#pragma unroll
        for (int t = 0; t < MT; ++t) xo[t] = (uint32_t)min(16 * t + row, rows_m - 1) * (uint32_t)K + 16u * unit;
#pragma unroll
        for (int r = 0; r < RB; ++r) wo[r] = (uint32_t)min(16 * r + row, rows_n - 1) * (uint32_t)K + 16u * unit;
        auto fetch = [&](i32x4* st, int s) {
            i32x4* img = st + wave * IMG;
#pragma unroll
            for (int r = 0; r < RB; ++r) load_lds16(rw, wo[r], (uint32_t)s * 64u, img + 64 * r);
#pragma unroll
            for (int t = 0; t < MT; ++t) load_lds16(rx, xo[t], (uint32_t)s * 64u, img + 64 * (RB + t));
            __builtin_amdgcn_sched_barrier(0);
        };
        const int at = lr * 4 + (lg ^ unit_swizzle(lr));
        // step s from its image
        auto step = [&](const i32x4* st, int s) {
            const i32x4* img = st + wave * IMG + at;
            i32x4 x[MT], w[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) w[r] = img[64 * r];
#pragma unroll
            for (int t = 0; t < MT; ++t) x[t] = img[64 * (RB + t)];
            // past the end of its row (K % 64 != 0) a load has read what follows it
            const bool live = (int64_t)s * 64 + 16 * lg < K;
#pragma unroll
            for (int t = 0; t < MT; ++t) x[t] = live ? x[t] : i32x4{0, 0, 0, 0};
            multiply(x, w);
            __builtin_amdgcn_sched_barrier(0);
        };
        // The loop has no branches, so that the loads in flight can be counted: loads past the wave's last
        // step repeat it and are not read.  An image is filled again only after the MFMAs that read it.
        constexpr int W = I8_WAVES, FLY = (D - 1) * (RB + MT);
        static_assert(FLY < 16, "the count fits the low four bits of vmcnt");
        i32x4* const ring[D] = {st0, st1, st2};
        int left = wave < steps ? (steps - wave + W - 1) / W : 0, s = wave;
        const int last = wave + (left - 1) * W;
        if (left > 0) {
#pragma unroll
            for (int j = 0; j < D - 1; ++j) fetch(ring[j], min(s + j * W, last));
        }
        for (; left >= D; left -= D, s += D * W) {
#pragma unroll
            for (int j = 0; j < D; ++j) {
                fetch(ring[(j + D - 1) % D], min(s + (j + D - 1) * W, last));
                __builtin_amdgcn_s_waitcnt(0x0F70 | FLY);                        // vmcnt(the loads of the D - 1 later steps)
                __builtin_amdgcn_sched_barrier(0);
                step(ring[j], s + j * W);
            }
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);                                            // vmcnt(0)
#pragma unroll
        for (int j = 0; j < D - 1; ++j)
            if (j < left) step(ring[j], s + j * W);
    } else {
        const int8_t *xp[MT], *wp[RB];
#pragma unroll
        for (int t = 0; t < MT; ++t) xp[t] = x0 + (int64_t)min(16 * t + lr, rows_m - 1) * K;
#pragma unroll
        for (int r = 0; r < RB; ++r) wp[r] = w0 + (int64_t)min(16 * r + lr, rows_n - 1) * K;
        struct Part {
            i32x4 x[MT], w[RB];
        };
        auto load = [&](int s) {
            const int64_t k = (int64_t)s * 64 + 16 * lg;
            Part f;
#pragma unroll
            for (int r = 0; r < RB; ++r) f.w[r] = load_16<DWORDS>(wp[r] + k);
#pragma unroll
            for (int t = 0; t < MT; ++t) f.x[t] = load_16<DWORDS>(xp[t] + k);
            return f;
        };
        // whole steps, the next one's loads under way; the last part step goes to the next wave in turn
        const int whole = (int)(K / 64), last = whole - 1;
        Part f0, f1;
        if (wave < whole) f0 = load(wave);
        for (int s = wave; s < whole; s += 2 * I8_WAVES) {
            f1 = load(min(s + I8_WAVES, last));
            multiply(f0.x, f0.w);
            f0 = load(min(s + 2 * I8_WAVES, last));
            if (s + I8_WAVES < whole) multiply(f1.x, f1.w);
        }
        if (whole < steps && whole % I8_WAVES == wave) {
            const int64_t k = (int64_t)whole * 64 + 16 * lg;
#pragma unroll
            for (int r = 0; r < RB; ++r) f0.w[r] = row_16<DWORDS>(wp[r], k, K);
#pragma unroll
            for (int t = 0; t < MT; ++t) f0.x[t] = row_16<DWORDS>(xp[t], k, K);
            multiply(f0.x, f0.w);
        }
    }
    // the eight partial tiles through LDS, one block of 16 channels after another
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        __syncthreads();
#pragma unroll
        for (int t = 0; t < MT; ++t) st0[(wave * MT + t) * 64 + lane] = acc[r][t];
        __syncthreads();
        for (int e = tid; e < MT * 64; e += 64 * I8_WAVES) {
            const int l = e & 63, t = e >> 6, n = 16 * r + (l & 15);
            i32x4 sum = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < I8_WAVES; ++w) sum += st0[(w * MT + t) * 64 + l];
            if (n >= rows_n) continue;
            const float gs = i8_scale(a.gamma[n0 + n]), bias = a.bias ? a.bias[n0 + n] : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = 16 * t + 4 * (l >> 4) + i;
                if (m < rows_m) i8_store(a, (m0 + m) * a.N + n0 + n, sum[i], i8_scale(a.beta[m0 + m]), gs, bias);
            }
        }
    }
}

template <int ROWS, int MT, int RB>
static hipError_t launch_i8_dec_rb(const I8Args& a, hipStream_t s) {
    const int64_t slices = (a.M + 16 * MT - 1) / (16 * MT), blocks = (a.N + 16 * RB - 1) / (16 * RB);
    hipLaunchKernelGGL((k_i8_dec<ROWS, MT, RB>), dim3((unsigned)(slices * blocks)), dim3(64 * I8_WAVES), 0, s, a, (int)slices);
    return hipGetLastError();
}

// One block of 16 channels a workgroup; two where 48 or 64 tokens leave room for one workgroup per compute
// unit only and there would be more than 256 (K = N = 4096, M = 48 (256 workgroups) 7.4 against 9.4 us with
// two blocks; K = N = 8192, M = 48 (512) 26.7 against 20.9; M = 16 15.5 against 17.9 us).
template <int ROWS, int MT>
static hipError_t launch_i8_dec_mt(const I8Args& a, hipStream_t s) {
    if constexpr (MT >= 3)
        if ((a.M + 16 * MT - 1) / (16 * MT) * ((a.N + 15) / 16) > 256) return launch_i8_dec_rb<ROWS, MT, 2>(a, s);
    return launch_i8_dec_rb<ROWS, MT, 1>(a, s);
}

template <int ROWS>
static hipError_t launch_i8_dec(const I8Args& a, hipStream_t s) {
    const int64_t tiles = (a.M + 15) / 16;
    return tiles == 1   ? launch_i8_dec_mt<ROWS, 1>(a, s)
           : tiles == 2 ? launch_i8_dec_mt<ROWS, 2>(a, s)
           : tiles == 3 ? launch_i8_dec_mt<ROWS, 3>(a, s)
                        : launch_i8_dec_mt<ROWS, 4>(a, s);
}

// ---- many tokens ----------------------------------------------------------------------------
// A workgroup of eight waves computes 64 MI tokens x 128 FN channels, a wave 32 MI x 32 FN of them in 32 x 32
// blocks, in steps of 128 k (rows of whole cache lines); three LDS stages (up to 48 KiB each), filled two
// steps ahead by loads that go past the registers (aligned rows), or two filled through registers.
// Unit u (16 bytes) of row r lies at slot u ^ ((r / 2) % 8) of its eight: no bank conflicts.
// Bound: power.  M = 2048, K = 11008, N = 4096: 91 us, 2.03 POPS (a library's plain int8 product of 8192^3:
// 2.04); the matrix cores are busy 59% of the cycles and the clock is down at 1.8 GHz.  The same tile with a
// step's loads and operand reads before its MFMAs took 108 us (38% busy, 2.15 GHz), through registers 114,
// with four waves of 64 x 128 110 us.
// 32x32x32 lane layout: A/B lane l holds row/column l % 32, k = 16 (l / 32) + j; accumulator r of
// lane l is row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
constexpr int IG_BK = 128;

template <int ROWS, int MI, int FN>
__global__ __launch_bounds__(512, 2) void k_i8_gemm(I8Args a, int tiles_m, int tiles_n) {
    constexpr bool ALIGNED = ROWS == ROWS_16, DWORDS = ROWS == ROWS_1;
    constexpr int IG_BM = 64 * MI, IG_BN = 128 * FN, OB = IG_BM * 8, UNITS = OB + IG_BN * 8;
    __shared__ i32x4 st0[UNITS];
    __shared__ i32x4 st1[UNITS];
    __shared__ i32x4 st2[ALIGNED ? UNITS : 1];
    __shared__ __align__(16) float bscale[IG_BM];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // a contiguous run of tiles for each XCD, four rows of tiles at a time
    const int T = tiles_m * tiles_n, xcd = blockIdx.x & 7, per = T >> 3, rem = T & 7;
    int t = xcd * per + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
    const int grp = t / (4 * tiles_n), gm = tiles_m - 4 * grp < 4 ? tiles_m - 4 * grp : 4;
    t -= grp * 4 * tiles_n;
    const int64_t m0 = (int64_t)(4 * grp + t % gm) * IG_BM, n0 = (int64_t)(t / gm) * IG_BN;
    const int64_t K = a.K;
    const int rows_m = (int)(a.M - m0 < IG_BM ? a.M - m0 : IG_BM), rows_n = (int)(a.N - n0 < IG_BN ? a.N - n0 : IG_BN);
    const int8_t* x0 = a.xq + m0 * K;
    const int8_t* w0 = a.wq + n0 * K;

    i32x16 acc[MI][FN];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = i32x16{};
    const int wi = wave & 1, wj = wave >> 1, lr = lane & 31, lg = lane >> 5, sw = (lr >> 1) & 7;
    // scales before the loop: the tokens' in LDS, the channels' in registers
    if (tid < IG_BM) bscale[tid] = tid < rows_m ? i8_scale(a.beta[m0 + tid]) : 0.0f;
    float gs[FN], bias[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int64_t n = n0 + min(32 * FN * wj + 32 * j + lr, rows_n - 1);
        gs[j] = i8_scale(a.gamma[n]);
        bias[j] = a.bias ? a.bias[n] : 0.0f;
    }
    struct Frag {
        i32x4 a[MI], b[FN];
    };
    // operands of k 32 kk .. 32 kk + 31 of the step in stage st
    auto read = [&](const i32x4* st, int kk) {
        const int u = 2 * kk + lg, at = u ^ sw;
        Frag f;
#pragma unroll
        for (int j = 0; j < FN; ++j) f.b[j] = st[OB + (32 * FN * wj + 32 * j + lr) * 8 + at];
#pragma unroll
        for (int i = 0; i < MI; ++i) f.a[i] = st[(32 * MI * wi + 32 * i + lr) * 8 + at];
        return f;
    };
    auto multiply = [&](const Frag& f) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    // load block q (8 rows): wave w takes MI w .. MI w + MI - 1 of x_q and 2 FN w .. 2 FN w + 2 FN - 1 of W_q
    auto block_row = [&](int q) { return 8 * q + (lane >> 3); };
    auto block_unit = [&](int q) { return (lane & 7) ^ ((block_row(q) >> 1) & 7); };
    if constexpr (ALIGNED) {
        const __amdgpu_buffer_rsrc_t rx = raw_buffer(x0, (uint32_t)rows_m * (uint32_t)K);
        const __amdgpu_buffer_rsrc_t rw = raw_buffer(w0, (uint32_t)rows_n * (uint32_t)K);
        uint32_t xo[MI], wo[2 * FN];
#pragma unroll
        for (int q = 0; q < MI; ++q)
            xo[q] = (uint32_t)min(block_row(MI * wave + q), rows_m - 1) * (uint32_t)K + 16u * block_unit(MI * wave + q);
#pragma unroll
        for (int q = 0; q < 2 * FN; ++q)
            wo[q] = (uint32_t)min(block_row(2 * FN * wave + q), rows_n - 1) * (uint32_t)K + 16u * block_unit(2 * FN * wave + q);
        // a third of a step's loads
        auto fetch = [&](i32x4* st, int s, int third) {
            const uint32_t so = (uint32_t)s * IG_BK;
            if (third == 0) {
#pragma unroll
                for (int q = 0; q < MI; ++q) load_lds16(rx, xo[q], so, st + 64 * (MI * wave + q));
            } else {
#pragma unroll
                for (int q = FN * (third - 1); q < FN * third; ++q) load_lds16(rw, wo[q], so, st + OB + 64 * (2 * FN * wave + q));
            }
        };
        // Step s in stage `cur`, its first operands in f0.  Operands are read one part ahead of their
        // MFMAs, across the turn too; the stage that a turn frees is loaded with the step after next
        // but one, a third at a time, so that the matrix cores have work while loads are issued.  Loads
        // past the last whole step repeat it and are not read.
        const int steps = (int)(K / IG_BK), last = steps - 1;
        auto step = [&](i32x4* cur, i32x4* nxt, i32x4* prv, int s, Frag& f0) {
            Frag f1 = read(cur, 1);
            fetch(prv, min(s + 2, last), 1);
            multiply(f0);
            f0 = read(cur, 2);
            fetch(prv, min(s + 2, last), 2);
            multiply(f1);
            f1 = read(cur, 3);
            multiply(f0);
            // step s + 1 has landed for every wave, and every wave holds the rest of step s in registers
            __builtin_amdgcn_s_waitcnt(0x0070 | (MI + 2 * FN)); // vmcnt(the loads of step s + 2) lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            f0 = read(nxt, 0);
            fetch(cur, min(s + 3, last), 0);
            multiply(f1);
        };
        if (steps > 0) {
#pragma unroll
            for (int q = 0; q < 3; ++q) fetch(st0, 0, q);
#pragma unroll
            for (int q = 0; q < 3; ++q) fetch(st1, min(1, last), q);
            fetch(st2, min(2, last), 0);
            __builtin_amdgcn_s_waitcnt(0x0070 | (2 * MI + 2 * FN)); // vmcnt(the loads after step 0's) lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            Frag f = read(st0, 0);
            int s = 0;
            for (; s + 3 <= steps; s += 3) {
                step(st0, st1, st2, s, f);
                step(st1, st2, st0, s + 1, f);
                step(st2, st0, st1, s + 2, f);
            }
            if (s < steps) step(st0, st1, st2, s, f);
            if (s + 1 < steps) step(st1, st2, st0, s + 1, f);
            __builtin_amdgcn_s_waitcnt(0x0070);            // nothing is in flight into the stages any more
        } else {
            __syncthreads();                               // the tokens' scales
        }
        // what is left of K, fewer than 128, straight into the operands
        for (int64_t k = (int64_t)steps * IG_BK; k < K; k += 32) {
            Frag f;
#pragma unroll
            for (int i = 0; i < MI; ++i) f.a[i] = row_16(x0 + (int64_t)min(32 * MI * wi + 32 * i + lr, rows_m - 1) * K, k + 16 * lg, K);
#pragma unroll
            for (int j = 0; j < FN; ++j) f.b[j] = row_16(w0 + (int64_t)min(32 * FN * wj + 32 * j + lr, rows_n - 1) * K, k + 16 * lg, K);
            multiply(f);
        }
    } else {
        const int8_t *xp[MI], *wp[2 * FN];
#pragma unroll
        for (int q = 0; q < MI; ++q) xp[q] = x0 + (int64_t)min(block_row(MI * wave + q), rows_m - 1) * K;
#pragma unroll
        for (int q = 0; q < 2 * FN; ++q) wp[q] = w0 + (int64_t)min(block_row(2 * FN * wave + q), rows_n - 1) * K;
        struct Regs {
            i32x4 v[MI + 2 * FN];
        };
        auto load = [&](int s) {
            const int64_t k = (int64_t)s * IG_BK;
            Regs r;
#pragma unroll
            for (int q = 0; q < MI; ++q) r.v[q] = load_16<DWORDS>(xp[q] + k + 16 * block_unit(MI * wave + q));
#pragma unroll
            for (int q = 0; q < 2 * FN; ++q) r.v[MI + q] = load_16<DWORDS>(wp[q] + k + 16 * block_unit(2 * FN * wave + q));
            return r;
        };
        auto put = [&](i32x4* st, const Regs& r) {
#pragma unroll
            for (int q = 0; q < MI; ++q) st[64 * (MI * wave + q) + lane] = r.v[q];
#pragma unroll
            for (int q = 0; q < 2 * FN; ++q) st[OB + 64 * (2 * FN * wave + q) + lane] = r.v[MI + q];
        };
        auto multiply_stage = [&](const i32x4* st) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) multiply(read(st, kk));
        };
        // The last part step first (sums of integers are exact in any order), through st0, while the first
        // whole steps' loads are under way; then whole steps in st1 and st0 in turn, loaded three ahead.
        const int whole = (int)(K / IG_BK), last = whole - 1;
        Regs r0, r1;
        if (whole > 0) {
            r0 = load(0);
            r1 = load(min(1, last));
        }
        if (K % IG_BK) {
            const int64_t k = (int64_t)whole * IG_BK;
            Regs r;
#pragma unroll
            for (int q = 0; q < MI; ++q) r.v[q] = row_16<DWORDS>(xp[q], k + 16 * block_unit(MI * wave + q), K);
#pragma unroll
            for (int q = 0; q < 2 * FN; ++q) r.v[MI + q] = row_16<DWORDS>(wp[q], k + 16 * block_unit(2 * FN * wave + q), K);
            put(st0, r);
            __syncthreads();
            multiply_stage(st0);
        } else {
            __syncthreads();                       // the tokens' scales
        }
        for (int s = 0; s < whole; s += 2) {
            put(st1, r0);                          // its last readers are past the barrier before this one
            r0 = load(min(s + 2, last));
            __syncthreads();
            multiply_stage(st1);
            if (s + 1 >= whole) break;
            put(st0, r1);
            r1 = load(min(s + 3, last));
            __syncthreads();
            multiply_stage(st0);
        }
    }
    // tokens 4 q .. 4 q + 3 of a block are four registers of a lane: their scales are one LDS read
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int m = 32 * MI * wi + 32 * i + 8 * q + 4 * lg;
            const float4 bs4 = *reinterpret_cast<const float4*>(&bscale[m]);
            const float bs[4] = {bs4.x, bs4.y, bs4.z, bs4.w};
            const int64_t at = (m0 + m) * a.N + n0 + 32 * FN * wj + lr;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (m + e >= rows_m) break;
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    if (32 * FN * wj + 32 * j + lr < rows_n)
                        i8_store(a, at + e * a.N + 32 * j, acc[i][j][4 * q + e], bs[e], gs[j], bias[j]);
            }
        }
}

template <int ROWS, int MI, int FN>
static hipError_t launch_i8_gemm_tile(const I8Args& a, hipStream_t s) {
    const int64_t tm = (a.M + 64 * MI - 1) / (64 * MI), tn = (a.N + 128 * FN - 1) / (128 * FN);
    hipLaunchKernelGGL((k_i8_gemm<ROWS, MI, FN>), dim3((unsigned)(tm * tn)), dim3(512), 0, s, a, (int)tm, (int)tn);
    return hipGetLastError();
}

// Tiles of 64 x 256: what the choices below count.
static int64_t i8_tiles(const I8Args& a) { return (a.M + 63) / 64 * ((a.N + 255) / 256); }

// The largest tile whose workgroups still fill the card.  64 x 128 while 64 x 256 makes at most 128 tiles, so
// that twice as many still run at once: K = N = 4096, M = 256 (64 tiles) 12.2 against 16.6 us, M = 512 (128)
// 15.5 against 18.1; K = 4096, N = 11008, M = 256 (172) 30.9 against 26.9.  64 x 256 while those run at once
// (256 slots): K = N = 4096, M = 1024 (256) 23.7 against 25.8 us with 128 x 256; K = 4096, N = 11008, M = 512
// (344) 51.7 against 33.6.
// Rows off dword boundaries are read dword by dword only in 64-token tiles: with many tiles the plain loads'
// time is hidden (64 x 256, M = 501, K = 1001, N = 1536 15.8 against 20.7 us; 128 x 256, M = 2048, K = 4099,
// N = 4096 60.1 against 55.9).
template <int ROWS>
static hipError_t launch_i8_gemm(const I8Args& a, hipStream_t s) {
    const int64_t tiles = i8_tiles(a);
    if (tiles <= 128) return launch_i8_gemm_tile<ROWS, 1, 1>(a, s);
    if (tiles <= 256) return launch_i8_gemm_tile<ROWS, 1, 2>(a, s);
    return launch_i8_gemm_tile<ROWS == ROWS_1 ? ROWS_4 : ROWS, 2, 2>(a, s);
}

// The streaming kernel while 64 x 256 makes at most 32 tiles, too few to read the weights at speed (against
// 64 x 128): K = N = 4096, M = 64 (16 tiles) 8.5 against 11.9 us, M = 128 (32) 11.7 against 12.1, M = 256 (64)
// 20.0 against 12.2; K = N = 8192, M = 64 (32) 23.3 against 30.1; K = 4096, N = 11008, M = 64 (43) 22.1 against
// 17.1; K = 4096, N = 32000, M = 16 (125) 26.4 against 21.5 us.
template <int ROWS>
static hipError_t launch_i8(const I8Args& a, hipStream_t s) {
    if (a.M == 1) return launch_i8_gemv<ROWS == ROWS_16>(a, s);
    if (i8_tiles(a) <= 32) return launch_i8_dec<ROWS>(a, s);
    return launch_i8_gemm<ROWS>(a, s);
}

hipError_t launch_forward_i8(const I8Args& a, hipStream_t s) {
    const uintptr_t low = (uintptr_t)a.xq | (uintptr_t)a.wq | (uintptr_t)a.K;
    return low % 16 == 0 ? launch_i8<ROWS_16>(a, s) : low % 4 == 0 ? launch_i8<ROWS_4>(a, s) : launch_i8<ROWS_1>(a, s);
}

}  // namespace bitlinear
