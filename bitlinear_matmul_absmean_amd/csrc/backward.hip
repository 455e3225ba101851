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
// hi + 2^-12 lo, two fp16 numbers: hi is the element rounded to 11 bits, lo the exact remainder, 2^12
// times it, rounded to 11 bits, together within 2^-23 of the element down to 2^-14, 2^-28 of the row's
// largest (2^-23 is what two fp32 roundings may lose; the products that follow are exact, where fp32's
// own are rounded once more).  2^-12 goes to the integer operand, which fp16 still holds exactly: without
// the factor lo was subnormal from 2^-17 of the largest down, and columns where the largest elements
// meet zeros lost their bits.  Two f16 MFMA products into one fp32 accumulator then give the product to
// fp32 accuracy at half the f16 matrix rate, several times the rate of fp32 products.
// Smaller elements have hi = 0 and 11 bits in lo (none below 2^-26), off by 2^-26 at most; fp16's subnormal
// numbers are left alone, since the matrix cores align sums as if those were 2^-14 (measured: sums of
// products near 2^-17 came out 2^-31 off).  What small elements lack is below 2^-23 of a sum unless the sum is
// tiny itself, where all larger elements meet zeros: to such sums it is added in fp32 (step 5).
//
// Operands lie in panels, the blocks that a step of the product reads, each contiguous and in the
// order of its LDS image, so that every load is 1 KiB of whole cache lines:
//   split gradients  [rows / 128][L / 32][hi, lo][128 rows][32 l] fp16, the 16-byte unit u of row r at
//                    position u ^ split_swizzle(r);
//   integer operand  [columns / 256][L / 32][256 columns][32 l] as bytes v + 128, the 16-byte unit u
//                    of column c at position u ^ (c / 8) % 2.
//
// Steps, each one launch over the whole problem:
//   1. k_grad_prep: the largest |d alpha| of every token and |d beta / 127| of every channel, and the
//      bias sums, tile by tile; the panels of the integer operands;
//   2. k_grad_reduce (more than 64 tokens): the tiles' maxima and sums put together;
//   3. k_grad_split: d once more, scaled and split, rows being tokens (dx) and channels (dW);
//   4. k_split_gemm: both products;
//   5. k_grad_finish: the parts of a sum added, where it was cut, and to tiny sums what their small elements
//      lack.
// Up to 16 tokens one pass in fp32 takes their place (k_grad_few), beyond, where the tiles are few, one that does
// steps 1 to 4 tile by tile in LDS (k_grad_mid).
//
// 2048 tokens, K = 4096, F = 11008 (gated): 1290 us: step 1 92, 2 5, 3 130 (copies of their bytes would
// take 83, 1, 132), 5 5, the products 1.05 ms.  (Without the factor 2^-12 and step 5: 1265.)
#include <limits.h>

#include "ffn.hpp"

namespace bitlinear {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Exponent s of the power of two that scales a row whose largest element is mx to [2^14, 2^15);
// clamped so that 2^s and 2^-s are normal numbers.
__device__ __forceinline__ int scale_exponent(float mx) {
    if (mx == 0.0f) return 0;
    const int s = 15 - __builtin_amdgcn_frexp_expf(mx);
    return s > 126 ? 126 : s < -126 ? -126 : s;
}
// Eight bytes v + 128 as the fp16 numbers v.
__device__ __forceinline__ f16x8 bytes_f16(uint32_t lo, uint32_t hi) {
    const f16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
    f16x2 r[4];
    r[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u)) - bias;
    r[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u)) - bias;
    r[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u)) - bias;
    r[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u)) - bias;
    f16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = r[i / 2][i % 2];
    return o;
}
// The same 2^-12 times (exact: fp16 is normal down to 2^-14), for the products with lo.
__device__ __forceinline__ f16x8 lower_operand(f16x8 v) { return v * (_Float16)0x1p-12f; }
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// d from the incoming gradient and the saved values: one projection d[0] = dy; gated d[0] = dh u a'(g),
// d[1] = dh a(g).  ACT 0: one projection.
template <int ACT>
__device__ __forceinline__ void grad_of(float dy, float g, float u, float (&d)[2]) {
    if constexpr (ACT == 0) {
        d[0] = dy;
    } else {
        float v, slope;
        act_grad<ACT>(g, v, slope);
        d[0] = dy * u * slope;
        d[1] = dy * v;
    }
}
// d of element i = (m, n).
template <int ACT>
__device__ __forceinline__ void grad_at(const BackwardArgs& a, int64_t i, float (&d)[2]) {
    grad_of<ACT>(a.dy[i], ACT == 0 ? 0.0f : a.g[i], ACT == 0 ? 0.0f : a.u[i], d);
}

constexpr int SG_BM = 128, SG_BN = 256, SG_BK = 32, SG_SLOTS = 512;

// Where row r keeps its four 16-byte units: 16 consecutive rows then spread one unit over all 64 banks.
__device__ __forceinline__ int split_swizzle(int r) { return ((r >> 2) & 3) ^ (((r >> 1) & 1) << 1); }
// Index of element (row, l) of the hi plane of split panels with sums of length L; lo lies 4096 on.
__device__ __forceinline__ int64_t split_at(int64_t row, int64_t l, int64_t L) {
    const int r = (int)(row & 127), c = (int)(l & 31);
    return ((row >> 7) * (L >> 5) + (l >> 5)) * 8192 + r * 32 + (((c >> 3) ^ split_swizzle(r)) << 3) + (c & 7);
}
// Index of the 16-byte unit that holds element (column, l) of integer panels.
__device__ __forceinline__ int64_t code_unit(int64_t col, int64_t l, int64_t L) {
    const int c = (int)(col & 255);
    return ((col >> 8) * (L >> 5) + (l >> 5)) * 512 + c * 2 + (((l >> 4) & 1) ^ ((c >> 3) & 1));
}

struct GradPlan {
    int64_t Np, Mp, Lx;            // N and M rounded up to 64, P Np
    int tm, tn;                    // tokens and columns of a maximum tile
    int64_t mt, ct;                // maximum tiles along the tokens, along the columns
    float *rpart, *cpart;          // largest |d alpha| [M, ct], |d beta / 127| [mt, P N] of a tile
    double* bpart;                 // sums of d [mt, P N] of a tile
    float *rmax, *cmax;            // [M], [P N]
    uint16_t *xs, *wsp;            // panels of the split gradients: M rows of Lx (dx), P N rows of Mp (dW)
    uint8_t *wt, *cd;              // panels of W_hat^T, K columns of Lx, and of x_q^T, K columns of Mp
    float *part_x, *part_w;        // sums cut into parts
    int parts_x, parts_w;
    int64_t st;                    // tiles of 128 columns (step 3)
    uint8_t* small_x;              // where elements below 2^-14 are: for every four tokens, in rows of tx bytes, for
    int64_t tx;                    // each tile of 128 columns of a projection a bit for each token; and for each
    uint64_t* small_w;             // projection, parity and tile and every four tokens a bit for each of 64 columns
    int64_t nb;                    // blocks of 128 columns k, rounded up to eight
    uint8_t *need_x, *need_w;      // the whole sums that step 5 looks at: for each row of dx and dW a byte for each block
    int *smalls;                   // [M + P N] small elements of a row: of tokens, of channels
    size_t bytes;
};

static int64_t product_tiles(int64_t I, int64_t J) { return ((I + SG_BM - 1) / SG_BM) * ((J + SG_BN - 1) / SG_BN); }

// Parts to cut a sum of length L into (`tiles` tiles of outputs).  The least cost of: the rounds of
// workgroups over the slots (a last round that leaves one workgroup to a compute unit runs in 0.6 of the
// time) times a part's share of the sum, plus the exchange of the parts (a part is written and read once
// for each output, 8 bytes, and the output written once more; 4 bytes take the time of 220 terms).  But no
// more parts than bring a workgroup under the time `even` that the workgroups of both products take
// together, evenly spread: the other product's fill the slots (2048 tokens, K = 4096, F = 11008: dx in one
// part 1327 us, in two 1369).  Parts of at least 256 terms, at most 32.
static int sum_parts(int64_t tiles, int64_t L, int64_t even) {
    int best = 1;
    double cost = 1e30;
    for (int s = 1; s <= 32 && (s == 1 || L / s >= 256); ++s) {
        const int64_t left = tiles * s % SG_SLOTS;
        const double rounds = (double)(tiles * s / SG_SLOTS) + (left == 0 ? 0.0 : left <= SG_SLOTS / 2 ? 0.6 : 1.0);
        const double c = (double)L * rounds * SG_SLOTS / (double)(tiles * s) + (s > 1 ? 220.0 * (2 * s + 1) : 0.0);
        if (c < cost) {
            cost = c;
            best = s;
        }
        if (L / s <= even) break;
    }
    return best;
}

static GradPlan grad_plan(int64_t M, int64_t K, int64_t N, bool gated, void* ws) {
    GradPlan p{};
    const int64_t P = gated ? 2 : 1;
    p.Np = (N + 63) / 64 * 64;
    p.Mp = (M + 63) / 64 * 64;
    p.Lx = P * p.Np;
    // up to 64 tokens one tile holds all of a column's, and nothing is left to put together but rows
    p.tn = M <= 64 ? 64 : 256;
    p.ct = (N + p.tn - 1) / p.tn;
    p.tm = M <= 64 || (M + 63) / 64 * p.ct >= 512 ? 64 : 16;
    p.mt = (M + p.tm - 1) / p.tm;
    const int64_t tx = product_tiles(M, K), tw = product_tiles(P * N, K), even = (tx * p.Lx + tw * p.Mp) / SG_SLOTS;
    p.parts_x = sum_parts(tx, p.Lx, even);
    p.parts_w = sum_parts(tw, p.Mp, even);
    uint8_t* base = static_cast<uint8_t*>(ws);
    size_t off = 0;
    auto take = [&](int64_t count, size_t size) {
        uint8_t* q = base ? base + off : nullptr;
        off += ((size_t)count * size + 255) / 256 * 256;
        return q;
    };
    p.rpart = reinterpret_cast<float*>(take(M * p.ct, 4));
    p.cpart = reinterpret_cast<float*>(take(p.mt * P * N, 4));
    p.bpart = reinterpret_cast<double*>(take(p.mt * P * N, 8));
    p.rmax = reinterpret_cast<float*>(take(M, 4));
    p.cmax = reinterpret_cast<float*>(take(P * N, 4));
    const int64_t K256 = (K + 255) / 256 * 256;
    p.xs = reinterpret_cast<uint16_t*>(take((M + 127) / 128 * 128 * p.Lx, 4));
    p.wsp = reinterpret_cast<uint16_t*>(take((P * N + 127) / 128 * 128 * p.Mp, 4));
    p.wt = take(K256 * p.Lx, 1);
    p.cd = take(K256 * p.Mp, 1);
    p.part_x = reinterpret_cast<float*>(take(p.parts_x > 1 ? p.parts_x * M * K : 0, 4));
    p.part_w = reinterpret_cast<float*>(take(p.parts_w > 1 ? p.parts_w * P * N * K : 0, 4));
    p.st = (N + 127) / 128;
    p.tx = (P * p.st + 3) / 4 * 4;
    p.small_x = take(p.Mp / 4 * p.tx, 1);
    p.small_w = reinterpret_cast<uint64_t*>(take(P * 2 * p.st * (p.Mp / 4), 8));
    p.nb = (K + 1023) / 1024 * 8;
    p.need_x = take(M * p.nb, 1);
    p.need_w = take(P * N * p.nb, 1);
    p.smalls = reinterpret_cast<int*>(take(M + P * N, 4));
    p.bytes = off;
    return p;
}


// ---- step 1 -------------------------------------------------------------------------------
// Maxima and sums.  A workgroup takes p.tm tokens x 64 C columns, a wave a quarter of the tokens, a
// lane C columns 64 apart (whole lines whatever the alignment).
template <int ACT, int C>
__device__ __forceinline__ void max_tile(const BackwardArgs& a, const GradPlan& p, int64_t b, uint8_t* lds) {
    constexpr int P = ACT == 0 ? 1 : 2;
    double (*cs)[P][256] = reinterpret_cast<double (*)[P][256]>(lds);
    float (*cm)[P][256] = reinterpret_cast<float (*)[P][256]>(lds + 4 * P * 256 * 8);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t tn = b % p.ct, tmi = b / p.ct, n0 = tn * 64 * C, m0 = tmi * p.tm;
    const float al[2] = {a.al0[0], ACT == 0 ? 0.0f : a.al1[0]};
    const bool bias = a.db0 || a.db1;
    float cmx[P][C];
    double sum[P][C];
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            cmx[q][c] = 0.0f;
            sum[q][c] = 0.0;
        }
    // TT tokens at a time, their loads under way together: rows and columns past the end read the last
    // ones and count for nothing
    constexpr int TT = C == 1 ? 16 : 4;
    const int per = p.tm / 4;
    for (int t0 = 0; t0 < per; t0 += TT) {
        const int64_t mb = m0 + per * wave + t0;
        if (mb >= a.M) break;
        float d[TT][C][2], bs[TT], rm[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int64_t m = mb + t < a.M ? mb + t : a.M - 1;
            bs[t] = a.beta[m] / 127.0f;
            rm[t] = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t n = n0 + 64 * c + lane;
                grad_at<ACT>(a, m * a.N + (n < a.N ? n : a.N - 1), d[t][c]);
            }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (mb + t < a.M && n0 + 64 * c + lane < a.N) {
#pragma unroll
                    for (int q = 0; q < P; ++q) {
                        rm[t] = fmaxf(rm[t], fabsf(d[t][c][q] * al[q]));
                        cmx[q][c] = fmaxf(cmx[q][c], fabsf(d[t][c][q] * bs[t]));
                        if (bias) sum[q][c] += (double)d[t][c][q];
                    }
                }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float v = wave_max_pos(rm[t]);
            if (lane == 0 && mb + t < a.M) p.rpart[(mb + t) * p.ct + tn] = v;
        }
    }
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            cm[wave][q][64 * c + lane] = cmx[q][c];
            if (bias) cs[wave][q][64 * c + lane] = sum[q][c];
        }
    __syncthreads();
    const int64_t n = n0 + threadIdx.x;
    if (threadIdx.x >= 64 * C || n >= a.N) return;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        float v = 0.0f;
        double s = 0.0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            v = fmaxf(v, cm[w][q][threadIdx.x]);
            if (bias) s += cs[w][q][threadIdx.x];
        }
        if (p.mt == 1) {
            p.cmax[q * a.N + n] = v;
            float* out = q ? a.db1 : a.db0;
            if (out) out[n] = (float)s;
        } else {
            p.cpart[(tmi * P + q) * a.N + n] = v;
            if (bias) p.bpart[(tmi * P + q) * a.N + n] = s;
        }
    }
}

// Four bytes at p + i of a row of `row` bytes, zeros past its end; no alignment is assumed.
__device__ __forceinline__ uint32_t row_dword(const uint8_t* __restrict__ p, int64_t i, int64_t row) {
    uint32_t v = 0;
    if (i + 4 <= row) {
        __builtin_memcpy(&v, p + i, 4);
    } else {
        for (int j = 0; j < 4; ++j)
            if (i + j < row) v |= (uint32_t)p[i + j] << (8 * j);
    }
    return v;
}

// A 64 x 64 byte tile, transposed through LDS.  Thread t holds dword t % 16 (four columns) of rows
// 4 (t / 16) .. 4 (t / 16) + 3, turns the 4 x 4 bytes round in registers and writes four columns' dwords
// (a column is 17 dwords, so that the lanes of a write and of a read spread over the banks); it gets back
// sixteen rows of one column, rows 16 (t % 4) .. of column t / 4.
__device__ __forceinline__ void turn_put(uint32_t* lds, u32x4 rows, int t) {
    const u32x4 cols = transpose4x4_perm(rows);
    const int c = 4 * (t & 15), r4 = t >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) lds[(c + j) * 17 + r4] = cols[j];
}
__device__ __forceinline__ u32x4 turn_get(const uint32_t* lds, int t) {
    const uint32_t* p = lds + (t >> 2) * 17 + 4 * (t & 3);
    return u32x4{p[0], p[1], p[2], p[3]};
}
__device__ __forceinline__ u32x4 turn_tile(uint32_t* lds, u32x4 rows) {
    turn_put(lds, rows, threadIdx.x);
    __syncthreads();
    return turn_get(lds, threadIdx.x);
}
// The thread's dwords of such a tile: bytes at .. at + 3 of rows r0 .. r0 + 3 of a matrix with rows of `row`
// bytes; zeros past a row's end, `fill` for rows past the last (whole: the tile has neither).
__device__ __forceinline__ u32x4 tile_rows(const uint8_t* __restrict__ p, int64_t r0, int64_t rows, int64_t at, int64_t row,
                                           uint32_t fill, bool whole) {
    u32x4 d;
    if (whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v;
            __builtin_memcpy(&v, p + (r0 + i) * row + at, 4);
            d[i] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = r0 + i < rows ? row_dword(p + (r0 + i) * row, at, row) : fill;
    }
    return d;
}
// Sixteen bytes of codes 0, 1, 2 (four to a byte) to the weights of code i as bytes 127, 128, 129.
__device__ __forceinline__ u32x4 code_bytes(u32x4 v, int i) { return ((v >> (uint32_t)(2 * i)) & 0x03030303u) + 0x7F7F7F7Fu; }

// Panels of W_hat^T, 64 weight rows x 256 columns k per workgroup: a lane expands the codes 0, 1, 2 of
// sixteen rows at four columns to the bytes 127, 128, 129.
__device__ __forceinline__ void weights_tile(const BackwardArgs& a, const GradPlan& p, int64_t b, int64_t kt, uint32_t* lds) {
    const int64_t k0 = b % kt * 256, l0 = b / kt * 64;
    const int q = l0 >= p.Np;
    const int64_t n0 = l0 - q * p.Np, rowb = a.K >> 2;
    const uint8_t* w = q ? a.w1 : a.w0;
    const int64_t r0 = n0 + 4 * (threadIdx.x >> 4), at = (k0 >> 2) + 4 * (threadIdx.x & 15);
    const u32x4 v = turn_tile(lds, tile_rows(w, r0, a.N, at, rowb, 0x55555555u, n0 + 64 <= a.N && (k0 >> 2) + 64 <= rowb));
    const int u = threadIdx.x & 3, c = threadIdx.x >> 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        reinterpret_cast<u32x4*>(p.wt)[code_unit(k0 + 4 * c + i, l0 + 16 * u, p.Lx)] = code_bytes(v, i);
    }
}

// Panels of x_q^T, 64 tokens x 64 columns per workgroup.
__device__ __forceinline__ void codes_tile(const BackwardArgs& a, const GradPlan& p, int64_t b, int64_t kt, uint32_t* lds) {
    const int64_t k0 = b % kt * 64, m0 = b / kt * 64;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(a.xq);
    const int64_t r0 = m0 + 4 * (threadIdx.x >> 4), at = k0 + 4 * (threadIdx.x & 15);
    const u32x4 v = turn_tile(lds, tile_rows(x, r0, a.M, at, a.K, 0u, m0 + 64 <= a.M && k0 + 64 <= a.K));
    const int u = threadIdx.x & 3, c = threadIdx.x >> 2;
    reinterpret_cast<u32x4*>(p.cd)[code_unit(k0 + c, m0 + 16 * u, p.Mp)] = v ^ 0x80808080u;
}

template <int ACT, int C>
__global__ __launch_bounds__(256) void k_grad_prep(BackwardArgs a, GradPlan p, int64_t maxima, int64_t weights, int64_t ktw,
                                                   int64_t ktc) {
    constexpr int P = ACT == 0 ? 1 : 2;
    __shared__ __align__(16) uint8_t lds[4 * P * 256 * 12];
    const int64_t b = blockIdx.x;
    for (int64_t i = b * 256 + threadIdx.x; i < a.M + P * a.N; i += (int64_t)gridDim.x * 256) p.smalls[i] = 0;
    if (b < maxima) max_tile<ACT, C>(a, p, b, lds);
    else if (b < maxima + weights) weights_tile(a, p, b - maxima, ktw, reinterpret_cast<uint32_t*>(lds));
    else codes_tile(a, p, b - maxima - weights, ktc, reinterpret_cast<uint32_t*>(lds));
}

// ---- step 2 (more than one tile of tokens): columns (a thread each), then rows (a wave each) ----
__global__ __launch_bounds__(256) void k_grad_reduce(BackwardArgs a, GradPlan p, int P, int64_t cblocks) {
    const int64_t NT = P * a.N;
    if (blockIdx.x < cblocks) {
        const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (n >= NT) return;
        float v = 0.0f;
#pragma unroll 8
        for (int64_t t = 0; t < p.mt; ++t) v = fmaxf(v, p.cpart[t * NT + n]);
        p.cmax[n] = v;
        float* out = n < a.N ? a.db0 : a.db1;
        if (!out) return;
        double s = 0.0;
#pragma unroll 8
        for (int64_t t = 0; t < p.mt; ++t) s += p.bpart[t * NT + n];
        out[n < a.N ? n : n - a.N] = (float)s;
    } else {
        const int64_t m = ((int64_t)blockIdx.x - cblocks) * 4 + (threadIdx.x >> 6);
        if (m >= a.M) return;
        const int lane = threadIdx.x & 63;
        float v = 0.0f;
        for (int64_t t = lane; t < p.ct; t += 64) v = fmaxf(v, p.rpart[m * p.ct + t]);
        v = wave_max_pos(v);
        if (lane == 0) p.rmax[m] = v;
    }
}

// ---- step 3 -------------------------------------------------------------------------------
__device__ __forceinline__ bool is_small(float v) { return fabsf(v) < 0x1p-14f && v != 0.0f; }
// Whether there is a small element among several: twice the bits of a number less one order them by size, zeros
// last (two instructions where a comparison each would take four).
__device__ __forceinline__ uint32_t size_bits(float v) { return 2 * __float_as_uint(v) - 1; }
constexpr uint32_t SMALL_BITS = 2u * (127 - 14) << 23;
__device__ __forceinline__ uint32_t split_f16(float v) {
    const _Float16 hi = fabsf(v) < 0x1p-14f ? (_Float16)0.0f : (_Float16)v;
    const _Float16 lo = fabsf(v) < 0x1p-26f ? (_Float16)0.0f : (_Float16)((v - (float)hi) * 0x1p12f);
    return (uint32_t)__builtin_bit_cast(uint16_t, hi) | (uint32_t)__builtin_bit_cast(uint16_t, lo) << 16;
}
// What a small element lacks when split (exact).
__device__ __forceinline__ float split_rest(float v) {
    return fabsf(v) < 0x1p-26f ? v : v - (float)(_Float16)(v * 0x1p12f) * 0x1p-12f;
}
// Sums below this many times the number of small elements are looked at in step 5: 2^23 times what one may lack,
// times the largest of the integer operand.
constexpr float NEED_X = 0x1p-3f, NEED_W = 0x1p-3f * 128.0f;

// Scaled and split gradients, 32 tokens x 128 columns per workgroup of eight waves; a wave takes four
// tokens, their loads under way together, a lane two neighbouring columns.  Rows of tokens are
// written as they come, rows of channels through LDS.  Padded columns and tokens are written as zeros.
template <int ACT>
__global__ __launch_bounds__(512) void k_grad_split(BackwardArgs a, GradPlan p, int ctiles) {
    constexpr int P = ACT == 0 ? 1 : 2;
    __shared__ uint32_t tile[P][128][33];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)(blockIdx.x % ctiles) * 128, m0 = (int64_t)(blockIdx.x / ctiles) * 32;
    const int64_t n = n0 + 2 * lane;
    const float al[2] = {a.al0[0], ACT == 0 ? 0.0f : a.al1[0]};
    float cscale[P][2];
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int c = 0; c < 2; ++c) cscale[q][c] = n + c < a.N ? pow2f(scale_exponent(p.cmax[q * a.N + n + c])) : 0.0f;
    // with one tile of tokens the rows' maxima are put together here, and kept for the product's scales
    // (lane l: token l / 16 of the wave, every sixteenth tile)
    float rmax[4];
    if (p.mt > 1) {
#pragma unroll
        for (int t = 0; t < 4; ++t) rmax[t] = m0 + 4 * wave + t < a.M ? p.rmax[m0 + 4 * wave + t] : 0.0f;
    } else {
        const int64_t m = m0 + 4 * wave + (lane >> 4);
        const float* part = p.rpart + (m < a.M ? m : a.M - 1) * p.ct;
        float v = 0.0f;
#pragma unroll 8
        for (int64_t t = lane & 15; t < p.ct; t += 16) v = fmaxf(v, part[t]);
        v = fmaxf(v, __shfl_xor(v, 1, 64));
        v = fmaxf(v, __shfl_xor(v, 2, 64));
        v = fmaxf(v, __shfl_xor(v, 4, 64));
        v = fmaxf(v, __shfl_xor(v, 8, 64));
        if (m < a.M && n0 == 0 && (lane & 15) == 0) p.rmax[m] = v;
#pragma unroll
        for (int t = 0; t < 4; ++t) rmax[t] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16 * t));
    }
    // tokens and columns past the end read the last ones and count as zeros
    float d[4][2][2], bs[4], rscale[4];                // d[token][column][projection]
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t m = m0 + 4 * wave + t, ml = m < a.M ? m : a.M - 1;
        bs[t] = a.beta[ml] / 127.0f;
        rscale[t] = pow2f(scale_exponent(rmax[t]));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            grad_at<ACT>(a, ml * a.N + (n + c < a.N ? n + c : a.N - 1), d[t][c]);
            if (m >= a.M || n + c >= a.N) d[t][c][0] = d[t][c][1] = 0.0f;
        }
    }
    uint32_t least = ~0u;                              // the smallest element
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t m = m0 + 4 * wave + t;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            if (a.dx && m < a.M && n < p.Np) {
                const float f0 = d[t][0][q] * al[q] * rscale[t], f1 = d[t][1][q] * al[q] * rscale[t];
                const uint32_t v0 = split_f16(f0), v1 = split_f16(f1);
                uint32_t* o = reinterpret_cast<uint32_t*>(p.xs + split_at(m, q * p.Np + n, p.Lx));
                o[0] = __builtin_amdgcn_perm(v1, v0, 0x05040100u);
                o[2048] = __builtin_amdgcn_perm(v1, v0, 0x07060302u);
                least = min(least, min(size_bits(f0), size_bits(f1)));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float f = d[t][c][q] * bs[t] * cscale[q][c];
                tile[q][2 * lane + c][4 * wave + t] = split_f16(f);
                least = min(least, size_bits(f));
            }
        }
    }
    uint32_t small_x[P] = {};                          // a bit for each of the wave's tokens with small elements
    uint64_t small_w[P][2] = {};                       // and for each of its columns
    if (__ballot(least < SMALL_BITS - 1)) {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            int of_column[2] = {0, 0};
            for (int t = 0; t < 4; ++t) {
                const int of_token = is_small(d[t][0][q] * al[q] * rscale[t]) + is_small(d[t][1][q] * al[q] * rscale[t]);
                small_x[q] |= __ballot(of_token) ? 1u << t : 0u;
                if (a.dx && of_token) atomicAdd(p.smalls + m0 + 4 * wave + t, of_token);
#pragma unroll
                for (int c = 0; c < 2; ++c) of_column[c] += is_small(d[t][c][q] * bs[t] * cscale[q][c]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                small_w[q][c] = __ballot(of_column[c]);
                if (a.dw0 && of_column[c]) atomicAdd(p.smalls + a.M + q * a.N + n + c, of_column[c]);
            }
        }
    }
    if (a.dx) {
#pragma unroll
        for (int q = 0; q < P; ++q)
            if (lane == 0) p.small_x[(m0 / 4 + wave) * p.tx + q * p.st + n0 / 128] = (uint8_t)small_x[q];
    }
    if (!a.dw0) return;
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (lane == 0) p.small_w[((2 * q + c) * p.st + n0 / 128) * (p.Mp / 4) + m0 / 4 + wave] = small_w[q][c];
    __syncthreads();
    const int u = threadIdx.x & 3, r = threadIdx.x >> 2;
    if (n0 + r >= a.N) return;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = tile[q][r][8 * u + j];
        u32x4 h, l;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[j] = __builtin_amdgcn_perm(v[2 * j + 1], v[2 * j], 0x05040100u);
            l[j] = __builtin_amdgcn_perm(v[2 * j + 1], v[2 * j], 0x07060302u);
        }
        u32x4* o = reinterpret_cast<u32x4*>(p.wsp + split_at(q * a.N + n0 + r, m0 + 8 * u, p.Mp));
        o[0] = h;
        o[512] = l;
    }
}

// ---- step 4 -------------------------------------------------------------------------------
struct SplitArgs {
    const uint16_t* a;             // panels of I rows of split gradients
    const uint8_t* b;              // panels of J columns of the integer operand
    const float* amax;             // [I] the rows' largest elements
    int64_t I, J, L;               // L a multiple of 64
    float *c0, *c1;                // rows below I0 go to c0 [I0, J], the others to c1
    int64_t I0;
    float* part;                   // parts > 1: [parts][I][J] unscaled sums
    int parts, tiles_i, tiles_j;
    uint8_t* need;                 // [I][nb]
    int64_t nb;
    const int* smalls;             // [I]
    float below;                   // sums below it times a row's small elements are marked
};

// C[i, j] = 2^-s_i sum_l (hi[i, l] + 2^-12 lo[i, l]) b[j, l].  A workgroup of four waves computes 128 x 256
// outputs, a wave 64 x 128 of them in 32 x 32 blocks (128 accumulator registers), in steps of 32 l.
// Three LDS stages (24 KiB each: a panel block of each operand) are filled two steps ahead by loads
// that go past the registers; two workgroups share a compute unit.  Bytes v + 128 become fp16 as
// 1024 + (v + 128), the byte under the exponent 0x64, minus 1152: two instructions for two values.
// Bound: power.  The 739 GFLOP of gradients at 2048 tokens, K = 4096, F = 11008 (1.48 TFLOP in fp16) take 1.04
// ms, 1.42 PFLOP/s of fp16 (a library's plain fp16 product of 8192^3: 1.48); the matrix cores are busy 75% of
// the cycles and the clock is down between 1.6 and 1.8 GHz.  (Of it 1 to 2% for the integers times 2^-12 and the
// look at rows with small elements.)  Before the panels and the byte operand
// (64-byte pieces of rows, fp16 on both sides, 32 KiB a step): 1.16 ms; the order of the MFMAs, 256 x 256
// tiles, a third stage there and operands read ahead across the barrier all measured level.
// In the first MFMA of a step lane group g (lanes 32 g ..) holds l 16 g .. 16 g + 7, in the second
// 16 g + 8 .. 16 g + 15, so that one read of 16 bytes brings both of the lane's integer operands.
__global__ __launch_bounds__(256, 2) void k_split_gemm(SplitArgs x, SplitArgs w) {
    // the workgroups of the first product, then those of the second
    const int TX = x.parts * x.tiles_i * x.tiles_j;
    const bool first = blockIdx.x < TX;
    const SplitArgs& a = first ? x : w;
    const int blk = first ? blockIdx.x : blockIdx.x - TX;
    constexpr int OL = 512, OB = 1024, UNITS = 1536;           // units: lo, b, a stage
    __shared__ i32x4 st0[UNITS];
    __shared__ i32x4 st1[UNITS];
    __shared__ i32x4 st2[UNITS];
    __shared__ __align__(16) float scale[SG_BM];               // 2^-s of the rows (1 for parts of a sum)
    __shared__ __align__(16) float limit[SG_BM];               // below it a sum of the row is marked
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // consecutive workgroups go to the eight XCDs in turn: give each XCD a contiguous run of tiles,
    // four rows of tiles at a time, so that its L2 holds the panels its workgroups share
    const int T = a.parts * a.tiles_i * a.tiles_j;
    const int xcd = blk & 7, per = T >> 3, rem = T & 7;
    int t = xcd * per + (xcd < rem ? xcd : rem) + (blk >> 3);
    const int part = t / (a.tiles_i * a.tiles_j);
    t -= part * a.tiles_i * a.tiles_j;
    const int grp = t / (4 * a.tiles_j), gi = a.tiles_i - 4 * grp < 4 ? a.tiles_i - 4 * grp : 4;
    t -= grp * 4 * a.tiles_j;
    const int ti = 4 * grp + t % gi, tj = t / gi;
    const int64_t i0 = (int64_t)ti * SG_BM, j0 = (int64_t)tj * SG_BN;
    const int KS = (int)(a.L / SG_BK);
    const int ks0 = (int)((int64_t)KS * part / a.parts), ks1 = (int)((int64_t)KS * (part + 1) / a.parts);

    const __amdgpu_buffer_rsrc_t ra = raw_buffer(a.a + (int64_t)ti * KS * 8192, (uint32_t)KS * 16384u);
    const __amdgpu_buffer_rsrc_t rb = raw_buffer(a.b + (int64_t)tj * KS * 8192, (uint32_t)KS * 8192u);
    const uint32_t voff = 16u * lane;
    const int last = ks1 - 1;
    auto fetch = [&](i32x4* st, int ks) {
        const uint32_t s = (uint32_t)(ks < last ? ks : last);
#pragma unroll
        for (int q = 0; q < 4; ++q) load_lds16(ra, voff, s * 16384u + 1024u * (4 * wave + q), st + 64 * (4 * wave + q));
#pragma unroll
        for (int q = 0; q < 2; ++q) load_lds16(rb, voff, s * 8192u + 1024u * (2 * wave + q), st + OB + 64 * (2 * wave + q));
        __builtin_amdgcn_sched_barrier(0);         // issued here, not where their data is needed
    };

    f32x16 acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
    const int wi = wave & 1, wj = wave >> 1, lr = lane & 31, lg = lane >> 5;
    const int sw = split_swizzle(lr), sb = lg ^ ((lr >> 3) & 1);
    auto multiply = [&](const i32x4* st) {
        i32x4 cb[4];
        f16x8 fh[2][2], fl[2][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) cb[j] = st[OB + (128 * wj + 32 * j + lr) * 2 + sb];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = (64 * wi + 32 * i + lr) * 4 + ((2 * lg + kk) ^ sw);
                fh[kk][i] = __builtin_bit_cast(f16x8, st[at]);
                fl[kk][i] = __builtin_bit_cast(f16x8, st[OL + at]);
            }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f16x8 fb = bytes_f16((uint32_t)cb[j][2 * kk], (uint32_t)cb[j][2 * kk + 1]), fd = lower_operand(fb);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fh[kk][i], fb, acc[i][j], 0, 0, 0);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fl[kk][i], fd, acc[i][j], 0, 0, 0);
                }
            }
    };
    // the loads of the stage to be read have landed, for every wave, and every read of the stage to
    // be filled is over; loads past the last step repeat it and are not read
    auto turn = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0070 | 6);    // vmcnt(6: the next stage's loads) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    int ks = ks0;
    fetch(st0, ks);
    fetch(st1, ks + 1);
    if (tid < SG_BM) limit[tid] = i0 + tid < a.I ? a.below * (float)a.smalls[i0 + tid] : 0.0f;
    if (tid < SG_BM) scale[tid] = a.parts > 1 ? 1.0f : pow2f(-scale_exponent(a.amax[i0 + tid < a.I ? i0 + tid : a.I - 1]));
    for (; ks + 3 <= ks1; ks += 3) {
        turn();
        fetch(st2, ks + 2);
        multiply(st0);
        turn();
        fetch(st0, ks + 3);
        multiply(st1);
        turn();
        fetch(st1, ks + 4);
        multiply(st2);
    }
    if (ks < ks1) {
        turn();
        multiply(st0);
    }
    if (ks + 1 < ks1) {
        __builtin_amdgcn_s_waitcnt(0x0070);
        __builtin_amdgcn_s_barrier();
        multiply(st1);
    }
    __builtin_amdgcn_s_waitcnt(0x0070);            // nothing is in flight into the stages any more

    // accumulator r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4 of the block, column l % 32
    const int64_t left = a.J - (j0 + 128 * wj + lr);           // columns from this lane's first to the end
    if (a.parts == 1) {                                        // rows with tiny sums, a lane each
        uint64_t tiny = 0;
        if (__ballot(limit[64 * wi + lane] > 0.0f)) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 l4 = *reinterpret_cast<const float4*>(&limit[64 * wi + 32 * i + 8 * q + 4 * lg]);
                    const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float least = INFINITY;
#pragma unroll
                        for (int j = 0; j < 4; ++j) least = fminf(least, 32 * j < left ? fabsf(acc[i][j][4 * q + e]) : INFINITY);
                        const uint64_t lanes = __ballot(least < l[e]);
                        const int row = 32 * i + 8 * q + e;
                        tiny |= (uint64_t)((uint32_t)lanes != 0) << row | (uint64_t)((lanes >> 32) != 0) << (row + 4);
                    }
                }
        }
        const int64_t row = i0 + 64 * wi + lane;
        if (row < a.I) a.need[row * a.nb + 2 * tj + wj] = (uint8_t)(tiny >> lane & 1u);
    }
    const int rows = (int)(a.I - i0 < SG_BM ? a.I - i0 : SG_BM);
    const int split = (int)(a.I0 - i0 < 0 ? 0 : a.I0 - i0 < SG_BM ? a.I0 - i0 : SG_BM);   // rows of c0 in the tile
    float* top = (a.parts > 1 ? a.part + (int64_t)part * a.I * a.J : a.c0) + i0 * a.J + j0 + 128 * wj + lr;
    float* bottom = a.parts > 1 || !a.c1 ? top : a.c1 + (i0 - a.I0) * a.J + j0 + 128 * wj + lr;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = 64 * wi + 32 * i + 8 * q + 4 * lg;
            const float4 inv4 = *reinterpret_cast<const float4*>(&scale[r]);
            const float inv[4] = {inv4.x, inv4.y, inv4.z, inv4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (r + e >= rows) break;
                float* out = (r + e < split ? top : bottom) + (int64_t)(r + e) * a.J;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (32 * j < left) out[32 * j] = acc[i][j][4 * q + e] * inv[e];
            }
        }
}

// ---- step 5: parts of sums, and what small elements lack in tiny sums --------------------------
// Where a sum was cut, a wave adds the parts of 128 columns of a row in their order, two a lane, and scales them
// back.  Where it was not, a workgroup looks at the marks of 64 pieces of rows, of 1024 columns each; that no sum
// is marked is the rule.  To tiny sums, a wave adds what small elements lack: it forms the elements of the
// tiles of the row that hold small ones again, a lane one or two, and adds to its columns, in fp32 and in the
// order of l, the rest of each small one times its integer.  Bound: a launch and a round of loads (5 us
// beside 1.27 ms) or the parts' bytes; where most sums are tiny and most elements small, a vector product's
// time.

// A lane's C codes of a row from column k on (sixteen, or two at an even k), zeros past its end, and
// s += e times what they stand for.
template <int C>
__device__ __forceinline__ uint32_t codes_at(const uint8_t* __restrict__ w, int64_t k, int64_t K) {
    if constexpr (C == 16) return row_dword(w, k >> 2, K >> 2);
    return k < K ? (uint32_t)w[k >> 2] >> (2 * (k & 3)) : 0u;
}
template <int C>
__device__ __forceinline__ u32x4 codes_at(const int8_t* __restrict__ x, int64_t k, int64_t K) {
    if constexpr (C == 16) return row_16(reinterpret_cast<const uint8_t*>(x), k, K);
    uint16_t v = 0;
    if (k < K) __builtin_memcpy(&v, x + k, 2);
    return u32x4{v, 0u, 0u, 0u};
}
template <int C>
__device__ __forceinline__ void add_codes(float (&s)[C], float e, uint32_t codes) {
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = __builtin_fmaf(e, (float)(int)(codes >> (2 * c) & 3u) - 1.0f, s[c]);
}
template <int C>
__device__ __forceinline__ void add_codes(float (&s)[C], float e, u32x4 codes) {
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = __builtin_fmaf(e, (float)(int8_t)(codes[c / 4] >> (8 * (c % 4))), s[c]);
}
// s += the products of the elements e of the lanes in `bits` with the rows of codes b0 + lane `step`.
template <int C, typename Codes>
__device__ __forceinline__ void add_rests(float (&s)[C], uint64_t bits, float e, const Codes* b0, int64_t step, int64_t k, int64_t K) {
    for (; bits; bits &= bits - 1) {
        const int l = __builtin_ctzll(bits);
        add_codes<C>(s, __int_as_float(__builtin_amdgcn_readlane(__float_as_int(e), l)), codes_at<C>(b0 + l * step, k, K));
    }
}

// Token m of dx: C columns a lane from k on.
template <int ACT, int C>
__device__ __forceinline__ void tail_token(const BackwardArgs& a, const GradPlan& p, int64_t m, int64_t k, float (&sum)[C]) {
    constexpr int P = ACT == 0 ? 1 : 2;
    const int lane = threadIdx.x & 63;
    const int64_t tiles = P * p.st, rowb = a.K >> 2;
    const uint32_t* marks = reinterpret_cast<const uint32_t*>(p.small_x + m / 4 * p.tx);
    const int s = scale_exponent(p.rmax[m]);
    for (int64_t t0 = 0; t0 < tiles; t0 += 256) {                  // four tiles a lane
        uint32_t mine = t0 + 4 * lane < tiles ? marks[t0 / 4 + lane] >> (m & 3) & 0x01010101u : 0u;
        const int64_t behind = t0 + 4 * lane + 4 - tiles;          // bytes past the last tile hold anything
        if (behind > 0 && behind < 4) mine &= 0xFFFFFFFFu >> (8 * behind);
        for (uint64_t lanes = __ballot(mine != 0); lanes; lanes &= lanes - 1) {
            const int from = __builtin_ctzll(lanes);
            for (uint32_t bytes = __builtin_amdgcn_readlane(mine, from); bytes; bytes &= bytes - 1) {
                const int64_t t = t0 + 4 * from + __builtin_ctz(bytes) / 8;
                const int q = t >= p.st;
                const float al = q ? a.al1[0] : a.al0[0];
                for (int h = 0; h < 2; ++h) {
                    const int64_t n0 = (t - q * p.st) * 128 + 64 * h, n = n0 + lane;
                    float d[2];
                    grad_at<ACT>(a, m * a.N + (n < a.N ? n : a.N - 1), d);
                    const float v = n < a.N ? (q ? d[1] : d[0]) * al * pow2f(s) : 0.0f;
                    add_rests<C>(sum, __ballot(is_small(v)), split_rest(v) * pow2f(-s), (q ? a.w1 : a.w0) + n0 * rowb, rowb, k, a.K);
                }
            }
        }
    }
}

// Channel n of projection q of dW.
template <int ACT, int C>
__device__ __forceinline__ void tail_channel(const BackwardArgs& a, const GradPlan& p, int q, int64_t n, int64_t k, float (&sum)[C]) {
    const int lane = threadIdx.x & 63;
    const int64_t fours = p.Mp / 4;
    const uint64_t* marks = p.small_w + ((2 * q + (n & 1)) * p.st + n / 128) * fours;
    const int s = scale_exponent(p.cmax[q * a.N + n]);
    for (int64_t t0 = 0; t0 < fours; t0 += 64) {                   // four tokens a lane
        uint64_t lanes = __ballot(t0 + lane < fours && (marks[t0 + lane] >> ((n & 127) / 2) & 1u));
        while (lanes) {                                            // 64 tokens from the first marked ones on
            const int from = __builtin_ctzll(lanes);
            lanes &= from < 48 ? ~0ull << (from + 16) : 0;
            const int64_t m0 = 4 * (t0 + from), m = m0 + lane, ml = m < a.M ? m : a.M - 1;
            float d[2];
            grad_at<ACT>(a, ml * a.N + n, d);
            const bool next = from > 48 && lane >= 4 * (64 - from);   // tokens of the next round
            const float v = m < a.M && !next ? (q ? d[1] : d[0]) * (a.beta[ml] / 127.0f) * pow2f(s) : 0.0f;
            add_rests<C>(sum, __ballot(is_small(v)), split_rest(v) * pow2f(-s), a.xq + m0 * a.K, a.K, k, a.K);
        }
    }
}

// Workgroups: first the sums in parts (xwaves waves for dx, then those for dW), then the pieces of the others
// (xpieces of dx, then those of dW).
template <int ACT>
__global__ __launch_bounds__(256) void k_grad_finish(BackwardArgs a, GradPlan p, SplitArgs x, SplitArgs w, int64_t xwaves, int64_t waves,
                                                     int64_t xpieces, int64_t pieces) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t sums = (waves + 3) / 4, blocks = (a.K + 127) / 128;
    if (blockIdx.x < sums) {
        int64_t id = (int64_t)blockIdx.x * 4 + wave;
        if (id >= waves) return;
        const bool first = id < xwaves;
        const SplitArgs& sa = first ? x : w;
        id -= first ? 0 : xwaves;
        const int64_t row = id / blocks, k = id % blocks * 128 + 2 * lane, n = sa.I * sa.J;
        const bool inside = k < a.K;
        const float* part = sa.part + row * a.K + (inside ? k : 0);
        float s[2] = {0.0f, 0.0f};
#pragma unroll 8
        for (int q = 0; q < sa.parts; ++q) {
            const float2 v = *reinterpret_cast<const float2*>(part + q * n);
            s[0] += v.x, s[1] += v.y;
        }
        const uint64_t tiny = __ballot(inside && fminf(fabsf(s[0]), fabsf(s[1])) < sa.below * (float)sa.smalls[row]);
        const float scale = pow2f(-scale_exponent(sa.amax[row]));
        s[0] *= scale, s[1] *= scale;
        const int q = !first && row >= a.N;
        if (tiny) {
            if (first) tail_token<ACT, 2>(a, p, row, k, s);
            else tail_channel<ACT, 2>(a, p, q, row - q * a.N, k, s);
        }
        if (inside) __builtin_memcpy((first ? a.dx : q ? a.dw1 : a.dw0) + (row - q * a.N) * a.K + k, s, 8);
        return;
    }
    const int64_t group = (int64_t)blockIdx.x - sums, pass = p.nb / 8, mine = group * 64 + lane;
    uint64_t marks = 0;                                            // the piece's eight blocks, those below K
    if (mine < pieces) {
        marks = *reinterpret_cast<const uint64_t*>(mine < xpieces ? p.need_x + 8 * mine : p.need_w + 8 * (mine - xpieces));
        const int64_t left = blocks - mine % pass * 8;
        if (left < 8) marks &= ~0ull >> (64 - 8 * left);
    }
    uint64_t bits = __ballot(marks != 0);
    for (int i = 0; bits; bits &= bits - 1, ++i) {                 // a wave every fourth
        if (i % 4 != wave) continue;
        const int64_t piece = group * 64 + __builtin_ctzll(bits);
        const bool first = piece < xpieces;
        const int64_t id = first ? piece : piece - xpieces, row = id / pass, k = id % pass * 1024 + 16 * lane;
        const int q = !first && row >= a.N;
        float* out = (first ? a.dx : q ? a.dw1 : a.dw0) + (row - q * a.N) * a.K;
        float s[16] = {};
#pragma unroll
        for (int c = 0; c < 16; c += 4)
            if (k + c < a.K) __builtin_memcpy(s + c, out + k + c, 16);
        if (first) tail_token<ACT, 16>(a, p, row, k, s);
        else tail_channel<ACT, 16>(a, p, q, row - q * a.N, k, s);
#pragma unroll
        for (int c = 0; c < 16; c += 4)
            if (k + c < a.K) __builtin_memcpy(out + k + c, s + c, 16);
    }
}

// ---- few tokens ---------------------------------------------------------------------------
// One pass in fp32: a workgroup takes 256 columns k and a chunk of the rows n of one projection, wave w the
// rows w, w + 4, ... of it, a lane four columns.  For a row it holds d of every token (through LDS) and
//     dW[n, k] = sum_m d[m, n] (x_q[m, k] beta[m] / 127),   written at once,
//     dx[m, k] += d[m, n] (alpha W[n, k]),                  held for the whole chunk,
// so that dW is written once and each weight read once, in its two bits.  The waves' dx are added through
// LDS, the chunks' by k_few_sum, in their order.
// Against the steps above (us): K = 1000, N = 1023, 1 token 7.8 and 19.8, 7 tokens 10.1 and 20.9, 16 tokens 13.6
// and 22.2; K = 4096, N = 11008, 4 tokens 36.8 and 76.0, 16 tokens 60.7 and 75.7; gated, F = 11008, 16 tokens
// 130 and 151.  Bound: writing dW (180 MB in the 36.8 us of 4 tokens) up to 8 tokens, beyond it the
// multiplications, 2 M + 3 instructions for a weight; more than 16 tokens do not fit the registers.
// 512 workgroups (two to a compute unit): 256 took 46.3 and 1024 38.1 us where 512 took 36.8.
constexpr int FEW_TOKENS = 16, MID_TOKENS = 64, FEW_K = 256, FEW_N = 64, FEW_GROUPS = 512;
struct FewPlan {
    int64_t kt, chunks, rows;      // column tiles; chunks of a projection, of `rows` rows
    int64_t groups;                // of 64 tokens (k_grad_mid)
    float* part;                   // dx [P chunks, M, K]
    float* wpart;                  // several groups: dW [groups, P N, K] and the bias sums [groups, P N]
    double* bpart;
    size_t bytes;
};
static FewPlan few_plan(int64_t M, int64_t K, int64_t N, bool gated, void* ws) {
    FewPlan p{};
    const int64_t P = gated ? 2 : 1;
    p.kt = (K + FEW_K - 1) / FEW_K;
    const int64_t rows = (P * N * p.kt + FEW_GROUPS - 1) / FEW_GROUPS;
    p.rows = M > FEW_TOKENS ? FEW_N : rows < 16 ? 16 : (rows + 3) / 4 * 4;
    p.chunks = (N + p.rows - 1) / p.rows;
    p.groups = (M + MID_TOKENS - 1) / MID_TOKENS;
    uint8_t* base = static_cast<uint8_t*>(ws);
    size_t off = 0;
    auto take = [&](int64_t bytes) {
        uint8_t* q = base ? base + off : nullptr;
        off += ((size_t)bytes + 255) / 256 * 256;
        return q;
    };
    p.part = reinterpret_cast<float*>(take(P * p.chunks * M * K * 4));
    p.wpart = reinterpret_cast<float*>(take(p.groups > 1 ? p.groups * P * N * K * 4 : 0));
    p.bpart = reinterpret_cast<double*>(take(p.groups > 1 ? p.groups * P * N * 8 : 0));
    p.bytes = off;
    return p;
}

template <int ACT, int MT>
__global__ __launch_bounds__(256) void k_grad_few(BackwardArgs a, FewPlan p) {
    __shared__ __align__(16) float d[FEW_N][MT];
    __shared__ __align__(16) float red[3][MT][FEW_K];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t tile = blockIdx.x % p.kt, ch = blockIdx.x / p.kt, rowb = a.K >> 2;
    const int q = ACT != 0 && ch >= p.chunks;
    const int64_t r0 = (ch - q * p.chunks) * p.rows, r1 = r0 + p.rows < a.N ? r0 + p.rows : a.N;
    const int64_t k = tile * FEW_K + 4 * lane, kl = k < a.K ? k : 0;       // kl: where the lane loads
    const uint8_t* w = (q ? a.w1 : a.w0) + (kl >> 2);
    float* dw = q ? a.dw1 : a.dw0;
    float* db = q ? a.db1 : a.db0;
    const float al = q ? a.al1[0] : a.al0[0];
    float x[MT][4], acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        uint32_t v = 0;
        float bs = 0.0f;
        if (a.dw0 && m < a.M) {
            __builtin_memcpy(&v, a.xq + m * a.K + kl, 4);
            bs = a.beta[m] / 127.0f;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            x[m][c] = (float)(int8_t)(v >> (8 * c)) * bs;
            acc[m][c] = 0.0f;
        }
    }
    for (int64_t n0 = r0; n0 < r1; n0 += FEW_N) {
        uint32_t codes[FEW_N / 4];
        if (a.dx) {
#pragma unroll
            for (int i = 0; i < FEW_N / 4; ++i) {
                const int64_t n = n0 + wave + 4 * i;
                codes[i] = w[(n < r1 ? n : r1 - 1) * rowb];
            }
        }
        __syncthreads();                               // the rows before have been read
#pragma unroll
        for (int e = tid; e < FEW_N * MT; e += 256) {
            const int j = e % FEW_N, m = e / FEW_N;
            float v[2] = {0.0f, 0.0f};
            if (n0 + j < r1 && m < a.M) grad_at<ACT>(a, m * a.N + n0 + j, v);
            d[j][m] = q ? v[1] : v[0];
        }
        __syncthreads();
        if (db && tile == 0 && tid < FEW_N && n0 + tid < r1) {
            double sum = 0.0;
#pragma unroll
            for (int m = 0; m < MT; ++m) sum += (double)d[tid][m];
            db[n0 + tid] = (float)sum;
        }
#pragma unroll
        for (int i = 0; i < FEW_N / 4; ++i) {
            const int j = wave + 4 * i;
            if (n0 + j >= r1) break;
            float dm[MT];
#pragma unroll
            for (int m = 0; m < MT; m += 4) {
                const float4 v = *reinterpret_cast<const float4*>(&d[j][m]);
                dm[m] = v.x, dm[m + 1] = v.y, dm[m + 2] = v.z, dm[m + 3] = v.w;
            }
            if (a.dx) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float t = __builtin_fmaf((float)((codes[i] >> (2 * c)) & 3u), al, -al);   // exact
#pragma unroll
                    for (int m = 0; m < MT; ++m) acc[m][c] = __builtin_fmaf(dm[m], t, acc[m][c]);
                }
            }
            if (dw) {
                float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[c] = __builtin_fmaf(dm[m], x[m][c], o[c]);
                if (k < a.K) __builtin_memcpy(dw + (n0 + j) * a.K + k, o, 16);
            }
        }
    }
    if (!a.dx) return;
    if (wave > 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
            *reinterpret_cast<float4*>(&red[wave - 1][m][4 * lane]) = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
    }
    __syncthreads();
    if (wave > 0 || k >= a.K) return;
    float* out = gridDim.x == p.kt ? a.dx : p.part + ch * a.M * a.K;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m >= a.M) break;
        float o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            o[c] = ((acc[m][c] + red[0][m][4 * lane + c]) + red[1][m][4 * lane + c]) + red[2][m][4 * lane + c];
        __builtin_memcpy(out + m * a.K + k, o, 16);
    }
}

// ---- some tokens, few tiles ---------------------------------------------------------------
// The products on the matrix cores without panels: a workgroup takes 256 columns k, 64 rows n of one
// projection and a group of 64 tokens.  It scales and splits its d as above, in both orders, into LDS, where x_q
// and W are turned and stay bytes v + 128; dx is written as a part for each 64 rows, dW at once or, with
// several groups, as a part for each (a scale is taken over a part's terms, and the part scaled back before it
// leaves); k_few_sum adds them.
// Small elements as above: where there are tiny sums too, the workgroup adds what the elements lack.
// Against the steps above (us): gated, K = 1024, F = 2731, 61 tokens (344 workgroups) 26.7 and 41.2; K = 512,
// N = 512, 64 tokens (16) 12.2 and 26.3; K = 2944, N = 5335 (1008), 32 tokens 36.2 and 45.4, 64 tokens 44.4 and
// 47.0; gated, K = 2048, F = 5504 (1376), 64 tokens 64.6 and 58.3: the parts of dx, as many bytes as dW.  With parts
// of dW: K = 512, N = 512, 250 tokens (64) 16.2 and 27.1; K = 1280, N = 1230, 256 tokens (400) 30.0 and 34.5; K = 1000,
// N = 1023, 500 tokens (512) 33.4 and 41.2; K = 2048, N = 2048, 250 tokens (1024) 56.9 and 38.4.
// Several tiles of rows in a workgroup halve those but hold twice the registers (gated, K = 1024, F = 2731, 61
// tokens 33 us).  Bound: at a single tile latency, loads, three barriers and some 800 instructions of a wave.
// LDS images: split gradients, rows of 64 values, the 16-byte unit u at position u ^ (row / 2) % 8; bytes,
// columns of 64, the 16-byte unit u at position u ^ split_swizzle(column).
constexpr int MID_TILES = 1024, MID_TILES_GROUPS = 512;
static_assert(16 * (int64_t)BITLINEAR_MAX_K + 4 * 32 < (int64_t)1 << 32, "a lane's offset in mid_store has 32 bits");

// acc[i] += sum_l (hi + 2^-12 lo)[row, l] b[column, l]: rows 32 i .. 32 i + 31 (i = 0 alone if !high), columns c0 ..
// c0 + 31, l 0 .. 63 (0 .. 31 if !deep); operands in lanes as k_split_gemm's.
__device__ __forceinline__ void mid_multiply(f32x16 (&acc)[2], const u32x4* hi, const u32x4* lo, const u32x4* b, int c0, bool high,
                                             bool deep) {
    const int lr = threadIdx.x & 31, lg = (threadIdx.x >> 5) & 1, c = c0 + lr;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (s && !deep) break;
        const u32x4 cb = b[4 * c + ((2 * s + lg) ^ split_swizzle(c))];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const f16x8 fb = bytes_f16(cb[2 * kk], cb[2 * kk + 1]), fd = lower_operand(fb);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i && !high) break;
                const int r = 32 * i + lr, at = 8 * r + ((4 * s + 2 * lg + kk) ^ ((r >> 1) & 7));
                acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, hi[at]), fb, acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, lo[at]), fd, acc[i], 0, 0, 0);
            }
        }
    }
}

// out[row, column] = acc scale[row], rows below `rows`, columns below `cols` (lane: column lane % 32 of rows
// 4 (lane / 32) .. of eight).  A running row and one lane offset of 32 bits: the addresses of every row would
// fill the registers.
__device__ __forceinline__ void mid_store(const f32x16 (&acc)[2], const float* scale, float* out, int64_t stride, int64_t rows,
                                          int64_t cols) {
    const int lr = threadIdx.x & 31, lg = (threadIdx.x >> 5) & 1;
    if (lr >= cols) return;
    const uint32_t off = 4u * (4u * lg * (uint32_t)stride + lr);
    const int left = (int)(rows < 64 ? rows : 64) - 4 * lg;
    auto rows_out = [&](auto inside) {
        char* row = reinterpret_cast<char*>(out);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4 v = *reinterpret_cast<const float4*>(&scale[32 * i + 8 * g + 4 * lg]);
                const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (inside(32 * i + 8 * g + e)) *reinterpret_cast<float*>(row + off) = acc[i][4 * g + e] * f[e];
                    row += 4 * stride;
                }
                row += 16 * stride;
            }
    };
    if (rows >= 64) rows_out([](int) { return true; });
    else rows_out([&](int r) { return r < left; });
}

// Whether one of the lane's sums is below `need` times its row's small elements, in the first `cols` columns.
__device__ __forceinline__ bool mid_tiny(const f32x16 (&acc)[2], const float* smalls, float need, int64_t cols) {
    const int lr = threadIdx.x & 31, lg = (threadIdx.x >> 5) & 1;
    float over = INFINITY;                             // the least |sum| - limit
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 v = *reinterpret_cast<const float4*>(&smalls[32 * i + 8 * g + 4 * lg]);
            const float n[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) over = fminf(over, __builtin_fmaf(n[e], -need, fabsf(acc[i][4 * g + e])));
        }
    return over < 0.0f && lr < cols;
}

template <int ACT>
__global__ __launch_bounds__(512, 4) void k_grad_mid(BackwardArgs a, FewPlan p) {
    // split gradients: hi and lo of d alpha, a row for a token, then of d beta / 127, a row for a channel
    __shared__ u32x4 sp[4][512];
    __shared__ u32x4 xb[1024], wb[1024];               // bytes of x_q^T and of W_hat^T
    __shared__ uint32_t turn[64 * 17];
    __shared__ float cmx[8][64];
    __shared__ double csum[8][64];
    __shared__ __align__(16) float rinv[64];
    __shared__ __align__(16) float cinv[64];
    __shared__ float rscale[64], cscale[64];           // scales of the tokens' d alpha and the channels' d beta / 127
    __shared__ __align__(16) float small_x[64], small_w[64];   // small elements of the tokens' d alpha, of the channels' d beta / 127
    __shared__ int again[2];                           // small elements' rests are to be added to dx, to dW
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = wave >> 2, tt = tid & 255;        // a tile of bytes is turned by 256 threads
    const uint32_t kt = (uint32_t)p.kt, chs = (uint32_t)p.chunks * (ACT == 0 ? 1 : 2), idx = blockIdx.x / kt;
    const int64_t tile = blockIdx.x % kt, ch = idx % chs, grp = idx / chs, m0 = MID_TOKENS * grp;
    const int64_t rowb = a.K >> 2, k0 = tile * FEW_K;
    const int M = (int)(a.M - m0 < MID_TOKENS ? a.M - m0 : MID_TOKENS);
    const int q = ACT != 0 && ch >= p.chunks;
    const int64_t n0 = (ch - q * p.chunks) * FEW_N;
    const uint8_t* w = q ? a.w1 : a.w0;
    const int8_t* xq = a.xq + m0 * a.K;
    const float *dy = a.dy + m0 * a.N, *sg = ACT == 0 ? nullptr : a.g + m0 * a.N, *su = ACT == 0 ? nullptr : a.u + m0 * a.N;
    float* dw = q ? a.dw1 : a.dw0;
    float* db = tile > 0 ? nullptr : q ? a.db1 : a.db0;
    if (dw && p.groups > 1) dw = p.wpart + (grp * (ACT == 0 ? 1 : 2) + q) * a.N * a.K;
    double* bp = p.bpart + (grp * (ACT == 0 ? 1 : 2) + q) * a.N;   // several groups: in db's place
    const float al = q ? a.al1[0] : a.al0[0];
    // tokens and rows past the end repeat the last (their d is zero), columns past it are not stored
    u32x4 x[2], wr{};
    if (dw) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int64_t k = k0 + 64 * (2 * half + c) + 4 * (tt & 15);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = 4 * (tt >> 4) + i;
                uint32_t v;
                __builtin_memcpy(&v, xq + (m < M ? m : M - 1) * a.K + (k < a.K ? k : 0), 4);
                x[c][i] = v;
            }
        }
    }
    // four bytes of W in four rows, zeros past a row's end
    if (a.dx && half == 0) {
        const int64_t at = (k0 >> 2) + 4 * (tt & 15), end = rowb - 4, from = at < end ? at : end;
        const int past = at - from < 4 ? (int)(at - from) : 0;     // bytes of the dword past the row's end
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = n0 + 4 * (tt >> 4) + i;
            const uint8_t* row = w + (n < a.N ? n : a.N - 1) * rowb;
            uint32_t v = 0;
            if (end >= 0) {
                __builtin_memcpy(&v, row + from, 4);
                v >>= 8 * past;
            } else if (at == 0) {
#pragma nounroll
                for (int b = 0; b < (int)rowb; ++b) v |= (uint32_t)row[b] << (8 * b);
            }
            wr[i] = v;
        }
    }
    // d of tokens 8 wave .. 8 wave + 7 in row n0 + lane, zeros past the ends; offsets below 2^31 bytes
    auto load_d = [&](float (&d)[8]) {
        const uint32_t n = (uint32_t)(n0 + lane < a.N ? n0 + lane : a.N - 1), N = (uint32_t)a.N;
        auto at = [](const float* p, uint32_t i) { return *reinterpret_cast<const float*>(reinterpret_cast<const char*>(p) + 4u * i); };
        float y[8], g[8], u[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int m = 8 * wave + t;
            const uint32_t i = (uint32_t)(m < M ? m : M - 1) * N + n;
            y[t] = at(dy, i);
            g[t] = ACT == 0 ? 0.0f : at(sg, i);
            u[t] = ACT == 0 ? 0.0f : at(su, i);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            float e[2];
            grad_of<ACT>(y[t], g[t], u[t], e);
            d[t] = n0 + lane < a.N && 8 * wave + t < M ? (q ? e[1] : e[0]) : 0.0f;
        }
    };
    float d[8];
    load_d(d);
    if (tid < 2) again[tid] = 0;
    if (tid < 64) small_x[tid] = small_w[tid] = 0.0f;
    // x_q: four tiles of 64 columns, turned in the split gradients' place; W
    uint32_t* room = reinterpret_cast<uint32_t*>(sp);
    if (dw) {
#pragma unroll
        for (int c = 0; c < 2; ++c) turn_put(room + 64 * 17 * (2 * half + c), x[c], tt);
    }
    if (a.dx && half == 0) turn_put(turn, wr, tt);
    // the tokens' and the channels' scales; beta / 127 of the wave's tokens (the same in every lane)
    float bs[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const int m = 8 * wave + t, s = scale_exponent(wave_max_pos(fabsf(d[t] * al)));
        bs[t] = m < M ? a.beta[m0 + m] / 127.0f : 0.0f;
        if (lane == 0) {
            rscale[m] = pow2f(s);
            rinv[m] = pow2f(-s);
        }
    }
    if (dw) {
        float v = 0.0f;
#pragma unroll
        for (int t = 0; t < 8; ++t) v = fmaxf(v, fabsf(d[t] * bs[t]));
        cmx[wave][lane] = v;
    }
    if (db) {
        double v = 0.0;
#pragma unroll
        for (int t = 0; t < 8; ++t) v += (double)d[t];
        csum[wave][lane] = v;
    }
    __syncthreads();
    u32x4 xt[2];
    if (dw) {
#pragma unroll
        for (int c = 0; c < 2; ++c) xt[c] = turn_get(room + 64 * 17 * (2 * half + c), tt) ^ 0x80808080u;
    }
    __syncthreads();                                   // the room is free
    if (dw) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int col = 64 * (2 * half + c) + (tt >> 2);
            xb[4 * col + ((tt & 3) ^ split_swizzle(col))] = xt[c];
        }
        float v = cmx[0][lane];
#pragma unroll
        for (int i = 1; i < 8; ++i) v = fmaxf(v, cmx[i][lane]);
        const int s = scale_exponent(v), at = 8 * lane + (wave ^ ((lane >> 1) & 7));
        const float cs = pow2f(s);
        if (wave == 0) {
            cscale[lane] = cs;
            cinv[lane] = pow2f(-s);
        }
        u32x4 hi, lo;
        uint32_t least = ~0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f0 = d[2 * e] * bs[2 * e] * cs, f1 = d[2 * e + 1] * bs[2 * e + 1] * cs;
            const uint32_t v0 = split_f16(f0), v1 = split_f16(f1);
            hi[e] = __builtin_amdgcn_perm(v1, v0, 0x05040100u);
            lo[e] = __builtin_amdgcn_perm(v1, v0, 0x07060302u);
            least = min(least, min(size_bits(f0), size_bits(f1)));
        }
        if (least < SMALL_BITS - 1) {
            float n = 0.0f;
#pragma unroll
            for (int t = 0; t < 8; ++t) n += is_small(d[t] * bs[t] * cs);
            atomicAdd(&small_w[lane], n);              // exact in any order
        }
        sp[2][at] = hi;
        sp[3][at] = lo;
    }
    if (a.dx) {
        uint16_t* hi = reinterpret_cast<uint16_t*>(sp[0]);
        uint16_t* lo = reinterpret_cast<uint16_t*>(sp[1]);
        uint32_t least = ~0u;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int m = 8 * wave + t, at = 8 * (8 * m + ((lane >> 3) ^ ((m >> 1) & 7))) + (lane & 7);
            const float f = d[t] * al * rscale[m];
            const uint32_t v = split_f16(f);
            hi[at] = (uint16_t)v;
            lo[at] = (uint16_t)(v >> 16);
            least = min(least, size_bits(f));
        }
        if (__ballot(least < SMALL_BITS - 1)) {
            for (int t = 0; t < 8; ++t) {
                const float n = (float)__popcll(__ballot(is_small(d[t] * al * rscale[8 * wave + t])));
                if (lane == 0) small_x[8 * wave + t] = n;
            }
        }
        const u32x4 v = turn_get(turn, tt);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = 4 * (tt >> 2) + 2 * half + i;
            wb[4 * c + ((tt & 3) ^ split_swizzle(c))] = code_bytes(v, 2 * half + i);
        }
    }
    if (db && tid < 64 && n0 + tid < a.N) {
        double v = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += csum[i][tid];
        if (p.groups > 1) bp[n0 + tid] = v;
        else db[n0 + tid] = (float)v;
    }
    __syncthreads();
    const int64_t left = a.K - (k0 + 32 * wave);       // columns from the wave's first to the end
    bool some_x = false, some_w = false;               // there are small elements
    if (a.dx) some_x = __ballot(small_x[lane] > 0.0f) != 0;
    if (dw) some_w = __ballot(small_w[lane] > 0.0f) != 0;
    if (a.dx) {
        f32x16 acc[2] = {};
        mid_multiply(acc, sp[0], sp[1], wb, 32 * wave, M > 32, true);
        if (some_x && mid_tiny(acc, small_x, NEED_X, left)) again[0] = 1;
        mid_store(acc, rinv, (chs == 1 ? a.dx : p.part + ch * a.M * a.K) + m0 * a.K + k0 + 32 * wave, a.K, M, left);
    }
    if (dw) {
        f32x16 acc[2] = {};
        mid_multiply(acc, sp[2], sp[3], xb, 32 * wave, true, M > 32);
        if (some_w && mid_tiny(acc, small_w, NEED_W, left)) again[1] = 1;
        mid_store(acc, cinv, dw + n0 * a.K + k0 + 32 * wave, a.K, a.N - n0, left);
    }
    if (!some_x && !some_w) return;
    __syncthreads();
    if (!again[0] && !again[1]) return;
    // tiny sums and small elements, rare: those are formed again, and what they lack when split is added
    // to what has been stored in the order of the sums, to dx by each wave in its own tokens, to dW by one wave
    // after another; a lane takes four columns (every lane stays: a rest is read from any of them)
    const int64_t k = k0 + 4 * lane, kl = k < a.K ? k : 0;
    load_d(d);
    if (again[0]) {
        float* out = (chs == 1 ? a.dx : p.part + ch * a.M * a.K) + m0 * a.K;
        for (int t = 0; t < 8; ++t) {
            const int m = 8 * wave + t;
            const float v = d[t] * al * rscale[m], rest = split_rest(v) * rinv[m];
            uint64_t bits = __ballot(is_small(v));
            if (!bits) continue;
            float s[4];
            __builtin_memcpy(s, out + m * a.K + kl, 16);
            for (; bits; bits &= bits - 1) {
                const int j = __builtin_ctzll(bits);
                const float e = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(rest), j));
                const uint32_t codes = w[(n0 + j) * rowb + (kl >> 2)];
#pragma unroll
                for (int c = 0; c < 4; ++c) s[c] = __builtin_fmaf(e, (float)(int)(codes >> (2 * c) & 3u) - 1.0f, s[c]);
            }
            if (k < a.K) __builtin_memcpy(out + m * a.K + k, s, 16);
        }
    }
    if (!again[1]) return;
    for (int i = 0; i < 8; ++i) {
        if (i == wave) {
            for (int t = 0; t < 8; ++t) {
                const int m = 8 * wave + t;
                const float v = d[t] * bs[t] * cscale[lane], rest = split_rest(v) * cinv[lane];
                for (uint64_t bits = __ballot(is_small(v)); bits; bits &= bits - 1) {
                    const int j = __builtin_ctzll(bits);
                    const float e = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(rest), j));
                    float* out = dw + (n0 + j) * a.K;
                    uint32_t codes;
                    float s[4];
                    __builtin_memcpy(&codes, xq + m * a.K + kl, 4);
                    __builtin_memcpy(s, out + kl, 16);
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[c] = __builtin_fmaf(e, (float)(int8_t)(codes >> (8 * c)), s[c]);
                    if (k < a.K) __builtin_memcpy(out + k, s, 16);
                }
            }
        }
        __syncthreads();                               // the next wave's elements may be of the same rows
    }
}

// Sums of parts, in their order: dx from the chunks', dW from the token groups', 256 elements per workgroup, a wave
// every fourth part; last the bias sums.
struct PartSum {
    const float* part;
    float* out;
    int64_t n, parts, stride, blocks;
};
__global__ __launch_bounds__(256) void k_few_sum(PartSum x, PartSum w0, PartSum w1, const double* __restrict__ bpart, float* db0,
                                                 float* db1, int64_t N, int64_t P, int64_t groups) {
    __shared__ __align__(16) float4 red[3][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t b = blockIdx.x;
    PartSum a = x;
    if (b >= a.blocks) {
        b -= a.blocks;
        a = w0;
    }
    if (b >= a.blocks) {
        b -= a.blocks;
        a = w1;
    }
    if (b >= a.blocks) {
        const int64_t i = (b - a.blocks) * 256 + threadIdx.x;
        float* out = i < N ? db0 : db1;
        if (i >= P * N || !out) return;
        double s = 0.0;
        for (int64_t g = 0; g < groups; ++g) s += bpart[g * P * N + i];
        out[i < N ? i : i - N] = (float)s;
        return;
    }
    const int64_t e = b * 256 + 4 * lane, el = e < a.n ? e : 0;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int64_t c = wave; c < a.parts; c += 4) {
        const float4 v = *reinterpret_cast<const float4*>(a.part + c * a.stride + el);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    if (wave > 0) red[wave - 1][lane] = s;
    __syncthreads();
    if (wave > 0 || e >= a.n) return;
#pragma unroll
    for (int w = 0; w < 3; ++w) {
        const float4 v = red[w][lane];
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    __builtin_memcpy(a.out + e, &s, 16);
}

static bool use_mid(int64_t M, int64_t K, int64_t N, bool gated) {
    const int64_t groups = (M + MID_TOKENS - 1) / MID_TOKENS;
    const int64_t tiles = ((K + FEW_K - 1) / FEW_K) * ((N + FEW_N - 1) / FEW_N) * (gated ? 2 : 1) * groups;
    return M > FEW_TOKENS && tiles <= (groups == 1 ? MID_TILES : MID_TILES_GROUPS);
}

// MT: tokens that k_grad_few holds, 0 for k_grad_mid.
template <int ACT, int MT>
static hipError_t launch_few(const BackwardArgs& a, hipStream_t s) {
    FewPlan p = few_plan(a.M, a.K, a.N, ACT != 0, a.ws);
    if (!a.dx && !a.dw0) p.kt = 1;                     // the bias sums alone
    const int64_t P = ACT == 0 ? 1 : 2, chunks = P * p.chunks, n = a.M * a.K;
    if constexpr (MT > 0)
        hipLaunchKernelGGL((k_grad_few<ACT, MT>), dim3((unsigned)(chunks * p.kt)), dim3(256), 0, s, a, p);
    else
        hipLaunchKernelGGL(k_grad_mid<ACT>, dim3((unsigned)(chunks * p.kt * p.groups)), dim3(512), 0, s, a, p);
    auto sum = [](const float* part, float* out, int64_t n, int64_t parts, int64_t stride) {
        return PartSum{part, out, n, parts, stride, out && parts > 1 ? (n + 255) / 256 : 0};
    };
    const PartSum x = sum(p.part, a.dx, n, chunks, n), w0 = sum(p.wpart, a.dw0, a.N * a.K, p.groups, P * a.N * a.K),
                  w1 = sum(p.wpart + a.N * a.K, a.dw1, a.N * a.K, p.groups, P * a.N * a.K);
    const int64_t bias = (a.db0 || a.db1) && p.groups > 1 ? (P * a.N + 255) / 256 : 0;
    if (x.blocks + w0.blocks + w1.blocks + bias)
        hipLaunchKernelGGL(k_few_sum, dim3((unsigned)(x.blocks + w0.blocks + w1.blocks + bias)), dim3(256), 0, s, x, w0, w1, p.bpart,
                           a.db0, a.db1, a.N, P, p.groups);
    return hipGetLastError();
}

size_t backward_workspace(int64_t M, int64_t K, int64_t N, bool gated) {
    return M <= FEW_TOKENS || use_mid(M, K, N, gated) ? few_plan(M, K, N, gated, nullptr).bytes
                                                      : grad_plan(M, K, N, gated, nullptr).bytes;
}

template <int ACT>
static hipError_t launch_grads(const BackwardArgs& a, hipStream_t s) {
    constexpr int P = ACT == 0 ? 1 : 2;
    if (a.M <= FEW_TOKENS) return a.M <= 4 ? launch_few<ACT, 4>(a, s) : a.M <= 8 ? launch_few<ACT, 8>(a, s) : launch_few<ACT, 16>(a, s);
    if (use_mid(a.M, a.K, a.N, P == 2)) return launch_few<ACT, 0>(a, s);
    const GradPlan p = grad_plan(a.M, a.K, a.N, P == 2, a.ws);
    auto blocks = [](int64_t n) { return dim3((unsigned)n); };
    const int64_t ktw = (a.K + 255) / 256, ktc = (a.K + 63) / 64;
    const int64_t maxima = p.mt * p.ct, weights = a.dx ? p.Lx / 64 * ktw : 0, codes = a.dw0 ? p.Mp / 64 * ktc : 0;
    if (p.tn == 64)
        hipLaunchKernelGGL((k_grad_prep<ACT, 1>), blocks(maxima + weights + codes), dim3(256), 0, s, a, p, maxima, weights, ktw, ktc);
    else
        hipLaunchKernelGGL((k_grad_prep<ACT, 4>), blocks(maxima + weights + codes), dim3(256), 0, s, a, p, maxima, weights, ktw, ktc);
    const int64_t cblocks = (P * a.N + 255) / 256;
    if (p.mt > 1) hipLaunchKernelGGL(k_grad_reduce, blocks(cblocks + (a.M + 3) / 4), dim3(256), 0, s, a, p, P, cblocks);
    if (!a.dx && !a.dw0) return hipGetLastError();
    const int64_t ct = (a.N + 127) / 128;
    hipLaunchKernelGGL(k_grad_split<ACT>, blocks(p.Mp / 32 * ct), dim3(512), 0, s, a, p, (int)ct);
    auto tiles = [](SplitArgs q) {
        q.tiles_i = (int)((q.I + SG_BM - 1) / SG_BM);
        q.tiles_j = (int)((q.J + SG_BN - 1) / SG_BN);
        return q;
    };
    SplitArgs x{}, w{};
    if (a.dx)
        x = tiles(SplitArgs{p.xs, p.wt, p.rmax, a.M, a.K, p.Lx, a.dx, nullptr, a.M, p.part_x, p.parts_x, 0, 0, p.need_x, p.nb,
                            p.smalls, NEED_X});
    if (a.dw0)
        w = tiles(SplitArgs{p.wsp, p.cd, p.cmax, P * a.N, a.K, p.Mp, a.dw0, a.dw1, a.N, p.part_w, p.parts_w, 0, 0, p.need_w, p.nb,
                            p.smalls + a.M, NEED_W});
    const int64_t grid = (int64_t)x.parts * x.tiles_i * x.tiles_j + (int64_t)w.parts * w.tiles_i * w.tiles_j;
    hipLaunchKernelGGL(k_split_gemm, blocks(grid), dim3(256), 0, s, x, w);
    const int64_t cols = (a.K + 127) / 128, xw = x.parts > 1 ? x.I * cols : 0, waves = xw + (w.parts > 1 ? w.I * cols : 0);
    const int64_t xp = x.parts == 1 ? x.I * (p.nb / 8) : 0, pieces = xp + (w.parts == 1 ? w.I * (p.nb / 8) : 0);
    hipLaunchKernelGGL(k_grad_finish<ACT>, blocks((waves + 3) / 4 + (pieces + 63) / 64), dim3(256), 0, s, a, p, x, w, xw, waves, xp,
                       pieces);
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
