// grouped_backward.hip -- gradients of the ternary BitLinears grouped by expert and of the gated block, gfx950.
//
// What is computed, row m of group e reading token r, for one projection or two (gate and up):
//     dx[m, k]     = sum_p sum_n (alpha_p,e d_p[m, n]) W_p,e[n, k]
//     dW_p,e[n, k] = sum_{m in e} (d_p[m, n] beta[r] / 127) x_q[r, k],   dbias_p,e[n] = sum_{m in e} d_p[m, n]
// with d = dy, or dg = dh u a'(g) and du = dh a(g), which a first kernel leaves in the workspace.
//
// Both products run on the bf16 matrix cores: an fp32 factor is the exact sum of three bf16 values (its upper
// eight significant bits, the next eight, the last eight), and the other factor, -1, 0, 1 or an int8 code,
// is a bf16 value, so that three products with exact terms and fp32 sums give a product of fp32 accuracy,
// whatever the sizes of the elements beside each other.
#include <type_traits>

#include "experts.hpp"
#include "ffn.hpp"

namespace bitlinear {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

size_t grouped_backward_workspace(int64_t M, int64_t K, int64_t N, int64_t E, bool gated) {
    return 256 + (gated ? (size_t)M * N * 8 : 0);
}

// dg and du, one element a thread at a time.
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

struct Products {
    GroupedBackwardArgs a;
    const float *d0, *d1;          // [M, N]: dy, or dg and du
};

// ---- the two products -----------------------------------------------------------------------
// A workgroup of eight waves computes 64 MI x 256 of dx (rows x k) or of a dW (n x k), a wave 32 MI x 64, in
// steps of 64 of the sum.  A stage in LDS is three planes of the split factor, 64 MI rows of 64 bf16 values,
// and 256 rows (one for each k) of the other; both are loaded from memory into registers while the stage
// before is multiplied, split or widened there, turned where the sum runs down the rows, and written in 16-byte
// units: unit u (8 of the sum) of row r at slot u ^ ((r / 2) % 8), which spreads reads and writes over all banks.
// Row of k: column 2 l + j of the wave's 64 lies in row 32 j + l, so that a lane ends with pairs of columns.
// 32x32x16 lane layout: A/B lane l holds row/column l % 32, 8 (l / 32) + j of the sum; accumulator r of lane l is
// row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
constexpr int GB_BN = 256;

template <int MI>
struct Grad {
    static constexpr int BM = 64 * MI, OB = 3 * BM * 8, UNITS = OB + GB_BN * 8;
};

// Eight floats as a unit of each of the three planes: truncation leaves exact remainders.
__device__ __forceinline__ void split_unit(const float (&v)[8], u32x4 (&pl)[3]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        uint32_t b[2][3];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t h = __float_as_uint(v[i + e]) & 0xFFFF0000u;
            const float r = v[i + e] - __uint_as_float(h);
            const uint32_t m = __float_as_uint(r) & 0xFFFF0000u;
            b[e][0] = h;
            b[e][1] = m;
            b[e][2] = __float_as_uint(r - __uint_as_float(m));
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) pl[q][i >> 1] = __builtin_amdgcn_perm(b[1][q], b[0][q], 0x07060302u);
    }
}

// The product of stages, two at a time: `load(s)` puts step s into registers, `put(st)` writes them to a stage.
template <int MI, typename Load, typename Put>
__device__ __forceinline__ void grad_sum(u32x4* st0, u32x4* st1, int steps, f32x16 (&acc)[MI][2], Load load, Put put) {
    constexpr int BM = Grad<MI>::BM, OB = Grad<MI>::OB;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = wave & 1, wj = wave >> 1, lr = lane & 31, lg = lane >> 5, sw = (lr >> 1) & 7;
    auto multiply = [&](const u32x4* st) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const int at = (2 * ks + lg) ^ sw;
            bf16x8 b[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) b[j] = __builtin_bit_cast(bf16x8, st[OB + (64 * wj + 32 * j + lr) * 8 + at]);
#pragma unroll
            for (int q = 2; q >= 0; --q)
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const bf16x8 f = __builtin_bit_cast(bf16x8, st[(q * BM + 32 * MI * wi + 32 * i + lr) * 8 + at]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, b[j], acc[i][j], 0, 0, 0);
                }
        }
    };
    if (steps == 0) return;
    load(0);
    put(st0);
    if (steps > 1) load(1);
    lds_barrier();
    for (int s = 0; s < steps; s += 2) {
        if (s + 1 < steps) put(st1);                   // its last readers are past the barrier before
        if (s + 2 < steps) load(s + 2);
        multiply(st0);
        lds_barrier();
        if (s + 1 >= steps) break;
        if (s + 2 < steps) put(st0);
        if (s + 3 < steps) load(s + 3);
        multiply(st1);
        lds_barrier();
    }
}

// rows x columns of `out` (row length K) from a wave's accumulators.
template <int MI>
__device__ __forceinline__ void grad_store(float* __restrict__ out, int64_t K, int rows, int64_t k0, const f32x16 (&acc)[MI][2]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t k = k0 + 64 * (wave >> 1) + 2 * (lane & 31);
    if (k >= K) return;                                // K is even
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int m = 32 * MI * (wave & 1) + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
            const float2 v = make_float2(acc[i][0][r], acc[i][1][r]);
            if (m < rows) __builtin_memcpy(out + (int64_t)m * K + k, &v, 8);
        }
}

// LDS row of k 4 c + j of the tile (c a lane, j < 4).
__device__ __forceinline__ int grad_row(int c, int j) { return 64 * (c >> 4) + 32 * (j & 1) + 2 * (c & 15) + (j >> 1); }

template <int MI>
__device__ __forceinline__ void dx_tile(const Products& p, u32x4* st0, u32x4* st1, const Slot& slot, int64_t k0) {
    constexpr int BM = Grad<MI>::BM, OB = Grad<MI>::OB;
    const GroupedBackwardArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t N = a.N, rowb = a.K >> 2, e = slot.e;
    const int per = (int)((N + 63) / 64), steps = per * (a.w1 ? 2 : 1);
    // of d: row tid / (8 / MI), MI units of 8; of W: rows 8 wave .., the lane's byte of 4 codes
    const int row = tid / (8 / MI), unit = (tid % (8 / MI)) * MI;
    const int64_t at = (slot.m0 + min(row, slot.rows - 1)) * N;
    const int64_t byte = min((k0 >> 2) + lane, rowb - 1);
    float v[MI][8], alpha;
    uint32_t w[8];
    auto load = [&](int s) {
        const bool second = s >= per;
        const int64_t n0 = (int64_t)(second ? s - per : s) * 64, n = n0 + 8 * unit;
        const float* d = (second ? p.d1 : p.d0) + at;
        const uint8_t* ww = (second ? a.w1 : a.w0) + e * N * rowb + byte;
        alpha = (second ? a.al1 : a.al0)[e];
        if (n0 + 64 <= N) {
#pragma unroll
            for (int i = 0; i < MI; ++i) __builtin_memcpy(v[i], d + n + 8 * i, 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = ww[(n0 + 8 * wave + i) * rowb];
        } else {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int x = 0; x < 8; ++x) v[i][x] = n + 8 * i + x < N ? d[n + 8 * i + x] : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = ww[min(n0 + 8 * wave + i, N - 1) * rowb];
        }
    };
    auto put = [&](u32x4* st) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            u32x4 pl[3];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[i][x] *= alpha;
            split_unit(v[i], pl);
#pragma unroll
            for (int q = 0; q < 3; ++q) st[(q * BM + row) * 8 + ((unit + i) ^ ((row >> 1) & 7))] = pl[q];
        }
        // codes of four n a dword; for each k their bf16 values from tables of the upper and lower bytes
        const uint32_t c0 = w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24, c1 = w[4] | w[5] << 8 | w[6] << 16 | w[7] << 24;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u32x4 o;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t c = ((h ? c1 : c0) >> (2 * j)) & 0x03030303u;
                const uint32_t hi = __builtin_amdgcn_perm(0u, 0x003F00BFu, c), lo = __builtin_amdgcn_perm(0u, 0x00800080u, c);
                o[2 * h] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
                o[2 * h + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
            }
            const int r = grad_row(lane, j);
            st[OB + r * 8 + (wave ^ ((r >> 1) & 7))] = o;
        }
    };
    f32x16 acc[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i) acc[i][0] = acc[i][1] = f32x16{};
    grad_sum<MI>(st0, st1, steps, acc, load, put);
    grad_store<MI>(a.dx + slot.m0 * a.K, a.K, slot.rows, k0, acc);
}

template <int MI>
__device__ __forceinline__ void dw_tile(const Products& p, u32x4* st0, u32x4* st1, int64_t e, bool second, int64_t n0, int64_t k0) {
    constexpr int BM = Grad<MI>::BM, OB = Grad<MI>::OB;
    const GroupedBackwardArgs& a = p.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t N = a.N, K = a.K;
    const Group g = group_rows(a.offsets, e, a.M);
    const int steps = g.hi > g.lo ? (int)((g.hi - g.lo + 63) / 64) : 0;
    const float* d = second ? p.d1 : p.d0;
    // the wave takes rows 8 wave .. of a step, a lane MI columns of d and four of x_q
    const int64_t n = n0 + MI * lane, k = min(k0 + 4 * lane, K - 4);
    const bool whole = n0 + BM <= N;
    int64_t cols[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) cols[i] = min(n + i, N - 1);
    // token of row lane % 8 of the wave's rows of a step: of the last row past the end
    auto row_of = [&](int s, int i) { return min(g.lo + (int64_t)s * 64 + 8 * wave + i, g.hi - 1); };
    auto tokens = [&](int s) { return (int)row_token(a.rows, row_of(s, lane & 7), a.T); };
    float v[8][MI], beta;
    uint32_t x[8];
    bool there;
    int token = steps ? tokens(0) : 0;
    auto load = [&](int s) {
        beta = token >= 0 ? a.beta[token] : 0.0f;
        there = g.lo + (int64_t)s * 64 + 8 * wave + (lane & 7) < g.hi;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float* dr = d + row_of(s, i) * N;
            if (MI == 2 && whole) {
                __builtin_memcpy(v[i], dr + n, 4 * MI);
            } else {
#pragma unroll
                for (int c = 0; c < MI; ++c) v[i][c] = dr[cols[c]];
            }
            const int t = __builtin_amdgcn_readlane(token, i);
            __builtin_memcpy(&x[i], a.xq + (int64_t)(t < 0 ? 0 : t) * K + k, 4);
        }
        token = tokens(s + 1);
    };
    auto put = [&](u32x4* st) {
        // beta / 127 of the rows; 0 for rows past the end and tokens that are not there
        const float f = there ? beta / 127.0f : 0.0f;
        float fi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) fi[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), i));
#pragma unroll
        for (int c = 0; c < MI; ++c) {
            float t[8];
            u32x4 pl[3];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = v[i][c] * fi[i];
            split_unit(t, pl);
            const int r = MI * lane + c;
#pragma unroll
            for (int q = 0; q < 3; ++q) st[(q * BM + r) * 8 + (wave ^ ((r >> 1) & 7))] = pl[q];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float lo = (float)(int8_t)(x[i] >> (8 * j)), hi = (float)(int8_t)(x[i + 1] >> (8 * j));
                o[i >> 1] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
            }
            const int r = grad_row(lane, j);
            st[OB + r * 8 + (wave ^ ((r >> 1) & 7))] = o;
        }
    };
    f32x16 acc[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i) acc[i][0] = acc[i][1] = f32x16{};
    grad_sum<MI>(st0, st1, steps, acc, load, put);
    const int rows = (int)(N - n0 < BM ? N - n0 : BM);
    grad_store<MI>((second ? a.dw1 : a.dw0) + (e * N + n0) * K, K, rows, k0, acc);
}

// dx's tiles first (`slots` x tiles_k of them at most), whose sums are the longer ones, then dW's, so that the
// short ones fill the card where dx's end.  Of each kind a contiguous run for every XCD.
template <int MI>
__global__ __launch_bounds__(512, 2) void k_grouped_gradients(Products p, int dx_wgs, int tiles_k, int tiles_n) {
    __shared__ u32x4 st0[Grad<MI>::UNITS];
    __shared__ u32x4 st1[Grad<MI>::UNITS];
    const GroupedBackwardArgs& a = p.a;
    auto run_of = [](int b, int T) { return (b & 7) * (T >> 3) + ((b & 7) < (T & 7) ? b & 7 : T & 7) + (b >> 3); };
    if ((int)blockIdx.x < dx_wgs) {
        int tiles_m;
        find_slot<Grad<MI>::BM, true>(a.offsets, (int)a.E, a.M, -1, &tiles_m);
        const int T = tiles_m * tiles_k;
        if ((int)blockIdx.x >= T) return;
        int t = run_of(blockIdx.x, T);
        const int grp = t / (4 * tiles_k), gm = tiles_m - 4 * grp < 4 ? tiles_m - 4 * grp : 4;
        t -= grp * 4 * tiles_k;
        dx_tile<MI>(p, st0, st1, find_slot<Grad<MI>::BM, false>(a.offsets, (int)a.E, a.M, 4 * grp + t % gm, nullptr),
                    (int64_t)(t / gm) * GB_BN);
    } else {
        const int two = a.w1 ? 2 : 1, T = (int)a.E * two * tiles_n * tiles_k, b = blockIdx.x - dx_wgs;
        if (b >= T) return;
        int t = run_of(b, T);
        const int tk = t % tiles_k;
        t /= tiles_k;
        const int tn = t % tiles_n;
        t /= tiles_n;
        dw_tile<MI>(p, st0, st1, t / two, t % two != 0, (int64_t)tn * Grad<MI>::BM, (int64_t)tk * GB_BN);
    }
}

// ---- bias gradients -------------------------------------------------------------------------
// A workgroup takes 64 columns of an expert's rows, 16 rows at a time; sums in fp64 in a fixed order.
__global__ __launch_bounds__(1024) void k_grouped_dbias(Products p) {
    __shared__ double part[16][64];
    const GroupedBackwardArgs& a = p.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n = (int64_t)blockIdx.x * 64 + lane, e = blockIdx.y;
    float* db = blockIdx.z ? a.db1 : a.db0;
    if (!db) return;
    const float* d = (blockIdx.z ? p.d1 : p.d0) + min(n, a.N - 1);
    const Group g = group_rows(a.offsets, e, a.M);
    double sum = 0.0;
#pragma unroll 8
    for (int64_t m = g.lo + wave; m < g.hi; m += 16) sum += (double)d[m * a.N];
    part[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && n < a.N) {
#pragma unroll
        for (int w = 1; w < 16; ++w) sum += part[w][lane];
        db[e * a.N + n] = (float)sum;
    }
}

// Workgroups of both products: dx's, a multiple of the XCDs, and dW's.
struct GradGrid {
    int64_t dx, dw, tiles_k, tiles_n;
};
template <int MI>
static GradGrid grad_grid(int64_t M, int64_t K, int64_t N, int64_t E, bool dx, int projections) {
    GradGrid g;
    g.tiles_k = (K + GB_BN - 1) / GB_BN;
    g.tiles_n = (N + Grad<MI>::BM - 1) / Grad<MI>::BM;
    g.dx = dx && M > 0 ? (most_slots(M, E, Grad<MI>::BM) * g.tiles_k + 7) / 8 * 8 : 0;
    g.dw = E * projections * g.tiles_n * g.tiles_k;
    return g;
}

template <int MI>
static hipError_t launch_gradients(const Products& p, hipStream_t s) {
    const GroupedBackwardArgs& a = p.a;
    const GradGrid g = grad_grid<MI>(a.M, a.K, a.N, a.E, a.dx, a.dw0 ? (a.w1 ? 2 : 1) : 0);
    if (g.dx + g.dw == 0) return hipSuccess;
    return launch_with_lds(k_grouped_gradients<MI>, dim3((unsigned)(g.dx + g.dw)), dim3(512), 0, s, p, (int)g.dx, (int)g.tiles_k, (int)g.tiles_n);
}

bool grouped_backward_fits(int64_t M, int64_t K, int64_t N, int64_t E) {
    const GradGrid g = grad_grid<1>(M, K, N, E, true, 2);
    return grid_fits(g.dx + g.dw, 512);
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
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        p.d0 = dg;
        p.d1 = du;
    }
    const hipError_t e = launch_gradients<2>(p, s);
    if (e != hipSuccess) return e;
    if (a.db0 || a.db1) {
        hipLaunchKernelGGL(k_grouped_dbias, dim3((unsigned)((a.N + 63) / 64), (unsigned)a.E, a.w1 ? 2u : 1u), dim3(1024), 0, s, p);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace bitlinear
