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
// A workgroup of eight waves computes BM x 256 of dx (rows x k) or of a dW (n x k), a wave 32 rows x 32 NJ columns,
// in steps of 64 of the sum.  A stage in LDS is three planes of the split factor, BM rows of 64 bf16 values, and
// 256 rows (one for each k) of the other; both are loaded from memory into registers two steps ahead, split or
// widened there, turned where the sum runs down the rows, and written in 16-byte units while the stage before
// is multiplied: unit u (8 of the sum) of row r at slot u ^ ((r / 2) % 8), which spreads reads and writes over all
// banks.  Row of k: column NJ l + j of a wave's columns lies in row 32 j + l of theirs, so that a lane ends with
// NJ neighbouring columns.
// 32x32x16 lane layout: A/B lane l holds row/column l % 32, 8 (l / 32) + j of the sum; accumulator r of lane l is
// row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
constexpr int GB_BN = 256;

template <int BM>
struct Grad {
    static constexpr int WM = BM / 32, NJ = WM, OB = 3 * BM * 8, UNITS = OB + GB_BN * 8;   // 8 / WM waves along k
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

// The sum over `steps` steps: load(r, s) starts step s on its way into registers r, put(r, st, part) writes a
// quarter of them to a stage.  Step s is multiplied while step s + 1 goes from registers to the other stage and
// step s + 2 is on its way from memory; past the last step the last one is repeated, and not read.
template <int BM, typename Regs, typename Load, typename Put>
__device__ __forceinline__ void grad_sum(u32x4* st0, u32x4* st1, int steps, f32x16 (&acc)[Grad<BM>::NJ], Load load, Put put) {
    constexpr int WM = Grad<BM>::WM, NJ = Grad<BM>::NJ, OB = Grad<BM>::OB;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = wave % WM, wj = wave / WM, lr = lane & 31, lg = lane >> 5, sw = (lr >> 1) & 7;
    struct Frag {
        bf16x8 a[3], b[NJ];
    };
    auto read = [&](const u32x4* st, int ks) {
        const int at = (2 * ks + lg) ^ sw;
        Frag f;
#pragma unroll
        for (int q = 2; q >= 0; --q) f.a[q] = __builtin_bit_cast(bf16x8, st[(q * BM + 32 * wi + lr) * 8 + at]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) f.b[j] = __builtin_bit_cast(bf16x8, st[OB + (32 * NJ * wj + 32 * j + lr) * 8 + at]);
        return f;
    };
    auto multiply = [&](const Frag& f) {
#pragma unroll
        for (int q = 2; q >= 0; --q)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[q], f.b[j], acc[j], 0, 0, 0);
    };
    if (steps == 0) return;
    const int last = steps - 1;
    // step s in `cur`, step s + 1 in registers r
    auto step = [&](const u32x4* cur, u32x4* nxt, const Regs& r) {
        Frag f = read(cur, 0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            Frag g;
            if (ks < 3) g = read(cur, ks + 1);
            put(r, nxt, ks);
            multiply(f);
            // reads first, then a product and what VALU work of the quarter falls to it, in turn
            __builtin_amdgcn_sched_group_barrier(0x100, 3 + NJ, 0);
#pragma unroll
            for (int i = 0; i < 3 * NJ; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x200, 3, 0);
            __builtin_amdgcn_sched_barrier(0);
            f = g;
        }
        lds_barrier();
    };
    Regs r0, r1;
    load(r0, 0);
    load(r1, min(1, last));
#pragma unroll
    for (int q = 0; q < 4; ++q) put(r0, st0, q);
    lds_barrier();
    for (int s = 0; s < steps; s += 2) {
        load(r0, min(s + 2, last));
        step(st0, st1, r1);
        if (s + 1 >= steps) break;
        load(r1, min(s + 3, last));
        step(st1, st0, r0);
    }
}

// `rows` rows of a tile of `out` (row length K, columns from k0) from a wave's accumulators.
template <int BM>
__device__ __forceinline__ void grad_store(float* __restrict__ out, int64_t K, int rows, int64_t k0, const f32x16 (&acc)[Grad<BM>::NJ]) {
    constexpr int WM = Grad<BM>::WM, NJ = Grad<BM>::NJ;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t k = k0 + 32 * NJ * (wave / WM) + NJ * (lane & 31);
    if (k >= K) return;                                // K is a multiple of 4
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int m = 32 * (wave % WM) + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        float v[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) v[j] = acc[j][r];
        if (m < rows) __builtin_memcpy(out + (int64_t)m * K + k, v, 4 * NJ);
    }
}

// LDS row of k 4 c + j of the tile (c a lane, j < 4).
template <int BM>
__device__ __forceinline__ int grad_row(int c, int j) {
    if constexpr (Grad<BM>::NJ == 4) return 128 * (c >> 5) + 32 * j + (c & 31);
    else return 64 * (c >> 4) + 32 * (j & 1) + 2 * (c & 15) + (j >> 1);
}

template <int BM>
__device__ __forceinline__ void dx_tile(const Products& p, u32x4* st0, u32x4* st1, const Slot& slot, int64_t k0) {
    constexpr int OB = Grad<BM>::OB, UN = BM / 64;     // units of a plane that a thread forms
    const GroupedBackwardArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t N = a.N, rowb = a.K >> 2, e = slot.e;
    const int per = (int)((N + 63) / 64), steps = per * (a.w1 ? 2 : 1);
    // of d: row tid / (8 / UN), UN units of 8; of W: rows 8 wave .., the lane's byte of 4 codes
    const int row = tid / (8 / UN), unit = (tid % (8 / UN)) * UN;
    const int64_t at = (slot.m0 + min(row, slot.rows - 1)) * N + 8 * unit;
    const uint32_t byte = (uint32_t)min((k0 >> 2) + lane, rowb - 1);
    struct Regs {
        float v[UN][8], alpha;
        uint32_t w[8];
    };
    auto load = [&](Regs& r, int s) {
        const bool second = s >= per;
        const int64_t n0 = (int64_t)(second ? s - per : s) * 64;
        const float* d = (second ? p.d1 : p.d0) + at + n0;
        const uint8_t* w = (second ? a.w1 : a.w0) + (e * N + n0 + 8 * wave) * rowb;
        r.alpha = (second ? a.al1 : a.al0)[e];
        if (n0 + 64 <= N) {
#pragma unroll
            for (int i = 0; i < UN; ++i) __builtin_memcpy(r.v[i], d + 8 * i, 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) r.w[i] = (w + i * rowb)[byte];
        } else {
            const int left = (int)(N - n0);
#pragma unroll
            for (int i = 0; i < UN; ++i)
#pragma unroll
                for (int x = 0; x < 8; ++x) r.v[i][x] = 8 * (unit + i) + x < left ? d[8 * i + x] : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) r.w[i] = (w + (min(8 * wave + i, left - 1) - 8 * wave) * rowb)[byte];
        }
    };
    auto put = [&](const Regs& r, u32x4* st, int part) {
        if (part < UN) {
            float t[8];
            u32x4 pl[3];
#pragma unroll
            for (int x = 0; x < 8; ++x) t[x] = r.v[part][x] * r.alpha;
            split_unit(t, pl);
#pragma unroll
            for (int q = 0; q < 3; ++q) st[(q * BM + row) * 8 + ((unit + part) ^ ((row >> 1) & 7))] = pl[q];
        }
        if (part < 2) return;
        // codes of four n a dword; for each k their bf16 values from tables of the upper and lower bytes
        const uint32_t c0 = r.w[0] | r.w[1] << 8 | r.w[2] << 16 | r.w[3] << 24, c1 = r.w[4] | r.w[5] << 8 | r.w[6] << 16 | r.w[7] << 24;
#pragma unroll
        for (int j = 2 * part - 4; j < 2 * part - 2; ++j) {
            u32x4 o;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t c = ((h ? c1 : c0) >> (2 * j)) & 0x03030303u;
                const uint32_t hi = __builtin_amdgcn_perm(0u, 0x003F00BFu, c), lo = __builtin_amdgcn_perm(0u, 0x00800080u, c);
                o[2 * h] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
                o[2 * h + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
            }
            const int k = grad_row<BM>(lane, j);
            st[OB + k * 8 + (wave ^ ((k >> 1) & 7))] = o;
        }
    };
    f32x16 acc[Grad<BM>::NJ];
#pragma unroll
    for (int j = 0; j < Grad<BM>::NJ; ++j) acc[j] = f32x16{};
    grad_sum<BM, Regs>(st0, st1, steps, acc, load, put);
    grad_store<BM>(a.dx + slot.m0 * a.K, a.K, slot.rows, k0, acc);
}

template <int BM>
__device__ __forceinline__ void dw_tile(const Products& p, u32x4* st0, u32x4* st1, int64_t e, bool second, int64_t n0, int64_t k0) {
    constexpr int OB = Grad<BM>::OB, UN = BM / 64;     // columns of d of a lane
    const GroupedBackwardArgs& a = p.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t N = a.N, K = a.K;
    const Group g = group_rows(a.offsets, e, a.M);
    const int rows = g.hi > g.lo ? (int)(g.hi - g.lo) : 0, steps = (rows + 63) / 64;
    const float* d = (second ? p.d1 : p.d0) + (g.lo + 8 * wave) * N + n0;
    const uint32_t width = (uint32_t)(N - n0) * 4;
    // the wave takes rows 8 wave .. of a step, a lane columns lane and lane + 64 of d and four of x_q
    const uint32_t k = (uint32_t)min(k0 + 4 * lane, K - 4);
    // tokens of rows lane % 8 of the wave's rows of a step (of the last row past the end)
    auto tokens = [&](int s) {
        const int64_t m = g.lo + min(64 * s + 8 * wave + (lane & 7), rows - 1);
        return a.rows ? a.rows[m] : m;
    };
    struct Regs {
        float v[UN][8], beta;
        uint32_t x[8];
        bool live;                                     // the row lies in the group, its token is there
    };
    int64_t next = steps ? tokens(0) : 0;              // tokens of the step that is loaded next
    auto load = [&](Regs& r, int s) {
        const bool there = next >= 0 && next < a.T;
        const uint64_t token = there ? (uint64_t)next : 0, off = token * (uint64_t)K;
        r.beta = a.beta[token];
        r.live = there && 64 * s + 8 * wave + (lane & 7) < rows;
        const float* ds = d + (int64_t)s * 64 * N;
        const int left = rows - 64 * s - 8 * wave;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // a buffer for what is left of each row: columns past it, and rows past the group's end, read zeros
            const __amdgpu_buffer_rsrc_t rd = raw_buffer(ds + i * N, i < left ? width : 0);
#pragma unroll
            for (int c = 0; c < UN; ++c)
                r.v[c][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rd, 4u * lane + 256u * c, 0, 0));
            const uint64_t o = (uint64_t)__builtin_amdgcn_readlane((uint32_t)(off >> 32), i) << 32 |
                               (uint32_t)__builtin_amdgcn_readlane((uint32_t)off, i);
            __builtin_memcpy(&r.x[i], a.xq + o + k, 4);
        }
        next = tokens(min(s + 1, steps - 1));
    };
    auto put = [&](const Regs& r, u32x4* st, int part) {
        if (part < UN) {
            const float f = r.live ? r.beta / 127.0f : 0.0f;
            float t[8];
            u32x4 pl[3];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = r.v[part][i] * __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), i));
            split_unit(t, pl);
            const int c = lane + 64 * part;
#pragma unroll
            for (int q = 0; q < 3; ++q) st[(q * BM + c) * 8 + (wave ^ ((c >> 1) & 7))] = pl[q];
        }
        if (part < 2) return;
#pragma unroll
        for (int j = 2 * part - 4; j < 2 * part - 2; ++j) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float lo = (float)(int8_t)(r.x[i] >> (8 * j)), hi = (float)(int8_t)(r.x[i + 1] >> (8 * j));
                o[i >> 1] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
            }
            const int c = grad_row<BM>(lane, j);
            st[OB + c * 8 + (wave ^ ((c >> 1) & 7))] = o;
        }
    };
    f32x16 acc[Grad<BM>::NJ];
#pragma unroll
    for (int j = 0; j < Grad<BM>::NJ; ++j) acc[j] = f32x16{};
    grad_sum<BM, Regs>(st0, st1, steps, acc, load, put);
    grad_store<BM>((second ? a.dw1 : a.dw0) + (e * N + n0) * K, K, (int)(N - n0 < BM ? N - n0 : BM), k0, acc);
}

// dx's tiles first (`dx_wgs` at most), whose sums are the longer ones, then dW's, so that the short ones fill the
// card where dx's end.  Each XCD gets a contiguous run of dx's tiles and of every expert's tiles of dW (whose work
// goes with the expert's rows).
template <int BM>
__global__ __launch_bounds__(512, 2) void k_grouped_gradients(Products p, int dx_wgs, int tiles_k, int tiles_n) {
    __shared__ u32x4 st0[Grad<BM>::UNITS];
    __shared__ u32x4 st1[Grad<BM>::UNITS];
    const GroupedBackwardArgs& a = p.a;
    auto run_of = [](int b, int T) { return (b & 7) * (T >> 3) + ((b & 7) < (T & 7) ? b & 7 : T & 7) + (b >> 3); };
    if ((int)blockIdx.x < dx_wgs) {
        int tiles_m;
        find_slot<BM, true>(a.offsets, (int)a.E, a.M, -1, &tiles_m);
        const int T = tiles_m * tiles_k;
        if ((int)blockIdx.x >= T) return;
        int t = run_of(blockIdx.x, T);
        const int grp = t / (4 * tiles_k), gm = tiles_m - 4 * grp < 4 ? tiles_m - 4 * grp : 4;
        t -= grp * 4 * tiles_k;
        dx_tile<BM>(p, st0, st1, find_slot<BM, false>(a.offsets, (int)a.E, a.M, 4 * grp + t % gm, nullptr), (int64_t)(t / gm) * GB_BN);
    } else {
        const int T = (a.w1 ? 2 : 1) * tiles_n * tiles_k, T8 = (T + 7) & ~7, b = blockIdx.x - dx_wgs;
        if (b % T8 >= T) return;
        const int t = run_of(b % T8, T), tn = t / tiles_k % tiles_n;
        dw_tile<BM>(p, st0, st1, b / T8, t >= tiles_n * tiles_k, (int64_t)tn * BM, (int64_t)(t % tiles_k) * GB_BN);
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
template <int BM>
static GradGrid grad_grid(int64_t M, int64_t K, int64_t N, int64_t E, bool dx, int projections) {
    GradGrid g;
    g.tiles_k = (K + GB_BN - 1) / GB_BN;
    g.tiles_n = (N + BM - 1) / BM;
    g.dx = dx && M > 0 ? (most_slots(M, E, BM) * g.tiles_k + 7) / 8 * 8 : 0;
    g.dw = E * ((projections * g.tiles_n * g.tiles_k + 7) / 8 * 8);
    return g;
}

template <int BM>
static hipError_t launch_gradients(const Products& p, hipStream_t s) {
    const GroupedBackwardArgs& a = p.a;
    const GradGrid g = grad_grid<BM>(a.M, a.K, a.N, a.E, a.dx, a.dw0 ? (a.w1 ? 2 : 1) : 0);
    if (g.dx + g.dw == 0) return hipSuccess;
    return launch_with_lds(k_grouped_gradients<BM>, dim3((unsigned)(g.dx + g.dw)), dim3(512), 0, s, p, (int)g.dx, (int)g.tiles_k, (int)g.tiles_n);
}

bool grouped_backward_fits(int64_t M, int64_t K, int64_t N, int64_t E) {
    const GradGrid g = grad_grid<64>(M, K, N, E, true, 2);
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
    const hipError_t e = launch_gradients<128>(p, s);
    if (e != hipSuccess) return e;
    if (a.db0 || a.db1) {
        hipLaunchKernelGGL(k_grouped_dbias, dim3((unsigned)((a.N + 63) / 64), (unsigned)a.E, a.w1 ? 2u : 1u), dim3(1024), 0, s, p);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace bitlinear
