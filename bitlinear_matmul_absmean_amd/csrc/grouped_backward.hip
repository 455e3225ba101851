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

// dg and du, one element a thread at a time.  Bound: the bytes (4096 x 2816: 41 us, 5.6 TB/s).
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
    int parts;                     // of dx's sums
    int slots;                     // most of its tiles of rows
    float* dx;                     // a.dx, or [parts, M, K] where there are several
    bool whole;                    // dW's rows are whole pieces of 64 bytes
};

// ---- the two products -----------------------------------------------------------------------
// A workgroup of eight waves computes 128 x 256 of dx (rows x k) or of a dW (n x k), a wave 32 rows x 128 columns,
// in steps of 64 of the sum.  A stage in LDS is three planes of the split factor, 128 rows of 64 bf16 values, and
// 256 rows (one for each k) of the other; both are loaded from memory into registers two steps ahead, split or
// widened there, turned where the sum runs down the rows, and written in 16-byte units while the stage before
// is multiplied: unit u (8 of the sum) of row r at slot u ^ grad_swizzle(r).  Row of k: column 4 l + j of a
// wave's columns lies in row 32 j + l of theirs, so that a lane ends with
// four neighbouring columns.
// 32x32x16 lane layout: A/B lane l holds row/column l % 32, 8 (l / 32) + j of the sum; accumulator r of lane l is
// row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
// Bound: the matrix cores, three MFMAs a product, and the clock: 4096 rows of 8 experts 2048 -> 2816 gated 520 us, 363
// TFLOP/s (1.09 PFLOP/s in bf16), 50% of cycles with an MFMA at 2.0 GHz; 2816 -> 2048 271 us.  fp32 products of a
// library reach 150.
constexpr int GB_BM = 128, GB_BN = 256, GB_NJ = 4, GB_OB = 3 * GB_BM * 8, GB_UNITS = GB_OB + GB_BN * 8;

// Eight lanes that write the same unit of neighbouring rows (128 bytes a cycle) meet eight different slots;
// sixteen that read it (256 bytes, two rows of a stage) as many pairs of a slot and a row's parity.
__device__ __forceinline__ int grad_swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Loads at base + off: the base (the same for the whole wave) in scalar registers, a lane's 32-bit offset in one
// vector register.  Any alignment of the type's elements.
typedef const __attribute__((address_space(1))) char* global_bytes;
__device__ __forceinline__ global_bytes scalar_base(const void* p) {
    uint64_t b = (uint64_t)p;
    asm("" : "+s"(b));                                 // keeps the sum with the lane's offset out of vector registers
    return (global_bytes)b;
}
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32u __attribute__((aligned(1)));

// Two floats as a dword of each of the three planes: truncation leaves exact remainders.
__device__ __forceinline__ void split_2(float v0, float v1, int at, u32x4 (&pl)[3]) {
    const float v[2] = {v0, v1};
    uint32_t b[2][3];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t h = __float_as_uint(v[e]) & 0xFFFF0000u;
        const float r = v[e] - __uint_as_float(h);
        const uint32_t m = __float_as_uint(r) & 0xFFFF0000u;
        b[e][0] = h;
        b[e][1] = m;
        b[e][2] = __float_as_uint(r - __uint_as_float(m));
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) pl[q][at] = __builtin_amdgcn_perm(b[1][q], b[0][q], 0x07060302u);
}

// The sum of `length` terms in `steps` steps.  load(s, part, j) starts a twelfth of step s on its way into registers (part < 3,
// j < 4), put(st, part, j) writes a twelfth of them to a stage.  A step's four parts of 16 of the sum each read the
// next part's operands, across the turn too, write a third of the next step and start a third of the step after
// it, three parts before it is needed; a quarter of that work goes with the three products of each 32 columns
// (scheduled apart, so that what it holds in registers stays small).  Past the last step the last one is repeated,
// and not used.  FEW: waves whose 32 rows lie past the tile's `rows` form no products (neighbouring waves, on other
// SIMDs, share the rows that there are).
template <bool FEW, typename Load, typename Put>
__device__ __forceinline__ void grad_sum(u32x4* st0, u32x4* st1, int steps, int length, int rows, f32x16 (&acc)[GB_NJ], Load load, Put put) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = wave >> 1, wj = wave & 1, lr = lane & 31, lg = lane >> 5, sw = grad_swizzle(lr);
    // operands of part ks (16 of the sum) of a stage
    struct Planes {
        bf16x8 a[3];
    };
    auto read_a = [&](const u32x4* st, int ks) {
        Planes f;
#pragma unroll
        for (int q = 2; q >= 0; --q) f.a[q] = __builtin_bit_cast(bf16x8, st[(q * GB_BM + 32 * wi + lr) * 8 + ((2 * ks + lg) ^ sw)]);
        return f;
    };
    auto read_b = [&](const u32x4* st, int ks, int j) {
        return __builtin_bit_cast(bf16x8, st[GB_OB + (128 * wj + 32 * j + lr) * 8 + ((2 * ks + lg) ^ sw)]);
    };
    bf16x8 b[GB_NJ];
    if (steps == 0) return;
    const int last = steps - 1;
    // a part's products with planes f, smallest first; the next part's operands (ks of st) take the place of
    // those that are done with
    auto part_of = [&](const Planes& f, const u32x4* st, int ks, auto work) {
#pragma unroll
        for (int j = 0; j < GB_NJ; ++j) {
            work(j);
            if (!FEW || 32 * wi < rows) {
#pragma unroll
                for (int q = 2; q >= 0; --q) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[q], b[j], acc[j], 0, 0, 0);
            }
            b[j] = read_b(st, ks, j);
            // a product and what VALU work falls to it, in turn
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // step s in `cur`, its first operands in f and b, step s + 1 in registers
    auto step = [&](const u32x4* cur, u32x4* nxt, int s, Planes& f) {
        const int after = min(s + 2, last);
        Planes g = read_a(cur, 1);
        part_of(f, cur, 1, [&](int j) { put(nxt, 0, j); });
        f = read_a(cur, 2);
        part_of(g, cur, 2, [&](int j) {
            put(nxt, 1, j);
            load(after, 0, j);
        });
        g = read_a(cur, 3);
        part_of(f, cur, 3, [&](int j) {
            put(nxt, 2, j);
            load(after, 1, j);
        });
        lds_barrier();                 // step s + 1 is whole, and every wave holds the rest of step s in registers
        f = read_a(nxt, 0);
        part_of(g, nxt, 0, [&](int j) { load(after, 2, j); });
    };
#pragma unroll
    for (int i = 0; i < 12; ++i) load(0, i >> 2, i & 3);
#pragma unroll
    for (int i = 0; i < 12; ++i) put(st0, i >> 2, i & 3);
    if (steps == 1) {                  // a short group: only the parts that hold something of the sum
        lds_barrier();
        for (int ks = 0; 16 * ks < length; ++ks) {
            const Planes f = read_a(st0, ks);
#pragma unroll
            for (int j = 0; j < GB_NJ; ++j) {
                b[j] = read_b(st0, ks, j);
#pragma unroll
                for (int q = 2; q >= 0; --q) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[q], b[j], acc[j], 0, 0, 0);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 12; ++i) load(min(1, last), i >> 2, i & 3);
    lds_barrier();
    Planes f = read_a(st0, 0);
#pragma unroll
    for (int j = 0; j < GB_NJ; ++j) b[j] = read_b(st0, 0, j);
    int s = 0;
    for (; s + 2 <= steps; s += 2) {
        step(st0, st1, s, f);
        step(st1, st0, s + 1, f);
    }
    if (s < steps) step(st0, st1, s, f);
}

// Rows m0 .. of the wave's 32 x 128 block, as far as `rows`, and columns from k.  STREAM: past the caches, which
// keeps d, x_q and the codes there (2048 tokens x 2 of 8 experts, 2816 -> 2048: 291 -> 271 us; 256 rows of 16 experts: 97
// -> 82).  dx always; dW, which is most of what is written, where its rows are whole pieces of 64 bytes: others are
// written in parts (256 rows of 16 experts, N = 2048: K = 1008 39.5 against 40.6 us cached, K = 1004 49.5 against 39.2).
// For dx alone the rows' ends hardly matter (N = 2048, past the caches / cached, us): K = 1004, 256 rows of 16 experts 19.9 /
// 19.3, 1024 of 8 29.6 / 29.9, 4096 of 8 67.9 / 69.0; K = 2816 and 2820, 4096 of 8: 141.7 / 142.1 and 143.4 / 143.3.  Parts of
// dx, which the next kernel reads, would gain most from the caches: 122 rows of 5 experts 1024 -> 2731 16.8 / 15.8.
template <bool STREAM>
__device__ __forceinline__ void block_store(float* __restrict__ out, int64_t K, int m0, int rows, int64_t k, const f32x16 (&acc)[GB_NJ]) {
    const int lane = threadIdx.x & 63;
    k += 4 * (lane & 31);
    if (k >= K) return;                                // K is a multiple of 4
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int m = m0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        const f32x4u v = {acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
        if (m < rows) {
            if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<f32x4u*>(out + (int64_t)m * K + k));
            else *reinterpret_cast<f32x4u*>(out + (int64_t)m * K + k) = v;
        }
    }
}

// `rows` rows of a tile of `out` (row length K, columns from k0) from a wave's accumulators.
template <bool STREAM>
__device__ __forceinline__ void grad_store(float* __restrict__ out, int64_t K, int rows, int64_t k0, const f32x16 (&acc)[GB_NJ]) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    block_store<STREAM>(out, K, 32 * (wave >> 1), rows, k0 + 128 * (wave & 1), acc);
}

// LDS row of k 4 c + j of the tile (c a lane, j < 4).
__device__ __forceinline__ int grad_row(int c, int j) { return 128 * (c >> 5) + 32 * j + (c & 31); }

// bf16 values of code j (of a byte's four) of eight rows: from tables of the upper and lower bytes.
__device__ __forceinline__ u32x4 code_values(const uint32_t (&codes)[2], int j) {
    u32x4 o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = (codes[h] >> (2 * j)) & 0x03030303u;
        const uint32_t hi = __builtin_amdgcn_perm(0u, 0x003F00BFu, c), lo = __builtin_amdgcn_perm(0u, 0x00800080u, c);
        o[2 * h] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
        o[2 * h + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
    }
    return o;
}

template <bool SHORT, bool FEW>
__device__ __forceinline__ void dx_tile(const Products& p, u32x4* st0, u32x4* st1, const Slot& slot, int64_t k0, int part) {
    const GroupedBackwardArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t N = a.N, rowb = a.K >> 2, e = slot.e;
    // part `part` of the sum's steps
    const int per = (int)((N + 63) / 64), all = per * (a.w1 ? 2 : 1);
    const int first = (int)((int64_t)all * part / p.parts), steps = (int)((int64_t)all * (part + 1) / p.parts) - first;
    // of d: row tid / 4, two units of 8; of W: rows 8 wave .., the lane's byte of 4 codes
    const int row = tid >> 2, unit = (tid & 3) * 2;
    const uint32_t at = ((uint32_t)min(row, slot.rows - 1) * (uint32_t)N + 8u * unit) * 4u;     // bytes
    const uint32_t byte = (uint32_t)min((k0 >> 2) + lane, rowb - 1);
    // A last part step takes the last 64 n, those that the step before has taken with weights of zero (an
    // element that is not finite has made its row so already); fewer than 64 n in all are guarded one by one.
    float v[2][8], alpha;
    uint32_t w[8];
    int taken;                                         // of the wave's eight n
    auto load = [&](int s, int part, int j) {
        s += first;
        const bool second = s >= per;
        const int64_t begin = (int64_t)(second ? s - per : s) * 64, n0 = SHORT ? 0 : min(begin, N - 64);
        if (part < 2) {
            const float* d = (second ? p.d1 : p.d0) + slot.m0 * N + n0;
            if constexpr (!SHORT) {
                if (j == 1 || j == 3) {
                    const f32x4u x = *(const __attribute__((address_space(1))) f32x4u*)(scalar_base(d) + at + 32 * part + 8 * (j - 1));
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[part][2 * (j - 1) + i] = x[i];
                }
            } else {
#pragma unroll
                for (int i = 2 * j; i < 2 * j + 2; ++i) v[part][i] = 8 * (unit + part) + i < N ? d[at / 4 + 8 * part + i] : 0.0f;
            }
            // (the second part of the step before is written by then)
            if (part == 0 && j == 3) alpha = (second ? a.al1 : a.al0)[e];
        } else {
            const uint8_t* ws = (second ? a.w1 : a.w0) + (e * N + n0) * rowb;
            if (j == 0) taken = (int)(begin - n0) - 8 * wave;
#pragma unroll
            for (int i = 2 * j; i < 2 * j + 2; ++i)
                w[i] = (uint8_t)scalar_base(ws + (SHORT ? min((int64_t)8 * wave + i, N - 1) : 8 * wave + i) * rowb)[byte];
        }
    };
    u32x4 pl[3];
    uint32_t codes[2];                                 // of four n each; 01 is a weight of zero
    auto put = [&](u32x4* st, int part, int j) {
        if (part < 2) {
            split_2(v[part][2 * j] * alpha, v[part][2 * j + 1] * alpha, j, pl);
            if (j == 3) {
#pragma unroll
                for (int q = 0; q < 3; ++q) st[(q * GB_BM + row) * 8 + ((unit + part) ^ grad_swizzle(row))] = pl[q];
            }
            return;
        }
        if (j == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int gone = taken - 4 * h;
                const uint32_t keep = gone >= 4 ? 0u : gone > 0 ? ~0u << 8 * gone : ~0u;
                codes[h] = ((w[4 * h] | w[4 * h + 1] << 8 | w[4 * h + 2] << 16 | w[4 * h + 3] << 24) & keep) | (0x55555555u & ~keep);
            }
        }
        const u32x4 o = code_values(codes, j);
        const int k = grad_row(lane, j);
        st[GB_OB + k * 8 + (wave ^ grad_swizzle(k))] = o;
    };
    f32x16 acc[GB_NJ];
#pragma unroll
    for (int j = 0; j < GB_NJ; ++j) acc[j] = f32x16{};
    grad_sum<FEW>(st0, st1, steps, 64 * steps, slot.rows, acc, load, put);
    grad_store<true>(p.dx + (part * a.M + slot.m0) * a.K, a.K, slot.rows, k0, acc);
}

__device__ __forceinline__ void dw_tile(const Products& p, u32x4* st0, u32x4* st1, int64_t e, bool second, int64_t n0, int64_t k0) {
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
        const int64_t r = *(a.rows ? a.rows + m : a.offsets);      // a load either way: the code has no branches
        return a.rows ? r : m;
    };
    float v[2][8], scale[8];
    uint32_t x[8], beta, live;                         // live: all ones where the row lies in the group and its token is there
    int64_t next = steps ? tokens(0) : 0;              // tokens of the step that is loaded next
    auto load = [&](int s, int part, int j) {
        const bool there = next >= 0 && next < a.T;
        const uint64_t token = there ? (uint64_t)next : 0;
        const int left = rows - 64 * s - 8 * wave;     // of the wave's eight rows
        if (part == 0 && j == 0) {
            beta = __float_as_uint(a.beta[token]);
            live = there && (lane & 7) < left ? ~0u : 0u;
        }
        const uint64_t off = token * (uint64_t)K;
#pragma unroll
        for (int i = 2 * j; i < 2 * j + 2; ++i) {
            if (part < 2) {
                // a buffer for what is left of each row: columns past it, and rows past the group's end, read zeros
                const __amdgpu_buffer_rsrc_t rd = raw_buffer(d + ((int64_t)s * 64 + i) * N, i < left ? width : 0);
                v[part][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rd, 4u * lane + 256u * part, 0, 0));
            } else {
                const uint64_t o = (uint64_t)__builtin_amdgcn_readlane((uint32_t)(off >> 32), i) << 32 |
                                   (uint32_t)__builtin_amdgcn_readlane((uint32_t)off, i);
                x[i] = *(const __attribute__((address_space(1))) u32u*)(scalar_base(a.xq + o) + k);
            }
        }
        if (part == 2 && j == 3) next = tokens(min(s + 1, steps - 1));
    };
    u32x4 pl[3];
    auto put = [&](u32x4* st, int part, int j) {
        if (part < 2) {
            if (part == 0 && j == 0) {
                const float f = __uint_as_float(beta & live) / 127.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) scale[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), i));
            }
            split_2(v[part][2 * j] * scale[2 * j], v[part][2 * j + 1] * scale[2 * j + 1], j, pl);
            if (j == 3) {
                const int c = lane + 64 * part;
#pragma unroll
                for (int q = 0; q < 3; ++q) st[(q * GB_BM + c) * 8 + (wave ^ grad_swizzle(c))] = pl[q];
            }
            return;
        }
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float lo = (float)(int8_t)(x[i] >> (8 * j)), hi = (float)(int8_t)(x[i + 1] >> (8 * j));
            o[i >> 1] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
        }
        const int c = grad_row(lane, j);
        st[GB_OB + c * 8 + (wave ^ grad_swizzle(c))] = o;
    };
    f32x16 acc[GB_NJ];
#pragma unroll
    for (int j = 0; j < GB_NJ; ++j) acc[j] = f32x16{};
    grad_sum<false>(st0, st1, steps, rows, GB_BM, acc, load, put);
    float* out = (second ? a.dw1 : a.dw0) + (e * N + n0) * K;
    const int there = (int)(N - n0 < GB_BM ? N - n0 : GB_BM);
    if (p.whole) grad_store<true>(out, K, there, k0, acc);
    else grad_store<false>(out, K, there, k0, acc);
}

// Bias gradients of 64 columns of an expert: a row a wave at a time, sums in fp64 in a fixed order.
template <int WAVES>
__device__ __forceinline__ void dbias_tile(const Products& p, void* lds, int64_t e, bool second, int64_t n0) {
    const GroupedBackwardArgs& a = p.a;
    float* db = second ? a.db1 : a.db0;
    if (!db) return;
    double* part = reinterpret_cast<double*>(lds);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n = n0 + lane;
    const float* d = (second ? p.d1 : p.d0) + min(n, a.N - 1);
    const Group g = group_rows(a.offsets, e, a.M);
    double sum = 0.0;
#pragma unroll 8
    for (int64_t m = g.lo + wave; m < g.hi; m += WAVES) sum += (double)d[m * a.N];
    part[64 * wave + lane] = sum;
    __syncthreads();
    if (wave != 0 || n >= a.N) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += part[64 * w + lane];
    db[e * a.N + n] = (float)sum;
}

// dx's tiles first (`dx_wgs` of each part at most), whose sums are the longer ones, then dW's, so that the short
// ones fill the card where dx's end; between them `db_wgs` of the bias gradients.  Each XCD gets a contiguous run of dx's tiles and of every expert's tiles of dW
// (whose work goes with the expert's rows).
__global__ __launch_bounds__(512, 2) void k_grouped_gradients(Products p, int dx_wgs, int db_wgs, int tiles_k, int tiles_n) {
    __shared__ u32x4 st0[GB_UNITS];
    __shared__ u32x4 st1[GB_UNITS];
    const GroupedBackwardArgs& a = p.a;
    auto run_of = [](int b, int T) { return (b & 7) * (T >> 3) + ((b & 7) < (T & 7) ? b & 7 : T & 7) + (b >> 3); };
    int b = blockIdx.x;
    if (b < p.parts * dx_wgs) {
        const int part = b / dx_wgs;
        b -= part * dx_wgs;
        int tiles_m;
        find_slot<GB_BM, true>(a.offsets, (int)a.E, a.M, -1, &tiles_m);
        tiles_m = min(tiles_m, p.slots);               // offsets that decrease may make more than were launched
        const int T = tiles_m * tiles_k;
        if (b >= T) return;
        int t = run_of(b, T);
        const int grp = t / (4 * tiles_k), gm = tiles_m - 4 * grp < 4 ? tiles_m - 4 * grp : 4;
        t -= grp * 4 * tiles_k;
        const Slot slot = find_slot<GB_BM, false>(a.offsets, (int)a.E, a.M, 4 * grp + t % gm, nullptr);
        const int64_t k0 = (int64_t)(t / gm) * GB_BN;
        if (a.N < 64) dx_tile<true, true>(p, st0, st1, slot, k0, part);
        else if (slot.rows <= 64) dx_tile<false, true>(p, st0, st1, slot, k0, part);
        else dx_tile<false, false>(p, st0, st1, slot, k0, part);
    } else if (b -= p.parts * dx_wgs; b < db_wgs) {
        const int per = (int)((a.N + 63) / 64), two = a.w1 ? 2 : 1, t = b / per;
        if (t < (int)a.E * two) dbias_tile<8>(p, st0, t / two, t % two != 0, (int64_t)(b % per) * 64);
    } else {
        const int T = (a.w1 ? 2 : 1) * tiles_n * tiles_k, T8 = (T + 7) & ~7;
        b -= db_wgs;
        if (b % T8 >= T) return;
        const int t = run_of(b % T8, T), tn = t / tiles_k % tiles_n;
        dw_tile(p, st0, st1, b / T8, t >= tiles_n * tiles_k, (int64_t)tn * GB_BM, (int64_t)(t % tiles_k) * GB_BN);
    }
}

// ---- short groups ----------------------------------------------------------------------------
// Waves on their own, with operands straight into registers: no stages, no barriers, so that several workgroups share
// a compute unit and many loads and stores are under way at once.  Bound: the bytes of dW (122 rows of 5 experts 1024 ->
// 2731 gated: 112 MB in 27 us, 19 for a fill of as many, behind 9 of dx), a launch where they are few.
//
// dx: a workgroup of four waves takes 32 rows x 128 k and a part of the sum, each wave a quarter of the part's steps
// of 16 n; the quarters are added at the end.  A lane reads eight n of its row of d, and the byte of four k of eight
// rows of codes.  Past the sum's end as in dx_tile.
template <bool NARROW>
__device__ __forceinline__ void dx_short(const Products& p, f32x4* lds, const Slot& slot, int64_t k0, int part) {
    const GroupedBackwardArgs& a = p.a;
    const int lane = threadIdx.x & 63, lr = lane & 31, lg = lane >> 5, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t N = a.N, rowb = a.K >> 2, e = slot.e;
    const int per = (int)((N + 15) / 16), all = per * (a.w1 ? 2 : 1), at = 4 * part + wave;
    const int first = (int)((int64_t)all * at / (4 * p.parts)), end = (int)((int64_t)all * (at + 1) / (4 * p.parts));
    const int64_t row = (slot.m0 + min(lr, slot.rows - 1)) * N, byte = min((k0 >> 2) + lr, rowb - 1);
    const float al[2] = {a.al0[e], a.w1 ? a.al1[e] : 0.0f};
    struct Part {
        float v[8];
        uint32_t w[8];
    };
    auto load = [&](int s) {
        Part f;
        const bool second = s >= per;
        const int64_t begin = (int64_t)(second ? s - per : s) * 16, n0 = (NARROW ? 0 : min(begin, N - 16)) + 8 * lg;
        const float* d = (second ? p.d1 : p.d0) + row + n0;
        const uint8_t* w = (second ? a.w1 : a.w0) + (e * N + n0) * rowb + byte;
        if constexpr (!NARROW) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x4u x = *reinterpret_cast<const f32x4u*>(d + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) f.v[4 * i + j] = x[j];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) f.w[i] = w[i * rowb];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool there = n0 + i < N;
                f.v[i] = there ? d[i] : 0.0f;
                f.w[i] = there ? w[i * rowb] : 0x55u;
            }
        }
        return f;
    };
    f32x16 acc[GB_NJ];
#pragma unroll
    for (int j = 0; j < GB_NJ; ++j) acc[j] = f32x16{};
    auto multiply = [&](const Part& f, int s) {
        const bool second = s >= per;
        const float alpha = second ? al[1] : al[0];
        u32x4 pl[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_2(f.v[2 * i] * alpha, f.v[2 * i + 1] * alpha, i, pl);
        uint32_t codes[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) codes[h] = f.w[4 * h] | f.w[4 * h + 1] << 8 | f.w[4 * h + 2] << 16 | f.w[4 * h + 3] << 24;
        const int64_t begin = (int64_t)(second ? s - per : s) * 16;
        if (!NARROW && begin > N - 16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int gone = (int)(begin - (N - 16)) - 8 * lg - 4 * h;
                const uint32_t keep = gone >= 4 ? 0u : gone > 0 ? ~0u << 8 * gone : ~0u;
                codes[h] = (codes[h] & keep) | (0x55555555u & ~keep);
            }
        }
#pragma unroll
        for (int j = 0; j < GB_NJ; ++j) {
            const u32x4 o = code_values(codes, j);
#pragma unroll
            for (int q = 2; q >= 0; --q)
                acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, pl[q]), __builtin_bit_cast(bf16x8, o), acc[j], 0, 0, 0);
        }
    };
    if (first < end) {
        Part f = load(first);
        for (int s = first; s < end; ++s) {
            const Part next = load(min(s + 1, end - 1));
            multiply(f, s);
            f = next;
        }
    }
    // waves 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                f32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = acc[c >> 2][4 * (c & 3) + i];
                lds[((wave - half) * 16 + c) * 64 + lane] = v;
            }
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const f32x4 v = lds[(wave * 16 + c) * 64 + lane];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c >> 2][4 * (c & 3) + i] += v[i];
            }
        }
        if (half > 1) __syncthreads();
    }
    if (wave == 0) block_store<true>(p.dx + (part * a.M + slot.m0) * a.K, a.K, 0, slot.rows, k0, acc);
}

// dW: a wave computes 32 n x 128 k, sixteen rows at a time: a lane reads its column n of eight rows of d, and four k of
// eight rows of x_q.
__device__ __forceinline__ void dw_short(const Products& p, int64_t e, bool second, int64_t n0, int64_t k0) {
    const GroupedBackwardArgs& a = p.a;
    const int lane = threadIdx.x & 63, lr = lane & 31, lg = lane >> 5;
    const int64_t N = a.N, K = a.K;
    const Group g = group_rows(a.offsets, e, a.M);
    const int rows = g.hi > g.lo ? (int)(g.hi - g.lo) : 0;
    const float* d = (second ? p.d1 : p.d0) + g.lo * N + min(n0 + lr, N - 1);
    const int8_t* x = a.xq + min(k0 + 4 * lr, K - 4);
    f32x16 acc[GB_NJ];
#pragma unroll
    for (int j = 0; j < GB_NJ; ++j) acc[j] = f32x16{};
    for (int m0 = 0; m0 < rows; m0 += 16) {
        float v[8], beta[8];
        uint32_t c[8];
        int64_t token[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = min(m0 + 8 * lg + i, rows - 1);
            token[i] = a.rows ? a.rows[g.lo + m] : g.lo + m;
            v[i] = d[(int64_t)m * N];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool there = token[i] >= 0 && token[i] < a.T;
            const int64_t r = there ? token[i] : 0;
            beta[i] = there && m0 + 8 * lg + i < rows ? a.beta[r] : 0.0f;
            __builtin_memcpy(&c[i], x + r * K, 4);
        }
        u32x4 pl[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_2(v[2 * i] * (beta[2 * i] / 127.0f), v[2 * i + 1] * (beta[2 * i + 1] / 127.0f), i, pl);
#pragma unroll
        for (int j = 0; j < GB_NJ; ++j) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float lo = (float)(int8_t)(c[i] >> (8 * j)), hi = (float)(int8_t)(c[i + 1] >> (8 * j));
                o[i >> 1] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
            }
#pragma unroll
            for (int q = 2; q >= 0; --q)
                acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, pl[q]), __builtin_bit_cast(bf16x8, o), acc[j], 0, 0, 0);
        }
    }
    float* out = (second ? a.dw1 : a.dw0) + (e * N + n0) * K;
    const int there = (int)(N - n0 < 32 ? N - n0 : 32);
    if (p.whole) block_store<true>(out, K, 0, there, k0, acc);
    else block_store<false>(out, K, 0, there, k0, acc);
}

// All gradients of short groups: dx's tiles, the bias gradients, dW's tiles, a tile a wave.
struct ShortGrid {
    int slots, dx, db, tiles_k, tiles_n;               // slots of 32 rows; workgroups of dx (each part) and db
};
__global__ __launch_bounds__(256, 4) void k_grouped_gradients_short(Products p, ShortGrid g) {
    __shared__ f32x4 lds[2048];
    const GroupedBackwardArgs& a = p.a;
    int b = blockIdx.x;
    if (b < p.parts * g.dx) {
        const int part = b / g.dx;
        b -= part * g.dx;
        const Slot slot = find_slot<32, false>(a.offsets, (int)a.E, a.M, b / g.tiles_k, nullptr);
        if (slot.rows == 0) return;
        const int64_t k0 = (int64_t)(b % g.tiles_k) * 128;
        if (a.N < 16) dx_short<true>(p, lds, slot, k0, part);
        else dx_short<false>(p, lds, slot, k0, part);
        return;
    }
    b -= p.parts * g.dx;
    const int two = a.w1 ? 2 : 1;
    if (b < g.db) {
        const int per = (int)((a.N + 63) / 64), t = b / per;
        dbias_tile<4>(p, lds, t / two, t % two != 0, (int64_t)(b % per) * 64);
        return;
    }
    const int64_t per = (int64_t)g.tiles_n * g.tiles_k;
    int64_t t = (int64_t)(b - g.db) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t e = t / (per * two);
    if (e >= a.E) return;
    t -= e * per * two;
    const bool second = t >= per;
    if (second) t -= per;
    dw_short(p, e, second, t / g.tiles_k * 32, t % g.tiles_k * 128);
}

// dx from its parts, in their order (122 x 1024, ten parts: 4 us): a row of a group x 1024 columns a workgroup.
__global__ __launch_bounds__(256) void k_grouped_dx_sum(Products p) {
    const GroupedBackwardArgs& a = p.a;
    const Slot slot = find_slot<1, false>(a.offsets, (int)a.E, a.M, (int)blockIdx.x, nullptr);
    const int64_t k = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4, size = a.M * a.K, at = slot.m0 * a.K + k;
    if (slot.rows == 0 || k >= a.K) return;
    float4 sum = *reinterpret_cast<const float4*>(p.dx + at);
#pragma unroll 8
    for (int q = 1; q < p.parts; ++q) {
        const float4 v = *reinterpret_cast<const float4*>(p.dx + q * size + at);
        sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
    }
    *reinterpret_cast<f32x4u*>(a.dx + at) = f32x4u{sum.x, sum.y, sum.z, sum.w};
}

// Workgroups of both products and the bias gradients: dx's of a part, db and dW's, all but dW's multiples of the XCDs;
// and the parts that dx's sums are cut into where its tiles are too few to fill the card.
struct GradGrid {
    int64_t dx, db, dw, slots, tiles_k, tiles_n, parts;
    bool is_short;
    int64_t all(bool split) const { return (split ? parts : 1) * dx + db + dw; }
};
// Short groups: at most 32 rows an expert, on average (the host does not read the offsets).  Where one expert has all the
// rows, its short sums read x_q again for every 32 n: 2048 rows of 64 experts 2048 -> 1408 519 us, 199 with even groups;
// 4096 of 160 1090 and 561.  Microseconds, the kernel of short groups against tiles of
// 128 x 256:  8 experts 2816 -> 2048: 32 rows 58 / 66, 64 rows 88 / 81;  16 experts 1024 -> 1024: 40 rows 34 / 37, 75
// rows 53 / 43;  8 experts gated 1024 -> 1408: 50 rows 55 / 50;  5 experts gated 1024 -> 2731: 24 rows 44 / 55.
// Parts of dx's sum: about 1024 workgroups, with at least eight steps of 16 n a wave (53 experts 564 -> 230: one part
// 26 us, two and their sum 31;  16 experts gated 2048 -> 2816 of four rows: three parts 171, one 219).
constexpr int64_t SHORT_ROWS = 32, SHORT_WGS = 1024;
static GradGrid grad_grid(int64_t M, int64_t K, int64_t N, int64_t E, int projections, bool dx = true, bool db = true, bool dw = true) {
    GradGrid g;
    g.is_short = M <= SHORT_ROWS * E;
    const int64_t rows = g.is_short ? 32 : GB_BM, columns = g.is_short ? 128 : GB_BN, n = g.is_short ? 32 : GB_BM, of = g.is_short ? 16 : 64;
    g.tiles_k = (K + columns - 1) / columns;
    g.tiles_n = (N + n - 1) / n;
    g.slots = most_slots(M, E, rows);
    const int64_t tiles = g.slots * g.tiles_k, steps = projections * ((N + of - 1) / of);
    g.dx = dx ? (g.is_short ? tiles : (tiles + 7) / 8 * 8) : 0;
    g.db = db ? E * projections * ((N + 63) / 64) : 0;
    g.dw = dw ? E * projections * g.tiles_n * g.tiles_k : 0;
    g.parts = 1;
    if (g.is_short) {
        g.dw = (g.dw + 3) / 4;
        if (tiles > 0 && tiles <= SHORT_WGS / 2) {
            g.parts = SHORT_WGS / tiles;
            if (g.parts > (steps + 31) / 32) g.parts = (steps + 31) / 32;
        }
        return g;
    }
    g.db = (g.db + 7) / 8 * 8;
    g.dw = dw ? E * ((projections * g.tiles_n * g.tiles_k + 7) / 8 * 8) : 0;
    if (tiles > 0 && tiles <= 128) {
        g.parts = 256 / tiles;
        if (g.parts > (steps + 1) / 2) g.parts = (steps + 1) / 2;
    }
    return g;
}

// dg and du of the gated block, then dx's parts.
static size_t gate_bytes(int64_t M, int64_t N, bool gated) { return gated ? ((size_t)M * N * 8 + 255) / 256 * 256 : 0; }
size_t grouped_backward_workspace(int64_t M, int64_t K, int64_t N, int64_t E, bool gated) {
    const GradGrid g = grad_grid(M, K, N, E, gated ? 2 : 1);
    return 256 + gate_bytes(M, N, gated) + (g.parts > 1 ? (size_t)g.parts * M * K * 4 : 0);
}

bool grouped_backward_fits(int64_t M, int64_t K, int64_t N, int64_t E) {
    const GradGrid g = grad_grid(M, K, N, E, 2);
    return grid_fits(g.all(true), g.is_short ? 256 : 512);
}

hipError_t launch_grouped_backward(const GroupedBackwardArgs& a, hipStream_t s) {
    Products p{a, a.dy, nullptr, 1, (int)most_slots(a.M, a.E, GB_BM), a.dx,
               a.K % 16 == 0 && ((uintptr_t)a.dw0 | (uintptr_t)a.dw1) % 64 == 0};
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
    const GradGrid g = grad_grid(a.M, a.K, a.N, a.E, a.w1 ? 2 : 1, a.dx && a.M > 0, a.db0 || a.db1, a.dw0);
    if (a.dx && g.parts > 1) {
        p.parts = (int)g.parts;
        p.dx = reinterpret_cast<float*>(static_cast<char*>(a.ws) + gate_bytes(a.M, a.N, a.w1));
    }
    const int64_t wgs = g.all(p.parts > 1);
    if (wgs > 0) {
        const dim3 grid((unsigned)wgs);
        if (g.is_short)
            hipLaunchKernelGGL(k_grouped_gradients_short, grid, dim3(256), 0, s, p,
                               ShortGrid{(int)g.slots, (int)g.dx, (int)g.db, (int)g.tiles_k, (int)g.tiles_n});
        else
            hipLaunchKernelGGL(k_grouped_gradients, grid, dim3(512), 0, s, p, (int)g.dx, (int)g.db, (int)g.tiles_k, (int)g.tiles_n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (p.parts > 1) {
        hipLaunchKernelGGL(k_grouped_dx_sum, dim3((unsigned)most_slots(a.M, a.E, 1), (unsigned)((a.K + 1023) / 1024)), dim3(256), 0, s, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace bitlinear
