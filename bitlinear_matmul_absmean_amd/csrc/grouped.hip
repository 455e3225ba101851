// grouped.hip -- ternary BitLinears grouped by expert, one projection or a gated block, gfx950.
//
// What is computed: rows sorted by expert, row m of group e reading token r = rows[m]:
//     acc[m, n] = sum_k x_q[r, k] W_e[n, k]                                   (int32, exact)
//     y[m, n]   = fp32(acc) * fp32(alpha_e beta[r] / 127)  (+ bias_e[n])
// and for the gated block h = a(gate) up of two such projections (one fp32 rounding).
//
// A group is cut into slots of a tile's rows; the host, which does not know the offsets, launches as many
// workgroups as there can be slots, and each finds its own from the offsets.  A workgroup multiplies its rows
// with two sets of weight rows: the gate and up rows of the same columns, whose product is then formed where
// the sums end, or two neighbouring sets of columns of the one projection.  Two kernels:
//   * few rows an expert: k_grouped_dec, the weight streams on the 16x16x64 int8 MFMA, for any K % 4 == 0 and any
//     alignment;
//   * else: k_grouped_gemm, LDS tiles on the 32x32x32 int8 MFMA, in a form for aligned rows (16-byte aligned
//     tensors, K % 64 == 0, T K < 2^32) and one for any.
#include <type_traits>

#include "experts.hpp"
#include "ffn.hpp"

namespace bitlinear {

static int64_t most_slots(const GroupedArgs& a, int64_t tile) { return most_slots(a.M, a.E, tile); }

// The GEMM's smallest tiles, 32 rows x 128 columns of 256 threads (the streaming kernel is taken for few).
bool grouped_fits(int64_t M, int64_t N, int64_t E) { return grid_fits(most_slots(M, E, 32) * ((N + 127) / 128), 256); }

// Element `at` (m N + n) of the gated block from its two sums.
template <int ACT>
__device__ __forceinline__ void gate_store(const GroupedArgs& a, int64_t at, float g, float u) {
    a.y[at] = act_value<ACT>(g) * u;
    if (a.g) {
        a.g[at] = g;
        a.u[at] = u;
    }
}

// ---- few rows an expert ---------------------------------------------------------------------
// A workgroup of WAVES waves computes 16 rows x 16 columns of both sets; wave w takes the steps of 256 k w, w + WAVES,
// ..., and the partial tiles are added at the end (integers: exact in any order).  In MFMA q of a step lane group g
// (lanes 16 g ..) holds weights 64 g + 16 q .. 64 g + 16 q + 15, dword q of the lane's 16 bytes of codes, expanded
// in weight order to signed bytes.  Operands go straight into registers, a step ahead; the first weights are on
// their way before the rows' tokens are known.
// 16x16x64 lane layout: A/B lane l holds row/column l % 16, k = 16 (l / 16) + j; accumulator r of
// lane l is row 4 (l / 16) + r, column l % 16.
// Bound: a chain of loads (offsets, tokens, x_q and beta) and one or two rounds of workgroups beside the weight stream:
// 64 rows of 16 experts 2816 -> 2048 7.8 us, 3.0 TB/s; one load of x_q a step for slots of up to four rows won half a microsecond there and lost as
// much at sixteen rows.
template <bool GATED, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_grouped_dec(GroupedArgs a, int slots) {
    __shared__ i32x4 part[WAVES * 2 * 64];
    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Slot slot = find_slot<16, false>(a.offsets, (int)a.E, a.M, (int)(blockIdx.x % slots), nullptr);
    const int rows_m = slot.rows;
    if (rows_m == 0) return;
    const int64_t K = a.K, rowb = K >> 2, e = slot.e, m0 = slot.m0;
    const int64_t n0 = (int64_t)(blockIdx.x / slots) * (GATED ? 16 : 32);
    // columns of the second set: up's, or the next 16 (which may lie past the end: then the first's again)
    const int rows_n = (int)(a.N - n0 < 16 ? a.N - n0 : 16);
    const int64_t n1 = GATED ? n0 : n0 + 16;
    const int rows_n1 = GATED ? rows_n : (int)(a.N - n1 < 0 ? 0 : a.N - n1 < 16 ? a.N - n1 : 16);
    const uint8_t* w0 = a.w0 + (e * a.N + n0) * rowb;
    const uint8_t* w1 = GATED ? a.w1 + (e * a.N + n0) * rowb : rows_n1 ? w0 + 16 * rowb : w0;
    const uint8_t *wp[2] = {w0 + (int64_t)min(lr, rows_n - 1) * rowb, w1 + (int64_t)min(lr, (rows_n1 ? rows_n1 : rows_n) - 1) * rowb};
    const int whole = (int)(K / 256);
    struct Part {
        i32x4 x[4];
        u32x4 w[2];
    };
    auto load_w = [&](Part& f, int s) {
#pragma unroll
        for (int p = 0; p < 2; ++p) f.w[p] = load_16(wp[p] + (int64_t)s * 64 + 16 * lg);
    };
    Part f;
    if (wave < whole) load_w(f, wave);
    // the lane's row lr (the last one past the end), its token, and beta: 0 for a token that is not there
    const int64_t r = row_token(a.rows, m0 + min(lr, rows_m - 1), a.T);
    const uint8_t* x = reinterpret_cast<const uint8_t*>(a.xq) + (r < 0 ? 0 : r) * K;
    const float beta = r < 0 ? 0.0f : a.beta[r];
    auto load_x = [&](Part& f, int s) {
#pragma unroll
        for (int q = 0; q < 4; ++q) f.x[q] = (i32x4)load_16(x + (int64_t)s * 256 + 64 * lg + 16 * q);
    };
    i32x4 acc[2] = {i32x4{0, 0, 0, 0}, i32x4{0, 0, 0, 0}};
    auto multiply = [&](const Part& f) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int p = 0; p < 2; ++p) acc[p] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.x[q], expand_signed_in_order(f.w[p][q]), acc[p], 0, 0, 0);
    };
    if (wave < whole) {
        load_x(f, wave);
        for (int s = wave; s < whole; s += WAVES) {
            Part next;
            load_w(next, min(s + WAVES, whole - 1));
            load_x(next, min(s + WAVES, whole - 1));
            multiply(f);
            f = next;
        }
    }
    if (K % 256 && whole % WAVES == wave) {                      // the last part step, to the next wave in turn
        const int64_t k = (int64_t)whole * 256 + 64 * lg;
#pragma unroll
        for (int p = 0; p < 2; ++p) f.w[p] = row_16(wp[p], k >> 2, rowb);
#pragma unroll
        for (int q = 0; q < 4; ++q) f.x[q] = (i32x4)row_16(x, k + 16 * q, K);
        multiply(f);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) part[(wave * 2 + p) * 64 + lane] = acc[p];
    __syncthreads();
    if (wave >= 4) return;
    // wave i takes element i of every lane: row 4 (l / 16) + i, column l % 16, of both sets
    const int i = wave, n = lr, m = 4 * lg + i;
    const float b = __shfl(beta, m, 64);
    // the sums of a token that is not there are those of zeros (a scale of zero alone would leave them their sign)
    const int some = (int)((uint32_t)__ballot(r < 0) >> m & 1) - 1;
    int s0 = 0, s1 = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const int* p = reinterpret_cast<const int*>(part + w * 2 * 64 + lane);
        s0 += p[i];
        s1 += p[i + 256];
    }
    s0 &= some;
    s1 &= some;
    if (m >= rows_m) return;
    const int64_t at = (m0 + m) * a.N + n0 + n, bn = e * a.N + n0 + n;
    float v0 = (float)s0 * dequant_scale(a.al0[e], b);
    if constexpr (GATED) {
        if (n >= rows_n) return;
        float v1 = (float)s1 * dequant_scale(a.al1[e], b);
        if (a.b0) v0 = v0 + a.b0[bn];
        if (a.b1) v1 = v1 + a.b1[bn];
        if (a.act == BITLINEAR_ACT_SILU) gate_store<BITLINEAR_ACT_SILU>(a, at, v0, v1);
        else if (a.act == BITLINEAR_ACT_GELU) gate_store<BITLINEAR_ACT_GELU>(a, at, v0, v1);
        else gate_store<BITLINEAR_ACT_RELU2>(a, at, v0, v1);
    } else {
        const float v1 = (float)s1 * dequant_scale(a.al0[e], b);
        if (n < rows_n) a.y[at] = a.b0 ? v0 + a.b0[bn] : v0;
        if (n < rows_n1) a.y[at + 16] = a.b0 ? v1 + a.b0[bn + 16] : v1;
    }
}

template <bool GATED, int WAVES>
static hipError_t launch_grouped_dec(const GroupedArgs& a, hipStream_t s) {
    const int64_t slots = most_slots(a, 16), blocks = (a.N + (GATED ? 15 : 31)) / (GATED ? 16 : 32);
    hipLaunchKernelGGL((k_grouped_dec<GATED, WAVES>), dim3((unsigned)(slots * blocks)), dim3(64 * WAVES), 0, s, a, (int)slots);
    return hipGetLastError();
}

// ---- many rows an expert --------------------------------------------------------------------
// A workgroup of four waves computes 32 FM rows x 128 columns of both sets, a wave all the rows x 32 columns of
// each: FM 32-row operands against one weight operand of each set, so that the expansion of a weight operand
// (17 instructions) serves FM MFMAs.  Steps of 128 k, three LDS stages (4 FM + 8 KiB each: 32 FM rows of x_q of
// 128 bytes, 256 weight rows of 32 bytes) filled two steps ahead by loads that go past the registers (aligned
// rows), or two filled through registers.  Unit u of x_q's row r lies at slot u ^ ((r / 2) % 8), unit u
// of weight row r at slot u ^ ((r / 8) % 2), so that an operand read spreads over all banks.
// In the two MFMAs of k 64 h .. 64 h + 63 (h = 0, 1) a lane group holds 32 codes, eight bytes of a
// weight row: the lane's unit h, of which group lg uses dwords 2 lg and 2 lg + 1.
// Bound: VALU instructions, 15 for each MFMA with FM = 2 (8.5 of the expansion, 5 of the gated epilogue at K = 2048):
// 8192 rows of 16 experts 2048 -> 2816 gated 126 us, 1.5 PFLOP/s in int8, 68% of cycles in VALU and 38% in MFMA.  FM = 4
// halves the expansion, but its 180 registers leave two workgroups a compute unit in place of three, and more of a tile's
// rows are empty: with the quantizer 137 us against 130.
constexpr int EG_BF = 128, EG_BK = 128;

// ACT 0: one projection, whose columns n0 + 128 .. are the second set.
template <int ACT, bool ALIGNED, int FM>
__global__ __launch_bounds__(256, 2) void k_grouped_gemm(GroupedArgs a, int most_m, int tiles_f) {
    constexpr bool GATED = ACT != 0;
    constexpr int BM = 32 * FM, OB = BM * 8, UNITS = OB + 2 * EG_BF * 2;
    __shared__ i32x4 st0[UNITS];
    __shared__ i32x4 st1[UNITS];
    __shared__ i32x4 st2[ALIGNED ? UNITS : 1];
    __shared__ __align__(16) float scale[3][BM];       // of the two sets; and what is added to a row's sums
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // of the tiles there are, a contiguous run for each XCD, four rows of tiles at a time
    int tiles_m;
    find_slot<BM, true>(a.offsets, (int)a.E, a.M, -1, &tiles_m);
    tiles_m = min(tiles_m, most_m);                    // offsets that decrease may make more than were launched
    const int T = tiles_m * tiles_f, xcd = blockIdx.x & 7, per = T >> 3, rem = T & 7;
    if ((int)blockIdx.x >= T) return;
    int t = xcd * per + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
    const int grp = t / (4 * tiles_f), gm = tiles_m - 4 * grp < 4 ? tiles_m - 4 * grp : 4;
    t -= grp * 4 * tiles_f;
    const Slot slot = find_slot<BM, false>(a.offsets, (int)a.E, a.M, 4 * grp + t % gm, nullptr);
    const int rows_m = slot.rows;
    const int64_t m0 = slot.m0, e = slot.e, n0 = (int64_t)(t / gm) * (GATED ? EG_BF : 2 * EG_BF);
    const int64_t K = a.K, rowb = K >> 2;
    const int rows_n = (int)(a.N - n0 < EG_BF ? a.N - n0 : EG_BF);
    const int64_t n1 = GATED ? n0 : n0 + EG_BF;
    const int rows_n1 = GATED ? rows_n : (int)(a.N - n1 < 0 ? 0 : a.N - n1 < EG_BF ? a.N - n1 : EG_BF);
    const uint8_t* w0 = a.w0 + (e * a.N + n0) * rowb;
    const uint8_t* w1 = GATED ? a.w1 + (e * a.N + n0) * rowb : rows_n1 ? w0 + EG_BF * rowb : w0;
    const int last_n = rows_n - 1, last_n1 = rows_n1 ? rows_n1 - 1 : rows_n - 1;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(a.xq);
    // token of row r of the tile (the last row's past the end; 0 for one that is not there)
    auto token = [&](int r) {
        const int64_t v = row_token(a.rows, m0 + min(r, rows_m - 1), a.T);
        return v < 0 ? (int64_t)0 : v;
    };
    if (tid < BM) {
        const int64_t r = row_token(a.rows, m0 + min(tid, rows_m - 1), a.T);
        const float beta = r < 0 ? 0.0f : a.beta[r];
        // A token that is not there is one of zeros, but token 0 is read for it: times a scale of zero its sums keep their
        // sign, which adding 0 takes away.  Adding -0 changes nothing.
        scale[2][tid] = r < 0 ? 0.0f : -0.0f;
        scale[0][tid] = dequant_scale(a.al0[e], beta);
        if (GATED) scale[1][tid] = dequant_scale(a.al1[e], beta);
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
            // weight rows of a stage: 128 of the first set, then 128 of the second
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
    // load block q of x_q: rows 8 q .. 8 q + 7 (wave w takes FM w .. FM w + FM - 1); of a set: rows 32 q .. 32 q
    // + 31 (wave w takes q = w of both)
    const int wrow = 32 * wave + (lane >> 1), wunit = (lane & 1) ^ ((wrow >> 3) & 1);
    auto xrow = [&](int q) { return 8 * (FM * wave + q) + (lane >> 3); };
    auto xunit = [&](int q) { return (lane & 7) ^ ((xrow(q) >> 1) & 7); };
    if constexpr (ALIGNED) {
        const __amdgpu_buffer_rsrc_t rx = raw_buffer(x, (uint32_t)(a.T * K));
        const __amdgpu_buffer_rsrc_t r0 = raw_buffer(w0, (uint32_t)rows_n * (uint32_t)rowb);
        const __amdgpu_buffer_rsrc_t r1 = raw_buffer(w1, (uint32_t)(last_n1 + 1) * (uint32_t)rowb);
        uint32_t xo[FM];
#pragma unroll
        for (int q = 0; q < FM; ++q) xo[q] = (uint32_t)token(xrow(q)) * (uint32_t)K + 16u * xunit(q);
        const uint32_t o0 = (uint32_t)min(wrow, last_n) * (uint32_t)rowb + 16u * wunit;
        const uint32_t o1 = (uint32_t)min(wrow, last_n1) * (uint32_t)rowb + 16u * wunit;
        const int steps = (int)(K / EG_BK), last = steps - 1;
        auto fetch = [&](i32x4* st, int s) {
            s = s < last ? s : last;
#pragma unroll
            for (int q = 0; q < FM; ++q) load_lds16(rx, xo[q], (uint32_t)s * EG_BK, st + 64 * (FM * wave + q));
            load_lds16(r0, o0, (uint32_t)s * (EG_BK / 4), st + OB + 64 * wave);
            load_lds16(r1, o1, (uint32_t)s * (EG_BK / 4), st + OB + 256 + 64 * wave);
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
        if (K % EG_BK) {
            // the last 64 k through st2, which nobody reads any more
            const int64_t k = (int64_t)steps * EG_BK;
#pragma unroll
            for (int j = 0; j < (FM + 1) / 2; ++j) {
                const int r = (tid >> 2) + 64 * j, u = tid & 3;
                if (r >= BM) break;
                st2[r * 8 + (u ^ ((r >> 1) & 7))] = *reinterpret_cast<const i32x4*>(x + token(r) * K + k + 16 * u);
            }
            const uint8_t* w = tid < 128 ? w0 + (int64_t)min(tid, last_n) * rowb : w1 + (int64_t)min(tid - 128, last_n1) * rowb;
            st2[OB + tid * 2 + ((tid >> 3) & 1)] = *reinterpret_cast<const i32x4*>(w + (k >> 2));
            __syncthreads();
            multiply(st2, 1);
        }
    } else {
        struct Regs {
            u32x4 v[FM + 2];
        };
        const uint8_t *wr0 = w0 + (int64_t)min(wrow, last_n) * rowb, *wr1 = w1 + (int64_t)min(wrow, last_n1) * rowb;
        const uint8_t* xp[FM];
#pragma unroll
        for (int q = 0; q < FM; ++q) xp[q] = x + token(xrow(q)) * K;
        auto load = [&](int s) {
            const int64_t k = (int64_t)s * EG_BK;
            Regs r;
#pragma unroll
            for (int q = 0; q < FM; ++q) r.v[q] = load_16(xp[q] + k + 16 * xunit(q));
            r.v[FM] = load_16(wr0 + (k >> 2) + 16 * wunit);
            r.v[FM + 1] = load_16(wr1 + (k >> 2) + 16 * wunit);
            return r;
        };
        auto put = [&](i32x4* st, const Regs& r) {
#pragma unroll
            for (int q = 0; q < FM; ++q) st[64 * (FM * wave + q) + lane] = (i32x4)r.v[q];
            st[OB + 64 * wave + lane] = (i32x4)r.v[FM];
            st[OB + 256 + 64 * wave + lane] = (i32x4)r.v[FM + 1];
        };
        // The last part step first (sums of integers are exact in any order), through st0, while the first
        // whole steps' loads are under way; then whole steps in st1 and st0 in turn, loaded two ahead.
        const int whole = (int)(K / EG_BK), last = whole - 1;
        Regs r0, r1;
        if (whole > 0) {
            r0 = load(0);
            r1 = load(min(1, last));
        }
        if (K % EG_BK) {
            const int64_t k = (int64_t)whole * EG_BK;
            Regs r;
#pragma unroll
            for (int q = 0; q < FM; ++q) r.v[q] = row_16(xp[q], k + 16 * xunit(q), K);
            r.v[FM] = row_16(wr0, (k >> 2) + 16 * wunit, rowb);
            r.v[FM + 1] = row_16(wr1, (k >> 2) + 16 * wunit, rowb);
            put(st0, r);
            __syncthreads();
            multiply(st0, 2);
        } else {
            __syncthreads();                                        // the rows' scales
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
    // accumulator r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4 of the block, column l % 32
    const int n = 32 * wave + lr;
    if (n >= rows_n) return;
    const bool second = n < rows_n1;
    const float* bias1 = GATED ? a.b1 : a.b0;
    float b0 = a.b0 ? a.b0[e * a.N + n0 + n] : -0.0f, b1 = bias1 && second ? bias1[e * a.N + n1 + n] : -0.0f;
    // both are there before the first store: waited for behind the stores' conditions they would be waited for at each,
    // and the stores before it with them
    asm volatile("" : "+v"(b0), "+v"(b1));
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int m = 32 * i + 8 * q + 4 * lg;
            const float4 s4 = *reinterpret_cast<const float4*>(&scale[0][m]);
            const float4 t4 = *reinterpret_cast<const float4*>(&scale[GATED ? 1 : 0][m]);
            const float4 z4 = *reinterpret_cast<const float4*>(&scale[2][m]);
            const float s0[4] = {s4.x, s4.y, s4.z, s4.w}, s1[4] = {t4.x, t4.y, t4.z, t4.w}, z[4] = {z4.x, z4.y, z4.z, z4.w};
            const int64_t at = (m0 + m) * a.N + n0 + n;
            float v0[4], v1[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                v0[c] = (float)acc[i][0][4 * q + c] * s0[c] + z[c] + b0;
                v1[c] = (float)acc[i][1][4 * q + c] * s1[c] + z[c] + b1;
            }
            if constexpr (!GATED) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (m + c < rows_m) {
                        a.y[at + c * a.N] = v0[c];
                        if (second) a.y[at + c * a.N + EG_BF] = v1[c];
                    }
            } else {
                float v[4];
                if constexpr (ACT == BITLINEAR_ACT_GELU) {
                    const float4 v4 = gelu4_f32(make_float4(v0[0], v0[1], v0[2], v0[3]));
                    v[0] = v4.x, v[1] = v4.y, v[2] = v4.z, v[3] = v4.w;
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = act_value<ACT>(v0[c]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (m + c < rows_m) a.y[at + c * a.N] = v[c] * v1[c];
                if (a.g) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (m + c < rows_m) {
                            a.g[at + c * a.N] = v0[c];
                            a.u[at + c * a.N] = v1[c];
                        }
                }
            }
        }
}

template <int ACT, bool ALIGNED, int FM>
static hipError_t launch_grouped_gemm_fm(const GroupedArgs& a, hipStream_t s) {
    constexpr int COLUMNS = ACT ? EG_BF : 2 * EG_BF;
    const int64_t tm = most_slots(a, 32 * FM), tf = (a.N + COLUMNS - 1) / COLUMNS;
    hipLaunchKernelGGL((k_grouped_gemm<ACT, ALIGNED, FM>), dim3((unsigned)(tm * tf)), dim3(256), 0, s, a, (int)tm, (int)tf);
    return hipGetLastError();
}

// Tiles of 32 rows where a group has few, or while those tiles are at most about as many as compute units; then 64,
// and 128 for long sums and many tiles.  Microseconds with 32 / 64 / 128 rows, for experts of so many rows (the
// number of tiles of 32 as counted below):
//   8 experts 4096 -> 11008, gated: 16 rows (688) 42.1 / 51.8 / 83.2;  32 (1032) 64.0 / 53.4 / 86.2
//   8 experts 2048 -> 2816: 64 rows (220) 13.6 / 17.0 / 22.7;  128 (396) 19.2 / 18.8 / 25.3;  gated 32 (264) 13.6 /
//     16.6 / 23.4;  gated 128 (792) 31.7 / 27.2 / 38.3;  gated 512 (2904) 86.2 / 64.1 / 73.8
//   16 experts 2816 -> 2048: 48 rows (256) 16.8 / 20.5 / 28.4;  64 (320) 22.9 / 21.5 / 28.9
//   8 experts 4096 -> 11008: 64 rows (860) 51.1 / 51.0 / 54.9;  128 (1548) 75.9 / 71.3 / 62.0;  512 (5676) 288 / 208 / 200
template <int ACT, bool ALIGNED>
static hipError_t launch_grouped_gemm(const GroupedArgs& a, hipStream_t s) {
    const int64_t used = a.E < a.M ? a.E : a.M, rows = a.M / used;
    const int64_t tiles = (a.M / 32 + used / 2) * ((a.N + (ACT ? EG_BF : 2 * EG_BF) - 1) / (ACT ? EG_BF : 2 * EG_BF));
    if (rows <= 24 || tiles <= 288) return launch_grouped_gemm_fm<ACT, ALIGNED, 1>(a, s);
    if (a.K >= 4096 && rows >= 96 && tiles >= 1280) return launch_grouped_gemm_fm<ACT, ALIGNED, 4>(a, s);
    return launch_grouped_gemm_fm<ACT, ALIGNED, 2>(a, s);
}

template <bool ALIGNED>
static hipError_t launch_grouped_tiles(const GroupedArgs& a, hipStream_t s) {
    if (!a.w1) return launch_grouped_gemm<0, ALIGNED>(a, s);
    switch (a.act) {
        case BITLINEAR_ACT_SILU: return launch_grouped_gemm<BITLINEAR_ACT_SILU, ALIGNED>(a, s);
        case BITLINEAR_ACT_GELU: return launch_grouped_gemm<BITLINEAR_ACT_GELU, ALIGNED>(a, s);
        default: return launch_grouped_gemm<BITLINEAR_ACT_RELU2, ALIGNED>(a, s);
    }
}

// The streaming kernel while its workgroups (slots of 16 rows as counted below, by blocks of columns) are few enough:
// a GEMM's time is about 5 us and 3.5 ns a unit of K while its tiles run at once, the streaming kernel's 3.5 us and 2
// ps (up to two rows an expert) to 3.5 ps a workgroup and unit of K.  Microseconds, streaming kernel against GEMM of 32
// rows (workgroups):  8 experts 2048 -> 2816, gated: 2 rows (1408) 9.4 / 11.3, 4 (1408) 11.6 / 11.6, 16 (2112) 22.9 /
// 12.0;  16 experts 2816 -> 2048: 8 rows (1024) 11.1 / 15.0, 16 (1536) 17.8 / 15.4;  64 experts 1024 -> 1024: 1 row
// (2048) 8.2 / 8.7, gated (4096) 12.0 / 9.7;  8 experts 4096 -> 11008: 1 row (2752) 23.9 / 20.7;  4 experts 512 -> 1024:
// 128 rows (1088) 6.5 / 7.6, 256 (2112) 9.8 / 7.9;  7 experts 1088 -> 1537: 32 rows (857) 7.7 / 9.8, 64 (1519) 11.4 / 10.1.
// Eight waves for up to two workgroups a compute unit, four beyond (microseconds, eight / four):  8 experts 11008 ->
// 4096: 2 rows in all (256 workgroups) 8.2 / 11.1, 4 rows (512) 12.9 / 13.4, 32 rows (1024) 27.2 / 24.8;  16 experts
// 2816 -> 2048: 4 rows (256) 4.4 / 4.9, 16 rows (1024) 11.7 / 9.3.
hipError_t launch_grouped(const GroupedArgs& a, hipStream_t s) {
    const int64_t used = a.E < a.M ? a.E : a.M, half_full = a.M / 16 + used / 2, slots = used > half_full ? used : half_full;
    const int64_t blocks = a.w1 ? (a.N + 15) / 16 : (a.N + 31) / 32;
    const int64_t most = a.M <= 2 * used ? ((int64_t)1 << 20) / a.K + 2048 : ((int64_t)1 << 19) / a.K + 1024;
    if (slots * blocks <= 512) return a.w1 ? launch_grouped_dec<true, 8>(a, s) : launch_grouped_dec<false, 8>(a, s);
    if (slots * blocks <= most) return a.w1 ? launch_grouped_dec<true, 4>(a, s) : launch_grouped_dec<false, 4>(a, s);
    const bool aligned = a.K % 64 == 0 && a.T <= 0xFFFFFFFFll / a.K && (uintptr_t)a.xq % 16 == 0 && (uintptr_t)a.w0 % 16 == 0 &&
                         (uintptr_t)a.w1 % 16 == 0;
    return aligned ? launch_grouped_tiles<true>(a, s) : launch_grouped_tiles<false>(a, s);
}

}  // namespace bitlinear
