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
// the sums end, or two neighbouring sets of columns of the one projection.  Two kernels, each in a form for
// aligned rows and one for any K % 4 == 0 and any alignment:
//   * few rows an expert: k_grouped_dec, the weight streams on the 16x16x64 int8 MFMA;
//   * else: k_grouped_gemm, LDS tiles on the 32x32x32 int8 MFMA.
#include <type_traits>

#include "experts.hpp"
#include "ffn.hpp"

namespace bitlinear {

static int64_t most_slots(const GroupedArgs& a, int64_t tile) { return most_slots(a.M, a.E, tile); }

// The GEMM's smallest tiles, 32 rows x 128 columns of 256 threads (the streaming kernel is taken where its fit).
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
// A workgroup of eight waves computes 16 MT rows x 16 columns of both sets; wave w takes the steps of 256 k
// w, w + 8, ..., and the partial tiles are added at the end (integers: exact in any order).  In MFMA q of a
// step lane group g (lanes 16 g ..) holds weights 64 g + 16 q .. 64 g + 16 q + 15, dword q of the lane's 16
// bytes of codes, expanded in weight order to signed bytes.
// Aligned rows (16-byte aligned tensors, K % 64 == 0, T K < 2^32): operands come through a wave's own LDS image,
// filled by loads that go past the registers; a step's image is read into registers, the next step's loads are
// started into it, and the MFMAs run while they are in flight.  Row R's 16-byte unit u of a step lies at
// position u ^ (R % 16) of its sixteen.  Otherwise operands are read straight into registers.
// 16x16x64 lane layout: A/B lane l holds row/column l % 16, k = 16 (l / 16) + j; accumulator r of
// lane l is row 4 (l / 16) + r, column l % 16.
constexpr int ED_WAVES = 8;

template <bool GATED, bool ALIGNED, int MT>
__global__ __launch_bounds__(64 * ED_WAVES) void k_grouped_dec(GroupedArgs a, int slots) {
    constexpr int IMG = (4 * MT + 2) * 64;                          // 16-byte units of a wave's image
    constexpr int TILES = 2 * MT * 64;                              // of a wave's partial tiles
    constexpr int PER = ALIGNED && IMG > TILES ? IMG : TILES;
    __shared__ i32x4 lds[ED_WAVES * PER];
    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Slot slot = find_slot<16 * MT, false>(a.offsets, (int)a.E, a.M, (int)(blockIdx.x % slots), nullptr);
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
    const int last_n = rows_n - 1, last_n1 = rows_n1 ? rows_n1 - 1 : rows_n - 1;
    // tokens of the rows, one a lane (of row 0 past the end)
    int token = 0;
    float beta = 0.0f;
    {
        const int64_t r = row_token(a.rows, m0 + min(lane, rows_m - 1), a.T);
        if (r >= 0) {
            token = (int)r;
            beta = a.beta[r];
        }
    }
    const int steps = (int)((K + 255) / 256);
    i32x4 acc[2][MT];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[p][t] = i32x4{0, 0, 0, 0};
    auto multiply = [&](const i32x4 (&xv)[MT][4], const u32x4 (&w)[2]) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const i32x4 b = expand_signed_in_order(w[p][q]);
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[p][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xv[t][q], b, acc[p][t], 0, 0, 0);
            }
    };
    const uint8_t *wp[2] = {w0 + (int64_t)min(lr, last_n) * rowb, w1 + (int64_t)min(lr, last_n1) * rowb};
    const uint8_t* xp[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xp[t] = reinterpret_cast<const uint8_t*>(a.xq) + (int64_t)__shfl(token, 16 * t + lr, 64) * K;
    // step s with its operands read straight into registers
    auto direct = [&](int s) {
        const int64_t k = (int64_t)s * 256 + 64 * lg;
        i32x4 xv[MT][4];
        u32x4 w[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) w[p] = row_16(wp[p], k >> 2, rowb);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) xv[t][q] = (i32x4)row_16(xp[t], k + 16 * q, K);
        multiply(xv, w);
    };
    if constexpr (ALIGNED) {
        const int whole = (int)(K / 256);                           // a last part step is read directly
        i32x4* img = lds + wave * IMG;
        const __amdgpu_buffer_rsrc_t rx = raw_buffer(a.xq, (uint32_t)(a.T * K));
        const __amdgpu_buffer_rsrc_t r0 = raw_buffer(w0, (uint32_t)rows_n * (uint32_t)rowb);
        const __amdgpu_buffer_rsrc_t r1 = raw_buffer(w1, (uint32_t)(last_n1 + 1) * (uint32_t)rowb);
        // load i of x: rows 4 i .. 4 i + 3, sixteen lanes each; of a set: lane (lr, lg) reads 64 codes of row
        // lr.  Rows past the end repeat the last one; groups of four rows past it are not loaded (what they
        // hold reaches only outputs that are not written).
        uint32_t xo[4 * MT];
#pragma unroll
        for (int i = 0; i < 4 * MT; ++i)
            xo[i] = (uint32_t)__shfl(token, 4 * i + lg, 64) * (uint32_t)K + 16u * (uint32_t)(lr ^ ((4 * i + lg) & 15));
        const uint32_t o0 = (uint32_t)min(lr, last_n) * (uint32_t)rowb + 16u * (uint32_t)lg;
        const uint32_t o1 = (uint32_t)min(lr, last_n1) * (uint32_t)rowb + 16u * (uint32_t)lg;
        auto fetch = [&](int s) {
            load_lds16(r0, o0, (uint32_t)s * 64u, img + 64 * (4 * MT));
            load_lds16(r1, o1, (uint32_t)s * 64u, img + 64 * (4 * MT + 1));
#pragma unroll
            for (int i = 0; i < 4 * MT; ++i)
                if (4 * i < rows_m) load_lds16(rx, xo[i], (uint32_t)s * 256u, img + 64 * i);
        };
        if (wave < whole) fetch(wave);
        for (int s = wave; s < whole; s += ED_WAVES) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0x0F70);                     // vmcnt(0): the image is whole
            __builtin_amdgcn_sched_barrier(0);
            i32x4 xv[MT][4];
            u32x4 w[2];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) xv[t][q] = img[(16 * t + lr) * 16 + ((4 * lg + q) ^ lr)];
#pragma unroll
            for (int p = 0; p < 2; ++p) w[p] = (u32x4)img[64 * (4 * MT + p) + lane];
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xC07F);                     // lgkmcnt(0): every read of it is over
            __builtin_amdgcn_sched_barrier(0);
            if (s + ED_WAVES < whole) fetch(s + ED_WAVES);
            multiply(xv, w);
        }
        if (whole < steps && whole % ED_WAVES == wave) direct(whole);
    } else {
        struct Part {
            i32x4 x[MT][4];
            u32x4 w[2];
        };
        auto load = [&](int s) {
            const int64_t k = (int64_t)s * 256 + 64 * lg;
            Part f;
#pragma unroll
            for (int p = 0; p < 2; ++p) f.w[p] = load_16(wp[p] + (k >> 2));
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) f.x[t][q] = (i32x4)load_16(xp[t] + k + 16 * q);
            return f;
        };
        // whole steps, the next one's loads under way; the last part step goes to the next wave in turn
        const int whole = (int)(K / 256);
        if (wave < whole) {
            Part f = load(wave);
            for (int s = wave; s < whole; s += ED_WAVES) {
                const Part next = load(min(s + ED_WAVES, whole - 1));
                multiply(f.x, f.w);
                f = next;
            }
        }
        if (whole < steps && whole % ED_WAVES == wave) direct(whole);
    }
    __syncthreads();                                                // every wave is done with its image
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int t = 0; t < MT; ++t) lds[(wave * 2 * MT + p * MT + t) * 64 + lane] = acc[p][t];
    __syncthreads();
    const float al0 = a.al0[e], al1 = GATED ? a.al1[e] : al0;
    // element i of row block t and column l % 16, of both sets; a wave's elements share t and i
    for (int x = tid; x < MT * 256; x += 64 * ED_WAVES) {
        const int l = x & 63, i = (x >> 6) & 3, t = x >> 8, n = l & 15, m = 16 * t + 4 * (l >> 4) + i;
        const float b = __shfl(beta, m, 64);
        int s0 = 0, s1 = 0;
#pragma unroll
        for (int w = 0; w < ED_WAVES; ++w) {
            const int* p = reinterpret_cast<const int*>(lds + (w * 2 * MT + t) * 64 + l);
            s0 += p[i];
            s1 += p[i + MT * 256];
        }
        if (m >= rows_m) continue;
        const int64_t at = (m0 + m) * a.N + n0 + n, bn = e * a.N + n0 + n;
        float v0 = (float)s0 * dequant_scale(al0, b), v1 = (float)s1 * dequant_scale(al1, b);
        if constexpr (GATED) {
            if (n >= rows_n) continue;
            if (a.b0) v0 = v0 + a.b0[bn];
            if (a.b1) v1 = v1 + a.b1[bn];
            if (a.act == BITLINEAR_ACT_SILU) gate_store<BITLINEAR_ACT_SILU>(a, at, v0, v1);
            else if (a.act == BITLINEAR_ACT_GELU) gate_store<BITLINEAR_ACT_GELU>(a, at, v0, v1);
            else gate_store<BITLINEAR_ACT_RELU2>(a, at, v0, v1);
        } else {
            if (n < rows_n) a.y[at] = a.b0 ? v0 + a.b0[bn] : v0;
            if (n < rows_n1) a.y[at + 16] = a.b0 ? v1 + a.b0[bn + 16] : v1;
        }
    }
}

template <bool GATED, bool ALIGNED, int MT>
static hipError_t launch_grouped_dec_mt(const GroupedArgs& a, hipStream_t s) {
    const int64_t slots = most_slots(a, 16 * MT), blocks = (a.N + (GATED ? 15 : 31)) / (GATED ? 16 : 32);
    hipLaunchKernelGGL((k_grouped_dec<GATED, ALIGNED, MT>), dim3((unsigned)(slots * blocks)), dim3(64 * ED_WAVES), 0, s, a, (int)slots);
    return hipGetLastError();
}

template <bool GATED, bool ALIGNED>
static hipError_t launch_grouped_dec(const GroupedArgs& a, hipStream_t s) {
    return a.M <= 8 * a.E ? launch_grouped_dec_mt<GATED, ALIGNED, 1>(a, s) : launch_grouped_dec_mt<GATED, ALIGNED, 2>(a, s);
}

// ---- many rows an expert --------------------------------------------------------------------
// A workgroup of four waves computes 32 FM rows x 128 columns of both sets, a wave all the rows x 32 columns of
// each: FM 32-row operands against one weight operand of each set, so that the expansion of a weight operand
// (17 instructions) serves FM MFMAs.  Steps of 128 k, three LDS stages (4 FM + 8 KiB each: 32 FM rows of x_q of
// 128 bytes, 256 weight rows of 32 bytes) filled two steps ahead by loads that go past the registers (aligned
// rows, as above), or two filled through registers.  Unit u of x_q's row r lies at slot u ^ ((r / 2) % 8), unit u
// of weight row r at slot u ^ ((r / 8) % 2), so that an operand read spreads over all banks.
// In the two MFMAs of k 64 h .. 64 h + 63 (h = 0, 1) a lane group holds 32 codes, eight bytes of a
// weight row: the lane's unit h, of which group lg uses dwords 2 lg and 2 lg + 1.
constexpr int EG_BF = 128, EG_BK = 128;

// ACT 0: one projection, whose columns n0 + 128 .. are the second set.
template <int ACT, bool ALIGNED, int FM>
__global__ __launch_bounds__(256, 2) void k_grouped_gemm(GroupedArgs a, int tiles_f) {
    constexpr bool GATED = ACT != 0;
    constexpr int BM = 32 * FM, OB = BM * 8, UNITS = OB + 2 * EG_BF * 2;
    __shared__ i32x4 st0[UNITS];
    __shared__ i32x4 st1[UNITS];
    __shared__ i32x4 st2[ALIGNED ? UNITS : 1];
    __shared__ __align__(16) float scale[2][BM];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // of the tiles there are, a contiguous run for each XCD, four rows of tiles at a time
    int tiles_m;
    find_slot<BM, true>(a.offsets, (int)a.E, a.M, -1, &tiles_m);
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
    const float b0 = a.b0 ? a.b0[e * a.N + n0 + n] : 0.0f, b1 = bias1 && second ? bias1[e * a.N + n1 + n] : 0.0f;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int m = 32 * i + 8 * q + 4 * lg;
            const float4 s4 = *reinterpret_cast<const float4*>(&scale[0][m]);
            const float4 t4 = *reinterpret_cast<const float4*>(&scale[GATED ? 1 : 0][m]);
            const float s0[4] = {s4.x, s4.y, s4.z, s4.w}, s1[4] = {t4.x, t4.y, t4.z, t4.w};
            const int64_t at = (m0 + m) * a.N + n0 + n;
            float v0[4], v1[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                v0[c] = (float)acc[i][0][4 * q + c] * s0[c];
                v1[c] = (float)acc[i][1][4 * q + c] * s1[c];
                if (a.b0) v0[c] = v0[c] + b0;
                if (bias1) v1[c] = v1[c] + b1;
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
    hipLaunchKernelGGL((k_grouped_gemm<ACT, ALIGNED, FM>), dim3((unsigned)(tm * tf)), dim3(256), 0, s, a, (int)tf);
    return hipGetLastError();
}

template <int ACT, bool ALIGNED>
static hipError_t launch_grouped_gemm(const GroupedArgs& a, hipStream_t s) {
    const int64_t rows = a.M / (a.E < a.M ? a.E : a.M);
    return rows <= 32   ? launch_grouped_gemm_fm<ACT, ALIGNED, 1>(a, s)
           : rows <= 64 ? launch_grouped_gemm_fm<ACT, ALIGNED, 2>(a, s)
                        : launch_grouped_gemm_fm<ACT, ALIGNED, 4>(a, s);
}

template <bool ALIGNED>
static hipError_t launch_grouped_rows(const GroupedArgs& a, hipStream_t s) {
    if (a.M <= 16 * a.E && grid_fits(most_slots(a, 16) * ((a.N + 15) / 16), 64 * ED_WAVES))
        return a.w1 ? launch_grouped_dec<true, ALIGNED>(a, s) : launch_grouped_dec<false, ALIGNED>(a, s);
    if (!a.w1) return launch_grouped_gemm<0, ALIGNED>(a, s);
    switch (a.act) {
        case BITLINEAR_ACT_SILU: return launch_grouped_gemm<BITLINEAR_ACT_SILU, ALIGNED>(a, s);
        case BITLINEAR_ACT_GELU: return launch_grouped_gemm<BITLINEAR_ACT_GELU, ALIGNED>(a, s);
        default: return launch_grouped_gemm<BITLINEAR_ACT_RELU2, ALIGNED>(a, s);
    }
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t s) {
    const bool aligned = a.K % 64 == 0 && a.T <= 0xFFFFFFFFll / a.K && (uintptr_t)a.xq % 16 == 0 && (uintptr_t)a.w0 % 16 == 0 &&
                         (uintptr_t)a.w1 % 16 == 0;
    return aligned ? launch_grouped_rows<true>(a, s) : launch_grouped_rows<false>(a, s);
}

}  // namespace bitlinear
