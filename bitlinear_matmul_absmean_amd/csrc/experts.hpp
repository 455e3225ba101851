// experts.hpp -- products grouped by expert, their gradients, and the fp8 product with block scales: helpers
// and launch declarations.
#pragma once

#include "bitlinear.h"
#include "common.hpp"

namespace bitlinear {

// Largest sizes of the grouped calls, and whether their launches hold them (a grid has fewer than 2^32 threads).
constexpr int64_t GROUPED_MAX_E = 4096, GROUPED_MAX_N = (int64_t)1 << 20, GROUPED_MAX_M = (int64_t)1 << 24;
inline bool grid_fits(int64_t workgroups, int64_t threads) { return workgroups <= 0xFFFFFFFFll / threads; }
bool grouped_fits(int64_t M, int64_t N, int64_t E);
bool grouped_backward_fits(int64_t M, int64_t K, int64_t N, int64_t E);

// Group e as rows [lo, hi): offsets outside 0 .. M are taken as 0 or M.
struct Group {
    int64_t lo, hi;
};
__device__ __forceinline__ Group group_rows(const int64_t* __restrict__ offsets, int64_t e, int64_t M) {
    const int64_t lo = offsets[e], hi = offsets[e + 1];
    return Group{lo < 0 ? 0 : lo > M ? M : lo, hi < 0 ? 0 : hi > M ? M : hi};
}

// Token of row m: -1 for an index outside 0 .. T - 1.
__device__ __forceinline__ int64_t row_token(const int64_t* __restrict__ rows, int64_t m, int64_t T) {
    if (!rows) return m;
    const int64_t r = rows[m];
    return r >= 0 && r < T ? r : -1;
}

// Slot `at` of `tile` rows, the slots of a group following those of the groups before it: its expert, first
// row and number of rows (0: there is no such slot).  Each lane takes one of 64 experts at a time; `total`
// receives the number of all slots if asked for.
struct Slot {
    int e, rows;
    int64_t m0;
};
template <int TILE, bool TOTAL>
__device__ __forceinline__ Slot find_slot(const int64_t* __restrict__ offsets, int E, int64_t M, int at, int* total) {
    const int lane = threadIdx.x & 63;
    Slot s{0, 0, 0};
    int before = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        int lo = 0, n = 0;
        if (e0 + lane < E) {
            const Group g = group_rows(offsets, e0 + lane, M);
            lo = (int)g.lo;
            n = g.hi > g.lo ? (int)(g.hi - g.lo) : 0;
        }
        const int mine = (n + TILE - 1) / TILE;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(upto, d, 64);
            upto += lane >= d ? v : 0;
        }
        const int all = __builtin_amdgcn_readlane(upto, 63);
        if (at >= before && at < before + all) {
            const int l = __builtin_ctzll(__ballot(before + upto > at));
            const int tile = at - before - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(mine, l));
            const int left = __builtin_amdgcn_readlane(n, l) - tile * TILE;
            s = Slot{e0 + l, left < TILE ? left : TILE, __builtin_amdgcn_readlane(lo, l) + (int64_t)tile * TILE};
            if (!TOTAL) break;
        }
        before += all;
    }
    if (TOTAL) *total = before;
    return s;
}

// Most slots of `tile` rows that M rows of E experts can make.
inline int64_t most_slots(int64_t M, int64_t E, int64_t tile) { return M / tile + (E < M ? E : M); }

struct GroupedArgs {
    const int8_t* xq;              // [T, K]
    const float* beta;             // [T]
    int64_t T, K;
    const int64_t* rows;           // [M] or null
    int64_t M;
    const int64_t* offsets;        // [E + 1]
    int64_t E;
    const uint8_t *w0, *w1;        // packed [E, N, K/4]: one projection (w1 null), or gate and up
    const float *al0, *al1;        // alpha [E]
    const float *b0, *b1;          // bias [E, N] or null
    int64_t N;
    int act;                       // gated: a bitlinear_activation
    float* y;                      // [M, N]: y, or h of the gated block
    float *g, *u;                  // gated: [M, N] or both null
};
hipError_t launch_grouped(const GroupedArgs& a, hipStream_t s);
// The gated block of one token with x quantized in the same launch (xq and beta are written, not read).
bool grouped_gemv_supports(const GroupedArgs& a, const float* x);
hipError_t launch_grouped_gemv(const GroupedArgs& a, const float* x, int8_t* xq, float* beta, hipStream_t s);

struct GroupedBackwardArgs {
    const float* dy;               // [M, N]; gated: dh
    const float *g, *u;            // gated: [M, N]; else null
    int act;
    int64_t M, K, N, T;
    const int8_t* xq;
    const float* beta;
    const int64_t *rows, *offsets;
    int64_t E;
    const uint8_t *w0, *w1;        // packed [E, N, K/4]; w1 null for one projection
    const float *al0, *al1;        // alpha [E]
    float* dx;                     // [M, K] or null
    float *dw0, *dw1;              // [E, N, K] or null
    float *db0, *db1;              // [E, N] or null
    void* ws;
};
size_t grouped_backward_workspace(int64_t M, int64_t K, int64_t N, int64_t E, bool gated);
hipError_t launch_grouped_backward(const GroupedBackwardArgs& a, hipStream_t s);

struct Fp8Args {
    const uint8_t* xq;             // e4m3 [M, K]
    const float* xs;               // [ceil(K / 128), M]
    int64_t M, K, N;
    const uint8_t* wq;             // e4m3 [N, K]
    const float* ws;               // [ceil(N / 128), ceil(K / 128)]
    const float* bias;             // [N] or null
    float* y;                      // [M, N]
};
// Largest K (256 rows of x_q or W_q within 32-bit offsets, blocks of 128 within a grid's second dimension),
// and M, N and M N (grids of fewer than 2^32 threads).
constexpr int64_t FP8_MAX_K = (int64_t)1 << 22, FP8_MAX_ROWS = (int64_t)1 << 26, FP8_MAX_Y = (int64_t)1 << 36;
hipError_t launch_quantize_act_fp8(const float* x, int64_t M, int64_t K, uint8_t* xq, float* xs, hipStream_t s);
hipError_t launch_quantize_weights_fp8(const float* W, int64_t N, int64_t K, uint8_t* wq, float* ws, hipStream_t s);
hipError_t launch_forward_fp8(const Fp8Args& a, hipStream_t s);

}  // namespace bitlinear
