/*
 * bitlinear.h -- C ABI of the MI355X (gfx950) BitNet b1.58 BitLinear library (W1.58A8).
 *
 * Page keys used in the citations below:
 *   [P1] 2kiu.com, article on 1.58-bit quantization and hardware co-optimization (block
 *        scales, §2.3 and §4.2).
 *   [P2] nxmr.cn tutorial "1.58 位大模型" (per-row absmean, add/sub form of the matmul, §1.1
 *        and §6.1 more compact encodings).
 *   [P3] chenxutan.com, "1.58-bit 大模型极限量化实战：从 BitNet 三值权重到单颗 CPU 跑起 100B 模型"
 *        (absmean / absmax formulas, BitLinear forward, 2-bit packing, §6.1 the BitMLP,
 *        §6.2 the rotation before absmax).
 *
 * The layer is split the way [P3 §3.2] describes BitLinear: weights are quantized once and
 * cached (bitlinear_quantize_weights); every call quantizes the activations
 * (bitlinear_quantize_act), runs the ternary x int8 integer matmul and applies the
 * alpha*beta/127 dequantization (bitlinear_forward).
 *
 * Conventions shared by every entry point
 *   - Memory: every array argument is DEVICE memory on the current HIP device, allocated and
 *     owned by the caller.  The library never allocates, frees or retains caller memory.  Its
 *     only state between calls is the per-thread code of the last HIP error (see
 *     bitlinear_last_hip_error); calls are reentrant.
 *   - Execution: every call validates its arguments on the host, enqueues its kernels on
 *     `stream` (0 = the null stream) and returns without synchronising.  Results are
 *     visible to later work on the same stream.
 *   - Errors: 0 (BITLINEAR_OK) or a negative bitlinear_status.  Argument validation happens
 *     before any HIP call, so an invalid call enqueues nothing.  BITLINEAR_ERR_HIP reports a
 *     launch error from the HIP runtime (hipGetLastError after the launch).
 *   - Layouts: row-major.  W is [N, K] (out_features x in_features, the nn.Linear
 *     convention [P3 §4.2]); x is [M, K] (M tokens); y = x W^T is [M, N].
 *   - Packed ternary weights: uint8 [N, K/4].  Weight W[n, k] is stored as the 2-bit code
 *     W_hat + 1 (00 -> -1, 01 -> 0, 10 -> +1; 11 is never written) [P3 §5.3], at bits
 *     2*(k%4) .. 2*(k%4)+1 of byte n*K/4 + k/4.  K must be a multiple of 4.
 *   - Non-finite inputs (NaN, Inf) give unspecified codes and outputs.
 */
#ifndef BITLINEAR_H
#define BITLINEAR_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BITLINEAR_ABI_VERSION 1

/* Largest K for which |acc| <= 127*K still fits int32. */
#define BITLINEAR_MAX_K 16909320

typedef enum bitlinear_status {
    BITLINEAR_OK = 0,
    BITLINEAR_ERR_INVALID_ARG = -1, /* null required pointer, size <= 0 */
    BITLINEAR_ERR_SHAPE = -2,       /* K % 4 != 0, K > BITLINEAR_MAX_K, size overflow */
    BITLINEAR_ERR_ALIGNMENT = -3,   /* a pointer lacks the alignment the call documents */
    BITLINEAR_ERR_WORKSPACE = -4,   /* workspace null or smaller than required */
    BITLINEAR_ERR_HIP = -5,         /* the HIP runtime reported an error at launch */
    BITLINEAR_ERR_SCRATCH = -6      /* beyond the fixed scratch of an allocation-free call */
} bitlinear_status;

/* Returns BITLINEAR_ABI_VERSION of the built library. */
int bitlinear_abi_version(void);

/* Static, human-readable name of a status code (never NULL). */
const char* bitlinear_status_string(int status);

/* The hipError_t of the last BITLINEAR_ERR_HIP returned on the calling thread (0 if none). */
int bitlinear_last_hip_error(void);

/*
 * Bytes of device workspace bitlinear_quantize_weights needs for an [N, K] tensor:
 * N fp64 row partial sums (0 for invalid sizes).
 */
size_t bitlinear_quantize_weights_workspace_size(int64_t N, int64_t K);

/*
 * Absmean ternary weight quantization with one scale per tensor [P3 §2.3, §4.1]:
 *     alpha = mean(|W|),  W_hat = clip(round(W / alpha), -1, 1),  packed 2 bits/weight.
 * |W| is summed in fp64 (fixed order: per-row partials, then a fixed tree over rows) and
 * alpha is rounded to fp32 once; W / alpha is an IEEE fp32 division; round() is
 * round-half-to-even.  An all-zero W gives alpha = 0 and every code 0 (weight 0).
 *
 *   W          [N, K] fp32, 16-byte aligned.                                (in)
 *   W_packed   [N, K/4] uint8 in the packed layout above, 4-byte aligned.   (out)
 *   alpha      [1] fp32.                                                    (out)
 *   workspace  >= bitlinear_quantize_weights_workspace_size(N, K) bytes,
 *              8-byte aligned; scratch, contents undefined on return.
 * Errors: INVALID_ARG (null pointer, N or K <= 0), SHAPE (K % 4, K too large, N*K
 * overflow), ALIGNMENT, WORKSPACE, HIP.
 */
int bitlinear_quantize_weights(const float* W, int64_t N, int64_t K, uint8_t* W_packed,
                               float* alpha, void* workspace, size_t workspace_bytes,
                               hipStream_t stream);

/*
 * bitlinear_quantize_weights without a workspace argument, for callers that cannot allocate
 * device memory (code under HIP graph capture, serving loops, harnesses that forbid
 * hipMalloc).  The fp64 row sums go to a fixed scratch array inside the library, one copy per
 * device, held until the process ends, of bitlinear_quantize_weights_noalloc_max_rows() rows
 * (262144, 2 MiB).  The call allocates nothing (no hipMalloc, hipFree or allocating library
 * routine); the first call on a device looks up the address of that device's scratch.
 * Results are identical to bitlinear_quantize_weights.  All calls on one device share its
 * scratch, so calls that overlap on one device (different streams, or different host
 * threads) race and give undefined results; calls ordered on one stream do not.
 *   Arguments as bitlinear_quantize_weights, without the workspace.
 * Errors: as bitlinear_quantize_weights, and SCRATCH when N exceeds the scratch rows.
 */
int bitlinear_quantize_weights_noalloc(const float* W, int64_t N, int64_t K, uint8_t* W_packed,
                                       float* alpha, hipStream_t stream);

/* Rows (N) the fixed scratch of bitlinear_quantize_weights_noalloc holds. */
size_t bitlinear_quantize_weights_noalloc_max_rows(void);

/*
 * Per-output-row variant [P2 §3.1, §4.2]: alpha_rows[n] = mean_k |W[n, k]| (fp64 sum of
 * the row, one fp32 rounding); row n is ternarized with alpha_rows[n].  Needs no workspace.
 *   alpha_rows [N] fp32 (out).  Other arguments and errors as bitlinear_quantize_weights.
 */
int bitlinear_quantize_weights_rows(const float* W, int64_t N, int64_t K, uint8_t* W_packed,
                                    float* alpha_rows, hipStream_t stream);

/*
 * Per-token absmax int8 activation quantization [P3 §2.4, §4.1]:
 *     beta[m] = max_k |x[m, k]| + 1e-8 (fp32 add, as the page's code guards the division),
 *     x_q[m, k] = clip(round(fp32(127 * x[m, k]) / beta[m]), -127, 127),
 * with an IEEE fp32 division and round-half-to-even.  An all-zero token gives
 * beta = 1e-8 and x_q = 0.
 *
 *   x     [M, K] fp32.       (in)     x_q  [M, K] int8.   (out)
 *   beta  [M] fp32.          (out)
 * Any K >= 1 is accepted; K % 4 == 0 with 16-byte aligned x and 4-byte aligned x_q takes
 * the vector path.  Errors: INVALID_ARG, SHAPE (M*K overflow), HIP.
 */
int bitlinear_quantize_act(const float* x, int64_t M, int64_t K, int8_t* x_q, float* beta,
                           hipStream_t stream);

/*
 * Ternary x int8 matmul with the dequantization epilogue [P3 §2.4, §2.5, §3.2; P2 §3.3]:
 *     acc[m, n] = sum_k x_q[m, k] * W_hat[n, k]
 *               = sum_{W_hat=+1} x_q - sum_{W_hat=-1} x_q      (int32, exact)
 *     y[m, n]   = fp32(acc[m, n]) * fp32(alpha * beta[m] / 127)  (+ bias[n])
 * where alpha*beta/127 is evaluated in fp64 and rounded to fp32 once, the product is one
 * fp32 rounding and the bias a separate fp32 addition.
 *
 *   x_q       [M, K] int8 (from bitlinear_quantize_act).   (in)
 *   beta      [M] fp32.                                     (in)
 *   W_packed  [N, K/4] uint8, packed layout above.          (in)
 *   alpha     [1] fp32 (from bitlinear_quantize_weights).   (in)
 *   bias      [N] fp32 or NULL.                             (in)
 *   y         [M, N] fp32.                                  (out)
 *   acc       [M, N] int32 or NULL; when given, receives the exact integer sums.  (out)
 * The kernel is chosen by shape: one token (two on matrices of 2^26 weights or more or with
 * K >= 8192) runs a VALU GEMV (dot4 on unpacked codes); up to 64 tokens a weight-streaming int8
 * MFMA kernel; more an int8 MFMA GEMM that unpacks the ternary tiles on chip.  The fast paths
 * need K % 64 == 0 and 16-byte aligned x_q and W_packed; other inputs run a generic kernel
 * with identical results.
 * Errors: INVALID_ARG, SHAPE (K % 4, K > BITLINEAR_MAX_K, size overflow), HIP.
 */
int bitlinear_forward(const int8_t* x_q, const float* beta, int64_t M, int64_t K,
                      const uint8_t* W_packed, const float* alpha, int64_t N, const float* bias,
                      float* y, int32_t* acc, hipStream_t stream);

/*
 * bitlinear_forward with one alpha per output row [P2 §3.1]: column n of y uses
 * alpha_rows[n] ([N] fp32, from bitlinear_quantize_weights_rows).  Same contract otherwise.
 */
int bitlinear_forward_rows(const int8_t* x_q, const float* beta, int64_t M, int64_t K,
                           const uint8_t* W_packed, const float* alpha_rows, int64_t N,
                           const float* bias, float* y, int32_t* acc, hipStream_t stream);

/*
 * Activation quantization and forward in one call [P3 §3.2 steps 2-4]: y from fp32 x,
 * with results identical to bitlinear_quantize_act followed by bitlinear_forward.
 * For M <= 4, K % 64 == 0, K <= 32768 and 16-byte aligned x, W_packed (and x_q if given)
 * it is one kernel that quantizes x on chip; otherwise it makes the two calls.  For three or
 * four tokens, and for two with K > 4096, the two calls are faster, and they are made
 * whenever x_q and beta are given.
 *
 *   x      [M, K] fp32.                                               (in)
 *   x_q    [M, K] int8 or NULL; receives the quantized activations.   (out)
 *   beta   [M] fp32 or NULL; receives the per-token scales.           (out)
 *   W_packed, alpha, N, bias, y, acc: as bitlinear_forward.
 * x_q and beta may be NULL only on the one-kernel path (else INVALID_ARG).
 * Errors: as bitlinear_forward.
 */
int bitlinear_forward_fused(const float* x, int64_t M, int64_t K, const uint8_t* W_packed,
                            const float* alpha, int64_t N, const float* bias, float* y,
                            int8_t* x_q, float* beta, int32_t* acc, hipStream_t stream);

/*
 * bitlinear_forward_fused with one alpha per output row [P2 §3.1]: column n of y uses
 * alpha_rows[n] ([N] fp32).  Besides per-row quantized weights this serves grouped
 * projections: the packed rows of several projections that read the same x (the q, k and v
 * of an attention block, or gate and up of an MLP) stacked into one [N1 + N2 + ..., K/4]
 * matrix, each projection's per-tensor alpha repeated over its rows, give in one launch the
 * outputs of the separate calls, bit for bit.  Same contract as bitlinear_forward_fused.
 */
int bitlinear_forward_fused_rows(const float* x, int64_t M, int64_t K, const uint8_t* W_packed,
                                 const float* alpha_rows, int64_t N, const float* bias, float* y,
                                 int8_t* x_q, float* beta, int32_t* acc, hipStream_t stream);

/*
 * Ternary weights packed five to a byte [P2 §1.1, §6.1] (1.6 bits per weight; the pages name
 * more compact encodings than 2 bits without a format).  Byte b of a row holds the codes
 * c = W_hat + 1 of weights 5b .. 5b+4 as sum_i c_i 3^i (0..242); a row takes
 * bitlinear_t5_row_bytes(K) = 16 ceil(K / 80) bytes; trits past K hold code 1 (weight 0).
 * Quantization is that of bitlinear_quantize_weights (same alpha, same codes), packed this
 * way: W_t5 is [N, bitlinear_t5_row_bytes(K)] uint8 (out); other arguments and errors as
 * bitlinear_quantize_weights.  K % 4 == 0, K <= 65536.
 */
size_t bitlinear_t5_row_bytes(int64_t K);
int bitlinear_quantize_weights_t5(const float* W, int64_t N, int64_t K, uint8_t* W_t5, float* alpha,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The 2-bit packing of bitlinear_quantize_weights ([N, K/4]) repacked five codes per byte
 * into W_t5 ([N, bitlinear_t5_row_bytes(K)]): the same codes.  Errors: INVALID_ARG, SHAPE, HIP. */
int bitlinear_repack_t5(const uint8_t* W_packed, int64_t N, int64_t K, uint8_t* W_t5, hipStream_t stream);

/*
 * bitlinear_forward on 5-trit packed weights (16-byte aligned W_t5): the same acc and y as
 * bitlinear_forward on the 2-bit packing of the same codes.  The kernel is a decode GEMV
 * (one token per grid row; more tokens re-read the weights).  No acc output.  Bytes above
 * 242 are never written by the packers; if present they give unspecified outputs.
 * Errors: INVALID_ARG, SHAPE (K > 65536, M > 65535, ...), ALIGNMENT, HIP.
 */
int bitlinear_forward_t5(const int8_t* x_q, const float* beta, int64_t M, int64_t K, const uint8_t* W_t5,
                         const float* alpha, int64_t N, const float* bias, float* y, hipStream_t stream);

/*
 * Block-scaled weights [P1 §2.3, §4.2]: one scale per block of 128 consecutive weights of a
 * row, alpha_blocks of shape [N, K/128]:
 *     alpha_blocks[n, b] = mean |W[n, 128b .. 128b+127]|   (fp64 sum, one fp32 rounding)
 *     W_hat[n, k]        = clip(round(W[n, k] / alpha_blocks[n, k/128]), -1, 1)
 * (fp32 division, round-half-to-even; an all-zero block has alpha 0 and codes 0), packed as
 * above.  W is read once.
 *   W [N, K] fp32, 16-byte aligned (in); W_packed [N, K/4] uint8 (out);
 *   alpha_blocks [N, K/128] fp32, 4-byte aligned (out).
 * Errors: INVALID_ARG, SHAPE (K % 128, sizes), ALIGNMENT, HIP.
 */
int bitlinear_quantize_weights_blocks(const float* W, int64_t N, int64_t K, uint8_t* W_packed,
                                      float* alpha_blocks, hipStream_t stream);

/*
 * Forward with block-scaled weights [P1 §2.3; P2 §3.3; P3 §2.4]:
 *     acc[m, n, b] = sum over k in block b of x_q[m, k] * W_hat[n, k]      (int32, exact)
 *     y[m, n]      = fp32(S * (beta[m] / 127))  (+ bias[n], a separate fp32 addition)
 *     S            = sum_b alpha_blocks[n, b] * acc[m, n, b]
 * with S and beta/127 in fp64.  The products alpha*acc are exact in fp64; the additions run
 * in an order fixed by the kernel, so y can differ from an fp64 sum taken in another order by
 * one fp32 rounding in rare cases (results are reproducible run to run).
 *   x_q [M, K] int8, beta [M] fp32 (from bitlinear_quantize_act); W_packed [N, K/4] uint8 and
 *   alpha_blocks [N, K/128] fp32 (from bitlinear_quantize_weights_blocks); bias [N] or NULL;
 *   y [M, N] fp32 (out).  x_q and W_packed 16-byte aligned, alpha_blocks 4-byte aligned.
 * K % 128 == 0, K <= 32768 and M <= 262140.  One or two tokens run a GEMV; 3 to 127 run an
 * int8 MFMA kernel over slices of up to 64 tokens (32 when K % 256 != 0),
 * each slice reading the codes once; 128 and more an int8 MFMA GEMM.
 * Errors: INVALID_ARG, SHAPE, ALIGNMENT, HIP.
 */
int bitlinear_forward_blocks(const int8_t* x_q, const float* beta, int64_t M, int64_t K,
                             const uint8_t* W_packed, const float* alpha_blocks, int64_t N,
                             const float* bias, float* y, hipStream_t stream);

/*
 * Randomized Hadamard rotation along K [P3 §6.2], the preprocessing that spreads an outlier
 * channel over all dimensions before the absmax.  For each row r of x and each block of B
 * consecutive columns (B = `block`, a power of two, 1 <= B <= 4096, K % B == 0):
 *     out[r, blk] = (d[blk] * x[r, blk]) . H_B / sqrt(B)
 * with d[k] = -1 where signs[k] < 0, +1 elsewhere (signs NULL: all +1), and H_B the Sylvester
 * Hadamard matrix (H_1 = [1], H_2n = [[H_n, H_n], [H_n, -H_n]]).  Evaluation, fixed so that
 * results are reproducible bit for bit: the sign flip is exact; the transform runs as fp32
 * butterflies (a, b) -> (a + b, a - b) on element pairs (j, j + h), h = 1, 2, 4, ..., B/2 in
 * that order; every result is then multiplied once by fp32(1/sqrt(B)) (exact for B a power
 * of 4).  The rotation is orthonormal (R R^T = I): rotating the rows of W with the same
 * block and signs (once, before bitlinear_quantize_weights) and every x keeps x . W^T.
 *
 *   x      [M, K] fp32, 16-byte aligned.            (in)
 *   signs  [K] int8, 4-byte aligned, or NULL.       (in; the caller draws them)
 *   out    [M, K] fp32, 16-byte aligned; may be x (in place), else must not overlap it. (out)
 * K % 4 == 0.  Errors: INVALID_ARG, SHAPE (block not a power of two in [1, 4096], K % block,
 * K % 4, size overflow), ALIGNMENT, HIP.
 */
int bitlinear_hadamard_rows(const float* x, int64_t M, int64_t K, int64_t block, const int8_t* signs,
                            float* out, hipStream_t stream);

/*
 * Rotation then activation quantization in one pass [P3 §6.2, §2.4]: x_q and beta are those
 * bitlinear_quantize_act gives for the rows rotated by bitlinear_hadamard_rows (same block
 * and signs), without writing the rotated rows.  Feed x_q and beta to bitlinear_forward with
 * weights quantized from rotated rows.
 *
 *   x      [M, K] fp32, 16-byte aligned.            (in)
 *   signs  [K] int8, 4-byte aligned, or NULL.       (in)
 *   x_q    [M, K] int8, 4-byte aligned.             (out)
 *   beta   [M] fp32.                                (out)
 * Errors as bitlinear_hadamard_rows.
 */
int bitlinear_quantize_act_hadamard(const float* x, int64_t M, int64_t K, int64_t block,
                                    const int8_t* signs, int8_t* x_q, float* beta, hipStream_t stream);

/*
 * BitMLP forward [P3 §6.1]: y = fc2(GELU(fc1(x))) with both layers BitLinear (per-tensor
 * alpha, weights from bitlinear_quantize_weights), fc1: d_model -> d_ff, fc2: d_ff -> d_model.
 * GELU is the erf form, 0.5 h (1 + erf(h / sqrt 2)), evaluated in fp64 and rounded to fp32
 * once, applied in fc1's dequantization epilogue; fc2 quantizes its fp32 input per token
 * like any activation.  Each layer runs as bitlinear_forward_fused would (one fused launch
 * for M <= 4, else quantize_act then forward), so results equal the two calls
 *     g = GELU(bitlinear_forward_fused(x, W1...)),  y = bitlinear_forward_fused(g, W2...).
 *
 *   x        [M, d_model] fp32.                                   (in)
 *   W1_packed [d_ff, d_model/4], alpha1 [1], bias1 [d_ff] or NULL. (in)
 *   W2_packed [d_model, d_ff/4], alpha2 [1], bias2 [d_model] or NULL. (in)
 *   y        [M, d_model] fp32.                                   (out)
 *   g        [M, d_ff] fp32: GELU(fc1(x)), fc2's input.            (out, required)
 *   x_q1, beta1 / x_q2, beta2: each layer's quantized input ([M, d] int8, [M] fp32), as
 *   the x_q / beta of bitlinear_forward_fused (required when M > 4 or unaligned).
 * Both layers are validated before anything is enqueued.  Errors as bitlinear_forward_fused.
 */
int bitlinear_mlp_forward(const float* x, int64_t M, int64_t d_model, int64_t d_ff,
                          const uint8_t* W1_packed, const float* alpha1, const float* bias1,
                          const uint8_t* W2_packed, const float* alpha2, const float* bias2,
                          float* y, float* g, int8_t* x_q1, float* beta1, int8_t* x_q2,
                          float* beta2, hipStream_t stream);

/*
 * Rotation, activation quantization and forward in one call [P3 §6.2, §2.4, §3.2]: y from
 * fp32 x with results identical to bitlinear_quantize_act_hadamard (same block and signs)
 * followed by bitlinear_forward on weights quantized from rotated rows.  One token with
 * K % 64 == 0, K <= 16384 and 16-byte aligned W_packed runs as a single launch (every
 * workgroup rotates and quantizes x, then streams its weight rows); other calls need x_q and
 * beta and run the two steps.  x_q / beta (may be NULL on the single-launch path) receive the
 * quantized rotated activations.  Errors as bitlinear_quantize_act_hadamard and
 * bitlinear_forward.
 */
int bitlinear_forward_fused_hadamard(const float* x, int64_t M, int64_t K, int64_t block, const int8_t* signs,
                                     const uint8_t* W_packed, const float* alpha, int64_t N, const float* bias,
                                     float* y, int8_t* x_q, float* beta, hipStream_t stream);

/* Activation a(g) of the gated feed-forward block. */
typedef enum bitlinear_activation {
    BITLINEAR_ACT_GELU = 1, /* g Phi(g), the erf form of bitlinear_mlp_forward */
    BITLINEAR_ACT_SILU = 2, /* g / (1 + exp(-g)) */
    BITLINEAR_ACT_RELU2 = 3 /* max(g, 0)^2 */
} bitlinear_activation;

/*
 * Gated feed-forward block, both projections, the activation and the product in one call:
 *     g = BitLinear(x; Wg, alpha_g, bias_g),  u = BitLinear(x; Wu, alpha_u, bias_u),
 *     h[m, n] = a(g[m, n]) * u[m, n].
 * x is quantized as by bitlinear_quantize_act; g and u equal bitlinear_forward's y for the two
 * matrices bit for bit; a(g) is evaluated in fp32 (SiLU within 7 * 2^-24 relative or 2^-120
 * absolute; GELU as bitlinear_mlp_forward; squared ReLU one rounding) and the product is one
 * fp32 rounding.  Where g overflows or a bias is not finite, a(g) is its limit (NaN for GELU at
 * -infinity) and NaN for NaN.  The block's down projection is a bitlinear_quantize_act of h and
 * any forward call.
 *
 *   x          [M, K] fp32.                                                  (in)
 *   Wg_packed, Wu_packed  [F, K/4] uint8; alpha_g, alpha_u [1]; bias_g, bias_u [F] or NULL. (in)
 *   act        a bitlinear_activation.
 *   h          [M, F] fp32.                                                  (out)
 *   g, u       [M, F] fp32, both or neither: kept for bitlinear_gated_backward. (out)
 *   x_q, beta  [M, K] int8, [M] fp32: receive the quantized activations.     (out, required)
 * K % 4 == 0; any alignment.  Outputs must not overlap inputs or each other.
 * Errors: INVALID_ARG (null pointer, size <= 0, unknown act, one of g and u), SHAPE, HIP.
 */
int bitlinear_gated_forward(const float* x, int64_t M, int64_t K, const uint8_t* Wg_packed, const float* alpha_g,
                            const float* bias_g, const uint8_t* Wu_packed, const float* alpha_u,
                            const float* bias_u, int64_t F, int act, float* h, float* g, float* u, int8_t* x_q,
                            float* beta, hipStream_t stream);

/*
 * Gradients of one BitLinear y = bitlinear_forward(x_q, beta, W_packed, alpha, bias), straight
 * through both quantizers [P3 §3.3]: x and the latent W get the gradients of the products with
 * the values that were used,
 *     dx[m, k]  = alpha sum_n dy[m, n] W_hat[n, k]
 *     dW[n, k]  = sum_m dy[m, n] (beta[m] / 127) x_q[m, k]
 *     dbias[n]  = sum_m dy[m, n].
 * dy alpha and dy beta / 127, rounded to fp32, enter products within 2^-23 of themselves, whatever
 * their size beside the others of a row (dx) or column (dW) if it matters to the sum: an element
 * below 2^-28 of the largest may enter with an error that is below 2^-23 of the sum it is a term
 * of.  The products are exact, and sums are taken in fp32 (dbias in fp64) in an order fixed by the
 * sizes and, where elements so small make up a sum, by the values; results are reproducible bit for
 * bit.  (Up to 16 tokens dy enters whole, and beta x_q / 127 rounded to fp32.)  The time depends on
 * the values only there: rows of little else than such elements, in sums that the larger ones do
 * not enter, take a vector product's time (75 ms for 2048 tokens, 4096 -> 11008, instead of 0.6).
 *
 *   dy        [M, N] fp32.                                                   (in)
 *   x_q       [M, K] int8, beta [M] fp32: as bitlinear_forward used them.    (in)
 *   W_packed  [N, K/4] uint8, alpha [1] fp32.                                (in)
 *   dx        [M, K] fp32 or NULL.     dW  [N, K] fp32 or NULL.              (out)
 *   dbias     [N] fp32 or NULL.                                              (out)
 *   workspace >= bitlinear_backward_workspace_size(M, K, N) bytes, 256-byte aligned; scratch,
 *             one for each call that may overlap another.  It grows with the tokens: dy in two
 *             layouts, x_q and W at a byte an element, and parts of sums (2048 tokens, 11008 ->
 *             4096: 137 MB; gated 4096 -> 11008: 471 MB).
 * K % 4 == 0, M and N <= 2097152; any alignment of the tensors.  At least one output is given;
 * outputs must not overlap inputs or each other.  Errors: INVALID_ARG, SHAPE, ALIGNMENT and WORKSPACE (the
 * workspace), HIP.
 */
size_t bitlinear_backward_workspace_size(int64_t M, int64_t K, int64_t N);
int bitlinear_backward(const float* dy, int64_t M, int64_t N, const int8_t* x_q, const float* beta, int64_t K,
                       const uint8_t* W_packed, const float* alpha, float* dx, float* dW, float* dbias,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of bitlinear_gated_forward from dh, the gradient of h, and the g, u, x_q and beta it
 * left.  With dg = dh u a'(g) and du = dh a(g) (fp32), dx is the sum of both projections' dx of
 * bitlinear_backward, and dWg, dWu, dbias_g, dbias_u are those of the two projections; the same
 * accuracy holds.  a' of squared ReLU is 2 max(g, 0); a and a' of g that is not finite are their
 * limits and NaN as in the forward pass.
 *
 *   dh, g, u  [M, F] fp32.                                                   (in)
 *   dx        [M, K] or NULL.   dWg, dWu  [F, K], both or neither.           (out)
 *   dbias_g, dbias_u  [F] or NULL, each.                                     (out)
 *   workspace >= bitlinear_gated_backward_workspace_size(M, K, F) bytes, as bitlinear_backward.
 * Errors: as bitlinear_backward, and INVALID_ARG for an unknown act or one of dWg and dWu.
 */
size_t bitlinear_gated_backward_workspace_size(int64_t M, int64_t K, int64_t F);
int bitlinear_gated_backward(const float* dh, const float* g, const float* u, int64_t M, int64_t F,
                             const int8_t* x_q, const float* beta, int64_t K, const uint8_t* Wg_packed,
                             const float* alpha_g, const uint8_t* Wu_packed, const float* alpha_u, int act,
                             float* dx, float* dWg, float* dWu, float* dbias_g, float* dbias_u, void* workspace,
                             size_t workspace_bytes, hipStream_t stream);

/*
 * Weights kept in 8 bits (output heads, projections too sensitive for three values), one absmax
 * scale per output channel: W_q and gamma are what bitlinear_quantize_act gives for the rows of W,
 *     gamma[n] = max_k |W[n, k]| + 1e-8,  W_q[n, k] = clip(round(fp32(127 W[n, k]) / gamma[n]), -127, 127).
 *   W [N, K] fp32 (in);  W_q [N, K] int8, gamma [N] fp32 (out).  Any K >= 1.
 * Errors: INVALID_ARG, SHAPE, HIP.
 */
int bitlinear_quantize_weights_i8(const float* W, int64_t N, int64_t K, int8_t* W_q, float* gamma,
                                  hipStream_t stream);

/*
 * int8 x int8 matmul with a scale for each token and each output channel:
 *     acc[m, n] = sum_k x_q[m, k] * W_q[n, k]                              (int32, exact)
 *     y[m, n]   = (fp32(acc) * fp32(beta[m] / 127)) * fp32(gamma[n] / 127)  (+ bias[n])
 * every step one fp32 rounding.  Codes lie in [-127, 127].
 *   x_q [M, K] int8, beta [M] fp32 (from bitlinear_quantize_act); W_q [N, K] int8, gamma [N]
 *   (from bitlinear_quantize_weights_i8); bias [N] or NULL.                  (in)
 *   y [M, N] fp32; acc [M, N] int32 or NULL.                                 (out)
 * K <= 133144 (so that acc fits); any alignment.  Errors: INVALID_ARG, SHAPE, HIP.
 */
int bitlinear_forward_i8(const int8_t* x_q, const float* beta, int64_t M, int64_t K, const int8_t* W_q,
                         const float* gamma, int64_t N, const float* bias, float* y, int32_t* acc,
                         hipStream_t stream);

/*
 * Weights and activations in 8-bit floating point (e4m3: sign, 4 exponent and 3 mantissa bits, largest
 * value 448, no infinities), one fp32 scale for each block of 128 along K:
 *     scale = fp32(absmax of the block / 448),  code = e4m3(clip(fp32(v / scale), -448, 448)),
 * rounded to nearest, ties to even.  A block of zeros (or whose scale is below the fp32 range) has
 * scale 0 and codes 0.  The last block of a row ends with the row.  NaN and infinities have the code
 * NaN (and an infinity makes its block's scale infinite); the products with them are then not finite.
 *   quantize_act_fp8:      blocks of one token x 128; x [M, K] fp32 (in); x_q [M, K] e4m3,
 *                          x_scale [ceil(K / 128), M] fp32 (out): the tokens' scales of a block lie
 *                          together, as a tile of tokens reads them.
 *   quantize_weights_fp8:  blocks of 128 x 128; W [N, K] fp32 (in); W_q [N, K] e4m3,
 *                          W_scale [ceil(N / 128), ceil(K / 128)] fp32 (out).
 * 1 <= K <= 4194304, M and N <= 67108864, M K and N K <= 2^40; any alignment of fp32 elements.
 * Errors: INVALID_ARG, SHAPE, HIP.
 */
int bitlinear_quantize_act_fp8(const float* x, int64_t M, int64_t K, uint8_t* x_q, float* x_scale,
                               hipStream_t stream);
int bitlinear_quantize_weights_fp8(const float* W, int64_t N, int64_t K, uint8_t* W_q, float* W_scale,
                                   hipStream_t stream);

/*
 * e4m3 x e4m3 matmul with a scale for each block of 128:
 *     y[m, n] = sum_b (x_scale[b, m] W_scale[n / 128, b]) sum_{k in block b} x_q[m, k] W_q[n, k]  (+ bias[n])
 * Products are exact; a block's sum, its product with the scales and the sum over blocks are taken in
 * fp32, in an order fixed by the sizes (and the alignment): results are reproducible bit for bit.
 *   x_q [M, K], x_scale [ceil(K / 128), M]; W_q [N, K], W_scale [ceil(N / 128), ceil(K / 128)], as the
 *   quantizers lay them out; bias [N] or NULL.                               (in)
 *   y [M, N] fp32.                                                           (out)
 * 1 <= K <= 4194304, M and N <= 67108864, M K and N K <= 2^40, M N <= 2^36; any alignment.
 * Errors: INVALID_ARG, SHAPE, HIP.
 */
int bitlinear_forward_fp8(const uint8_t* x_q, const float* x_scale, int64_t M, int64_t K, const uint8_t* W_q,
                          const float* W_scale, int64_t N, const float* bias, float* y, hipStream_t stream);

/*
 * Products grouped by expert (the experts of a mixture layer): E BitLinears of one shape over M rows that
 * lie sorted by expert, any number of rows for each, none among them.  Group e is the rows
 * offsets[e] .. offsets[e + 1] - 1; row m reads token r = rows[m], or r = m where rows is NULL:
 *     y[m, n] = bitlinear_forward(x_q[r], beta[r], W_packed[e], alpha[e], bias[e])[n],
 * bit for bit.  Rows outside every group are left as they were in y.
 *
 *   x_q       [T, K] int8, beta [T] fp32: the tokens, from bitlinear_quantize_act.   (in)
 *   rows      [M] int64 token of each row, or NULL (then T == M).  A token may occur any number of
 *             times; an index outside 0 .. T - 1 reads a token of zeros (x_q = 0, beta = 0).  (in)
 *   offsets   [E + 1] int64, on the device, not decreasing, within 0 .. M; beyond, they are taken as
 *             0 or M, and a group that ends before it begins as empty.  Offsets that decrease, so that
 *             groups share rows, leave unspecified values in the outputs and touch nothing else.  (in)
 *   W_packed  [E, N, K/4] uint8; alpha [E]; bias [E, N] or NULL.              (in)
 *   y         [M, N] fp32.                                                   (out)
 * K % 4 == 0, E <= 4096, N <= 2^20, M <= 2^24, T < 2^31, T K and T N <= 2^40, E N K <= 2^42, and no more work than a
 * launch holds: M N <= 2^35 and min(E, M) N <= 2^29, with N counted in multiples of 128, always do.  Any alignment of
 * elements of their type.  M == 0 is a call without rows, for which x_q, beta, rows and y may be NULL.
 * Outputs must not overlap inputs.  The host reads no device memory: the call can be captured into a graph
 * and replayed with other offsets and rows.
 * Errors: INVALID_ARG (null pointer, size < 0, K, N or E == 0, T == 0 with rows), SHAPE (T != M where rows is NULL and M > 0), HIP.
 */
int bitlinear_grouped_forward(const int8_t* x_q, const float* beta, int64_t T, int64_t K, const int64_t* rows,
                              int64_t M, const int64_t* offsets, int64_t E, const uint8_t* W_packed,
                              const float* alpha, int64_t N, const float* bias, float* y, hipStream_t stream);

/*
 * bitlinear_gated_forward grouped by expert: the T tokens x are quantized as by bitlinear_quantize_act, and
 * row m of h (and g, u) is the gated block of token r under expert e's gate and up projections.
 *   x [T, K] fp32; rows, offsets as bitlinear_grouped_forward.              (in)
 *   Wg_packed, Wu_packed [E, F, K/4]; alpha_g, alpha_u [E]; bias_g, bias_u [E, F] or NULL.  (in)
 *   h [M, F]; g, u [M, F], both or neither; x_q [T, K], beta [T]: the quantized tokens.     (out)
 * Errors: as bitlinear_grouped_forward, and INVALID_ARG for an unknown act or one of g and u.
 */
int bitlinear_grouped_gated_forward(const float* x, int64_t T, int64_t K, const int64_t* rows, int64_t M,
                                    const int64_t* offsets, int64_t E, const uint8_t* Wg_packed,
                                    const float* alpha_g, const float* bias_g, const uint8_t* Wu_packed,
                                    const float* alpha_u, const float* bias_u, int64_t F, int act, float* h,
                                    float* g, float* u, int8_t* x_q, float* beta, hipStream_t stream);

/*
 * Gradients of bitlinear_grouped_forward, straight through both quantizers: with e the group of m and
 * r its token,
 *     dx[m, k]    = alpha[e] sum_n dy[m, n] W_hat[e, n, k]           (of the row; a token's is the sum of its rows')
 *     dW[e, n, k] = sum_{m in e} dy[m, n] (beta[r] / 127) x_q[r, k]
 *     dbias[e, n] = sum_{m in e} dy[m, n].
 * fp32(dy alpha) and fp32(dy fp32(beta / 127)) enter the products whole (but for what lies below 2^-126),
 * the products are exact, and sums are taken in fp32 (dbias in fp64) in an order fixed by the sizes and the
 * offsets: results are reproducible bit for bit.  An expert without rows has dW and dbias 0; rows outside
 * every group are left as they were in dx and add nothing to dW.  A gradient that is not finite makes its
 * row of dx and its row dW[e, n] not finite, and no others.
 *
 *   dy [M, N] fp32; x_q, beta, rows, offsets, W_packed, alpha as the forward call used them.     (in)
 *   dx [M, K], dW [E, N, K], dbias [E, N], each or NULL, one at least.                           (out)
 *   workspace >= bitlinear_grouped_backward_workspace_size(M, K, N, E) bytes, 256-byte aligned; scratch,
 *             one for each call that may overlap another.
 * Sizes as the forward call's, and no more work than a launch holds: E N K <= 2^36, E N <= 2^26, E K <= 2^27 and
 * M K <= 2^35, with N counted in multiples of 128 and K of 256, always do.  (Whichever gradients are asked for; the
 * workspace size of what does not fit is 0.)  Errors: as the forward call, SHAPE (does not fit), ALIGNMENT and WORKSPACE
 * (the workspace).
 */
size_t bitlinear_grouped_backward_workspace_size(int64_t M, int64_t K, int64_t N, int64_t E);
int bitlinear_grouped_backward(const float* dy, int64_t M, int64_t N, const int8_t* x_q, const float* beta, int64_t T,
                               int64_t K, const int64_t* rows, const int64_t* offsets, int64_t E,
                               const uint8_t* W_packed, const float* alpha, float* dx, float* dW, float* dbias,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of bitlinear_grouped_gated_forward from dh and the g, u, x_q and beta it left: with
 * dg = dh u a'(g) and du = dh a(g) (fp32, as bitlinear_gated_backward), dx is the sum of both projections'
 * and dWg, dWu, dbias_g, dbias_u are theirs, as bitlinear_grouped_backward.
 *   dh, g, u [M, F].   dx [M, K] or NULL; dWg, dWu [E, F, K], both or neither; dbias_g, dbias_u [E, F] or NULL.
 *   workspace >= bitlinear_grouped_gated_backward_workspace_size(M, K, F, E) bytes: dg and du.
 * Errors: as bitlinear_grouped_backward, and INVALID_ARG for an unknown act or one of dWg and dWu.
 */
size_t bitlinear_grouped_gated_backward_workspace_size(int64_t M, int64_t K, int64_t F, int64_t E);
int bitlinear_grouped_gated_backward(const float* dh, const float* g, const float* u, int64_t M, int64_t F,
                                     const int8_t* x_q, const float* beta, int64_t T, int64_t K, const int64_t* rows,
                                     const int64_t* offsets, int64_t E, const uint8_t* Wg_packed,
                                     const float* alpha_g, const uint8_t* Wu_packed, const float* alpha_u, int act,
                                     float* dx, float* dWg, float* dWu, float* dbias_g, float* dbias_u,
                                     void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Kernel(s) bitlinear_forward_fused launches for these arguments ("gemv_fused" or
 * "quantize_act+forward"; a non-NULL x_q stands for x_q and beta given); a static string. */
const char* bitlinear_forward_fused_kernel(int64_t M, int64_t K, int64_t N, const float* x,
                                           const uint8_t* W_packed, const int8_t* x_q);

/*
 * Name of the kernel bitlinear_forward launches for these arguments ("gemv_dot4",
 * "decode_mfma_i8", "gemm_mfma_i8" or "generic"); a static string, for profiling and reports.
 */
const char* bitlinear_forward_kernel(int64_t M, int64_t K, int64_t N, const int8_t* x_q,
                                     const uint8_t* W_packed);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_H */
