/*
 * bit_moe_expert_gb300 -- 8-bit floating point with block scales: quantisation,
 * products, expert layers, and the RMS norm that feeds them.
 *
 * Format: E4M3 codes (sign, four exponent bits, three mantissa bits: up to 448,
 * 0x7F and 0xFF NaN, no infinities) times an fp32 scale per block of 128.
 *   weights      [E][N][K]: one scale per block of 128 rows x 128 columns of a
 *                matrix (a checkpoint's layout: nothing is reordered);
 *   activations  [rows][K]: one scale per 128 columns of a row.
 * The last block of a row or column may be short: K is a multiple of 16, N any.
 * Scales are any fp32 numbers; the quantisation here makes powers of two, so
 * that a code's one rounding is all that it loses.
 *
 * Products are exact but for fp32 accumulation: the codes' products of a block
 * of 128 columns are added up on the tensor cores, multiplied by the product of
 * the two scales (which must lie in fp32's range) and added to the blocks before
 * it, all in fp32.  A product's order of additions depends on the path that its
 * sizes take, not on timing: the same call gives the same bits.  NaN codes and
 * scales make NaN results of the rows and columns that they belong to.
 *
 * The conventions of moe.h hold: device pointers, 16-byte aligned, owned by the
 * caller; nothing allocated; asynchronous on `stream`; capturable; checks on the
 * host before any launch; workspaces zero-filled once, 256-byte aligned, one
 * call in flight per workspace, device-side errors in their status word
 * (moe_check_status).  Products read weights (codes and scales) before waiting
 * for the previous kernel on the stream; after moe_blk_quantize_weights and the
 * moe_blk_dequant calls, which let no kernel start before they have completed,
 * they may follow directly.  Weights that any other kernel wrote are separated
 * as moe.h says.
 */
#ifndef BIT_MOE_EXPERT_GB300_MOE_BLK_H
#define BIT_MOE_EXPERT_GB300_MOE_BLK_H

#include "moe_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Codes and scales.
 *   weights      q uint8 [E][N][K], s float [E][ceil(N/128)][ceil(K/128)]
 *   activations  q uint8 [rows][K], s float [ceil(K/128)][R], R = rows rounded up
 *                to a multiple of 4: the scales of one block of columns are
 *                neighbours.  What the last R - rows of each hold does not
 *                matter; a call that writes scales may write them. */
typedef struct {
  uint8_t* q;
  float* s;
} moe_blk_mat;

/* X [rows][K] of type `type`, rows ldx elements apart -> activations *out.
 * Per block: a = max |x|, scale 2^e with the least e >= -126 for which a <= 448
 * 2^e, code = x 2^-e rounded to the nearest E4M3 value, ties to the even code.
 * A block with a NaN or an infinity gets a NaN scale and NaN codes for its NaNs.
 * Preconditions: rows >= 0, K a positive multiple of 16, ldx >= K, X and the
 * row pitch multiples of 16 bytes. */
moe_status moe_blk_quantize(const void* X, moe_dtype type, int rows, int K, long long ldx, const moe_blk_mat* out,
                            moe_stream stream);

/* W [E][N][K] of type `type` (contiguous) -> weights *out, by the same rule over
 * blocks of 128 x 128. */
moe_status moe_blk_quantize_weights(const void* W, moe_dtype type, int E, int N, int K, const moe_blk_mat* out,
                                    moe_stream stream);

/* The values of activations a -> X [rows][K], of weights m -> W [E][N][K]
 * (contiguous): code times scale in fp32, rounded to `type`.  (A magnitude next
 * to 2^128 may have been quantised up to it: infinity.) */
moe_status moe_blk_dequant(const moe_blk_mat* a, int rows, int K, moe_dtype type, void* X, moe_stream stream);
moe_status moe_blk_dequant_weights(const moe_blk_mat* m, int E, int N, int K, moe_dtype type, void* W,
                                   moe_stream stream);

/* Y [M][N] of type y_type (rounded once from the fp32 sum; rows N elements
 * apart) = activations A [M][K] times weights W [N][K] transposed.  ws: at
 * least 256 bytes (the status word).  M = 0 does nothing. */
moe_status moe_blk_matmul(const moe_blk_mat* A, int M, const moe_blk_mat* W, int N, int K, void* Y, moe_dtype y_type,
                          void* ws, size_t ws_bytes, moe_stream stream);

/* Workspace bytes of moe_blk_linear (the quantised X); 0 for a bad size. */
size_t moe_blk_linear_workspace_bytes(int T, int N, int K);

/* A linear layer: moe_blk_quantize(X [T][K]), then moe_blk_matmul.  (One token
 * may be quantised within the product, whose sums are then added in another
 * order than that of moe_blk_matmul.) */
moe_status moe_blk_linear(const void* X, moe_dtype x_type, int T, int K, long long ldx, const moe_blk_mat* W, int N,
                          void* Y, moe_dtype y_type, void* ws, size_t ws_bytes, moe_stream stream);

/* Root-mean-square norm of T rows of d columns, with the residual's addition
 * before it:
 *   r = x + residual, rounded to the residual's type and written to
 *       residual_out (which may be `residual`); r = x without a residual
 *   y = r / sqrt(mean(r^2) + eps) * gamma
 * y goes to Y (y_type), to the activations *out (quantised as by
 * moe_blk_quantize, from the unrounded y), or to both; the one that is not
 * wanted is NULL.
 *   X          [T][d] of x_type, rows ldx elements apart
 *   residual   NULL, or [T][d] contiguous; residual_type is x_type or MOE_FP32
 *   gamma      [d], bf16 or fp32 (gamma_type)
 * Y may be X itself where their types are the same and ldx = d.
 *
 * y is off by less than 2^-21 of itself; where that leaves a code or a scale
 * open, y is evaluated to about 2^-27 (2^-24 where a few values make up the
 * row's sum of squares).  A row whose sum of squares is not finite in
 * fp32 (or 0, with eps = 0) is NaN.  (That is where mean(r^2) + eps is at least
 * 2^-80, the squares of smaller numbers lose bits in fp32, and where neither y
 * nor r / sqrt(..) is below fp32's normal numbers.)  A y past fp32's range is
 * infinite, and so its block's scale NaN.
 * Preconditions: T >= 0 (0 does nothing), d a positive multiple of 16 up to
 * 32768 (MOE_ERR_UNSUPPORTED above), eps >= 0 and finite, X and the row pitch
 * multiples of 16 bytes. */
moe_status moe_rmsnorm(const void* X, moe_dtype x_type, int T, int d, long long ldx, const void* residual,
                       void* residual_out, moe_dtype residual_type, const void* gamma, moe_dtype gamma_type, float eps,
                       void* Y, moe_dtype y_type, const moe_blk_mat* out, moe_stream stream);

/* One expert set: gate and up [E][I][d], down [E][d][I]. */
typedef struct {
  moe_blk_mat gate;
  moe_blk_mat up;
  moe_blk_mat down;
  int n_experts;
} moe_blk_experts;

/* Workspace bytes of moe_blk_forward; block_rows: the routing's tile height. */
size_t moe_blk_forward_workspace_bytes(int T, int d, int I, int E, int k, int I_shared, int block_rows);

/* The expert layer on such weights -> bf16 Y [T][d]:
 *   Y[t] = sum_j w[t][j] FFN_{ids[t][j]}(x_t) + FFN_shared(x_t)
 *   FFN(x) = Q(silu(Q(x) Wg^T) * (Q(x) Wu^T)) Wd^T
 * with Q() the rounding of moe_blk_quantize; the products, SwiGLU and the sums
 * over experts are in fp32, and Y is rounded to bf16 once.
 *   X, XQ   bf16 X [T][d], or the activations XQ [T][d] that moe_rmsnorm or
 *           moe_blk_quantize wrote, taken as they are: one of them, the other
 *           NULL
 * Other arguments as for moe_forward; d, I and I_shared multiples of 32.  In
 * tables of the caller's own a token may take an expert more than once (for T <=
 * 8 a tile then has at most 8 rows: MOE_ERR_INVALID_ARG in the status word
 * above, by some of the paths that sizes take).
 * MOE_ERR_UNSUPPORTED also where moe_route_max_blocks times ceil(max(d, I) /
 * 128), plus the shared expert's tiles likewise, is above 2^30. */
moe_status moe_blk_forward(const uint16_t* X, const moe_blk_mat* XQ, int T, int d, int I, int k,
                           const moe_blk_experts* routed, const moe_blk_experts* shared, int I_shared,
                           const moe_routing* r, uint16_t* Y, void* ws, size_t ws_bytes, moe_stream stream);

size_t moe_blk_layer_workspace_bytes(int T, int d, int I, int E, int k, int I_shared, int block_rows);

/* moe_route_scored, then moe_blk_forward, with the same arguments and results. */
moe_status moe_blk_layer(const float* logits, const moe_scoring* scoring, const uint16_t* X, const moe_blk_mat* XQ,
                         int T, int d, int I, int k, int block_rows, const moe_blk_experts* routed,
                         const moe_blk_experts* shared, int I_shared, moe_routing* r, uint16_t* Y, void* ws,
                         size_t ws_bytes, moe_stream stream);

#ifdef __cplusplus
}
#endif
#endif
