/*
 * bit_moe_expert_gb300 -- MXFP4: microscaled 4-bit floating point, its products
 * and expert layers.
 *
 * Format (OCP Microscaling Formats, MXFP4): 32 consecutive values along K share
 * one E8M0 scale, a byte s that stands for 2^(s-127) (255 for NaN); each value
 * is an E2M1 code (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2,
 * 3, 4, 6 and their negatives) times the scale.  4.25 bits per value.
 *
 * Products run on the block-scaled tensor cores (both operands MXFP4, the
 * scales applied by the multiply, fp32 accumulation), so activations are
 * quantised too: x -> MXFP4 by moe_mx_quantize's rule, in every call and for
 * every token count, which makes a token's result independent of the batch it
 * comes in.
 *
 * The conventions of moe.h hold: device pointers, 16-byte aligned, owned by the
 * caller; nothing allocated; asynchronous on `stream`; capturable; checks on the
 * host before any launch; workspaces zero-filled once, 256-byte aligned, one
 * call in flight per workspace, device-side errors in their status word
 * (moe_check_status).  Products read weights before waiting for the previous
 * kernel on the stream; after moe_mx_quantize, moe_mx_prepack_scales and
 * moe_mx_dequant, which let no kernel start before they have completed, they may
 * follow directly.  Weights that any other kernel wrote are separated as moe.h
 * says.
 */
#ifndef BIT_MOE_EXPERT_GB300_MOE_MX_H
#define BIT_MOE_EXPERT_GB300_MOE_MX_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations and results. */
typedef enum { MOE_BF16 = 0, MOE_FP16 = 1, MOE_FP32 = 2 } moe_dtype;

/* A stack of E MXFP4 matrices of N rows and K columns (K a multiple of 32):
 *   q   uint8 [E][N][K/2]  two codes a byte, the lower column in the low
 *                          nibble (a checkpoint's row-major layout)
 *   sp  uint8 [E][ceil(N/128)][ceil(K/128)][512]  the scales in the order that
 *                          tensor memory takes them: one 512-byte piece holds
 *                          128 rows x 4 blocks of 32 columns, the byte of row r,
 *                          block b of the piece at 16 (r % 32) + 4 (r / 32) + b.
 *                          Bytes of blocks past K must not be 255 (they are
 *                          written as 0); bytes of rows past N are not used.
 *                          Build it from row-major scales [E][N][K/32] with
 *                          moe_mx_prepack_scales; moe_mx_quantize writes it. */
typedef struct {
  uint8_t* q;
  uint8_t* sp;
} moe_mx_mat;

/* Bytes of sp; 0 for a bad size. */
size_t moe_mx_scale_bytes(int E, int N, int K);

/* Row-major E8M0 scales [E][N][K/32] -> sp.  MOE_ERR_INVALID_ARG on a bad size
 * or pointer.  (Codes need no reordering.) */
moe_status moe_mx_prepack_scales(const uint8_t* scale, int E, int N, int K, uint8_t* sp, moe_stream stream);

/* X [rows][K] of type `type`, rows ldx elements apart -> *out (E = 1, N = rows).
 * Per block: a = max |x|, e = clamp(floor(log2 a) - 2, -127, 127) (-127 for a =
 * 0), code = x 2^-e rounded to the nearest E2M1 value, ties to the even code,
 * magnitudes above 6 to 6.  A block with a NaN or an infinity gets the scale
 * 255: its values, and every product with it, are NaN.
 * Preconditions: rows >= 0, K a positive multiple of 32, ldx >= K, X and the
 * row pitch multiples of 16 bytes. */
moe_status moe_mx_quantize(const void* X, moe_dtype type, int rows, int K, long long ldx, const moe_mx_mat* out,
                           moe_stream stream);

/* W [E][N][K] of type `type` (bf16: exact unless the value leaves bf16's range;
 * fp32: exact; fp16 is not offered: MOE_ERR_UNSUPPORTED) = the values of m. */
moe_status moe_mx_dequant(const moe_mx_mat* m, int E, int N, int K, moe_dtype type, void* W, moe_stream stream);

/* Y [M][N] of type y_type (bf16 or fp32; rounded once from the fp32 sum; rows N
 * elements apart) = A [M][K] times W [N][K] transposed, both MXFP4.  ws: at
 * least 256 bytes (the status word).  M = 0 does nothing. */
moe_status moe_mx_matmul(const moe_mx_mat* A, int M, const moe_mx_mat* W, int N, int K, void* Y, moe_dtype y_type,
                         void* ws, size_t ws_bytes, moe_stream stream);

/* Workspace bytes of moe_mx_linear (the quantised X); 0 for a bad size. */
size_t moe_mx_linear_workspace_bytes(int T, int N, int K);

/* A linear layer with MXFP4 weights W [N][K]: moe_mx_quantize(X [T][K]) into
 * the workspace, then moe_mx_matmul. */
moe_status moe_mx_linear(const void* X, moe_dtype x_type, int T, int K, long long ldx, const moe_mx_mat* W, int N,
                         void* Y, moe_dtype y_type, void* ws, size_t ws_bytes, moe_stream stream);

/* One expert set: gate and up [E][I][d], down [E][d][I]. */
typedef struct {
  moe_mx_mat gate;
  moe_mx_mat up;
  moe_mx_mat down;
  int n_experts;
} moe_mx_experts;

/* Workspace bytes of moe_mx_forward; block_rows: the routing's tile height. */
size_t moe_mx_forward_workspace_bytes(int T, int d, int I, int E, int k, int I_shared, int block_rows);

/* The expert layer on MXFP4 weights, bf16 X [T][d] -> bf16 Y [T][d]:
 *   Y[t] = sum_j w[t][j] FFN_{ids[t][j]}(x_t) + FFN_shared(x_t)
 *   FFN(x) = MX(silu(MX(x) Wg^T) * (MX(x) Wu^T)) Wd^T
 * with MX() the rounding of moe_mx_quantize; the products, SwiGLU and the sums
 * over experts (in slot order, the shared expert last) are in fp32, the second
 * MX() takes the fp32 SwiGLU (in it, silu of a value below -87.3 is 0), and Y is
 * rounded to bf16 once.
 * Arguments as for moe_forward; d, I and I_shared multiples of 32.
 * MOE_ERR_UNSUPPORTED also where moe_route_max_blocks times ceil(max(d, I) /
 * 128), plus the shared expert's tiles likewise, is above 2^30. */
moe_status moe_mx_forward(const uint16_t* X, int T, int d, int I, int k, const moe_mx_experts* routed,
                          const moe_mx_experts* shared, int I_shared, const moe_routing* r, uint16_t* Y, void* ws,
                          size_t ws_bytes, moe_stream stream);

size_t moe_mx_layer_workspace_bytes(int T, int d, int I, int E, int k, int I_shared, int block_rows);

/* moe_route_scored, then moe_mx_forward, with the same arguments and results. */
moe_status moe_mx_layer(const float* logits, const moe_scoring* scoring, const uint16_t* X, int T, int d, int I, int k,
                        int block_rows, const moe_mx_experts* routed, const moe_mx_experts* shared, int I_shared,
                        moe_routing* r, uint16_t* Y, void* ws, size_t ws_bytes, moe_stream stream);

#ifdef __cplusplus
}
#endif
#endif
