// Launch entry points of the kernels, called by the host boundary (api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "status.h"

namespace bm {

// Kernel kinds for the optional per-kernel timing (moe_profile.h).
enum KernelKind {
  kKRoute = 0,
  kKDecode,    // the fused decode kernel (gate/up + down)
  kKRouter,    // the router projection
  kKXGather,
  kKGemmGateUp,
  kKGemmDown,
  kKCombine,
  kKPrepack,
  kKTopkWide,  // exact top-K of wide rows
  kKMxQuantize,  // MXFP4 quantisation (with or without the scatter to the routing's rows)
  kKMxGemm,      // MXFP4 dense product
  kKMxGateUp,
  kKMxDown,
  kKNorm,         // RMS norm
  kKBlkQuantize,  // block-scaled 8-bit quantisation (with or without the scatter to the routing's rows) and its inverse
  kKBlkGemm,      // block-scaled dense product
  kKBlkGateUp,
  kKBlkDown,
  kKernelKinds
};
void timer_begin(int id, cudaStream_t s);
void timer_end(int id, cudaStream_t s);

struct RouteOut {
  int32_t* ids;
  float* w;
  int32_t* counts;
  int32_t* offsets;
  int32_t* perm;
  int32_t* inv_perm;
  int32_t* block_map;
  int32_t* num_blocks;
};

// One-time launch set-up, per device and kernel, thread-safe: raise the
// kernel's dynamic shared-memory limit to at least `bytes`; the kernel's
// resident CTAs per SM at (threads, smem).
cudaError_t set_max_dynamic_smem(const void* func, int bytes);
cudaError_t occupancy_per_sm(const void* func, int threads, size_t smem, int* per_sm);

// x / n for 0 <= x, n <= 1024 as (x * small_inverse(n)) >> 20: with m = ceil(2^20 / n), x m / 2^20 exceeds x / n by
// x (m n - 2^20) / (2^20 n) < 1/n, since x (n - 1) < 2^20.
inline uint32_t small_inverse(int n) { return ((1u << 20) + n - 1) / n; }

// How a row is scored (include/moe.h, moe_scoring).
struct RouteScore {
  const float* bias;  // [E] or null
  int sigmoid, n_group, topk_group, group_top, renormalize;
  float scale;
  // set by launch_route, so that the kernel divides nothing:
  int per_lane;     // experts per lane: lane l holds per_lane l .. per_lane l + per_lane - 1
  int group_size;   // E / n_group
  int group_shift;  // every group is 2^group_shift whole lanes; -1 where it is not
  uint32_t group_inv;  // small_inverse(group_size)
};

size_t route_hist_elems(int T, int E);
// status: where device-side errors go (null: the workspace header's status word);
// score: null for the softmax over the selected logits
cudaError_t launch_route(const float* logits, int T, int E, int k, int block_rows, const RouteOut& out, void* ws,
                         cudaStream_t stream, bool pdl, uint32_t* status = nullptr,
                         const RouteScore* score = nullptr);
cudaError_t launch_prepack_codes(const uint32_t* q, int E, int N, int K, int bits, uint32_t* qp,
                                 cudaStream_t stream);
cudaError_t launch_prepack(const uint16_t* scale, const uint16_t* bias, int E, int N, int K, uint32_t* sb,
                           cudaStream_t stream);
// fp16 weights W [E][N][K] = q * scale + bias of one prepacked matrix (bits per code 2, 3 or 4)
cudaError_t launch_dequant(const uint32_t* qp, const uint32_t* sb, int E, int N, int K, int bits, uint16_t* W,
                           cudaStream_t stream);

// Router projection: logits [T][E] fp32 = X [T][d] bf16 times Wr [E][d] bf16
// transposed (d a multiple of 32).  With `maps` (router_tc_shape true), the
// tensor-core path: TMA tiles, tcgen05 MMAs, K split over a 4-CTA cluster.
constexpr int kRouterTcE = 128;     // experts per CTA (the MMA's M)
constexpr int kRouterTcT = 64;      // tokens per CTA (the MMA's N)
constexpr int kRouterTcSplit = 4;   // CTAs of a cluster, each a quarter of K
struct RouterMaps {
  CUtensorMap x;   // X [T][d] bf16, box (64, kRouterTcT), 128-byte swizzle
  CUtensorMap wr;  // Wr [E][d] bf16, box (64, kRouterTcE), 128-byte swizzle
};
bool router_tc_shape(int T, int d, int E);
cudaError_t launch_router(const uint16_t* X, int T, int d, const uint16_t* Wr, int E, float* logits,
                          const RouterMaps* maps, cudaStream_t stream, bool pdl);

// Exact top-K (K <= 64) of each row of logits [T][V] (V <= 2^20): values and
// indices [T][K], descending, a lower index first among equal values.
size_t topk_wide_smem_bytes(int V, int K);
cudaError_t launch_topk_wide(const float* logits, int T, int V, int K, float* values, int32_t* indices,
                             int num_sms, cudaStream_t stream, bool pdl);

// ---------------------------------------------------------------- decode GEMV
constexpr int kDecodeRowsGU = 32;      // gate/up rows per item (phase 1)
constexpr int kDecodeChunkGroups = 8;  // 64-column groups per gate/up stage
constexpr int kDecodeRowsDown = 16;    // output rows per block (phase 2)

// Tensor maps of one expert set for the decode kernel.
struct DecodeMaps {
  CUtensorMap q_gate, q_up;    // codes [E][d/64][I*wpg], box (32 rows * wpg words, kDecodeChunkGroups groups, 1)
  CUtensorMap sb_gate, sb_up;  // group parameters [E][d/64][I], box (32 rows, d/64 groups, 1)
  CUtensorMap q_down;          // codes [E][I/64][d*wpg], box (16 rows * wpg words, I/64 groups, 1)
  CUtensorMap sb_down;         // group parameters [E][I/64][d], box (16 rows, I/64 groups, 1)
};

struct DecodeArgs {
  const uint16_t* X;      // [T][d] bf16
  const int32_t* ids;     // [T][k] (routing read from memory)
  const float* w;         // [T][k]
  const float* logits;    // [T][E]: when not null the kernel routes its own tokens (E <= 256) and its last
                          // CTA writes every routing output to `out`
  RouteOut out;           // routing outputs written by the kernel (logits != null)
  int block_rows;         // tile height of the block map it writes
  uint16_t* Y;            // [T][d] bf16
  uint8_t* hbuf;          // h records of the call's slots, decode_scratch_bytes, 16-byte aligned
  // gate and up codes of the routed experts and of the shared expert (the prepacked [E][d/64][I][wpg] arrays),
  // read directly into registers when every CTA has at most one phase-1 item
  const uint32_t *qg_r, *qu_r, *qg_s, *qu_s;
  uint32_t* status;
  int T, d, I, k, I_shared, E, num_sms;
  int bits;  // bits per weight code: 4 or 2
};

bool decode_supported(int T, int d, int I, int I_shared, int k);
size_t decode_scratch_bytes(int T, int I, int I_shared);  // global scratch: the h records
cudaError_t launch_decode(const DecodeArgs& a, const DecodeMaps* routed, const DecodeMaps* shared, void* ws,
                          cudaStream_t stream, bool pdl);
// Test hooks of the decode kernel: the limit of the wait at its barrier over
// the grid in SM clock cycles (<= 0: the default of about 2 s), and one CTA
// (-1: none) whose arrival at that barrier is skipped, so that the wait runs
// out.
cudaError_t decode_debug(long long wait_limit_cycles, int drop_cta);

// ---------------------------------------------------------------- prefill GEMM
constexpr int kGemmBM = 128;   // weight rows per tile (MMA M)
constexpr int kGemmBK = 64;    // K of one quantisation group
constexpr int kGemmGroupsGU = 2;    // quantisation groups per pipeline stage, gate/up GEMM
constexpr int kGemmGroupsDown = 2;  // ... down GEMM
constexpr int kGemmBN = 128;   // max tokens per tile (MMA N)

struct GemmMaps {
  // codes, box (wpg words, 128 rows, groups per stage); 32-byte swizzle for 4-bit codes.  3-bit codes: box
  // (64 rows x 3 units, 1)
  CUtensorMap q_gate, q_up, q_down;
  CUtensorMap sb_gate, sb_up, sb_down;  // group parameters, box (128 rows, groups per stage, 1)
};

struct GemmArgs {
  const int32_t* perm;        // [A]
  const int32_t* inv_perm;    // [A]
  const int32_t* block_map;   // [nb][3]
  const int32_t* num_blocks;  // [1]
  const float* w;             // [A]
  float* ypart;               // [A + T][d] fp32 expert outputs: routed rows in permuted order, then shared rows
  uint16_t* h_routed;         // [A][I] fp16
  uint16_t* h_shared;         // [T][I_shared] fp16
  const uint16_t* X;          // [T][d] bf16 input
  uint16_t* Xh;               // [A + T][d] fp16 gathered rows of X (tensor-core operand)
  uint16_t* Y;                // [T][d] bf16
  uint32_t* status;
  int T, d, I, k, I_shared, E, num_sms, max_blocks;
  int bits;  // bits per weight code: 4, 3 or 2
};

struct GemmActMaps {
  CUtensorMap x;         // gathered X [A + T][d] fp16, box (64, kGemmBN), 128-byte swizzle
  CUtensorMap h_routed;  // H [A][I] fp16, box (64, kGemmBN), 128-byte swizzle
  CUtensorMap h_shared;  // H [T][I_shared] fp16, same box
  CUtensorMap ypart;     // expert outputs [A + T][d] fp32, box (32, 16): the down GEMM's stores
};

cudaError_t launch_gemm(const GemmArgs& a, const GemmMaps* routed, const GemmMaps* shared, const GemmActMaps* act,
                        cudaStream_t stream, bool pdl);

// ---------------------------------------------------------------- host helpers of api.cu
bool encode_mx_codes(CUtensorMap* map, const uint8_t* q, long long rows, int row_bytes, int box_rows);
bool encode_mx_weights(CUtensorMap* map, const uint8_t* q, int E, int N, int row_bytes, int box_rows);
bool encode_mx_scales(CUtensorMap* map, const uint8_t* sp, long long pieces);
// a result [rows][cols] of 2- or 4-byte elements: boxes of 64 bytes of 32 rows (for stores), 64-byte swizzle
bool encode_out_boxes(CUtensorMap* map, const void* y, int elem_bytes, long long rows, int cols);
bool pdl_enabled();  // the environment variable MOE_PDL
int device_sms();    // 0: no device
// moe_route_scored's checks of everything but the workspace, and its launch.
moe_status check_scored(const float* logits, const moe_scoring* sc, int T, int E, int k, int block_rows,
                        const moe_routing* out);
moe_status route_scored(const float* logits, const moe_scoring* sc, int T, int E, int k, int block_rows,
                        moe_routing* out, void* ws, moe_stream stream);

// ---------------------------------------------------------------- MXFP4
constexpr int kMxBlock = 32;       // values along K that share a scale
constexpr int kMxPieceRows = 128;  // one 512-byte piece of packed scales: 128 rows x 4 blocks
constexpr int kMxPieceK = 128;
constexpr int kMxPieceBytes = 512;
inline size_t mx_pieces(long long rows, int K) {
  return static_cast<size_t>((rows + kMxPieceRows - 1) / kMxPieceRows) * ((K + kMxPieceK - 1) / kMxPieceK);
}

cudaError_t launch_mx_prepack(const uint8_t* scale, int E, int N, int K, uint8_t* sp, cudaStream_t stream);
// type: 0 bf16, 1 fp16, 2 fp32; early: the next kernel may start beside this one (the result is no weights)
cudaError_t launch_mx_quantize(const void* X, int type, int rows, int K, long long ldx, uint8_t* q, uint8_t* sp,
                               bool early, cudaStream_t stream, bool pdl);
cudaError_t launch_mx_dequant(const uint8_t* q, const uint8_t* sp, int E, int N, int K, int type, void* W,
                              cudaStream_t stream, bool pdl);

// Where the quantised rows of an expert layer go: assignment a = t k + j to row
// inv_perm[a], its scales to that row's tile (entry b of the block map holds
// slot b of the scales, rows counted from the tile's first); with a shared
// expert token t also to row T k + t, slots max_blocks + t / shared_rows.
struct MxScatter {
  const int32_t* inv_perm;
  const int32_t* block_map;
  const int32_t* num_blocks;
  uint32_t* status;
  int T, k, max_blocks, shared_rows;  // shared_rows = 0: no shared expert
  bool x_ready;                       // X was complete before the kernel before this one
};
// Y[t] = bf16(sum_j w[t][j] ypart[inv_perm[t k + j]] + ypart[T k + t]), the second term with has_shared.
cudaError_t launch_mx_combine(float* ypart, const int32_t* inv_perm, const float* w, int T, int d, int k,
                              bool has_shared, uint16_t* Y, uint32_t* status, int num_sms, cudaStream_t stream);
cudaError_t launch_mx_scatter(const uint16_t* X, int d, const MxScatter& s, uint8_t* q, uint8_t* sp,
                              cudaStream_t stream, bool pdl);

constexpr int kMxBM = 128;      // rows of the MMA's M operand
constexpr int kMxStageK = 256;  // K of a pipeline stage: one 128-byte line of codes a row
constexpr int kMxMaxBN = 128;   // tokens of an expert tile at most
constexpr int kMxMaxCols = 1 << 20;        // columns of a matrix; of an expert's matrices also rows
constexpr long long kMxMaxItems = 1 << 30;  // items (tiles times M tiles) of an expert product: 32-bit indexes

struct MxLinearArgs {
  const uint8_t *sp_w, *sp_x;  // packed scales of the weights and of the tokens
  void* Y;                     // [M][N]
  uint32_t* status;
  int M, N, K;
  int bn;  // height of the tokens' tiles: 64, 128, 256, or a multiple of 16 up to 128 that holds all M
  int num_sms, y_fp32;
};
struct MxLinearMaps {
  CUtensorMap w;  // codes [1][N][K/2], box (128 bytes, 128 rows, 1)
  CUtensorMap x;  // codes [M][K/2], box (128 bytes, bn rows)
};
// The same product by pairs of CTAs, 256 weight rows x 256 tokens a pair.
constexpr int kMxPair = 1 << 16;  // MxLinearArgs::bn of this form; no height of a tile
struct MxPairMaps {
  CUtensorMap w, x;    // codes, boxes of 128 rows
  CUtensorMap sw, sx;  // packed scales as [pieces][128] words, box (128, 2)
};
cudaError_t launch_mx_pair(const MxLinearArgs& a, const MxPairMaps& maps, cudaStream_t stream, bool pdl);
cudaError_t launch_mx_linear(const MxLinearArgs& a, const MxLinearMaps& maps, cudaStream_t stream, bool pdl);

struct MxExpertArgs {
  const int32_t* block_map;
  const int32_t* num_blocks;
  const uint8_t *sp_gate_r, *sp_up_r, *sp_down_r, *sp_gate_s, *sp_up_s, *sp_down_s;  // weights' packed scales
  const uint8_t* sp_x;         // X's, by tile slot
  uint8_t *sp_h_r, *sp_h_s;    // h's: by routed slot, by shared tile
  uint8_t *q_h_r, *q_h_s;      // h's codes [A][I/2], [T][I_shared/2]
  float* ypart;                // [A + T][d]
  uint32_t* status;
  const int32_t* inv_perm;
  const float* w;              // [T][k]
  uint16_t* Y;                 // [T][d] bf16
  int T, d, I, k, I_shared, E, num_sms, max_blocks;
  int bn_r, bn_s;              // tile heights in MMA columns (multiples of 16): routed, shared
};
struct MxExpertMaps {
  CUtensorMap gate_r, up_r, down_r, gate_s, up_s, down_s;  // codes [E][N][K/2], box (128 bytes, 128 rows, 1)
  CUtensorMap x_r, x_s;        // X's codes [A + T][d/2], box (128 bytes, bn_r / bn_s rows)
  CUtensorMap h_r, h_s;        // h's codes
};
// Few tokens: the activations are quantised inside the products, by every CTA
// again.  That pays while it is short beside the launch that it saves:
//   linear layer    up to kMxFewValues values of X: 8 x 2048 5.1 us against 5.9
//                   with X quantised by a kernel of its own, 2 x 8192 10.1
//                   against 12.4; 8 x 4096 8.7 against 8.0, 16 x 2048 7.4 against 5.9
//   expert layer    up to kMxFewItems CTAs of the gate/up product, as many as this
//                   GPU has SMs: d = 2048, I = 512, 8 + 1 experts: one token 15.2
//                   us against 18.0, 2 tokens 17.4 against 19.0, 4 tokens 27.7
//                   against 23.4.  A constant: the workspace's layout goes by it
//                   and is asked for without a device.
constexpr int kMxFewT = 32;  // tokens at most (accumulator columns)
constexpr int kMxFewValues = 16384;
constexpr int kMxFewItems = 152;
struct MxFewLinearArgs {
  const void* X;       // [T][K], rows ldx elements apart
  const uint8_t* sp;   // packed scales of W [N][K]
  void* Y;             // [T][N]
  uint32_t* status;
  long long ldx;
  int T, N, K, y_fp32;
};
bool mx_few_linear_fits(int T, int K);
// type of X as for launch_mx_quantize; w: codes of W [1][N][K/2], box (128 bytes, 128 rows, 1)
cudaError_t launch_mx_few_linear(const MxFewLinearArgs& a, int type, const CUtensorMap& w, cudaStream_t stream, bool pdl);

struct MxFewArgs {
  const uint16_t* X;         // [T][d] bf16
  const int32_t *perm, *inv_perm, *block_map, *num_blocks;
  const float* w;            // [T][k]
  const uint8_t *sp_gate_r, *sp_up_r, *sp_down_r, *sp_gate_s, *sp_up_s, *sp_down_s;
  float* gu;                 // [A + T][2][max(I, I_shared)]: gate and up of every row
  float* ypart;              // [A + T][d]
  uint16_t* Y;               // [T][d] bf16
  uint32_t* arrived;         // [ceil(d / 128)] arrival counters, zero between calls
  uint32_t* status;
  int T, d, I, k, I_shared, E;
  int tiles, bn;             // tiles of the routed experts launched (mx_few_tiles), MMA columns of a tile
};
int mx_few_tiles(int T, int k, int max_blocks);
bool mx_few_fits(int T, int d, int I, int I_shared, int k, int max_blocks);
cudaError_t launch_mx_few_experts(const MxFewArgs& a, const MxExpertMaps& maps, cudaStream_t stream, bool pdl);

cudaError_t launch_mx_experts(const MxExpertArgs& a, const MxExpertMaps& maps, cudaStream_t stream);

// ---------------------------------------------------------------- block-scaled 8-bit floating point
constexpr int kBlk = 128;               // rows and columns of a block of weights, columns of one of activations
constexpr int kBlkMaxCols = 1 << 20;    // columns of a matrix; of an expert's matrices also rows
constexpr long long kBlkMaxItems = 1 << 30;
constexpr int kNormMaxCols = 32768;
__host__ __device__ constexpr int blk_count(int n) { return (n + kBlk - 1) / kBlk; }
// pitch of the activations' scales
__host__ __device__ constexpr long long blk_scale_rows(long long rows) { return (rows + 3) & ~3ll; }
inline size_t blk_weight_scales(int N, int K) { return static_cast<size_t>(blk_count(N)) * blk_count(K); }

// types: 0 bf16, 1 fp16, 2 fp32
cudaError_t launch_blk_quantize(const void* X, int type, int rows, int K, long long ldx, uint8_t* q, float* s,
                                cudaStream_t stream, bool pdl);
cudaError_t launch_blk_dequant(const uint8_t* q, const float* s, int rows, int K, int type, void* X, cudaStream_t stream,
                               bool pdl);
cudaError_t launch_blk_quantize_weights(const void* W, int type, int E, int N, int K, uint8_t* q, float* s,
                                        cudaStream_t stream, bool pdl);
cudaError_t launch_blk_dequant_weights(const uint8_t* q, const float* s, int E, int N, int K, int type, void* W,
                                       cudaStream_t stream, bool pdl);

struct RmsNorm {
  const void* x;
  const void* residual;  // null: none
  void* residual_out;
  const void* gamma;
  void* y;               // null: none
  uint8_t* q;            // null: none
  float* s;
  long long ldx;
  float eps;
  int T, d, x_type, residual_type, gamma_fp32, y_type;
};
cudaError_t launch_rmsnorm(const RmsNorm& n, cudaStream_t stream, bool pdl);

// Activations of a product: values of a type, rows ldx elements apart, or codes and scales.
constexpr int kBlkCodes = 3;  // the "type" of codes
struct BlkX {
  const void* x;
  const float* s;  // codes: the scales [ceil(K/128)][pitch]
  long long ldx, pitch;
  int type;
};
// Few tokens: weights straight into the registers of warp-level MMAs.  One token of any type, or up to kBlkFewLinear
// that are codes; experts up to kBlkFewT (an MMA's columns).
constexpr int kBlkFewT = 8;
constexpr int kBlkFewLinear = 32;
struct BlkFewLinearArgs {
  BlkX x;
  const uint8_t* w;
  const float* sw;
  void* y;
  int T, N, K, y_type;
};
cudaError_t launch_blk_few_linear(const BlkFewLinearArgs& a, cudaStream_t stream, bool pdl);

struct BlkWeights {
  const uint8_t *gate, *up, *down;
  const float *s_gate, *s_up, *s_down;
};
struct BlkFewArgs {
  BlkX x;
  BlkWeights routed, shared;
  const int32_t *perm, *block_map, *num_blocks;
  const float* w;
  float* h;    // [A + T][max(I, I_shared)]
  uint16_t* y;
  uint32_t* status;
  int T, d, I, k, I_shared, E;
  int tiles;  // tiles of the routed experts launched
  int split;  // CTAs, a cluster, that share a down tile's work
};
// A few-token down product covers this many columns of Y a CTA.
constexpr int kBlkFewRows = 16;
cudaError_t launch_blk_few_experts(const BlkFewArgs& a, cudaStream_t stream, bool pdl);

// Tensor-core products.
struct BlkLinearArgs {
  const float *sw, *sx;  // scales of the weights, and of the tokens [ceil(K/128)][sx_pitch]
  void* y;               // [M][N]
  uint32_t* status;
  long long sx_pitch;
  int M, N, K, y_type;
  int bn;  // height of the tokens' tiles: a multiple of 16 up to 128 (wide: 128)
  int num_sms;
  int split;    // narrow: CTAs, a cluster, that share a tile's blocks of columns
  int y_boxed;  // wide: maps.y is there
};
struct BlkLinearMaps {
  CUtensorMap w;  // codes [1][N][K], box (128 bytes, 128 rows, 1)
  CUtensorMap x;  // codes [M][K], box (128 bytes, bn rows)
  CUtensorMap y;  // wide: the result, box (64 bytes, 32 rows)
};
cudaError_t launch_blk_linear(const BlkLinearArgs& a, const BlkLinearMaps& maps, cudaStream_t stream, bool pdl);

struct BlkExpertArgs {
  const int32_t *block_map, *num_blocks, *inv_perm;
  const float* w;              // [T][k]
  BlkWeights routed, shared;
  // scales of a tile's tokens, [slot][ceil(columns/128)][pitch]: X's (the shared expert's slots after max_blocks), h's
  float *sx, *sh_r, *sh_s;
  uint8_t *h_r, *h_s;          // h's codes [A][I], [T][I_shared]
  float* ypart;                // [A + T][d]
  uint16_t* y;                 // [T][d] bf16
  uint32_t* status;
  int T, d, I, k, I_shared, E, num_sms, max_blocks;
  int bn_r, bn_s, pitch;       // tile heights in MMA columns (multiples of 16): routed, shared, the larger
};
struct BlkExpertMaps {
  CUtensorMap gate_r, up_r, down_r, gate_s, up_s, down_s;  // codes [E][N][K], box (128 bytes, 128 rows, 1)
  CUtensorMap x_r, x_s;        // X's codes [A + T][d], box (128 bytes, bn_r / bn_s rows)
  CUtensorMap h_r, h_s;        // h's codes
  CUtensorMap ypart;           // wide: the experts' rows, box (64 bytes, 32 rows)
};
// Tiles of more than kBlkNarrow tokens: the tokens on the MMA's M side.
constexpr int kBlkNarrow = 64;
cudaError_t launch_blk_wide_linear(const BlkLinearArgs& a, const BlkLinearMaps& maps, cudaStream_t stream, bool pdl);
cudaError_t launch_blk_wide_experts(const BlkExpertArgs& a, const BlkExpertMaps& maps, cudaStream_t stream, bool pdl);
cudaError_t launch_blk_experts(const BlkExpertArgs& a, const BlkExpertMaps& maps, cudaStream_t stream, bool pdl);

// X's rows, quantised once, to the rows of their assignments; s as for
// launch_mx_scatter, the scales to [slot][ceil(d/128)][pitch] of sx.
cudaError_t launch_blk_scatter(const BlkX& x, int d, const MxScatter& s, int pitch, uint8_t* q, float* sx,
                               cudaStream_t stream, bool pdl);

}  // namespace bm
