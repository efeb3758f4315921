// Host side of include/moe_mx.h: argument checks, workspace layouts, tensor
// maps and launches.  Nothing here allocates device memory or synchronises.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "moe_mx.h"

namespace bm {
namespace {

constexpr int kMaxRows = 1 << 30;  // rows (row indexes and TMA coordinates are 32-bit)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ws_ok(const void* ws, size_t have, size_t need) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && need > 0 && have >= need;
}
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int round16(int x) { return (x + 15) & ~15; }

bool size_ok(int N, int K) { return N >= 1 && K >= kMxBlock && K % kMxBlock == 0 && K <= kMxMaxCols; }
bool mat_ok(const moe_mx_mat& m) { return m.q && m.sp && aligned16(m.q) && aligned16(m.sp); }
bool experts_ok(const moe_mx_experts* ex) {
  return ex && mat_ok(ex->gate) && mat_ok(ex->up) && mat_ok(ex->down) && ex->n_experts >= 1;
}
int type_bytes(moe_dtype t) { return t == MOE_FP32 ? 4 : 2; }
bool type_ok(moe_dtype t) { return t == MOE_BF16 || t == MOE_FP16 || t == MOE_FP32; }

size_t scale_bytes(long long rows, int K) { return mx_pieces(rows, K) * kMxPieceBytes; }

moe_status check_x(const void* X, moe_dtype type, int rows, int K, long long ldx) {
  if (rows < 0 || !size_ok(1, K) || !type_ok(type) || ldx < K || (ldx * type_bytes(type)) % 16 != 0)
    return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (rows > 0 && (!X || !aligned16(X))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_matmul(int M, const moe_mx_mat* W, int N, int K, const void* Y, moe_dtype y_type) {
  if (M < 0 || !size_ok(N, K) || !W || !mat_ok(*W) || !type_ok(y_type)) return MOE_ERR_INVALID_ARG;
  if (y_type == MOE_FP16 || M > kMaxRows || N > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (M > 0 && (!Y || !aligned16(Y))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Height of the dense product's token tiles, by a modelled time in clocks: a
// CTA's tiles in turn, each a stage of K = 256 after another at the rate its
// bytes arrive and are read, then the epilogue.  Measured (bf16 Y, 64 / 128 / 256
// high, quantisation included): 256 x 2048 -> 2048 6.1 / 6.8 / 8.5 us, 512 x 4096
// -> 8192 21.3 / 14.8 / 13.6 us, 333 x 2816 -> 1001 7.2 / 7.5 / 9.1 us, 1024 x
// 2048 -> 2048 8.9 / 8.3 / 9.2 us: the model picks the least of each.
//
// Returns kMxPair, tiles of 256 x 256 by pairs of CTAs, where tiles of 256 are best,
// each pair has a second one (the first starts later than a CTA's own) and their
// stages outweigh the epilogue.  Measured (fp32 Y, the product alone, one CTA / a
// pair): 8192 x 8192 -> 8192 180 / 158 us, 16384 x 2048 -> 4096 75.3 / 62.7 us,
// 4096 x 4096 -> 4096 32.7 / 30.3 us, 5001 x 1056 -> 4099 31.3 / 27.8 us, 2048 x
// 4096 -> 4096 17.3 / 17.4 us; without a second tile 512 x 8192 -> 8192 14.6 / 15.4
// us, 2048 x 2048 -> 2048 7.9 / 8.8 us; of few stages 2048 x 1024 -> 4096 9.6 / 9.9
// us, 16384 x 512 -> 8192 85.5 / 91.0 us.
int linear_tile(int M, int N, int K, int num_sms) {
  int best = 0;
  double least = 0;
  const int stages = (K + kMxStageK - 1) / kMxStageK;
  auto tiles = [&](int rows, int cols) {
    return static_cast<long long>((N + rows - 1) / rows) * ((M + cols - 1) / cols);
  };
  for (int bn : {64, 128, 256, M <= kMxMaxBN ? round16(M) : 64}) {
    const double turns = static_cast<double>((tiles(kMxBM, bn) + num_sms - 1) / num_sms);
    const double clocks = turns * (stages * (290 + 2.3 * bn) + 1500 + 8 * bn);
    if (best == 0 || clocks < least) {
      least = clocks;
      best = bn;
    }
  }
  if (best == 256 && stages > 4 && tiles(2 * kMxBM, 256) > num_sms / 2) return kMxPair;
  return best;
}

moe_status matmul(const moe_mx_mat& A, int M, const moe_mx_mat& W, int N, int K, void* Y, moe_dtype y_type,
                  uint32_t* status, moe_stream stream) {
  MxLinearArgs a{};
  a.sp_w = W.sp;
  a.sp_x = A.sp;
  a.Y = Y;
  a.status = status;
  a.M = M;
  a.N = N;
  a.K = K;
  a.num_sms = device_sms();
  if (a.num_sms <= 0) return MOE_ERR_CUDA;
  a.bn = linear_tile(M, N, K, a.num_sms);
  a.y_fp32 = y_type == MOE_FP32;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  if (a.bn == kMxPair) {
    MxPairMaps maps;
    if (encode_mx_weights(&maps.w, W.q, 1, N, K / 2, kMxBM) && encode_mx_codes(&maps.x, A.q, M, K / 2, kMxBM) &&
        encode_mx_scales(&maps.sw, W.sp, static_cast<long long>(mx_pieces(N, K))) &&
        encode_mx_scales(&maps.sx, A.sp, static_cast<long long>(mx_pieces(M, K))))
      e = launch_mx_pair(a, maps, st, pdl_enabled());
  } else {
    MxLinearMaps maps;
    if (encode_mx_weights(&maps.w, W.q, 1, N, K / 2, kMxBM) && encode_mx_codes(&maps.x, A.q, M, K / 2, a.bn))
      e = launch_mx_linear(a, maps, st, pdl_enabled());
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Tile heights of an expert call in MMA columns.  The shared expert's tiles are
// as high as the routed ones allow: up to 96 rows the gate/up product keeps two
// accumulators (2 x 2 x 96 columns of 512, and the scales).
int routed_rows(int block_rows) { return round16(block_rows); }
int shared_tile_rows(int T, int block_rows) {
  const int most = routed_rows(block_rows) <= 96 ? 96 : kMxMaxBN;
  return round16(T < most ? T : most);
}

struct ExpertLayout {
  size_t q_x, sp_x, q_h_r, q_h_s, sp_h_r, sp_h_s, ypart, gu, total;
  int max_blocks, bn_r, bn_s;
  bool few;  // the products for few tokens
};

ExpertLayout expert_layout(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  ExpertLayout L{};
  L.max_blocks = moe_route_max_blocks(T, E, k, block_rows);
  L.bn_r = routed_rows(block_rows);
  L.bn_s = shared_tile_rows(T < 1 ? 1 : T, block_rows);
  const size_t A = static_cast<size_t>(T) * k, rows = A + (I_shared > 0 ? T : 0);
  const size_t tiles_s = I_shared > 0 ? (T + L.bn_s - 1) / L.bn_s : 0;
  size_t o = sizeof(WsHeader);
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o = round256(o + bytes);
    return at;
  };
  L.few = mx_few_fits(T, d, I, I_shared, k, L.max_blocks);
  L.ypart = take(rows * d * 4);
  if (L.few) {
    L.gu = take(rows * 2 * (I > I_shared ? I : I_shared) * 4);
    L.total = o;
    return L;
  }
  L.q_x = take(rows * (d / 2));
  L.sp_x = take((L.max_blocks + tiles_s) * scale_bytes(1, d));
  L.q_h_r = take(A * (I / 2));
  L.q_h_s = take(static_cast<size_t>(T) * (I_shared / 2));
  L.sp_h_r = take(L.max_blocks * scale_bytes(1, I));
  L.sp_h_s = take(I_shared > 0 ? tiles_s * scale_bytes(1, I_shared) : 0);
  L.total = o;
  return L;
}

bool sizes_valid(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  return T >= 0 && size_ok(1, d) && size_ok(1, I) && (I_shared == 0 || size_ok(1, I_shared)) && E >= 1 && k >= 1 &&
         block_rows >= 1 && block_rows <= kMaxBlockRows;
}

moe_status check_experts(const uint16_t* X, int T, int d, int I, int k, const moe_mx_experts* routed,
                         const moe_mx_experts* shared, int I_shared, const uint16_t* Y) {
  if (T < 0 || k < 1 || !size_ok(1, d) || !size_ok(1, I) || I_shared < 0 || I_shared % kMxBlock || I_shared > kMxMaxCols)
    return MOE_ERR_INVALID_ARG;
  if ((shared != nullptr) != (I_shared > 0)) return MOE_ERR_INVALID_ARG;
  if (!experts_ok(routed) || (shared && (!experts_ok(shared) || shared->n_experts != 1))) return MOE_ERR_INVALID_ARG;
  const int E = routed->n_experts;
  if (E > kMaxE || k > kMaxK || k > E) return MOE_ERR_UNSUPPORTED;
  // rows of the tensor maps and the launch's items are 32-bit
  if (static_cast<long long>(T) * (k + 1) > (1ll << 30) || static_cast<long long>(E) * (d > I ? d : I) > (1ll << 30))
    return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!X || !Y || !aligned16(X) || !aligned16(Y))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Whether the products' items can be counted; everything else has been checked.
bool items_ok(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  auto m_tiles = [](int a, int b) { return static_cast<long long>((a > b ? a : b) + kMxBM - 1) / kMxBM; };
  long long items = moe_route_max_blocks(T, E, k, block_rows) * m_tiles(d, I);
  if (I_shared > 0) {
    const int rows = shared_tile_rows(T < 1 ? 1 : T, block_rows);
    items += (T + rows - 1) / rows * m_tiles(d, I_shared);
  }
  return items <= kMxMaxItems;
}

template <typename A>
void set_scales(A* a, const moe_mx_experts* routed, const moe_mx_experts* shared) {
  a->sp_gate_r = routed->gate.sp;
  a->sp_up_r = routed->up.sp;
  a->sp_down_r = routed->down.sp;
  a->sp_gate_s = shared ? shared->gate.sp : nullptr;
  a->sp_up_s = shared ? shared->up.sp : nullptr;
  a->sp_down_s = shared ? shared->down.sp : nullptr;
}

moe_status forward(const uint16_t* X, int T, int d, int I, int k, const moe_mx_experts* routed,
                   const moe_mx_experts* shared, int I_shared, const moe_routing* r, uint16_t* Y, void* ws,
                   bool after_routing, moe_stream stream) {
  if (T == 0) return MOE_OK;
  const int E = routed->n_experts;
  const ExpertLayout L = expert_layout(T, d, I, E, k, I_shared, r->block_rows);
  uint8_t* w = static_cast<uint8_t*>(ws);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int num_sms = device_sms();
  if (num_sms <= 0) return MOE_ERR_CUDA;

  const long long A = static_cast<long long>(T) * k, rows = A + (shared ? T : 0);
  uint32_t* status = &static_cast<WsHeader*>(ws)->status;
  float* ypart = reinterpret_cast<float*>(w + L.ypart);
  MxExpertMaps maps;
  bool ok = encode_mx_weights(&maps.gate_r, routed->gate.q, E, I, d / 2, kMxBM) &&
            encode_mx_weights(&maps.up_r, routed->up.q, E, I, d / 2, kMxBM) &&
            encode_mx_weights(&maps.down_r, routed->down.q, E, d, I / 2, kMxBM);
  if (shared)
    ok = ok && encode_mx_weights(&maps.gate_s, shared->gate.q, 1, I_shared, d / 2, kMxBM) &&
         encode_mx_weights(&maps.up_s, shared->up.q, 1, I_shared, d / 2, kMxBM) &&
         encode_mx_weights(&maps.down_s, shared->down.q, 1, d, I_shared / 2, kMxBM);
  else  // never read without a shared expert
    maps.gate_s = maps.up_s = maps.down_s = maps.gate_r;
  if (!ok) return MOE_ERR_CUDA;

  if (L.few) {
    maps.x_r = maps.x_s = maps.h_r = maps.h_s = maps.gate_r;  // not read
    MxFewArgs a{};
    a.X = X;
    a.perm = r->perm;
    a.inv_perm = r->inv_perm;
    a.block_map = r->block_map;
    a.num_blocks = r->num_blocks;
    a.w = r->w;
    set_scales(&a, routed, shared);
    a.gu = reinterpret_cast<float*>(w + L.gu);
    a.ypart = ypart;
    a.Y = Y;
    a.arrived = static_cast<WsHeader*>(ws)->mx_arrived;
    a.status = status;
    a.T = T;
    a.d = d;
    a.I = I;
    a.k = k;
    a.I_shared = I_shared;
    a.E = E;
    a.tiles = mx_few_tiles(T, k, L.max_blocks);
    a.bn = round16(T);
    return launch_mx_few_experts(a, maps, st, pdl_enabled()) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }

  MxExpertArgs a{};
  a.block_map = r->block_map;
  a.num_blocks = r->num_blocks;
  set_scales(&a, routed, shared);
  a.sp_x = w + L.sp_x;
  a.sp_h_r = w + L.sp_h_r;
  a.sp_h_s = w + L.sp_h_s;
  a.q_h_r = w + L.q_h_r;
  a.q_h_s = w + L.q_h_s;
  a.ypart = ypart;
  a.status = status;
  a.T = T;
  a.d = d;
  a.I = I;
  a.k = k;
  a.I_shared = I_shared;
  a.E = E;
  a.num_sms = num_sms;
  a.max_blocks = L.max_blocks;
  a.bn_r = L.bn_r;
  a.bn_s = L.bn_s;
  a.inv_perm = r->inv_perm;
  a.w = r->w;
  a.Y = Y;
  ok = encode_mx_codes(&maps.x_r, w + L.q_x, rows, d / 2, L.bn_r) && encode_mx_codes(&maps.h_r, a.q_h_r, A, I / 2, L.bn_r);
  if (shared)
    ok = ok && encode_mx_codes(&maps.x_s, w + L.q_x, rows, d / 2, L.bn_s) &&
         encode_mx_codes(&maps.h_s, a.q_h_s, T, I_shared / 2, L.bn_s);
  else
    maps.x_s = maps.h_s = maps.x_r;
  if (!ok) return MOE_ERR_CUDA;

  const MxScatter sc{r->inv_perm, r->block_map, r->num_blocks, a.status, T, k, L.max_blocks,
                     shared ? L.bn_s : 0, after_routing};
  if (launch_mx_scatter(X, d, sc, w + L.q_x, w + L.sp_x, st, pdl_enabled()) != cudaSuccess ||
      launch_mx_experts(a, maps, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // namespace
}  // namespace bm

using namespace bm;

extern "C" {

size_t moe_mx_scale_bytes(int E, int N, int K) {
  if (E < 1 || !size_ok(N, K)) return 0;
  return static_cast<size_t>(E) * scale_bytes(N, K);
}

moe_status moe_mx_prepack_scales(const uint8_t* scale, int E, int N, int K, uint8_t* sp, moe_stream stream) {
  if (E < 1 || !size_ok(N, K) || !scale || !sp || !aligned16(sp)) return MOE_ERR_INVALID_ARG;
  return launch_mx_prepack(scale, E, N, K, sp, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                                      : MOE_ERR_CUDA;
}

moe_status moe_mx_quantize(const void* X, moe_dtype type, int rows, int K, long long ldx, const moe_mx_mat* out,
                           moe_stream stream) {
  const moe_status st = check_x(X, type, rows, K, ldx);
  if (st != MOE_OK) return st;
  if (!out || !mat_ok(*out)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  return launch_mx_quantize(X, type, rows, K, ldx, out->q, out->sp, false, reinterpret_cast<cudaStream_t>(stream),
                            pdl_enabled()) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_mx_dequant(const moe_mx_mat* m, int E, int N, int K, moe_dtype type, void* W, moe_stream stream) {
  if (!m || !mat_ok(*m) || E < 1 || !size_ok(N, K) || !type_ok(type) || !W || !aligned16(W)) return MOE_ERR_INVALID_ARG;
  if (type == MOE_FP16 || E > 65535 || N > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return launch_mx_dequant(m->q, m->sp, E, N, K, type, W, reinterpret_cast<cudaStream_t>(stream),
                           pdl_enabled()) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_mx_matmul(const moe_mx_mat* A, int M, const moe_mx_mat* W, int N, int K, void* Y, moe_dtype y_type,
                         void* ws, size_t ws_bytes, moe_stream stream) {
  const moe_status st = check_matmul(M, W, N, K, Y, y_type);
  if (st != MOE_OK) return st;
  if (!A || !mat_ok(*A)) return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, sizeof(WsHeader))) return MOE_ERR_WORKSPACE;
  if (M == 0) return MOE_OK;
  return matmul(*A, M, *W, N, K, Y, y_type, &static_cast<WsHeader*>(ws)->status, stream);
}

size_t moe_mx_linear_workspace_bytes(int T, int N, int K) {
  if (T < 0 || !size_ok(N, K)) return 0;
  return sizeof(WsHeader) + round256(static_cast<size_t>(T) * (K / 2)) + round256(scale_bytes(T, K));
}

moe_status moe_mx_linear(const void* X, moe_dtype x_type, int T, int K, long long ldx, const moe_mx_mat* W, int N,
                         void* Y, moe_dtype y_type, void* ws, size_t ws_bytes, moe_stream stream) {
  moe_status st = check_x(X, x_type, T, K, ldx);
  if (st != MOE_OK) return st;
  st = check_matmul(T, W, N, K, Y, y_type);
  if (st != MOE_OK) return st;
  if (!ws_ok(ws, ws_bytes, moe_mx_linear_workspace_bytes(T, N, K))) return MOE_ERR_WORKSPACE;
  if (T == 0) return MOE_OK;
  uint32_t* status = &static_cast<WsHeader*>(ws)->status;
  if (mx_few_linear_fits(T, K)) {
    const MxFewLinearArgs a{X, W->sp, Y, status, ldx, T, N, K, y_type == MOE_FP32};
    CUtensorMap map;
    if (!encode_mx_weights(&map, W->q, 1, N, K / 2, kMxBM) ||
        launch_mx_few_linear(a, x_type, map, reinterpret_cast<cudaStream_t>(stream), pdl_enabled()) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  uint8_t* w = static_cast<uint8_t*>(ws) + sizeof(WsHeader);
  const moe_mx_mat xq{w, w + round256(static_cast<size_t>(T) * (K / 2))};
  if (launch_mx_quantize(X, x_type, T, K, ldx, xq.q, xq.sp, true, reinterpret_cast<cudaStream_t>(stream),
                         pdl_enabled()) != cudaSuccess)
    return MOE_ERR_CUDA;
  return matmul(xq, T, *W, N, K, Y, y_type, status, stream);
}

size_t moe_mx_forward_workspace_bytes(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  if (!sizes_valid(T, d, I, E, k, I_shared, block_rows)) return 0;
  return expert_layout(T, d, I, E, k, I_shared, block_rows).total;
}

moe_status moe_mx_forward(const uint16_t* X, int T, int d, int I, int k, const moe_mx_experts* routed,
                          const moe_mx_experts* shared, int I_shared, const moe_routing* r, uint16_t* Y, void* ws,
                          size_t ws_bytes, moe_stream stream) {
  const moe_status st = check_experts(X, T, d, I, k, routed, shared, I_shared, Y);
  if (st != MOE_OK) return st;
  if (!r) return MOE_ERR_INVALID_ARG;
  if (r->block_rows < 1 || r->block_rows > kMaxBlockRows) return MOE_ERR_UNSUPPORTED;
  if (!items_ok(T, d, I, routed->n_experts, k, I_shared, r->block_rows)) return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!r->w || !r->perm || !r->inv_perm || !r->block_map || !r->num_blocks)) return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes,
             moe_mx_forward_workspace_bytes(T, d, I, routed->n_experts, k, I_shared, r->block_rows)))
    return MOE_ERR_WORKSPACE;
  return forward(X, T, d, I, k, routed, shared, I_shared, r, Y, ws, false, stream);
}

size_t moe_mx_layer_workspace_bytes(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  const size_t f = moe_mx_forward_workspace_bytes(T, d, I, E, k, I_shared, block_rows);
  const size_t r = moe_route_workspace_bytes(T, E, k);
  return f && r ? (f > r ? f : r) : 0;
}

moe_status moe_mx_layer(const float* logits, const moe_scoring* scoring, const uint16_t* X, int T, int d, int I, int k,
                        int block_rows, const moe_mx_experts* routed, const moe_mx_experts* shared, int I_shared,
                        moe_routing* r, uint16_t* Y, void* ws, size_t ws_bytes, moe_stream stream) {
  moe_status st = check_experts(X, T, d, I, k, routed, shared, I_shared, Y);
  if (st != MOE_OK) return st;
  const int E = routed->n_experts;
  st = check_scored(logits, scoring, T, E, k, block_rows, r);
  if (st != MOE_OK) return st;
  if (!items_ok(T, d, I, E, k, I_shared, block_rows)) return MOE_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, moe_mx_layer_workspace_bytes(T, d, I, E, k, I_shared, block_rows))) return MOE_ERR_WORKSPACE;
  // one header for both, and after it the same room: the products start when the routing has completed
  st = route_scored(logits, scoring, T, E, k, block_rows, r, ws, stream);
  if (st != MOE_OK) return st;
  return forward(X, T, d, I, k, routed, shared, I_shared, r, Y, ws, true, stream);
}

}  // extern "C"
