// Host side of include/moe_blk.h: argument checks, workspace layouts and
// launches.  Nothing here allocates device memory or synchronises.
#include <cuda_runtime.h>

#include <cmath>

#include "kernels.h"
#include "moe_blk.h"

namespace bm {
namespace {

constexpr int kMaxRows = 1 << 30;  // rows (row indexes and TMA coordinates are 32-bit)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ws_ok(const void* ws, size_t have, size_t need) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && need > 0 && have >= need;
}
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
cudaStream_t cuda(moe_stream s) { return reinterpret_cast<cudaStream_t>(s); }
moe_status done(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool cols_ok(int K) { return K >= 16 && K % 16 == 0 && K <= kBlkMaxCols; }
bool size_ok(int N, int K) { return N >= 1 && cols_ok(K); }
bool mat_ok(const moe_blk_mat* m) { return m && m->q && m->s && aligned16(m->q) && aligned16(m->s); }
bool experts_ok(const moe_blk_experts* ex) {
  return ex && mat_ok(&ex->gate) && mat_ok(&ex->up) && mat_ok(&ex->down) && ex->n_experts >= 1;
}
int type_bytes(moe_dtype t) { return t == MOE_FP32 ? 4 : 2; }
bool type_ok(moe_dtype t) { return t == MOE_BF16 || t == MOE_FP16 || t == MOE_FP32; }
size_t act_scale_bytes(long long rows, int K) { return static_cast<size_t>(blk_scale_rows(rows)) * blk_count(K) * 4; }

moe_status check_x(const void* X, moe_dtype type, int rows, int K, long long ldx) {
  if (rows < 0 || !cols_ok(K) || !type_ok(type) || ldx < K || (ldx * type_bytes(type)) % 16 != 0)
    return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (rows > 0 && (!X || !aligned16(X))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_weights(const void* W, moe_dtype type, int E, int N, int K, const moe_blk_mat* m) {
  if (E < 1 || !size_ok(N, K) || !type_ok(type) || !W || !aligned16(W) || !mat_ok(m)) return MOE_ERR_INVALID_ARG;
  if (N > kMaxRows || static_cast<double>(E) * blk_weight_scales(N, K) > 2147483647.0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_matmul(int M, const moe_blk_mat* W, int N, int K, const void* Y, moe_dtype y_type) {
  if (M < 0 || !size_ok(N, K) || !mat_ok(W) || !type_ok(y_type)) return MOE_ERR_INVALID_ARG;
  if (M > kMaxRows || N > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (M > 0 && (!Y || !aligned16(Y))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status few_linear(const BlkX& x, int M, const moe_blk_mat* W, int N, int K, void* Y, moe_dtype y_type, moe_stream stream) {
  const BlkFewLinearArgs a{x, W->q, W->s, Y, M, N, K, y_type};
  return done(launch_blk_few_linear(a, cuda(stream), pdl_enabled()));
}

int round16(int x) { return (x + 15) & ~15; }

// How a dense product is computed, by modelled times in microseconds (a kernel of its own on the GPU).
struct LinearPlan {
  bool few;   // the products for few tokens
  int bn;     // else the height of the tiles of tokens (more than kBlkNarrow: the wide kernel's)
  int split;  // and the CTAs that share a tile's blocks of 128 columns
  double time;
};
constexpr double kStream = 5.5e6;  // the weights' bytes a microsecond, as fast as these kernels get them
LinearPlan linear_plan(int M, int N, int K, int num_sms) {
  const int blocks = blk_count(K);
  const double stream = static_cast<double>(N) * K / kStream;
  LinearPlan best{};
  double time = 1e30;
  auto consider = [&](double t, bool few, int bn, int split) {
    if (t >= time) return;
    time = t;
    best = LinearPlan{few, bn, split, t};
  };
  if (M <= kBlkFewLinear) {
    // a CTA's eight warps take a block each in turn.  Measured, 2048 -> 2048 / 5120 -> 1024 / 8192 -> 8192: 8 tokens 2.9 /
    // 5.0 / 18.9 us, 16 tokens 3.1 / 5.7 / 22.2, 32 tokens 4.4 / 9.9 / 38
    const double ctas = 0.9 * N / (16.0 * num_sms);  // an SM's, which share its loads
    const double per_block = M <= 8 ? 0.7 : M <= 16 ? 0.87 : 1.7;
    consider(1.4 + per_block * blocks / 8 * (ctas > 1 ? ctas : 1), true, 0, 1);
  }
  auto tiles = [&](int rows, int cols) { return static_cast<long long>((N + rows - 1) / rows) * ((M + cols - 1) / cols); };
  auto turns = [&](long long n) { return static_cast<double>((n + num_sms - 1) / num_sms); };
  // Tiles of up to 16 / 32 / 64 tokens (and 128 weight rows): 0.235 / 0.25 / 0.33 us a block.  A cluster's CTAs lie in one
  // GPC and join their sums in 2 us.  Measured, tokens x K -> N, tile / CTAs: 333 x 2816 -> 1001 32/1 8.0, 64/1 9.0, 64/2 8.1,
  // 64/3 (144 CTAs, which do not all fit their GPCs) 12.1; 64 x 2048 -> 2048 64/1 7.1, 64/4 5.1, 64/8 10.3; 64 x 8192 ->
  // 1024 64/1 21.9, 64/4 8.7, 64/8 7.1; 16 x 8192 -> 8192 16/1 18.2, 16/2 14.7
  for (int most = 16; most <= kBlkNarrow; most *= 2) {
    const int bn = round16(M) < most ? round16(M) : most;
    const double per_block = bn <= 16 ? 0.235 : bn <= 32 ? 0.25 : 0.33;
    const long long n = tiles(kBlk, bn);
    for (int split = 1; split <= 8 && split <= blocks; split *= 2) {
      // CTAs whose clusters of 2 / 4 / 8 find a place at once
      const int room = split == 2 ? num_sms : split == 4 ? num_sms - num_sms / 8 : num_sms / 2;
      if (split > 1 && n * split > room) break;
      const double work = turns(n * split) * (per_block * ((blocks + split - 1) / split) + 0.4);
      consider(1.7 + (work > stream ? work : stream) + (split > 1 ? 2.0 : 0.0), false, bn, split);
    }
    if (bn < most) break;
  }
  // 128 tokens x 256 weight rows: 256 x 8192 -> 8192 32.7 us (64/1 43.9), 300 x 2048 -> 4096 10.3 (64/1 12.7)
  if (M > kBlkNarrow) consider(1.8 + turns(tiles(2 * kBlk, 128)) * (0.44 * blocks + 1.2), false, 128, 1);
  return best;
}

// Whether one token of a linear layer is quantised in the warps that multiply it (a launch less, but each CTA's eight warps
// go through all of K) rather than by a launch before the product.  Measured, K -> N, so / the other way: 2048 -> 2048 1.9 /
// 4.0 us, 2048 -> 24576 12.7 / 14.6, 8192 -> 512 6.5 / 7.5, 8192 -> 8192 16.6 / 16.1, 4096 -> 60000 48 / 45, 16384 -> 1024
// 14.0 / 9.7, 16384 -> 16384 64 / 45, 65536 -> 128 54 / 20
bool one_launch_wins(int N, int K, int num_sms) {
  const double ctas = 0.9 * N / (16.0 * num_sms), time = 1.0 + 0.6 * blk_count(K) / 8 * (ctas > 1 ? ctas : 1);
  // (no plan takes less than 1.7 us and the weights' stream, but the same warps': those sizes need no look at the others)
  return time <= 3.7 + static_cast<double>(N) * K / kStream || time <= linear_plan(1, N, K, num_sms).time + 2.0;
}

moe_status matmul(const moe_blk_mat& A, int M, const moe_blk_mat* W, int N, int K, void* Y, moe_dtype y_type,
                  uint32_t* status, moe_stream stream) {
  const int num_sms = device_sms();
  if (num_sms <= 0) return MOE_ERR_CUDA;
  const LinearPlan plan = linear_plan(M, N, K, num_sms);
  if (plan.few) return few_linear(BlkX{A.q, A.s, K, blk_scale_rows(M), kBlkCodes}, M, W, N, K, Y, y_type, stream);
  BlkLinearArgs a{};
  a.sw = W->s;
  a.sx = A.s;
  a.y = Y;
  a.status = status;
  a.sx_pitch = blk_scale_rows(M);
  a.M = M;
  a.N = N;
  a.K = K;
  a.y_type = y_type;
  a.num_sms = num_sms;
  a.bn = plan.bn;
  a.split = plan.split;
  const bool wide = a.bn > kBlkNarrow;
  BlkLinearMaps maps;
  if (!encode_mx_weights(&maps.w, W->q, 1, N, K, kBlk) || !encode_mx_codes(&maps.x, A.q, M, K, a.bn)) return MOE_ERR_CUDA;
  if (!wide) {
    maps.y = maps.x;  // not read
    return done(launch_blk_linear(a, maps, cuda(stream), pdl_enabled()));
  }
  const int bytes = type_bytes(y_type);
  a.y_boxed = static_cast<long long>(N) * bytes % 16 == 0;
  maps.y = maps.x;
  if (a.y_boxed && !encode_out_boxes(&maps.y, Y, bytes, M, N)) return MOE_ERR_CUDA;
  return done(launch_blk_wide_linear(a, maps, cuda(stream), pdl_enabled()));
}

// Tile heights of an expert call in MMA columns.
int routed_rows(int T, int k, int block_rows) {
  const long long most = T < 1 ? 1 : static_cast<long long>(T) * k;  // a tile's rows are assignments
  return round16(most < block_rows ? static_cast<int>(most) : block_rows);
}
int shared_tile_rows(int T, int block_rows) {
  const int rows = round16(block_rows), most = round16(T < 1 ? 1 : T);
  return most < rows ? most : rows;
}

// The experts' rules below take the SMs of the GPU that this is compiled for, where a dense product's plan asks the device:
// they decide the workspace's layout, which a host may ask for on another device, or without one.
constexpr int kSms = 152;
long long few_units(int T, int I, int k, int I_shared) { return static_cast<long long>(T) * k * blk_count(I) + blk_count(I_shared); }
// CTAs, a cluster, that share the down product's work on their columns: while there is work for their 16 warps each, and room
// for the clusters (see linear_plan).
int few_split(int T, int d, int I, int k, int I_shared) {
  const int ctas = (d + kBlkFewRows - 1) / kBlkFewRows;
  const long long units = few_units(T, I, k, I_shared);
  int split = 1;
  for (int next = 2; next <= 8; next *= 2) {
    const int room = next == 2 ? kSms : next == 4 ? kSms - kSms / 8 : kSms / 2;
    if (ctas * next > room || units <= 16 * split) break;
    split = next;
  }
  return split;
}

// Whether the products for few tokens are the faster ones: two launches instead of four, but a down product whose CTAs (16
// columns of Y, one an SM) go through every assignment's blocks of h.  Those, times the CTAs' turns, against the
// difference measured (us; T, d, I, k, s: a shared expert): 16 (6, 1600, 128, 2) -4.4; 32 (8, 1024, 256, 2) -1.7; 68 (2, 2048,
// 512, 8, s) -0.9; 72 (1, 2560, 704, 5, s) -0.7; 96 (8, 1856, 288, 4) 2.7; 100 (3, 2048, 512, 8, s) 2.1; 108 (4, 2560, 704, 2, s)
// 2.7; 132 (2, 2048, 1408, 6) 5.8; 156 (1, 2560, 704, 12, s) 5.3; 288 (1, 4096, 2048, 8, s) 18.5.
bool few_experts_win(int T, int d, int I, int k, int I_shared) {
  if (T > kBlkFewT) return false;
  const int turns = (d / kBlkFewRows + kSms - 1) / kSms;
  // (one or two tokens gain from CTAs that share the work, 1, 1152, 704, 12: 15.5 against 16.9 us; of more the gate/up product
  // takes longer than that gives, 4, 320, 416, 7, s: 13.4 against 11.4)
  return few_units(T, I, k, I_shared) * turns <= 72 * (T <= 2 ? few_split(T, d, I, k, I_shared) : 1);
}

struct ExpertLayout {
  size_t h, q_x, sx, h_r, h_s, sh_r, sh_s, ypart, total;
  int max_blocks, bn_r, bn_s, pitch;
  bool few;  // the products for few tokens
};

ExpertLayout expert_layout(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  ExpertLayout L{};
  L.max_blocks = moe_route_max_blocks(T, E, k, block_rows);
  L.bn_r = routed_rows(T, k, block_rows);
  L.bn_s = shared_tile_rows(T, block_rows);
  L.pitch = L.bn_r > L.bn_s ? L.bn_r : L.bn_s;
  const size_t A = static_cast<size_t>(T) * k, rows = A + (I_shared > 0 ? T : 0);
  const size_t tiles_s = I_shared > 0 ? (T + L.bn_s - 1) / L.bn_s : 0;
  size_t o = sizeof(WsHeader);
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o = round256(o + bytes);
    return at;
  };
  L.few = few_experts_win(T, d, I, k, I_shared);
  const size_t h_bytes = static_cast<size_t>(I > I_shared ? I : I_shared) * 4;
  if (L.few) {
    L.h = take(rows * h_bytes);
    L.total = o;
    return L;
  }
  L.ypart = take(rows * d * 4);
  L.q_x = take(rows * d);
  L.sx = take((L.max_blocks + tiles_s) * blk_count(d) * L.pitch * 4);
  L.h_r = take(A * I);
  L.h_s = take(static_cast<size_t>(T) * I_shared);
  L.sh_r = take(static_cast<size_t>(L.max_blocks) * blk_count(I) * L.pitch * 4);
  L.sh_s = take(tiles_s * blk_count(I_shared) * L.pitch * 4);
  // a workspace for T tokens is one for fewer: the few tokens' fp32 h may be larger than all of the above
  for (size_t t = 1; t <= kBlkFewT && few_experts_win(static_cast<int>(t), d, I, k, I_shared); ++t) {
    const size_t few = sizeof(WsHeader) + round256(t * (k + (I_shared > 0 ? 1 : 0)) * h_bytes);
    if (few > o) o = few;
  }
  L.total = o;
  return L;
}

bool expert_cols_ok(int n) { return n >= 32 && n % 32 == 0 && n <= kBlkMaxCols; }
bool sizes_valid(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  return T >= 0 && T <= kMaxRows && expert_cols_ok(d) && expert_cols_ok(I) && (I_shared == 0 || expert_cols_ok(I_shared)) && E >= 1 && k >= 1 &&
         block_rows >= 1 && block_rows <= kMaxBlockRows;
}

moe_status check_experts(const uint16_t* X, const moe_blk_mat* XQ, int T, int d, int I, int k, const moe_blk_experts* routed,
                         const moe_blk_experts* shared, int I_shared, const uint16_t* Y) {
  if (T < 0 || k < 1 || !expert_cols_ok(d) || !expert_cols_ok(I) || (I_shared != 0 && !expert_cols_ok(I_shared)))
    return MOE_ERR_INVALID_ARG;
  if ((shared != nullptr) != (I_shared > 0)) return MOE_ERR_INVALID_ARG;
  if (!experts_ok(routed) || (shared && (!experts_ok(shared) || shared->n_experts != 1))) return MOE_ERR_INVALID_ARG;
  const int E = routed->n_experts;
  if (E > kMaxE || k > kMaxK || k > E) return MOE_ERR_UNSUPPORTED;
  // rows of the tensor maps and the launch's items are 32-bit
  if (static_cast<long long>(T) * (k + 1) > (1ll << 30) || static_cast<long long>(E) * (d > I ? d : I) > (1ll << 30))
    return MOE_ERR_UNSUPPORTED;
  if ((X != nullptr) == (XQ != nullptr) && T > 0) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!Y || !aligned16(Y) || (X && !aligned16(X)) || (XQ && !mat_ok(XQ)))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Whether the products' items can be counted; everything else has been checked.
bool items_ok(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  auto m_tiles = [](int a, int b) { return static_cast<long long>(blk_count(a > b ? a : b)); };
  long long items = moe_route_max_blocks(T, E, k, block_rows) * m_tiles(d, I);
  if (I_shared > 0) {
    const int rows = shared_tile_rows(T, block_rows);
    items += (T + rows - 1) / rows * m_tiles(d, I_shared);
  }
  return items <= kBlkMaxItems;
}

BlkWeights weights(const moe_blk_experts* ex) {
  if (!ex) return BlkWeights{};
  return BlkWeights{ex->gate.q, ex->up.q, ex->down.q, ex->gate.s, ex->up.s, ex->down.s};
}

moe_status forward(const uint16_t* X, const moe_blk_mat* XQ, int T, int d, int I, int k, const moe_blk_experts* routed,
                   const moe_blk_experts* shared, int I_shared, const moe_routing* r, uint16_t* Y, void* ws,
                   bool after_routing, moe_stream stream) {
  if (T == 0) return MOE_OK;
  const int E = routed->n_experts;
  const ExpertLayout L = expert_layout(T, d, I, E, k, I_shared, r->block_rows);
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint32_t* status = &static_cast<WsHeader*>(ws)->status;
  const int num_sms = device_sms();
  if (num_sms <= 0) return MOE_ERR_CUDA;
  const BlkX x = X ? BlkX{X, nullptr, d, 0, MOE_BF16} : BlkX{XQ->q, XQ->s, d, blk_scale_rows(T), kBlkCodes};
  if (L.few) {
    BlkFewArgs a{};
    a.x = x;
    a.routed = weights(routed);
    a.shared = weights(shared);
    a.perm = r->perm;
    a.block_map = r->block_map;
    a.num_blocks = r->num_blocks;
    a.w = r->w;
    a.h = reinterpret_cast<float*>(w + L.h);
    a.y = Y;
    a.status = status;
    a.T = T;
    a.d = d;
    a.I = I;
    a.k = k;
    a.I_shared = I_shared;
    a.E = E;
    a.tiles = T * k < L.max_blocks ? T * k : L.max_blocks;
    a.split = few_split(T, d, I, k, I_shared);
    return done(launch_blk_few_experts(a, cuda(stream), pdl_enabled()));
  }

  const long long A = static_cast<long long>(T) * k, rows = A + (shared ? T : 0);
  BlkExpertArgs a{};
  a.block_map = r->block_map;
  a.num_blocks = r->num_blocks;
  a.inv_perm = r->inv_perm;
  a.w = r->w;
  a.routed = weights(routed);
  a.shared = weights(shared);
  a.sx = reinterpret_cast<float*>(w + L.sx);
  a.sh_r = reinterpret_cast<float*>(w + L.sh_r);
  a.sh_s = reinterpret_cast<float*>(w + L.sh_s);
  a.h_r = w + L.h_r;
  a.h_s = w + L.h_s;
  a.ypart = reinterpret_cast<float*>(w + L.ypart);
  a.y = Y;
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
  a.pitch = L.pitch;
  BlkExpertMaps maps;
  bool ok = encode_mx_weights(&maps.gate_r, routed->gate.q, E, I, d, kBlk) &&
            encode_mx_weights(&maps.up_r, routed->up.q, E, I, d, kBlk) &&
            encode_mx_weights(&maps.down_r, routed->down.q, E, d, I, kBlk) &&
            encode_mx_codes(&maps.x_r, w + L.q_x, rows, d, L.bn_r) && encode_mx_codes(&maps.h_r, a.h_r, A, I, L.bn_r);
  if (shared) {
    ok = ok && encode_mx_weights(&maps.gate_s, shared->gate.q, 1, I_shared, d, kBlk) &&
         encode_mx_weights(&maps.up_s, shared->up.q, 1, I_shared, d, kBlk) &&
         encode_mx_weights(&maps.down_s, shared->down.q, 1, d, I_shared, kBlk) &&
         encode_mx_codes(&maps.x_s, w + L.q_x, rows, d, L.bn_s) && encode_mx_codes(&maps.h_s, a.h_s, T, I_shared, L.bn_s);
  } else {  // never read
    maps.gate_s = maps.up_s = maps.down_s = maps.gate_r;
    maps.x_s = maps.h_s = maps.x_r;
  }
  const bool wide = L.pitch > kBlkNarrow;
  maps.ypart = maps.x_r;
  if (wide) ok = ok && encode_out_boxes(&maps.ypart, a.ypart, 4, rows, d);
  if (!ok) return MOE_ERR_CUDA;
  const MxScatter sc{r->inv_perm, r->block_map, r->num_blocks, status, T, k, L.max_blocks, shared ? L.bn_s : 0, after_routing};
  if (launch_blk_scatter(x, d, sc, L.pitch, w + L.q_x, a.sx, cuda(stream), pdl_enabled()) != cudaSuccess) return MOE_ERR_CUDA;
  return done(wide ? launch_blk_wide_experts(a, maps, cuda(stream), pdl_enabled())
                   : launch_blk_experts(a, maps, cuda(stream), pdl_enabled()));
}

}  // namespace
}  // namespace bm

using namespace bm;

extern "C" {

moe_status moe_blk_quantize(const void* X, moe_dtype type, int rows, int K, long long ldx, const moe_blk_mat* out,
                            moe_stream stream) {
  const moe_status st = check_x(X, type, rows, K, ldx);
  if (st != MOE_OK || rows == 0) return st;
  if (!mat_ok(out)) return MOE_ERR_INVALID_ARG;
  return done(launch_blk_quantize(X, type, rows, K, ldx, out->q, out->s, cuda(stream), pdl_enabled()));
}

moe_status moe_blk_quantize_weights(const void* W, moe_dtype type, int E, int N, int K, const moe_blk_mat* out,
                                    moe_stream stream) {
  const moe_status st = check_weights(W, type, E, N, K, out);
  if (st != MOE_OK) return st;
  return done(launch_blk_quantize_weights(W, type, E, N, K, out->q, out->s, cuda(stream), pdl_enabled()));
}

moe_status moe_blk_dequant(const moe_blk_mat* a, int rows, int K, moe_dtype type, void* X, moe_stream stream) {
  const moe_status st = check_x(X, type, rows, K, K);
  if (st != MOE_OK || rows == 0) return st;
  if (!mat_ok(a)) return MOE_ERR_INVALID_ARG;
  return done(launch_blk_dequant(a->q, a->s, rows, K, type, X, cuda(stream), pdl_enabled()));
}

moe_status moe_blk_dequant_weights(const moe_blk_mat* m, int E, int N, int K, moe_dtype type, void* W, moe_stream stream) {
  const moe_status st = check_weights(W, type, E, N, K, m);
  if (st != MOE_OK) return st;
  return done(launch_blk_dequant_weights(m->q, m->s, E, N, K, type, W, cuda(stream), pdl_enabled()));
}

moe_status moe_blk_matmul(const moe_blk_mat* A, int M, const moe_blk_mat* W, int N, int K, void* Y, moe_dtype y_type,
                          void* ws, size_t ws_bytes, moe_stream stream) {
  const moe_status st = check_matmul(M, W, N, K, Y, y_type);
  if (st != MOE_OK) return st;
  if (!ws_ok(ws, ws_bytes, sizeof(WsHeader))) return MOE_ERR_WORKSPACE;
  if (M == 0) return MOE_OK;
  if (!mat_ok(A)) return MOE_ERR_INVALID_ARG;
  return matmul(*A, M, W, N, K, Y, y_type, &static_cast<WsHeader*>(ws)->status, stream);
}

size_t moe_blk_linear_workspace_bytes(int T, int N, int K) {
  if (T < 0 || !size_ok(N, K)) return 0;
  return sizeof(WsHeader) + round256(static_cast<size_t>(T) * K) + round256(act_scale_bytes(T, K));
}

moe_status moe_blk_linear(const void* X, moe_dtype x_type, int T, int K, long long ldx, const moe_blk_mat* W, int N,
                          void* Y, moe_dtype y_type, void* ws, size_t ws_bytes, moe_stream stream) {
  moe_status st = check_x(X, x_type, T, K, ldx);
  if (st != MOE_OK) return st;
  st = check_matmul(T, W, N, K, Y, y_type);
  if (st != MOE_OK) return st;
  if (!ws_ok(ws, ws_bytes, moe_blk_linear_workspace_bytes(T, N, K))) return MOE_ERR_WORKSPACE;
  if (T == 0) return MOE_OK;
  uint8_t* w = static_cast<uint8_t*>(ws) + sizeof(WsHeader);
  const moe_blk_mat xq{w, reinterpret_cast<float*>(w + round256(static_cast<size_t>(T) * K))};
  if (T == 1) {
    const int num_sms = device_sms();
    if (num_sms <= 0) return MOE_ERR_CUDA;
    if (one_launch_wins(N, K, num_sms)) return few_linear(BlkX{X, nullptr, ldx, 0, x_type}, T, W, N, K, Y, y_type, stream);
  }
  if (launch_blk_quantize(X, x_type, T, K, ldx, xq.q, xq.s, cuda(stream), pdl_enabled()) != cudaSuccess) return MOE_ERR_CUDA;
  return matmul(xq, T, W, N, K, Y, y_type, &static_cast<WsHeader*>(ws)->status, stream);
}

moe_status moe_rmsnorm(const void* X, moe_dtype x_type, int T, int d, long long ldx, const void* residual,
                       void* residual_out, moe_dtype residual_type, const void* gamma, moe_dtype gamma_type, float eps,
                       void* Y, moe_dtype y_type, const moe_blk_mat* out, moe_stream stream) {
  const moe_status st = check_x(X, x_type, T, d, ldx);
  if (st != MOE_OK) return st;
  if (!gamma || !aligned16(gamma) || (gamma_type != MOE_BF16 && gamma_type != MOE_FP32)) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return d > kNormMaxCols ? MOE_ERR_UNSUPPORTED : MOE_OK;
  if ((residual != nullptr) != (residual_out != nullptr)) return MOE_ERR_INVALID_ARG;
  if (residual && (!aligned16(residual) || !aligned16(residual_out) || (residual_type != x_type && residual_type != MOE_FP32)))
    return MOE_ERR_INVALID_ARG;
  if (!Y && !out) return MOE_ERR_INVALID_ARG;
  if (Y && (!aligned16(Y) || !type_ok(y_type))) return MOE_ERR_INVALID_ARG;
  if (out && !mat_ok(out)) return MOE_ERR_INVALID_ARG;
  if (d > kNormMaxCols) return MOE_ERR_UNSUPPORTED;
  RmsNorm n{};
  n.x = X;
  n.residual = residual;
  n.residual_out = residual_out;
  n.gamma = gamma;
  n.y = Y;
  n.q = out ? out->q : nullptr;
  n.s = out ? out->s : nullptr;
  n.ldx = ldx;
  n.eps = eps;
  n.T = T;
  n.d = d;
  n.x_type = x_type;
  n.residual_type = residual_type;
  n.gamma_fp32 = gamma_type == MOE_FP32;
  n.y_type = y_type;
  return done(launch_rmsnorm(n, cuda(stream), pdl_enabled()));
}

size_t moe_blk_forward_workspace_bytes(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  if (!sizes_valid(T, d, I, E, k, I_shared, block_rows)) return 0;
  return expert_layout(T, d, I, E, k, I_shared, block_rows).total;
}

moe_status moe_blk_forward(const uint16_t* X, const moe_blk_mat* XQ, int T, int d, int I, int k,
                           const moe_blk_experts* routed, const moe_blk_experts* shared, int I_shared,
                           const moe_routing* r, uint16_t* Y, void* ws, size_t ws_bytes, moe_stream stream) {
  const moe_status st = check_experts(X, XQ, T, d, I, k, routed, shared, I_shared, Y);
  if (st != MOE_OK) return st;
  if (!r) return MOE_ERR_INVALID_ARG;
  if (r->block_rows < 1 || r->block_rows > kMaxBlockRows) return MOE_ERR_UNSUPPORTED;
  if (!items_ok(T, d, I, routed->n_experts, k, I_shared, r->block_rows)) return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!r->w || !r->perm || !r->inv_perm || !r->block_map || !r->num_blocks)) return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, moe_blk_forward_workspace_bytes(T, d, I, routed->n_experts, k, I_shared, r->block_rows)))
    return MOE_ERR_WORKSPACE;
  return forward(X, XQ, T, d, I, k, routed, shared, I_shared, r, Y, ws, false, stream);
}

size_t moe_blk_layer_workspace_bytes(int T, int d, int I, int E, int k, int I_shared, int block_rows) {
  const size_t f = moe_blk_forward_workspace_bytes(T, d, I, E, k, I_shared, block_rows);
  const size_t r = moe_route_workspace_bytes(T, E, k);
  return f && r ? (f > r ? f : r) : 0;
}

moe_status moe_blk_layer(const float* logits, const moe_scoring* scoring, const uint16_t* X, const moe_blk_mat* XQ,
                         int T, int d, int I, int k, int block_rows, const moe_blk_experts* routed,
                         const moe_blk_experts* shared, int I_shared, moe_routing* r, uint16_t* Y, void* ws,
                         size_t ws_bytes, moe_stream stream) {
  moe_status st = check_experts(X, XQ, T, d, I, k, routed, shared, I_shared, Y);
  if (st != MOE_OK) return st;
  const int E = routed->n_experts;
  st = check_scored(logits, scoring, T, E, k, block_rows, r);
  if (st != MOE_OK) return st;
  if (!items_ok(T, d, I, E, k, I_shared, block_rows)) return MOE_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, moe_blk_layer_workspace_bytes(T, d, I, E, k, I_shared, block_rows))) return MOE_ERR_WORKSPACE;
  // one header for both, and after it the same room: the products start when the routing has completed
  st = route_scored(logits, scoring, T, E, k, block_rows, r, ws, stream);
  if (st != MOE_OK) return st;
  return forward(X, XQ, T, d, I, k, routed, shared, I_shared, r, Y, ws, true, stream);
}

}  // extern "C"
