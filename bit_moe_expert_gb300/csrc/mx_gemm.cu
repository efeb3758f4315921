// MXFP4 products on the block-scaled tensor cores: dense (Y = A W^T) and the
// expert layer's grouped gate/up and down products.
//
// D[m][n] = sum_k sa[m][k/32] sb[n][k/32] a[m][k] b[n][k], a and b E2M1 codes.
// tcgen05.mma kind::mxf4 takes the codes two to a byte from shared memory and
// the E8M0 scales from tensor memory, multiplies by them inside the MMA and
// accumulates in fp32: nothing is dequantised by other instructions.  A stage of
// the pipeline is K = 256: one 128-byte line of codes a row (the widest swizzle
// atom), two 512-byte pieces of scales per 128 rows, four MMAs of K = 64.
//
// The weights are the M = 128 side and the tokens the N side: an expert with few
// tokens streams its weights once and pads only tokens (tiles of 16..128), and
// the dense product's epilogue has neighbouring columns of Y in neighbouring
// lanes, whatever the width of Y (tokens on the M side, with 16-byte stores per
// lane, took 216 us instead of 205 at 8192^3).  Dense tiles are 64, 128 or 256
// tokens high.
//
// Roles (one persistent CTA per SM): warps 0 and 1 the weights' and the
// activations' loads, warp 2 MMA issuer (copies a stage's scales from shared to
// tensor memory, then multiplies: the tensor pipeline keeps the order), warps
// 3 on epilogue, two or four per quarter of the tensor-memory lanes.  Every wait
// is bounded and records MOE_ERR_TIMEOUT.
//
// Measured, each kernel alone between events: experts of d = 2048, I = 512, 8 of 256
// + shared, 512 tokens in tiles of 32: gate/up 44 us for 285 MB of weights, down 31
// us for 143 MB and 38 MB of rows (bound by memory); 4096 tokens in tiles of 128: 65
// us, and 76 us with 302 MB of rows written.  Inside a layer they overlap with their
// neighbours.  Dense: 333 x 2816 -> 1001 5 us, 512 x 4096 -> 8192 10 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "kernels.h"
#include "mx.cuh"
#include "ptx.cuh"

namespace bm {
namespace {

enum Mode { kLinear, kGateUp, kDown };

constexpr int kWeightsWarp = 0;
constexpr int kActivationsWarp = 1;
constexpr int kMmaWarp = 2;
constexpr int kEpiWarp0 = 3;
// A launch's variant.  kRowTiles: 128-row groups of scales of the tokens (tiles of
// up to 128, or of 256).  kHold: there is room for one accumulator only, so the
// epilogue takes its columns into registers and releases it before it works on
// them (8192^3 200 -> 195 us, 4096^3 42.4 -> 37.5, both before the pairs below;
// gate/up of 4096 tokens in tiles of 128 75.5 -> 65, the layer 224 -> 213); with
// more accumulators nothing waits for it, and the registers would keep the CTA from
// starting beside the previous kernel's (256 x 2048 -> 2048 6.1 -> 7.1 us).
template <int kMode_, int kRowTiles_, bool kHold_>
struct Variant {
  static constexpr int kMode = kMode_, kRowTiles = kRowTiles_;
  static constexpr bool kHold = kHold_;
  // epilogue warps, a multiple of four (one per quarter of the tensor-memory lanes)
  static constexpr int kEpiWarps = kMode == kGateUp || kHold ? 16 : 8;
  static constexpr int kParts = kEpiWarps / 4;  // shares of the columns
  static constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
  // what one turn of the epilogue's loop takes: groups of eight (gate/up) or 16 columns
  static constexpr int kGroup = kMode == kGateUp ? 8 : 16;
  static constexpr int kHeld = kHold ? 128 * kRowTiles / (kGroup * kParts) : 1;
};
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 12;
constexpr int kMaxAccs = 8;
constexpr int kCodeBytesM = kMxBM * 128;   // one matrix's codes of a stage
constexpr int kPairBytes = 2 * kMxPieceBytes;  // a stage's scales of 128 rows
constexpr int kSmemLimit = 227 * 1024;
constexpr int kEntries = 256;  // items of a CTA, from its first, whose Entry is in shared memory
constexpr int kSmemFixed = 1024 /* barriers */ + 16 * kEntries + 1024 /* alignment */;

// How a launch divides shared and tensor memory; bn: the N side's columns at most.
struct Plan {
  int bn, row_tiles, stages, stage_bytes, acc_bufs;
};

__host__ __device__ constexpr int scale_cols(int mats, int row_tiles) { return 8 * (mats + row_tiles); }

Plan make_plan(int mats, int bn) {
  Plan p;
  p.bn = bn;
  p.row_tiles = (bn + kMxPieceRows - 1) / kMxPieceRows;
  p.stage_bytes = mats * (kCodeBytesM + kPairBytes) + bn * 128 + p.row_tiles * kPairBytes;
  p.stages = (kSmemLimit - kSmemFixed) / p.stage_bytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  // further accumulators let the epilogue of one item run beside the next ones' products
  p.acc_bufs = (static_cast<int>(kTmemCols) - 2 * scale_cols(mats, p.row_tiles)) / (mats * bn);
  if (p.acc_bufs > kMaxAccs) p.acc_bufs = kMaxAccs;
  return p;
}

struct Item {
  const CUtensorMap *m0, *m1, *n;  // codes of the weights (one or two matrices) and of the tokens
  const uint8_t *sm0, *sm1, *sn;   // their scales: the item's first pieces
  int e, row_m, row_n;             // matrix of the M side; first rows of the codes
  int mt, rows, K, box;            // M tile, valid N rows, depth, N rows that the TMA box brings
  int row0, slot;                  // experts: first row among the assignments (or tokens), tile slot
  int groups;                      // 128-row groups of scales on the N side
  bool shared, ok;
};

// This CTA's items: local index i stands for item first + i * step, dealt out in
// turn, so that CTAs running together read neighbouring tiles (runs of
// consecutive items per CTA cost the 512-token layer's gate/up product 65
// instead of 53 us).
struct Sched {
  int mt_r, mt_s;  // M tiles of a routed and of a shared tile
  int n_routed;    // expert products: items below are routed
  int first, n, step;
};

// What an item's id stands for, as every role needs it.
struct Entry {
  int e, row0;    // expert (-1: malformed) and first row; dense: 0 and the M tile
  int slot;       // entry of the block map, the shared expert's tile of tokens, or the dense product's N tile
  uint32_t what;  // experts: M tile + 2^16 rows + 2^31 for the shared expert
};
constexpr uint32_t kEntryShared = 1u << 31;
static_assert(kMxMaxCols / kMxBM <= 1 << 16 && kMxMaxBN < 1 << 15, "an Entry's M tile and rows");
template <int kMode>
struct Args {
  using type = MxExpertArgs;
  using maps = MxExpertMaps;
};
template <>
struct Args<kLinear> {
  using type = MxLinearArgs;
  using maps = MxLinearMaps;
};

__device__ __forceinline__ int pieces_of(int K) { return (K + kMxPieceK - 1) / kMxPieceK; }

__device__ __forceinline__ Sched make_sched(const MxLinearArgs& a, const Plan& p, bool) {
  Sched s{};
  s.mt_r = (a.N + kMxBM - 1) / kMxBM;
  const int total = s.mt_r * ((a.M + p.bn - 1) / p.bn);
  s.first = blockIdx.x;
  s.step = gridDim.x;
  s.n = (total - s.first + s.step - 1) / s.step;
  return s;
}

__device__ __forceinline__ Entry make_entry(const MxLinearArgs&, const Sched& s, int it) {
  return Entry{0, it % s.mt_r, it / s.mt_r, 0};
}

__device__ __forceinline__ Item get_item(const MxLinearArgs& a, const MxLinearMaps& maps, const Plan& p,
                                         const Entry& en, bool) {
  Item m{};
  const int pieces = pieces_of(a.K);
  m.mt = en.row0;
  const int nt = en.slot;
  m.m0 = &maps.w;
  m.n = &maps.x;
  m.row_m = m.mt * kMxBM;
  m.row_n = nt * p.bn;
  m.rows = min(p.bn, a.M - m.row_n);
  m.K = a.K;
  m.box = p.bn;
  m.sm0 = a.sp_w + static_cast<size_t>(m.mt) * pieces * kMxPieceBytes;
  m.sn = a.sp_x + static_cast<size_t>(m.row_n / kMxPieceRows) * pieces * kMxPieceBytes;
  m.groups = (m.rows + kMxPieceRows - 1) / kMxPieceRows;
  m.ok = true;
  return m;
}

__device__ __forceinline__ Sched make_sched(const MxExpertArgs& a, const Plan&, bool gate_up) {
  Sched s{};
  int nb = *reinterpret_cast<const volatile int32_t*>(a.num_blocks);
  if (nb < 1 || nb > min(a.max_blocks, a.T * a.k)) {  // every tile holds an assignment
    if (threadIdx.x == 0) record_status(a.status, MOE_ERR_INVALID_ARG);
    nb = 0;
  }
  s.mt_r = ((gate_up ? a.I : a.d) + kMxBM - 1) / kMxBM;
  s.mt_s = ((gate_up ? a.I_shared : a.d) + kMxBM - 1) / kMxBM;
  s.n_routed = nb * s.mt_r;
  const int total = s.n_routed + (a.I_shared > 0 ? (a.T + a.bn_s - 1) / a.bn_s * s.mt_s : 0);
  s.first = blockIdx.x;
  s.step = gridDim.x;
  s.n = (total - s.first + s.step - 1) / s.step;
  return s;
}

__device__ __forceinline__ Entry make_entry(const MxExpertArgs& a, const Sched& s, int it) {
  Entry en;
  if (it < s.n_routed) {
    en.slot = it / s.mt_r;
    const volatile int32_t* b = a.block_map + 3 * static_cast<size_t>(en.slot);
    en.e = b[0];
    en.row0 = b[1];
    const int rows = b[2];
    const bool ok = en.e >= 0 && en.e < a.E && rows >= 1 && rows <= a.bn_r && en.row0 >= 0 &&
                    en.row0 <= a.T * a.k - rows;
    if (!ok) en.e = -1;
    en.what = static_cast<uint32_t>(it - en.slot * s.mt_r) | static_cast<uint32_t>(rows) << 16;
  } else {
    const int j = it - s.n_routed;
    en.slot = j / s.mt_s;
    en.e = 0;
    en.row0 = en.slot * a.bn_s;
    en.what = kEntryShared | static_cast<uint32_t>(j - en.slot * s.mt_s) |
              static_cast<uint32_t>(min(a.bn_s, a.T - en.row0)) << 16;
  }
  return en;
}

__device__ __forceinline__ Item get_item(const MxExpertArgs& a, const MxExpertMaps& maps, const Plan&, const Entry& en,
                                         bool gate_up) {
  Item m{};
  m.ok = en.e >= 0;
  if (!m.ok) return m;
  const int e = en.e;
  m.row0 = en.row0;
  m.rows = static_cast<int>(en.what >> 16 & 0x7FFFu);
  m.shared = (en.what & kEntryShared) != 0;
  m.mt = static_cast<int>(en.what & 0xFFFFu);
  m.slot = en.slot;
  const int I = m.shared ? a.I_shared : a.I;
  const int N = gate_up ? I : a.d;
  m.K = gate_up ? a.d : I;
  m.box = m.shared ? a.bn_s : a.bn_r;
  if (m.shared) {
    m.m0 = gate_up ? &maps.gate_s : &maps.down_s;
    m.m1 = &maps.up_s;
    m.n = gate_up ? &maps.x_s : &maps.h_s;
    m.sm0 = gate_up ? a.sp_gate_s : a.sp_down_s;
    m.sm1 = a.sp_up_s;
    m.row_n = gate_up ? a.T * a.k + m.row0 : m.row0;
  } else {
    m.m0 = gate_up ? &maps.gate_r : &maps.down_r;
    m.m1 = &maps.up_r;
    m.n = gate_up ? &maps.x_r : &maps.h_r;
    m.sm0 = gate_up ? a.sp_gate_r : a.sp_down_r;
    m.sm1 = a.sp_up_r;
    m.row_n = m.row0;
  }
  m.groups = 1;
  const int pieces = pieces_of(m.K);
  const size_t tile = (static_cast<size_t>(e) * ((N + kMxPieceRows - 1) / kMxPieceRows) + m.mt) * pieces * kMxPieceBytes;
  m.sm0 += tile;
  m.sm1 += tile;
  m.row_m = m.mt * kMxBM;
  m.e = e;
  const uint8_t* sn = gate_up ? a.sp_x : (m.shared ? a.sp_h_s : a.sp_h_r);
  m.sn = sn + static_cast<size_t>(gate_up && m.shared ? a.max_blocks + m.slot : m.slot) * pieces * kMxPieceBytes;
  return m;
}

__device__ __forceinline__ int tile_n(int rows) { return (rows + 15) & ~15; }

// An 8 x 8 matrix of 4-bit elements, row l in lane l of each group of eight
// lanes (element j in bits 4j): transposed by exchanging halves, bytes, nibbles.
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t v, int lane) {
  uint32_t t = __shfl_xor_sync(0xffffffffu, v, 4);
  v = (lane & 4) ? (v & 0xFFFF0000u) | (t >> 16) : (v & 0x0000FFFFu) | (t << 16);
  t = __shfl_xor_sync(0xffffffffu, v, 2);
  v = (lane & 2) ? (v & 0xFF00FF00u) | ((t >> 8) & 0x00FF00FFu) : (v & 0x00FF00FFu) | ((t & 0x00FF00FFu) << 8);
  t = __shfl_xor_sync(0xffffffffu, v, 1);
  v = (lane & 1) ? (v & 0xF0F0F0F0u) | ((t >> 4) & 0x0F0F0F0Fu) : (v & 0x0F0F0F0Fu) | ((t & 0x0F0F0F0Fu) << 4);
  return v;
}

// gate/up: h = silu(gate) * up in fp32, quantised here.  A warp's 32 lanes are 32
// consecutive columns of h, one block, so a token's largest magnitude is one
// reduction over the lanes; eight tokens' codes are turned by a nibble
// transposition into words of eight columns of one token.  (Two tokens' exponents
// to a word and shuffles that halve the words, 11 for eight tokens, came out 2 us
// slower than a reduction each at 4096 tokens; without any of this arithmetic and
// its stores the product takes 60 instead of 65.)
template <typename V, typename Release>
__device__ __forceinline__ void epilogue_gate_up(const MxExpertArgs& a, const Item& m, const Plan& p, uint32_t tbase,
                                                 int bn, int lanegrp, int colpart, int lane, Release release) {
  const int I = m.shared ? a.I_shared : a.I;
  const int n0 = m.mt * kMxBM + 32 * lanegrp;
  const int pieces = pieces_of(I);
  uint8_t* hq = (m.shared ? a.q_h_s : a.q_h_r) + static_cast<size_t>(m.row0) * (I / 2) + n0 / 2 + 4 * (lane >> 3);
  uint8_t* hs = (m.shared ? a.sp_h_s : a.sp_h_r) +
                (static_cast<size_t>(m.slot) * pieces + m.mt) * kMxPieceBytes + lanegrp;
  const bool valid = n0 < I;  // the same for the whole warp; past I the piece's scale bytes are zeros
  int first = 8 * colpart;
  do {  // with kHold, one turn
    uint32_t g[V::kHeld][8], u[V::kHeld][8];
#pragma unroll
    for (int i = 0; i < V::kHeld; ++i) {
      const int c0 = first + 8 * V::kParts * i;
      if (c0 < bn) {
        tmem_ld8(tbase + c0, g[i]);
        tmem_ld8(tbase + p.bn + c0, u[i]);
      }
    }
    tc_wait_ld();
    if (V::kHold) release();
#pragma unroll
    for (int i = 0; i < V::kHeld; ++i) {
      const int c0 = first + 8 * V::kParts * i;
      if (c0 >= m.rows) break;
      float h[8];
      uint32_t largest = 0;  // of token lane % 8: its exponent
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        h[c] = mx_swiglu(__uint_as_float(g[i][c]), __uint_as_float(u[i][c]));
        const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(h[c]) & 0x7F800000u);
        if ((lane & 7) == c) largest = e;
        h[c] *= __uint_as_float(0x80000000u - max(e, 2u << 23));  // mx_inverse_scale of its byte, but for 255
      }
      const uint32_t code = transpose_nibbles(f32x8_to_e2m1x8(h), lane);
      const int r = c0 + (lane & 7);
      if (r < m.rows) {
        if (valid) *reinterpret_cast<uint32_t*>(hq + static_cast<size_t>(r) * (I / 2)) = code;
        if (lane < 8) hs[(r % 32) * 16 + (r / 32) * 4] = valid ? static_cast<uint8_t>(mx_scale_byte(largest)) : 0;
      }
    }
    first += 8 * V::kParts * V::kHeld;
  } while (!V::kHold && first < bn);
  if (!V::kHold) release();
}

// Sixteen rows of a lane's column of the result, of which `valid` exist; `at`:
// the first one's element, the others `pitch` apart.
template <typename Store>
__device__ __forceinline__ void store_rows(size_t at, size_t pitch, int valid, const uint32_t (&v)[16], Store store) {
  if (valid >= 16) {
#pragma unroll
    for (int c = 0; c < 16; ++c, at += pitch) store(at, __uint_as_float(v[c]));
  } else {
#pragma unroll
    for (int c = 0; c < 16; ++c, at += pitch)
      if (c < valid) store(at, __uint_as_float(v[c]));
  }
}
struct OutF32 {
  float* y;
  __device__ __forceinline__ void rows(size_t at, size_t pitch, int valid, const uint32_t (&v)[16]) const {
    store_rows(at, pitch, valid, v, [&](size_t i, float x) { y[i] = x; });
  }
};
struct OutLinear {
  void* y;
  int fp32;
  __device__ __forceinline__ void rows(size_t at, size_t pitch, int valid, const uint32_t (&v)[16]) const {
    if (fp32)
      store_rows(at, pitch, valid, v, [&](size_t i, float x) { static_cast<float*>(y)[i] = x; });
    else
      store_rows(at, pitch, valid, v, [&](size_t i, float x) { static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(x); });
  }
};

// down and dense: a lane's column n of the tile's rows, from row `row0` of the
// result on; 32 lanes write neighbouring columns of a row.
template <typename V, typename Out, typename Release>
__device__ __forceinline__ void epilogue_rows(Out out, size_t row0, int n, int N, int rows, uint32_t tbase, int bn,
                                              int colpart, Release release) {
  const size_t pitch = N;
  int first = 16 * colpart;
  do {  // with kHold, one turn
    uint32_t v[V::kHeld][16];
#pragma unroll
    for (int i = 0; i < V::kHeld; ++i) {
      const int c0 = first + 16 * V::kParts * i;
      if (c0 < bn) tmem_ld16(tbase + c0, v[i]);
    }
    tc_wait_ld();
    if (V::kHold) release();
    if (n < N) {
#pragma unroll
      for (int i = 0; i < V::kHeld; ++i) {
        const int c0 = first + 16 * V::kParts * i;
        if (c0 < rows) out.rows((row0 + c0) * pitch + n, pitch, rows - c0, v[i]);
      }
    }
    first += 16 * V::kParts * V::kHeld;
  } while (!V::kHold && first < bn);
  if (!V::kHold) release();
}

template <typename V, typename Release>
__device__ __forceinline__ void epilogue(const MxExpertArgs& a, const Item& m, const Plan& p, uint32_t tbase, int bn,
                                         int lanegrp, int colpart, int lane, Release release) {
  if constexpr (V::kMode == kGateUp) {
    epilogue_gate_up<V>(a, m, p, tbase, bn, lanegrp, colpart, lane, release);
  } else {
    // fp32 rows of the experts' outputs, routed ones in permuted order, then the shared expert's in token order
    epilogue_rows<V>(OutF32{a.ypart}, static_cast<size_t>(m.shared ? a.T * a.k : 0) + m.row0,
                     m.mt * kMxBM + 32 * lanegrp + lane, a.d, m.rows, tbase, bn, colpart, release);
  }
}

template <typename V, typename Release>
__device__ __forceinline__ void epilogue(const MxLinearArgs& a, const Item& m, const Plan&, uint32_t tbase, int bn,
                                         int lanegrp, int colpart, int lane, Release release) {
  const int n = m.row_m + 32 * lanegrp + lane;
  epilogue_rows<V>(OutLinear{a.Y, a.y_fp32}, m.row_n, n, a.N, m.rows, tbase, bn, colpart, release);
}

template <typename V>
__global__ void __launch_bounds__(V::kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ typename Args<V::kMode>::maps maps,
                   const __grid_constant__ typename Args<V::kMode>::type a, const Plan p) {
  constexpr int kMode = V::kMode, kRowTiles = V::kRowTiles;
  constexpr int kMats = kMode == kGateUp ? 2 : 1;
  constexpr bool kGU = kMode == kGateUp;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(stages + p.stages * p.stage_bytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + kMaxAccs;
  uint64_t* done = acc_empty + kMaxAccs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Entry* entries = reinterpret_cast<Entry*>(stages + p.stages * p.stage_bytes + 1024);
  static_assert(sizeof(Entry) == 16, "room of the entries");

  // the same in all lanes, so that the roles' branches are known to be uniform
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  // The routing has completed by now (the kernel before this one lets this one
  // start only after its own wait), so only the activations are waited for.
  const Sched s = make_sched(a, p, kGU);
  for (int i = threadIdx.x; i < min(s.n, kEntries); i += V::kThreads) entries[i] = make_entry(a, s, s.first + i * s.step);
  auto item = [&](int i) {
    return get_item(a, maps, p, i < kEntries ? entries[i] : make_entry(a, s, s.first + i * s.step), kGU);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 2);  // the weights' and the activations' expect_tx; their bytes complete the phase
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < p.acc_bufs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], V::kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&]() {
    record_status(a.status, MOE_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == kWeightsWarp || warp == kActivationsWarp) {
    // one thread for the weights, which starts before the wait, and one for the activations
    if (lane == 0) {
      const bool weights = warp == kWeightsWarp;
      if (!weights) pdl_wait();
      int stage = 0, filled = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; i < s.n && ok; ++i) {
        const Item m = item(i);
        if (!m.ok) continue;
        const int pieces = pieces_of(m.K);
        const uint32_t codes = weights ? kMats * kCodeBytesM : m.box * 128;
        const int scales = weights ? kMats : m.groups;
        const size_t group = static_cast<size_t>(pieces) * kMxPieceBytes;
        const uint8_t *s0 = weights ? m.sm0 : m.sn, *s1 = weights ? m.sm1 : m.sn + group;
        for (int k0 = 0; k0 < pieces; k0 += 2, ++filled) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          uint8_t* st = stages + stage * p.stage_bytes + (weights ? 0 : kMats * kCodeBytesM);
          uint8_t* sf = stages + stage * p.stage_bytes + kMats * kCodeBytesM + p.bn * 128 + (weights ? 0 : kMats * kPairBytes);
          uint64_t* bar = &full[stage];
          const uint32_t sbytes = min(2, pieces - k0) * kMxPieceBytes;
          mbar_arrive_expect_tx(bar, codes + scales * sbytes);
          if (weights) {
            tma_load_3d(st, m.m0, bar, k0 * 64, m.row_m, m.e);
            if (kGU) tma_load_3d(st + kCodeBytesM, m.m1, bar, k0 * 64, m.row_m, m.e);
          } else {
            tma_load_2d(st, m.n, bar, k0 * 64, m.row_n);
          }
          bulk_g2s(sf, s0, sbytes, bar);
          if (scales > 1) bulk_g2s(sf + kPairBytes, s1, sbytes, bar);
          s0 += kPairBytes;
          s1 += kPairBytes;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // never leave while a load into this CTA's shared memory may be in flight
      for (int i = 0; i < min(filled, p.stages); ++i) {
        stage = stage == 0 ? p.stages - 1 : stage - 1;
        if (stage == p.stages - 1) phase ^= 1;
        if (!mbar_wait(&full[stage], phase, nullptr)) record_status(a.status, MOE_ERR_TIMEOUT);
      }
      if (weights) pdl_wait();
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    pdl_wait();
    pdl_launch_dependents();
    // One thread issues everything; what it issues is computed by the whole warp
    // from values that are the same in all lanes (votes, shuffles from lane 0),
    // which lets the compiler keep descriptors and addresses in uniform
    // registers.  The issue loop is what bounds short products otherwise: at
    // K = 512 a stage took 1,000 cycles to issue.
    const uint32_t stage0 = smem_u32(stages);
    // tensor memory: the accumulators, then two sets of a stage's scales
    const uint32_t sf_tmem = tmem + p.acc_bufs * kMats * p.bn;
    constexpr int kScaleCols = scale_cols(kMats, kRowTiles);
    const uint64_t ad0 = smem_desc_sw128_kmajor(stage0);
    const uint64_t bd0 = smem_desc_sw128_kmajor(stage0 + kMats * kCodeBytesM);
    const uint64_t sd0 = smem_desc_scales(stage0 + kMats * kCodeBytesM + p.bn * 128);
    const uint32_t stage_step = static_cast<uint32_t>(p.stage_bytes) >> 4;  // in the descriptors' address fields
    int stage = 0, accb = 0;
    uint32_t phase = 0, accphase = 0, set = 0, at = 0;
    const bool leader = elect_one();
    for (int i = 0; i < s.n; ++i) {
      const Item m = item(i);
      const int rows = __shfl_sync(0xffffffffu, m.ok ? m.rows : 0, 0);
      if (rows == 0) continue;
      const int n64 = (__shfl_sync(0xffffffffu, m.K, 0) + 63) / 64;
      const int bn = tile_n(rows);
      // a tile that starts inside a 128-row piece (64 rows high) finds its scales further on, 32 rows a column
      const uint32_t shift = kMode == kLinear ? __shfl_sync(0xffffffffu, m.row_n % kMxPieceRows, 0) / 32 : 0;
      const uint32_t idesc0 = idesc_mxfp(kMxBM, bn, 0), idesc1 = idesc_mxfp(kMxBM, bn, 2);
      mbar_wait_issue(&acc_empty[accb], accphase ^ 1, abort_flag, a.status);
      tc_fence_after();
      const uint32_t d = tmem + accb * kMats * p.bn;
      for (int k = 0; k < n64; k += 4) {
        mbar_wait_issue(&full[stage], phase, abort_flag, a.status);
        tc_fence_after();
        const uint64_t ad = ad0 + at, bd = bd0 + at, sd = sd0 + at;
        const uint32_t ta = sf_tmem + set * kScaleCols, tb = ta + 8 * kMats;
        const uint32_t tbm = tb + shift;
        if (leader) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (j == 1 && k + 2 >= n64) break;
#pragma unroll
            for (int mat = 0; mat < kMats; ++mat)
              tc_cp_scales(ta + 8 * mat + 4 * j, sd + mat * (kPairBytes >> 4) + j * (kMxPieceBytes >> 4));
#pragma unroll
            for (int g = 0; g < kRowTiles; ++g)
              tc_cp_scales(tb + 4 * kRowTiles * j + 4 * g, sd + (kMats + g) * (kPairBytes >> 4) + j * (kMxPieceBytes >> 4));
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk > 0 && k + kk >= n64) break;
#pragma unroll
            for (int mat = 0; mat < kMats; ++mat)
              tc_mma_mxfp(d + mat * p.bn, ad + mat * (kCodeBytesM >> 4) + 2 * kk, bd + 2 * kk, (kk & 1) ? idesc1 : idesc0,
                          ta + 8 * mat + 4 * (kk >> 1), tbm + 4 * kRowTiles * (kk >> 1), (k > 0 || kk > 0) ? 1u : 0u);
          }
          tc_commit(&empty[stage]);
          if (k + 4 >= n64) tc_commit(&acc_full[accb]);
        }
        set ^= 1;
        at += stage_step;
        if (++stage == p.stages) {
          stage = 0;
          at = 0;
          phase ^= 1;
        }
      }
      if (++accb == p.acc_bufs) {
        accb = 0;
        accphase ^= 1;
      }
    }
    // every MMA has completed before tensor memory is released
    __syncwarp();
    if (leader) {
      tc_commit(done);
      if (!mbar_wait(done, 0, nullptr)) record_status(a.status, MOE_ERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    pdl_wait();
    pdl_launch_dependents();
    const int lanegrp = warp & 3;
    const int colpart = (warp - kEpiWarp0) >> 2;
    int accb = 0;
    uint32_t accphase = 0;
    for (int i = 0; i < s.n; ++i) {
      const Item m = item(i);
      if (!m.ok) {
        if (lane == 0) record_status(a.status, MOE_ERR_INVALID_ARG);
        continue;
      }
      if (!mbar_wait_warp(&acc_full[accb], accphase, abort_flag)) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const uint32_t tbase = tmem + (static_cast<uint32_t>(lanegrp * 32) << 16) + accb * kMats * p.bn;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[accb]);
      };
      epilogue<V>(a, m, p, tbase, tile_n(m.rows), lanegrp, colpart, lane, release);
      if (++accb == p.acc_bufs) {
        accb = 0;
        accphase ^= 1;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ pairs of CTAs
// The dense product's tile of 128 x 256 is bound by shared memory (48 KB of MMA
// reads and 51 KB of loads a stage, 790 clocks at 128 bytes a clock, against 512
// of MMA).  A pair of CTAs (a cluster of two, on two SMs that share a tensor
// operation: cta_group::2) takes 256 weight rows x 256 tokens: each holds half of
// the weight rows and half of the tokens, and the MMA reads the other half from
// the peer, so a CTA's stage is 32 KB of reads and 35 KB of loads, and the 510
// clocks measured are the MMA's (8192 x 8192 -> 8192, fp32 Y: 180 -> 158 us; the
// first six stages of a tile still take about 900 each).  linear_tile says where it
// pays.
//
// Rank 0 issues copies and MMAs for both.  Every load of the pair completes on
// rank 0's barrier `full`, which rank 0 alone arms, for the bytes of both; a commit
// arrives at `empty` (and `acc_full`) of both ranks; both ranks' epilogue warps arrive
// at rank 0's `acc_empty`.
constexpr int kPairRows = 2 * kMxBM;
constexpr int kPairHalf = kMxBM * 128;  // a CTA's half of an operand's codes of a stage
constexpr int kPairStage = 2 * kPairHalf + 3 * kPairBytes;
constexpr int kPairStages = 6;
constexpr int kPairSmem = kPairStages * kPairStage + 1024 + 1024;
constexpr int kPairScaleCols = 8 + 16;  // of a stage: this CTA's weight rows, all tokens
using PairVariant = Variant<kLinear, 2, true>;
static_assert(kPairSmem <= kSmemLimit, "shared memory of a pair's CTA");

__global__ void __launch_bounds__(PairVariant::kThreads, 1)
    mx_pair_kernel(const __grid_constant__ MxPairMaps maps, const __grid_constant__ MxLinearArgs a) {
  using V = PairVariant;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(stages + kPairStages * kPairStage);
  uint64_t* empty = full + kPairStages;
  uint64_t* acc_full = empty + kPairStages;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* done = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&full[i], 2);  // rank 0's weights' and activations' expect_tx, for the bytes of both ranks
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * V::kEpiWarps);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc_pair(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_arrive_release();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int pieces = pieces_of(a.K);
  const int mts = (a.N + kPairRows - 1) / kPairRows;
  const int items = mts * ((a.M + kPairRows - 1) / kPairRows);
  const int step = static_cast<int>(gridDim.x >> 1), first = static_cast<int>(blockIdx.x >> 1);
  auto fail = [&]() {
    record_status(a.status, MOE_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == kWeightsWarp || warp == kActivationsWarp) {
    const bool weights = warp == kWeightsWarp;
    if (lane == 0) {
      if (!weights) pdl_wait();
      int stage = 0;
      uint32_t phase = 0, filled = 0;
      bool ok = true;
      for (int it = first; it < items && ok; it += step) {
        const int mt = it % mts, nt = it / mts;
        for (int k0 = 0; k0 < pieces; k0 += 2, ++filled) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          uint8_t* st = stages + stage * kPairStage;
          uint8_t* sf = st + 2 * kPairHalf;
          const uint32_t bar = mapa_shared(&full[stage], 0);
          if (weights) {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (kPairHalf + kPairBytes));
            tma_load_3d_pair(st, &maps.w, bar, k0 * 64, mt * kPairRows + rank * kMxBM, 0);
            tma_load_2d_pair(sf, &maps.sw, bar, 0, (2 * mt + rank) * pieces + k0);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (kPairHalf + 2 * kPairBytes));
            tma_load_2d_pair(st + kPairHalf, &maps.x, bar, k0 * 64, nt * kPairRows + rank * kMxBM);
            tma_load_2d_pair(sf + kPairBytes, &maps.sx, bar, 0, 2 * nt * pieces + k0);
            tma_load_2d_pair(sf + 2 * kPairBytes, &maps.sx, bar, 0, (2 * nt + 1) * pieces + k0);
          }
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // never leave while a load into this CTA's shared memory may be in flight: the commit of a stage's MMAs, which
      // waited for its loads, frees it
      const int n = filled < kPairStages ? static_cast<int>(filled) : kPairStages;
      for (int i = 0; i < n && ok; ++i) {
        stage = stage == 0 ? kPairStages - 1 : stage - 1;
        if (stage == kPairStages - 1) phase ^= 1;
        if (!mbar_wait(&empty[stage], phase, abort_flag)) {
          fail();
          ok = false;
        }
      }
      if (!ok) {  // what counts a copy's bytes is rank 0's: wait as long as no copy takes (a millisecond)
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000) {
        }
      }
      if (weights) pdl_wait();
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    pdl_wait();
    pdl_launch_dependents();
    if (rank == 0) {
      const uint32_t stage0 = smem_u32(stages);
      const uint64_t ad0 = smem_desc_sw128_kmajor(stage0), bd0 = smem_desc_sw128_kmajor(stage0 + kPairHalf);
      const uint64_t sd0 = smem_desc_scales(stage0 + 2 * kPairHalf);
      const uint32_t idesc0 = idesc_mxfp(kPairRows, 256, 0), idesc1 = idesc_mxfp(kPairRows, 256, 2);
      const int n64 = (a.K + 63) / 64;
      const bool leader = elect_one();
      int stage = 0;
      uint32_t phase = 0, accphase = 0, set = 0, at = 0;
      for (int it = first; it < items; it += step) {
        mbar_wait_issue(acc_empty, accphase ^ 1, abort_flag, a.status);
        tc_fence_after();
        for (int k = 0; k < n64; k += 4) {
          mbar_wait_issue(&full[stage], phase, abort_flag, a.status);
          tc_fence_after();
          const uint64_t ad = ad0 + at, bd = bd0 + at, sd = sd0 + at;
          const uint32_t ta = tmem + 256 + set * kPairScaleCols, tb = ta + 8;
          if (leader) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (j == 1 && k + 2 >= n64) break;
              const uint64_t sj = sd + j * (kMxPieceBytes >> 4);
              tc_cp_scales_pair(ta + 4 * j, sj);
              tc_cp_scales_pair(tb + 8 * j, sj + (kPairBytes >> 4));
              tc_cp_scales_pair(tb + 8 * j + 4, sj + 2 * (kPairBytes >> 4));
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk > 0 && k + kk >= n64) break;
              tc_mma_mxfp_pair(tmem, ad + 2 * kk, bd + 2 * kk, (kk & 1) ? idesc1 : idesc0, ta + 4 * (kk >> 1),
                               tb + 8 * (kk >> 1), (k > 0 || kk > 0) ? 1u : 0u);
            }
            tc_commit_pair(&empty[stage]);
            if (k + 4 >= n64) tc_commit_pair(acc_full);
          }
          set ^= 1;
          at += kPairStage >> 4;
          if (++stage == kPairStages) {
            stage = 0;
            at = 0;
            phase ^= 1;
          }
        }
        accphase ^= 1;
      }
      __syncwarp();
      if (leader) tc_commit_pair(done);
    }
    // every MMA has completed, and the last arrival at both ranks has come, before tensor memory is released
    __syncwarp();
    if (lane == 0 && !mbar_wait(done, 0, nullptr)) record_status(a.status, MOE_ERR_TIMEOUT);
    __syncwarp();
  } else {
    pdl_wait();
    pdl_launch_dependents();
    const int lanegrp = warp & 3, colpart = (warp - kEpiWarp0) >> 2;
    const uint32_t acc_empty0 = mapa_shared(acc_empty, 0);
    uint32_t accphase = 0;
    for (int it = first; it < items; it += step) {
      if (!mbar_wait_warp(acc_full, accphase, abort_flag)) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty0);
      };
      const int mt = it % mts, nt = it / mts;
      const int n = mt * kPairRows + rank * kMxBM + 32 * lanegrp + lane;
      epilogue_rows<V>(OutLinear{a.Y, a.y_fp32}, nt * kPairRows, n, a.N, min(kPairRows, a.M - nt * kPairRows),
                       tmem + (static_cast<uint32_t>(lanegrp * 32) << 16), kPairRows, colpart, release);
      accphase ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA leaves, or frees tensor memory, while the other may still reach its barriers or operands
  cluster_arrive_release();
  cluster_wait();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

template <typename V>
cudaError_t launch(int kind, const typename Args<V::kMode>::maps& maps, const typename Args<V::kMode>::type& a,
                   const Plan& p, int grid, cudaStream_t stream, bool pdl) {
  const int smem = p.stages * p.stage_bytes + kSmemFixed;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(mx_gemm_kernel<V>), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(V::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  timer_begin(kind, stream);
  e = cudaLaunchKernelEx(&cfg, mx_gemm_kernel<V>, maps, a, p);
  timer_end(kind, stream);
  return e;
}

}  // namespace

cudaError_t launch_mx_linear(const MxLinearArgs& a, const MxLinearMaps& maps, cudaStream_t stream, bool pdl) {
  const Plan p = make_plan(1, a.bn);
  const long long items = static_cast<long long>((a.N + kMxBM - 1) / kMxBM) * ((a.M + a.bn - 1) / a.bn);
  if (items > (1ll << 30)) return cudaErrorInvalidValue;
  const int grid = static_cast<int>(items < a.num_sms ? items : a.num_sms);
  return p.row_tiles == 1 ? launch<Variant<kLinear, 1, false>>(kKMxGemm, maps, a, p, grid, stream, pdl)
                          : launch<Variant<kLinear, 2, true>>(kKMxGemm, maps, a, p, grid, stream, pdl);
}

namespace {
// Pairs of mx_pair_kernel that the device runs at once (SMs that a cluster can
// take in twos), found once per device.
cudaError_t pairs_resident(int* most) {
  static std::mutex mu;
  static int known[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] == 0) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(PairVariant::kThreads);
    cfg.dynamicSmemBytes = kPairSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, mx_pair_kernel, &cfg);
    if (e != cudaSuccess) return e;
    known[dev] = n;
  }
  *most = known[dev];
  return cudaSuccess;
}
}  // namespace

cudaError_t launch_mx_pair(const MxLinearArgs& a, const MxPairMaps& maps, cudaStream_t stream, bool pdl) {
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(mx_pair_kernel), kPairSmem);
  if (e != cudaSuccess) return e;
  const long long items = static_cast<long long>((a.N + kPairRows - 1) / kPairRows) * ((a.M + kPairRows - 1) / kPairRows);
  if (items > (1ll << 30)) return cudaErrorInvalidValue;
  int most = 0;  // pairs that run at once
  e = pairs_resident(&most);
  if (e != cudaSuccess) return e;
  if (most < 1) return cudaErrorInvalidConfiguration;
  const int pairs = static_cast<int>(items < most ? items : most);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(PairVariant::kThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  timer_begin(kKMxGemm, stream);
  e = cudaLaunchKernelEx(&cfg, mx_pair_kernel, maps, a);
  timer_end(kKMxGemm, stream);
  return e;
}

cudaError_t launch_mx_experts(const MxExpertArgs& a, const MxExpertMaps& maps, cudaStream_t stream) {
  const int bn = a.I_shared > 0 && a.bn_s > a.bn_r ? a.bn_s : a.bn_r;
  const Plan p = make_plan(2, bn);
  cudaError_t e = p.acc_bufs == 1 ? launch<Variant<kGateUp, 1, true>>(kKMxGateUp, maps, a, p, a.num_sms, stream, true)
                                  : launch<Variant<kGateUp, 1, false>>(kKMxGateUp, maps, a, p, a.num_sms, stream, true);
  if (e != cudaSuccess) return e;
  e = launch<Variant<kDown, 1, false>>(kKMxDown, maps, a, make_plan(1, bn), a.num_sms, stream, true);
  if (e != cudaSuccess) return e;
  return launch_mx_combine(a.ypart, a.inv_perm, a.w, a.T, a.d, a.k, a.I_shared > 0, a.Y, a.status, a.num_sms, stream);
}

}  // namespace bm
