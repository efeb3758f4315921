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
// The expert layer puts the weights on the M = 128 side and a tile's tokens
// (16..128) on the N side, so that an expert with few tokens streams its
// weights once and pads only tokens.  The dense product does the same for few
// tokens; for many, tokens are the M side, whose tensor-memory lanes then hold
// rows of Y, and 256 columns of Y a tile halve the reads of the tokens' codes.
//
// Roles (one persistent CTA per SM): warp 0 TMA producer, warp 1 MMA issuer
// (copies a stage's scales from shared to tensor memory, then multiplies: the
// tensor pipeline keeps the order), warps 2-9 epilogue, two per quarter of the
// tensor-memory lanes.  Every wait is bounded and records MOE_ERR_TIMEOUT.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "mx.cuh"
#include "ptx.cuh"

namespace bm {
namespace {

enum Mode { kLinear, kGateUp, kDown };

constexpr int kProducerWarp = 0;
constexpr int kMmaWarp = 1;
constexpr int kEpiWarp0 = 2;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 12;
constexpr int kCodeBytesM = kMxBM * 128;   // one matrix's codes of a stage
constexpr int kPairBytes = 2 * kMxPieceBytes;  // a stage's scales of 128 rows
constexpr int kSmemLimit = 227 * 1024;
constexpr int kSmemFixed = 1024 /* barriers */ + 1024 /* alignment */;

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
  // a second accumulator lets the epilogue of one item run beside the next one's products
  p.acc_bufs = 2 * mats * bn + 2 * scale_cols(mats, p.row_tiles) <= static_cast<int>(kTmemCols) ? 2 : 1;
  return p;
}

struct Item {
  const CUtensorMap *m0, *m1, *n;  // codes of the M side's matrices and of the N side
  const uint8_t *sm0, *sm1, *sn;   // their scales: the item's first pieces
  int row_m, row_n;                // first rows of the codes
  int mt, rows, K, box;            // M tile, valid N rows, depth, N rows that the TMA box brings
  int row0, slot;                  // experts: first row among the assignments (or tokens), tile slot
  bool shared, ok;
};

struct Sched {
  int nb, mt_r, mt_s, n_routed, n_total;
};

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
  s.mt_r = (a.rows_m + kMxBM - 1) / kMxBM;
  s.n_total = s.mt_r * ((a.rows_n + p.bn - 1) / p.bn);
  return s;
}

__device__ __forceinline__ Item get_item(const MxLinearArgs& a, const MxLinearMaps& maps, const Plan& p, const Sched& s,
                                         int it, bool) {
  Item m{};
  const int pieces = pieces_of(a.K);
  m.mt = it % s.mt_r;
  const int nt = it / s.mt_r;
  m.m0 = &maps.m;
  m.n = &maps.n;
  m.row_m = m.mt * kMxBM;
  m.row_n = nt * p.bn;
  m.rows = min(p.bn, a.rows_n - m.row_n);
  m.K = a.K;
  m.box = p.bn;
  m.sm0 = a.sp_m + static_cast<size_t>(m.mt) * pieces * kMxPieceBytes;
  m.sn = a.sp_n + static_cast<size_t>(m.row_n / kMxPieceRows) * pieces * kMxPieceBytes;
  m.ok = true;
  return m;
}

__device__ __forceinline__ Sched make_sched(const MxExpertArgs& a, const Plan&, bool gate_up) {
  Sched s{};
  s.nb = *a.num_blocks;
  if (s.nb < 0 || s.nb > a.max_blocks) {
    if (threadIdx.x == 0) record_status(a.status, MOE_ERR_INVALID_ARG);
    s.nb = 0;
  }
  s.mt_r = ((gate_up ? a.I : a.d) + kMxBM - 1) / kMxBM;
  s.mt_s = ((gate_up ? a.I_shared : a.d) + kMxBM - 1) / kMxBM;
  s.n_routed = s.nb * s.mt_r;
  s.n_total = s.n_routed + (a.I_shared > 0 ? (a.T + a.bn_s - 1) / a.bn_s * s.mt_s : 0);
  return s;
}

__device__ __forceinline__ Item get_item(const MxExpertArgs& a, const MxExpertMaps& maps, const Plan&, const Sched& s,
                                         int it, bool gate_up) {
  Item m{};
  int e, N;
  if (it < s.n_routed) {
    const int blk = it / s.mt_r;
    m.mt = it % s.mt_r;
    e = __ldg(a.block_map + 3 * blk);
    m.row0 = __ldg(a.block_map + 3 * blk + 1);
    m.rows = __ldg(a.block_map + 3 * blk + 2);
    m.slot = blk;
    m.box = a.bn_r;
    N = gate_up ? a.I : a.d;
    m.K = gate_up ? a.d : a.I;
    m.ok = e >= 0 && e < a.E && m.rows >= 1 && m.rows <= a.bn_r && m.row0 >= 0 && m.row0 + m.rows <= a.T * a.k;
    if (!m.ok) return m;
    m.m0 = gate_up ? &maps.gate_r : &maps.down_r;
    m.m1 = &maps.up_r;
    m.n = gate_up ? &maps.x_r : &maps.h_r;
    m.sm0 = gate_up ? a.sp_gate_r : a.sp_down_r;
    m.sm1 = a.sp_up_r;
    m.row_n = m.row0;
  } else {
    const int j = it - s.n_routed;
    m.shared = true;
    m.slot = j / s.mt_s;
    m.mt = j % s.mt_s;
    e = 0;
    m.row0 = m.slot * a.bn_s;
    m.rows = min(a.bn_s, a.T - m.row0);
    m.box = a.bn_s;
    N = gate_up ? a.I_shared : a.d;
    m.K = gate_up ? a.d : a.I_shared;
    m.ok = true;
    m.m0 = gate_up ? &maps.gate_s : &maps.down_s;
    m.m1 = &maps.up_s;
    m.n = gate_up ? &maps.x_s : &maps.h_s;
    m.sm0 = gate_up ? a.sp_gate_s : a.sp_down_s;
    m.sm1 = a.sp_up_s;
    m.row_n = gate_up ? a.T * a.k + m.row0 : m.row0;
  }
  const int pieces = pieces_of(m.K);
  const size_t tile = (static_cast<size_t>(e) * ((N + kMxPieceRows - 1) / kMxPieceRows) + m.mt) * pieces * kMxPieceBytes;
  m.sm0 += tile;
  m.sm1 += tile;
  m.row_m = e * N + m.mt * kMxBM;
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
// transposition into words of eight columns of one token.
__device__ __forceinline__ void epilogue(const MxExpertArgs& a, const Item& m, const Plan& p, uint32_t tbase, int bn,
                                         int lanegrp, int colpart, int lane, std::integral_constant<int, kGateUp>) {
  const int I = m.shared ? a.I_shared : a.I;
  const int n0 = m.mt * kMxBM + 32 * lanegrp;
  const int pieces = pieces_of(I);
  uint8_t* hq = (m.shared ? a.q_h_s : a.q_h_r) + static_cast<size_t>(m.row0) * (I / 2) + n0 / 2 + 4 * (lane >> 3);
  uint8_t* hs = (m.shared ? a.sp_h_s : a.sp_h_r) +
                (static_cast<size_t>(m.slot) * pieces + m.mt) * kMxPieceBytes + lanegrp;
  const bool valid = n0 < I;  // the same for the whole warp; past I the piece's scale bytes are zeros
  for (int c0 = 8 * colpart; c0 < bn; c0 += 8 * (kEpiWarps / 4)) {
    uint32_t g[8], u[8];
    tmem_ld8(tbase + c0, g);
    tmem_ld8(tbase + p.bn + c0, u);
    tc_wait_ld();
    uint32_t code = 0, bytes[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
      float h[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float v = mx_swiglu(__uint_as_float(g[c + i]), __uint_as_float(u[c + i]));
        const uint32_t byte = mx_warp_scale_byte(v);
        bytes[c >> 2] |= byte << (8 * ((c + i) & 3));
        h[i] = v * mx_inverse_scale(byte);
      }
      code |= f32x2_to_e2m1x2(h[0], h[1]) << (4 * c);
    }
    code = transpose_nibbles(code, lane);
    const int r = c0 + (lane & 7);
    if (r < m.rows) {
      if (valid) *reinterpret_cast<uint32_t*>(hq + static_cast<size_t>(r) * (I / 2)) = code;
      if (lane < 8) {
        const uint32_t word = (lane & 4) ? bytes[1] : bytes[0];
        hs[(r % 32) * 16 + (r / 32) * 4] = valid ? static_cast<uint8_t>(word >> (8 * (lane & 3))) : 0;
      }
    }
  }
}

// down: fp32 rows of the experts' outputs, routed ones in permuted order, then
// the shared expert's in token order; 32 lanes write one 128-byte line.
__device__ __forceinline__ void epilogue(const MxExpertArgs& a, const Item& m, const Plan& p, uint32_t tbase, int bn,
                                         int lanegrp, int colpart, int lane, std::integral_constant<int, kDown>) {
  const int n = m.mt * kMxBM + 32 * lanegrp + lane;
  float* y = a.ypart + (static_cast<size_t>(m.shared ? a.T * a.k : 0) + m.row0) * a.d + n;
  for (int c0 = 16 * colpart; c0 < bn; c0 += 16 * (kEpiWarps / 4)) {
    uint32_t v[16];
    tmem_ld16(tbase + c0, v);
    tc_wait_ld();
    if (n < a.d) {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (c0 + c < m.rows) y[static_cast<size_t>(c0 + c) * a.d] = __uint_as_float(v[c]);
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t*>(&b);
}

// dense: Y rounded once.  With tokens on the M side (stride_n 1) a lane owns 16
// consecutive elements of a row, stored as 16-byte words where the rows are
// aligned to them; otherwise the lanes' elements are the neighbours.
__device__ __forceinline__ void epilogue(const MxLinearArgs& a, const Item& m, const Plan& p, uint32_t tbase, int bn,
                                         int lanegrp, int colpart, int lane, std::integral_constant<int, kLinear>) {
  const int r = m.row_m + 32 * lanegrp + lane;
  const bool wide = a.stride_n == 1 && a.stride_m % (a.y_fp32 ? 4 : 8) == 0;
  for (int c0 = 16 * colpart; c0 < bn; c0 += 16 * (kEpiWarps / 4)) {
    uint32_t v[16];
    tmem_ld16(tbase + c0, v);
    tc_wait_ld();
    if (r >= a.rows_m) continue;
    const size_t at = static_cast<size_t>(r) * a.stride_m + static_cast<size_t>(m.row_n + c0) * a.stride_n;
    if (a.y_fp32) {
      float* y = static_cast<float*>(a.Y) + at;
      if (wide && c0 + 16 <= m.rows) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          reinterpret_cast<uint4*>(y)[c] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c0 + c < m.rows) y[c * a.stride_n] = __uint_as_float(v[c]);
      }
    } else {
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.Y) + at;
      if (wide && c0 + 16 <= m.rows) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          reinterpret_cast<uint4*>(y)[c] = make_uint4(bf16x2(v[8 * c], v[8 * c + 1]), bf16x2(v[8 * c + 2], v[8 * c + 3]),
                                                      bf16x2(v[8 * c + 4], v[8 * c + 5]), bf16x2(v[8 * c + 6], v[8 * c + 7]));
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c0 + c < m.rows) y[c * a.stride_n] = __float2bfloat16_rn(__uint_as_float(v[c]));
      }
    }
  }
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ typename Args<kMode>::maps maps,
                   const __grid_constant__ typename Args<kMode>::type a, const Plan p) {
  constexpr int kMats = kMode == kGateUp ? 2 : 1;
  constexpr bool kGU = kMode == kGateUp;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(stages + p.stages * p.stage_bytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps);
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

  pdl_wait();
  pdl_launch_dependents();

  const Sched s = make_sched(a, p, kGU);
  auto fail = [&]() {
    record_status(a.status, MOE_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == kProducerWarp) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, used_mask = 0, last_parity = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < s.n_total && ok; it += gridDim.x) {
        const Item m = get_item(a, maps, p, s, it, kGU);
        if (!m.ok) continue;
        const int pieces = pieces_of(m.K);
        // 128-row groups of the N side that exist (the dense product's last tile may have one less)
        const int groups = (m.rows + kMxPieceRows - 1) / kMxPieceRows;
        for (int k0 = 0; k0 < pieces; k0 += 2) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          uint8_t* st = stages + stage * p.stage_bytes;
          uint8_t* sf = st + kMats * kCodeBytesM + p.bn * 128;
          const uint32_t sbytes = min(2, pieces - k0) * kMxPieceBytes;
          uint64_t* bar = &full[stage];
          mbar_arrive_expect_tx(bar, kMats * kCodeBytesM + m.box * 128 + (kMats + groups) * sbytes);
          tma_load_2d(st, m.m0, bar, k0 * 64, m.row_m);
          if (kGU) tma_load_2d(st + kCodeBytesM, m.m1, bar, k0 * 64, m.row_m);
          tma_load_2d(st + kMats * kCodeBytesM, m.n, bar, k0 * 64, m.row_n);
          const size_t at = static_cast<size_t>(k0) * kMxPieceBytes;
          bulk_g2s(sf, m.sm0 + at, sbytes, bar);
          if (kGU) bulk_g2s(sf + kPairBytes, m.sm1 + at, sbytes, bar);
          for (int g = 0; g < groups; ++g)
            bulk_g2s(sf + (kMats + g) * kPairBytes, m.sn + static_cast<size_t>(g) * pieces * kMxPieceBytes + at, sbytes,
                     bar);
          used_mask |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // never leave while a load into this CTA's shared memory may be in flight
      for (int i = 0; i < p.stages; ++i)
        if ((used_mask >> i) & 1u) {
          if (!mbar_wait(&full[i], (last_parity >> i) & 1u, nullptr)) record_status(a.status, MOE_ERR_TIMEOUT);
        }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    const uint32_t stage0 = smem_u32(stages);
    // tensor memory: the accumulators, then two sets of a stage's scales
    const uint32_t sf_tmem = tmem + p.acc_bufs * kMats * p.bn;
    int stage = 0, accb = 0;
    uint32_t phase = 0, accphase = 0, set = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < s.n_total && ok; it += gridDim.x) {
      const Item m = get_item(a, maps, p, s, it, kGU);
      if (!m.ok) continue;
      const int bn = tile_n(m.rows);
      if (!mbar_wait(&acc_empty[accb], accphase ^ 1, abort_flag)) {
        fail();
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + accb * kMats * p.bn;
      const int n64 = (m.K + 63) / 64;
      const int pieces = pieces_of(m.K);
      for (int k0 = 0; k0 < pieces; k0 += 2) {
        if (!mbar_wait(&full[stage], phase, abort_flag)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t st = stage0 + stage * p.stage_bytes;
          const uint32_t sf = st + kMats * kCodeBytesM + p.bn * 128;
          const uint32_t ts = sf_tmem + set * scale_cols(kMats, p.row_tiles);
          const int np = min(2, pieces - k0);
          for (int j = 0; j < np; ++j) {
            const uint64_t sd = smem_desc_scales(sf + j * kMxPieceBytes);
#pragma unroll
            for (int i = 0; i < kMats; ++i)
              tc_cp_scales(ts + 8 * i + 4 * j, sd + static_cast<uint64_t>(i * (kPairBytes >> 4)));
            for (int g = 0; g < p.row_tiles; ++g)
              tc_cp_scales(ts + 8 * kMats + 4 * p.row_tiles * j + 4 * g,
                           sd + static_cast<uint64_t>((kMats + g) * (kPairBytes >> 4)));
          }
          const uint64_t ad = smem_desc_sw128_kmajor(st);
          const uint64_t bd = smem_desc_sw128_kmajor(st + kMats * kCodeBytesM);
          const int nk = min(4, n64 - 2 * k0);
          for (int kk = 0; kk < nk; ++kk) {
            const uint32_t idesc = idesc_mxfp(kMxBM, bn, 2 * (kk & 1));
            const uint32_t tb = ts + 8 * kMats + 4 * p.row_tiles * (kk >> 1);
            const uint32_t acc = (k0 | kk) ? 1u : 0u;
#pragma unroll
            for (int i = 0; i < kMats; ++i)
              tc_mma_mxfp(d + i * p.bn, ad + static_cast<uint64_t>(i * (kCodeBytesM >> 4) + 2 * kk), bd + 2 * kk, idesc,
                          ts + 8 * i + 4 * (kk >> 1), tb, acc);
          }
          tc_commit(&empty[stage]);
        }
        __syncwarp();
        set ^= 1;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(&acc_full[accb]);
      __syncwarp();
      if (++accb == p.acc_bufs) {
        accb = 0;
        accphase ^= 1;
      }
    }
    // every MMA has completed before tensor memory is released
    if (elect_one()) {
      tc_commit(done);
      if (!mbar_wait(done, 0, nullptr)) record_status(a.status, MOE_ERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    const int lanegrp = warp & 3;
    const int colpart = (warp - kEpiWarp0) >> 2;
    int accb = 0;
    uint32_t accphase = 0;
    for (int it = blockIdx.x; it < s.n_total; it += gridDim.x) {
      const Item m = get_item(a, maps, p, s, it, kGU);
      if (!m.ok) {
        if (lane == 0) record_status(a.status, MOE_ERR_INVALID_ARG);
        continue;
      }
      if (!mbar_wait(&acc_full[accb], accphase, abort_flag)) {
        if (lane == 0) fail();
        break;
      }
      __syncwarp();
      tc_fence_after();
      const uint32_t tbase = tmem + (static_cast<uint32_t>(lanegrp * 32) << 16) + accb * kMats * p.bn;
      epilogue(a, m, p, tbase, tile_n(m.rows), lanegrp, colpart, lane, std::integral_constant<int, kMode>{});
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[accb]);
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

template <int kMode>
cudaError_t launch(int kind, const typename Args<kMode>::maps& maps, const typename Args<kMode>::type& a, const Plan& p,
                   int grid, cudaStream_t stream, bool pdl) {
  const int smem = p.stages * p.stage_bytes + kSmemFixed;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(mx_gemm_kernel<kMode>), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  timer_begin(kind, stream);
  e = cudaLaunchKernelEx(&cfg, mx_gemm_kernel<kMode>, maps, a, p);
  timer_end(kind, stream);
  return e;
}

}  // namespace

cudaError_t launch_mx_linear(const MxLinearArgs& a, const MxLinearMaps& maps, cudaStream_t stream, bool pdl) {
  const Plan p = make_plan(1, a.bn);
  const long long items = static_cast<long long>((a.rows_m + kMxBM - 1) / kMxBM) * ((a.rows_n + a.bn - 1) / a.bn);
  if (items > (1ll << 30)) return cudaErrorInvalidValue;
  return launch<kLinear>(kKMxGemm, maps, a, p, static_cast<int>(items < a.num_sms ? items : a.num_sms), stream, pdl);
}

cudaError_t launch_mx_experts(const MxExpertArgs& a, const MxExpertMaps& maps, cudaStream_t stream) {
  const int bn = a.I_shared > 0 && a.bn_s > a.bn_r ? a.bn_s : a.bn_r;
  const cudaError_t e = launch<kGateUp>(kKMxGateUp, maps, a, make_plan(2, bn), a.num_sms, stream, true);
  if (e != cudaSuccess) return e;
  return launch<kDown>(kKMxDown, maps, a, make_plan(1, bn), a.num_sms, stream, true);
}

}  // namespace bm
