// MXFP4 products for few tokens (one decoded token to a few): what bounds
// them is the weights' stream and the number of dependent launches, so the
// activations are quantised inside the products.  A CTA takes one tile of 128
// weight rows over all of K; its loads are in flight while eight warps turn the
// tokens' activations into the N operand in shared memory (codes in the 128-byte
// swizzle the MMA reads, scales in pieces), which costs every CTA the same few
// kilobytes from L2 that a quantised copy would.
//
// Linear layer: one launch.  Expert layer: two after the routing,
//   gate/up  one matrix a CTA (gate or up), fp32 results to memory;
//   down     the prologue forms h = MX(silu(gate) up) of the tile's rows; the
//            last CTA to finish among those of the same 128 columns of Y (a
//            counter, no wait) adds the experts' rows up in slot order.
// K is not split: a token's sums are the bits that larger batches give.
//
// Weights are asked for before the wait for the previous kernel where their
// address is known by then: a linear layer's, the shared expert's, and in the
// down product the routed experts' too, since the gate/up kernel lets its
// successor start only after its own wait, when the routing has completed.
//
// Bound by latency.  One token, in a CUDA graph: 2048 -> 2048 3.2 us (2.2 MB,
// 0.33 us of memory); an expert layer of 8 + 1 experts, d = 2048, I = 512, with
// scored routing 15.2 us (15 MB, 2.2 us).
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
constexpr int kWorkWarp0 = 2;  // prologue and epilogue
constexpr int kWorkWarps = 8;
constexpr int kThreads = (kWorkWarp0 + kWorkWarps) * 32;
constexpr uint32_t kBarWork = 1;  // named barrier of the work warps
constexpr int kMaxRing = 8;       // stages of weights in flight (K = 256 each)
constexpr int kABytes = kMxBM * 128;
constexpr int kPairBytes = 2 * kMxPieceBytes;
constexpr int kSmemFixed = 1024 + 1024;  // barriers, alignment
constexpr int kSmemLimit = 227 * 1024;
// tensor memory: accumulator, two sets of a stage's scales of the weights and of the tokens
constexpr uint32_t kTmemCols = 64;
constexpr uint32_t kTmemSA = 32, kTmemSB = 48;
static_assert(kMxFewT <= static_cast<int>(kTmemSA), "one accumulator column a token");

struct Plan {
  int bn, stages, ring;  // stages: of K = 256, at most, in an item
  __host__ __device__ int b_bytes() const { return bn * 128; }
  // The tokens' scales: at most 32 rows, so of the four words of 16 bytes that
  // a copy to tensor memory takes per row, two are a stage's two pieces along K
  // instead of groups of 32 rows: one copy a stage, not two (a copy holds the
  // tensor pipeline up for about 65 clocks).
  __host__ __device__ int sb_bytes() const { return stages * kMxPieceBytes; }
  __host__ __device__ int smem() const {
    return ring * (kABytes + kPairBytes) + stages * b_bytes() + sb_bytes() + kSmemFixed;
  }
};

Plan make_plan(int bn, int K) {
  Plan p{bn, (K + kMxStageK - 1) / kMxStageK, 0};
  p.ring = p.stages < kMaxRing ? p.stages : kMaxRing;
  while (p.ring > 2 && p.smem() > kSmemLimit) --p.ring;
  return p;
}

struct Item {
  const CUtensorMap* map;
  const uint8_t* scales;  // the weight tile's first piece
  int e, row_m, mt, K;    // matrix and first row of the weights, tile of 128 rows, depth
  int rows, row0, N;      // tokens of the tile, the first one's row, weight rows of the matrix
  int mat;                // gate/up: 0 gate, 1 up
  bool shared, ok, some;  // some: false past the last item
};

struct LinearParams {
  MxFewLinearArgs a;
  CUtensorMap w;
};
struct ExpertParams {
  MxFewArgs a;
  MxExpertMaps maps;
};
template <int kMode>
struct Params {
  using type = ExpertParams;
};
template <>
struct Params<kLinear> {
  using type = LinearParams;
};

__device__ __forceinline__ int pieces_of(int K) { return (K + kMxPieceK - 1) / kMxPieceK; }

template <int kMode>
__device__ __forceinline__ Item get_item(const LinearParams& p) {
  Item m{};
  m.mt = blockIdx.x;
  m.map = &p.w;
  m.K = p.a.K;
  m.N = p.a.N;
  m.rows = p.a.T;
  m.row_m = m.mt * kMxBM;
  m.scales = p.a.sp + static_cast<size_t>(m.mt) * pieces_of(m.K) * kMxPieceBytes;
  m.ok = m.some = true;
  return m;
}

// Tiles of the experts' rows: the shared expert's first, then the block map's, of
// which a routing has at least one and as many as are launched at most; none of a
// malformed one.
__device__ __forceinline__ int routed_tiles(const MxFewArgs& a) {
  const int nb = *reinterpret_cast<const volatile int32_t*>(a.num_blocks);
  return nb < 1 || nb > a.tiles ? 0 : nb;
}

template <int kMode>
__device__ __forceinline__ Item get_item(const ExpertParams& p) {
  const MxFewArgs& a = p.a;
  constexpr bool kGU = kMode == kGateUp;
  constexpr int kMats = kGU ? 2 : 1;
  Item m{};
  int i = blockIdx.x;
  const int mt_s = a.I_shared > 0 ? ((kGU ? a.I_shared : a.d) + kMxBM - 1) / kMxBM : 0;
  const int mt_r = ((kGU ? a.I : a.d) + kMxBM - 1) / kMxBM;
  int e = 0;
  if (i < mt_s * kMats) {
    m.shared = m.ok = m.some = true;
    m.rows = a.T;
    m.row0 = 0;
    m.N = kGU ? a.I_shared : a.d;
    m.K = kGU ? a.d : a.I_shared;
  } else {
    i -= mt_s * kMats;
    const int tile = i / (mt_r * kMats);
    i -= tile * (mt_r * kMats);
    // the entry exists (the block map has room for all tiles launched), whether valid or not: one round trip for all of it
    const volatile int32_t* b = a.block_map + 3 * tile;
    e = b[0];
    m.row0 = b[1];
    m.rows = b[2];
    m.some = tile < routed_tiles(a);
    if (!m.some) return m;
    m.N = kGU ? a.I : a.d;
    m.K = kGU ? a.d : a.I;
    m.ok = e >= 0 && e < a.E && m.rows >= 1 && m.rows <= a.bn && m.row0 >= 0 && m.row0 <= a.T * a.k - m.rows;
  }
  m.mat = i % kMats;
  m.mt = i / kMats;
  if (!m.ok) return m;
  const MxExpertMaps& t = p.maps;
  if (kGU) {
    m.map = m.mat ? (m.shared ? &t.up_s : &t.up_r) : (m.shared ? &t.gate_s : &t.gate_r);
    m.scales = m.mat ? (m.shared ? a.sp_up_s : a.sp_up_r) : (m.shared ? a.sp_gate_s : a.sp_gate_r);
  } else {
    m.map = m.shared ? &t.down_s : &t.down_r;
    m.scales = m.shared ? a.sp_down_s : a.sp_down_r;
  }
  m.row_m = m.mt * kMxBM;
  m.e = e;
  m.scales += (static_cast<size_t>(e) * ((m.N + kMxPieceRows - 1) / kMxPieceRows) + m.mt) * pieces_of(m.K) * kMxPieceBytes;
  return m;
}

// One warp's 256 values of row r, stage s of the N operand.
__device__ __forceinline__ void put_row(uint8_t* b, uint8_t* sf, const Plan& p, int r, int s, uint32_t code, uint32_t scales,
                                        int lane) {
  *reinterpret_cast<uint32_t*>(b + s * p.b_bytes() + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + 4 * (lane & 3)) = code;
  if ((lane & 15) == 0)
    *reinterpret_cast<uint32_t*>(sf + s * kMxPieceBytes + r * 16 + 8 * (lane >> 4)) = scales;
}

// The N operand from activations: row r of the tile is row_of(r).
template <int kType, typename RowOf>
__device__ __forceinline__ void quantise_rows(uint8_t* b, uint8_t* sf, const Plan& p, const Item& m, int warp, int lane,
                                              RowOf row_of) {
  const int stages = (m.K + kMxStageK - 1) / kMxStageK;
  constexpr int kU = 4;  // units of a row and a stage in flight
  for (int u0 = warp; u0 < m.rows * stages; u0 += kU * kWorkWarps) {
    Load8<kType> x[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = u0 + i * kWorkWarps, c = (u % stages) * kMxStageK + 8 * lane;
      if (u < m.rows * stages && c < m.K) x[i].load(row_of(u / stages), c); else x[i].zero();
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = u0 + i * kWorkWarps;
      if (u >= m.rows * stages) break;
      uint32_t scales;
      const uint32_t code = quantize8(x[i], scales, lane);
      put_row(b, sf, p, u / stages, u % stages, code, scales, lane);
    }
  }
}

template <int kMode, int kType>
__device__ __forceinline__ void prologue(const LinearParams& p, uint8_t* b, uint8_t* sf, const Plan& plan, const Item& m,
                                         int warp, int lane) {
  const char* x = static_cast<const char*>(p.a.X);
  const size_t pitch = static_cast<size_t>(p.a.ldx) * (kType == kFp32 ? 4 : 2);
  quantise_rows<kType>(b, sf, plan, m, warp, lane, [&](int r) { return x + r * pitch; });
}

template <int kMode, int kType>
__device__ __forceinline__ void prologue(const ExpertParams& p, uint8_t* b, uint8_t* sf, const Plan& plan, const Item& m,
                                         int warp, int lane) {
  const MxFewArgs& a = p.a;
  if constexpr (kMode == kGateUp) {
    quantise_rows<kBf16>(b, sf, plan, m, warp, lane, [&](int r) {
      int t = m.shared ? r : __ldg(a.perm + m.row0 + r) / a.k;
      if (t < 0 || t >= a.T) {  // a malformed permutation
        record_status(a.status, MOE_ERR_INVALID_ARG);
        t = 0;
      }
      return a.X + static_cast<size_t>(t) * a.d;
    });
  } else {
    // h: a warp per row and block of 32 columns, one column a lane; blocks past
    // I in the last pair that an MMA reads are zeros
    const int pitch = max(a.I, a.I_shared);
    const int blocks = m.K / kMxBlock, blocks_up = (blocks + 1) & ~1;
    const float* gu = a.gu + static_cast<size_t>(m.shared ? a.T * a.k : m.row0) * 2 * pitch + lane;
    constexpr int kU = 4;
    for (int u0 = warp; u0 < m.rows * blocks_up; u0 += kU * kWorkWarps) {
      float g[kU], up[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int u = u0 + i * kWorkWarps, r = u / blocks_up, c = u % blocks_up;
        const bool in = u < m.rows * blocks_up && c < blocks;
        const float* at = gu + static_cast<size_t>(r) * 2 * pitch + c * kMxBlock;
        g[i] = in ? __ldcg(at) : 0.0f;
        up[i] = in ? __ldcg(at + pitch) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int u = u0 + i * kWorkWarps, r = u / blocks_up, c = u % blocks_up;
        if (u >= m.rows * blocks_up) break;
        const float v = mx_swiglu(g[i], up[i]);
        const uint32_t byte = c < blocks ? mx_warp_scale_byte(v) : 0u;
        uint32_t code = (f32x2_to_e2m1x2(v * mx_inverse_scale(byte), 0.0f) & 15u) << (4 * (lane & 7));
        code |= __shfl_xor_sync(0xffffffffu, code, 1);
        code |= __shfl_xor_sync(0xffffffffu, code, 2);
        code |= __shfl_xor_sync(0xffffffffu, code, 4);
        const int s = c >> 3, chunk = c & 7;  // 32 codes: one 16-byte chunk of the stage's line
        if ((lane & 7) == 0)
          *reinterpret_cast<uint32_t*>(b + s * plan.b_bytes() + r * 128 + ((chunk ^ (r & 7)) << 4) + 4 * (lane >> 3)) = code;
        if (lane == 0) sf[s * kMxPieceBytes + r * 16 + 8 * (chunk >> 2) + (chunk & 3)] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// Accumulator column c of this lane's weight row: 16 columns at c0 are in v.
template <int kMode>
__device__ __forceinline__ void store16(const LinearParams& p, const Item& m, int n, int c0, const uint32_t (&v)[16]) {
  const size_t at = static_cast<size_t>(c0) * p.a.N + n;
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    if (c0 + c >= m.rows) break;
    const float y = __uint_as_float(v[c]);
    if (p.a.y_fp32)
      static_cast<float*>(p.a.Y)[at + static_cast<size_t>(c) * p.a.N] = y;
    else
      static_cast<__nv_bfloat16*>(p.a.Y)[at + static_cast<size_t>(c) * p.a.N] = __float2bfloat16_rn(y);
  }
}
template <int kMode>
__device__ __forceinline__ void store16(const ExpertParams& p, const Item& m, int n, int c0, const uint32_t (&v)[16]) {
  const MxFewArgs& a = p.a;
  const int pitch = max(a.I, a.I_shared);
  const size_t row = static_cast<size_t>(m.shared ? a.T * a.k : 0) + m.row0 + c0;
  float* y = kMode == kGateUp ? a.gu + (row * 2 + m.mat) * pitch + n : a.ypart + row * a.d + n;
  const size_t step = kMode == kGateUp ? 2 * static_cast<size_t>(pitch) : a.d;
#pragma unroll
  for (int c = 0; c < 16; ++c)
    if (c0 + c < m.rows) y[c * step] = __uint_as_float(v[c]);
}

// Up to eight of a token's slots: their rows (-1: none) and weights.
struct Slots {
  int row[8];
  float w[8];
  // those of thread i's first token from slot j0 on
  __device__ __forceinline__ void load(const MxFewArgs& a, int i, int j0 = 0) {
    const int t = i / kMxBM, A = a.T * a.k;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = t < a.T && j0 + u < a.k;
      row[u] = in ? __ldg(a.inv_perm + t * a.k + j0 + u) : -1;
      w[u] = in ? __ldg(a.w + t * a.k + j0 + u) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (t >= a.T || j0 + u >= a.k) continue;
      if (row[u] < 0 || row[u] >= A) {  // a malformed permutation
        record_status(a.status, MOE_ERR_INVALID_ARG);
        row[u] = -1;
      }
    }
  }
};

// Y's columns 128 mt .. 128 mt + 127 of every token: the experts' rows in slot
// order, the shared expert's last (combine_kernel's arithmetic).  `slots`: the
// first token's first slots, loaded ahead.
__device__ __forceinline__ void combine_columns(const MxFewArgs& a, int mt, int i0, Slots& slots) {
  const size_t A = static_cast<size_t>(a.T) * a.k;
  for (int i = i0; i < a.T * kMxBM; i += kWorkWarps * 32) {
    const int t = i / kMxBM, n = mt * kMxBM + i % kMxBM;
    float acc = 0.0f;
    const bool in = n < a.d;
    const float sh = in && a.I_shared > 0 ? __ldcg(a.ypart + (A + t) * a.d + n) : 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
      if (i != i0 || j0 > 0) slots.load(a, i, j0);
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = in && slots.row[u] >= 0 ? __ldcg(a.ypart + static_cast<size_t>(slots.row[u]) * a.d + n) : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (slots.row[u] >= 0) acc = fmaf(slots.w[u], v[u], acc);
    }
    if (a.I_shared > 0) acc += sh;
    if (in) a.Y[static_cast<size_t>(t) * a.d + n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc));
  }
}

__device__ __forceinline__ int shared_items(const LinearParams&) { return 0; }
__device__ __forceinline__ int shared_items(const ExpertParams& p) {  // of the gate/up product
  return 2 * ((p.a.I_shared + kMxBM - 1) / kMxBM);
}

// Lane 0's value.
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return (static_cast<uint64_t>(__shfl_sync(0xffffffffu, static_cast<uint32_t>(v >> 32), 0)) << 32) |
         __shfl_sync(0xffffffffu, static_cast<uint32_t>(v), 0);
}

template <int kMode, int kType>
__global__ void __launch_bounds__(kThreads, 2)
    mx_few_kernel(const __grid_constant__ typename Params<kMode>::type p, const Plan plan) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* b = ring + plan.ring * kABytes;
  uint8_t* sa = b + plan.stages * plan.b_bytes();
  uint8_t* sb = sa + plan.ring * kPairBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sb + plan.sb_bytes());
  uint64_t* empty = full + kMaxRing;
  uint64_t* b_full = empty + kMaxRing;
  uint64_t* acc_full = b_full + 1;
  uint64_t* done = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* last_flag = const_cast<int*>(abort_flag) + 1;

  // the same in all lanes, so that the roles' branches are known to be uniform
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < plan.ring; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(b_full, kWorkWarps);
    mbar_init(acc_full, 1);
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
  uint32_t* status = p.a.status;
  auto fail = [&]() {
    record_status(status, MOE_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  // The routed experts of the gate/up product are known only after the wait.
  const bool early = kMode != kGateUp || static_cast<int>(blockIdx.x) < shared_items(p);
  if (!early || warp != kProducerWarp) {
    if (kMode != kDown) pdl_wait();
  }
  // (the down product's routing has completed: see above)
  const Item m = get_item<kMode>(p);
  if (kMode == kDown && warp != kProducerWarp) pdl_wait();
  if (warp != kProducerWarp) pdl_launch_dependents();

  if (warp == kProducerWarp) {
    // one thread issues; what it issues is the same in all lanes (uniform registers)
    const int n = __shfl_sync(0xffffffffu, m.some && m.ok ? pieces_of(m.K) : 0, 0);
    const int row_m = __shfl_sync(0xffffffffu, m.row_m, 0), e = __shfl_sync(0xffffffffu, m.e, 0);
    const CUtensorMap* map = reinterpret_cast<const CUtensorMap*>(uniform64(reinterpret_cast<uint64_t>(m.map)));
    const uint8_t* scales = reinterpret_cast<const uint8_t*>(uniform64(reinterpret_cast<uint64_t>(m.scales)));
    int stage = 0, filled = 0;
    uint32_t phase = 0;
    for (int k0 = 0; k0 < n; k0 += 2, ++filled) {
      if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
        fail();
        break;
      }
      if (elect_one()) {
        const uint32_t sbytes = min(2, n - k0) * kMxPieceBytes;
        mbar_arrive_expect_tx(&full[stage], kABytes + sbytes);
        tma_load_3d(ring + stage * kABytes, map, &full[stage], k0 * 64, row_m, e);
        bulk_g2s(sa + stage * kPairBytes, scales + static_cast<size_t>(k0) * kMxPieceBytes, sbytes, &full[stage]);
      }
      __syncwarp();
      if (++stage == plan.ring) {
        stage = 0;
        phase ^= 1;
      }
    }
    // never leave while a load into this CTA's shared memory may be in flight
    for (int i = 0; i < min(filled, plan.ring); ++i) {
      stage = stage == 0 ? plan.ring - 1 : stage - 1;
      if (stage == plan.ring - 1) phase ^= 1;
      if (!mbar_wait(&full[stage], phase, nullptr)) record_status(status, MOE_ERR_TIMEOUT);
    }
    if (early) pdl_wait();
  } else {
    if (warp == kMmaWarp) {
      // issued by one thread, computed by the warp from values that are the same
      // in all lanes (uniform registers)
      const int rows = __shfl_sync(0xffffffffu, m.some && m.ok ? m.rows : 0, 0);
      if (rows > 0) {
        const int n64 = (__shfl_sync(0xffffffffu, m.K, 0) + 63) / 64;
        const int bn = (rows + 15) & ~15;
        const uint32_t idesc0 = idesc_mxfp(kMxBM, bn, 0), idesc1 = idesc_mxfp(kMxBM, bn, 2);
        const uint64_t ad0 = smem_desc_sw128_kmajor(smem_u32(ring)), bd0 = smem_desc_sw128_kmajor(smem_u32(b));
        const uint64_t sa0 = smem_desc_scales(smem_u32(sa)), sb0 = smem_desc_scales(smem_u32(sb));
        int stage = 0;
        uint32_t phase = 0;
        const bool leader = elect_one();
        mbar_wait_issue(b_full, 0, abort_flag, status);
        // two stages a turn, one in each set of scales: a turn's own cost (waits,
        // branches, addresses: some 300 clocks) is more than the MMAs'
        for (int k = 0; k < n64; k += 8) {
          int st[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            st[h] = stage;
            if (h == 1 && k + 4 >= n64) break;
            mbar_wait_issue(&full[stage], phase, abort_flag, status);
            if (++stage == plan.ring) {
              stage = 0;
              phase ^= 1;
            }
          }
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int kh = k + 4 * h, s = kh >> 2;
              if (h == 1 && kh >= n64) break;
              const uint64_t ad = ad0 + st[h] * (kABytes >> 4), bd = bd0 + static_cast<uint32_t>(s * plan.b_bytes() >> 4);
              const uint64_t ad_s = sa0 + st[h] * (kPairBytes >> 4);
              const uint32_t ta = tmem + kTmemSA + 8 * h, tb = tmem + kTmemSB + 4 * h;
              tc_cp_scales(ta, ad_s);
              if (kh + 2 < n64) tc_cp_scales(ta + 4, ad_s + (kMxPieceBytes >> 4));
              tc_cp_scales(tb, sb0 + s * (kMxPieceBytes >> 4));
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if (kk > 0 && kh + kk >= n64) break;
                tc_mma_mxfp(tmem, ad + 2 * kk, bd + 2 * kk, (kk & 1) ? idesc1 : idesc0, ta + 4 * (kk >> 1),
                            tb + 2 * (kk >> 1), (kh > 0 || kk > 0) ? 1u : 0u);
              }
              tc_commit(&empty[st[h]]);
            }
            if (k + 8 >= n64) tc_commit(acc_full);
          }
        }
        // every MMA has completed before tensor memory is released
        __syncwarp();
        if (leader) {
          tc_commit(done);
          if (!mbar_wait(done, 0, nullptr)) record_status(status, MOE_ERR_TIMEOUT);
        }
        __syncwarp();
      }
    } else if (m.some) {
      const int ww = warp - kWorkWarp0;
      bool done = false;
      Slots slots;  // of the first token that this thread may have to sum up (down product)
      if (m.ok) {
        prologue<kMode, kType>(p, b, sb, plan, m, ww, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_full);
        if constexpr (kMode == kDown) slots.load(p.a, ww * 32 + lane);  // beside the MMAs
        done = mbar_wait(acc_full, 0, abort_flag);
        __syncwarp();
        if (done) {
          tc_fence_after();
          const int lanegrp = warp & 3, c0 = 16 * (ww >> 2);
          const int n = m.mt * kMxBM + 32 * lanegrp + lane;
          if (c0 < m.rows) {  // the same for the whole warp
            uint32_t v[16];
            tmem_ld16(tmem + (static_cast<uint32_t>(lanegrp * 32) << 16) + c0, v);
            tc_wait_ld();
            if (n < m.N) store16<kMode>(p, m, n, c0, v);
          }
          tc_fence_before();
        } else if (lane == 0) {
          fail();
        }
      } else if (lane == 0) {
        record_status(status, MOE_ERR_INVALID_ARG);
      }
      if constexpr (kMode == kDown) {
        // every product of these columns counts itself, a skipped one too; the
        // counter's release and acquire cover the other threads' stores and
        // loads through the barriers around it
        const uint32_t all = routed_tiles(p.a) + (p.a.I_shared > 0 ? 1 : 0);
        if (!m.ok) slots.load(p.a, ww * 32 + lane);
        bar_sync_or(kBarWork, kWorkWarps * 32, false);
        if (ww == 0 && lane == 0) {
          const bool last = atom_add_acq_rel_gpu(&p.a.arrived[m.mt], 1u) == all - 1;
          if (last) p.a.arrived[m.mt] = 0;  // ready for the next call
          *last_flag = last;
        }
        bar_sync_or(kBarWork, kWorkWarps * 32, false);
        if (*last_flag) combine_columns(p.a, m.mt, ww * 32 + lane, slots);
      }
    } else if constexpr (kMode != kLinear) {  // past the last item
      if (threadIdx.x == kWorkWarp0 * 32 && routed_tiles(p.a) == 0) record_status(status, MOE_ERR_INVALID_ARG);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int kMode, int kType>
cudaError_t launch(int kind, const typename Params<kMode>::type& p, const Plan& plan, int grid, cudaStream_t stream,
                   bool pdl) {
  const auto kernel = mx_few_kernel<kMode, kType>;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), plan.smem());
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = plan.smem();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  timer_begin(kind, stream);
  e = cudaLaunchKernelEx(&cfg, kernel, p, plan);
  timer_end(kind, stream);
  return e;
}

int round16(int x) { return (x + 15) & ~15; }
bool fits(int bn, int K) {
  const Plan p = make_plan(bn, K);
  return p.smem() <= kSmemLimit;
}

}  // namespace

bool mx_few_linear_fits(int T, int K) {
  return T <= kMxFewT && static_cast<long long>(T) * K <= kMxFewValues && fits(round16(T), K);
}

cudaError_t launch_mx_few_linear(const MxFewLinearArgs& a, int type, const CUtensorMap& w, cudaStream_t stream, bool pdl) {
  const LinearParams p{a, w};
  const Plan plan = make_plan(round16(a.T), a.K);
  const int grid = (a.N + kMxBM - 1) / kMxBM;
  if (type == kBf16) return launch<kLinear, kBf16>(kKMxGemm, p, plan, grid, stream, pdl);
  if (type == kFp16) return launch<kLinear, kFp16>(kKMxGemm, p, plan, grid, stream, pdl);
  return launch<kLinear, kFp32>(kKMxGemm, p, plan, grid, stream, pdl);
}

// Tiles of the routed experts at most (every tile holds an assignment).
int mx_few_tiles(int T, int k, int max_blocks) { return T * k < max_blocks ? T * k : max_blocks; }

namespace {
// The gate/up product's CTAs.
long long few_items(int I, int I_shared, int tiles) {
  const long long mt = (I + kMxBM - 1) / kMxBM, mt_s = (I_shared + kMxBM - 1) / kMxBM;
  return 2 * (tiles * mt + mt_s);
}
}  // namespace

bool mx_few_fits(int T, int d, int I, int I_shared, int k, int max_blocks) {
  const int bn = round16(T);
  return T <= kMxFewT && few_items(I, I_shared, mx_few_tiles(T, k, max_blocks)) <= kMxFewItems &&
         (d + kMxBM - 1) / kMxBM <= static_cast<int>(sizeof(WsHeader::mx_arrived) / 4) && fits(bn, d) &&
         fits(bn, I > I_shared ? I : I_shared);
}

cudaError_t launch_mx_few_experts(const MxFewArgs& a, const MxExpertMaps& maps, cudaStream_t stream, bool pdl) {
  const ExpertParams p{a, maps};
  const int mt_d = (a.d + kMxBM - 1) / kMxBM;
  const cudaError_t e = launch<kGateUp, kBf16>(kKMxGateUp, p, make_plan(a.bn, a.d),
                                               static_cast<int>(few_items(a.I, a.I_shared, a.tiles)), stream, pdl);
  if (e != cudaSuccess) return e;
  const int I = a.I > a.I_shared ? a.I : a.I_shared;
  return launch<kDown, kBf16>(kKMxDown, p, make_plan(a.bn, I), mt_d * (a.tiles + (a.I_shared > 0 ? 1 : 0)), stream, pdl);
}

}  // namespace bm
