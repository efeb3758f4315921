// Block-scaled 8-bit products on the tensor cores: dense (Y = A W^T) and the
// expert layer's grouped gate/up and down products.
//
// D[n][m] = sum_kb sw[kb] sa[m][kb] sum_{k in kb} w[n][k] a[m][k]: a scale holds for
// 128 columns, so tcgen05.mma (kind::f8f6f4, E4M3, fp32) adds up one block of 128
// columns into an accumulator of its own, and warps with the running sums in
// registers read it, multiply it by the two scales' product and add it (packed fp32
// operations) while the next blocks multiply into other accumulators.  The scales
// are any fp32 numbers; nothing of them reaches the tensor cores.
//
// The weights are the M = 128 side (a tile's rows share their scale) and the tokens
// the N side: an expert with few tokens streams its weights once and pads only
// tokens, and the epilogues have neighbouring columns of a row in neighbouring
// lanes.  A stage of the pipeline is K = 128: one 128-byte line of codes a row (the
// widest swizzle atom) and the tokens' scales, four MMAs of K = 32.
//
// Roles (one persistent CTA per SM): warps 0, 1 and 3 the loads of the weights, of
// the activations and of their scales, warp 2 the MMAs' issue, warps 4 to 11 the sums: two per
// quarter of the tensor-memory lanes, the tokens' groups in turn.  Every wait is
// bounded and records MOE_ERR_TIMEOUT.
//
// A block after another takes 0.23 to 0.33 us, for the most part the way from MMA
// to sums.  So a dense product of few tiles divides each tile's blocks among the
// CTAs of a cluster, which leave their sums in shared memory and add them up, every
// CTA some tokens', in the CTAs' order.
#include <cuda_runtime.h>

#include "blk_items.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace bm {
namespace {

constexpr int kWeightsWarp = 0;
constexpr int kActivationsWarp = 1;
constexpr int kMmaWarp = 2;
constexpr int kScalesWarp = 3;
constexpr int kSumWarp0 = 4;
constexpr int kSumWarps = 8;
constexpr int kParts = kSumWarps / 4;  // shares of the tokens
constexpr int kThreads = (kSumWarp0 + kSumWarps) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 12;
constexpr int kMaxAccs = 8;
constexpr int kMatBytes = kBlk * 128;  // one matrix's codes of a stage
constexpr int kSmemLimit = 227 * 1024;
constexpr int kEntries = 256;          // items of a CTA, from its first, whose Entry is in shared memory
constexpr int kSmemFixed = 1024 /* barriers */ + 16 * kEntries + 2 * 4 * 4 * kMaxTile /* maxima */ + 1024 /* alignment */;

// A launch's variant; kBN: tokens of a tile at most, which the sums' registers are for.
template <int kMode_, int kBN_>
struct Variant {
  static constexpr int kMode = kMode_, kBN = kBN_;
  static constexpr int kMats = kMode == kGateUp ? 2 : 1;
  static constexpr int kGroup = kBN == 16 ? 8 : 16;                // tokens that a warp takes at a time
  static constexpr int kGroups = kBN / (kGroup * kParts);          // of a warp
};

// How a launch divides shared and tensor memory; bn: the tiles' height in columns.
struct Plan {
  int bn, stages, stage_bytes, accs, scale_slots;
};
Plan make_plan(int mats, int bn) {
  Plan p;
  p.bn = bn;
  const int most = static_cast<int>(kTmemCols) / (mats * bn);
  p.stage_bytes = mats * kMatBytes + bn * 128;
  for (p.stages = kMaxStages;; --p.stages) {
    p.accs = most < p.stages ? most : p.stages;  // no more than stages: see where the sums wait
    if (p.accs > kMaxAccs) p.accs = kMaxAccs;
    // the scales of a block are read until its accumulator is free again, which may be `accs` stages after the
    // stage's codes: a ring of their own
    p.scale_slots = p.stages + p.accs;
    if (p.stages * p.stage_bytes + p.scale_slots * bn * 4 + kSmemFixed <= kSmemLimit) return p;
  }
}
int plan_smem(const Plan& p) { return p.stages * p.stage_bytes + p.scale_slots * p.bn * 4 + kSmemFixed; }

__device__ __forceinline__ int tile_n(int rows) { return (rows + 15) & ~15; }

// A warp's sums: two tokens to a register pair, for each of its groups.
template <typename V>
struct Sums {
  uint64_t v[V::kMats][V::kGroups][V::kGroup / 2];
  __device__ __forceinline__ float get(int mat, int g, int c) const {
    float lo, hi;
    unpack2(v[mat][g][c >> 1], lo, hi);
    return c & 1 ? hi : lo;
  }
};

// Four bytes of four lanes (4i .. 4i+3), byte j of lane i to byte i of lane j.
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t v, int lane) {
  uint32_t t = __shfl_xor_sync(0xffffffffu, v, 2);
  v = (lane & 2) ? __byte_perm(v, t, 0x3276) : __byte_perm(v, t, 0x5410);
  t = __shfl_xor_sync(0xffffffffu, v, 1);
  return (lane & 1) ? __byte_perm(v, t, 0x3715) : __byte_perm(v, t, 0x6240);
}

// A lane's column of a tile's rows: the first one's place, the others `pitch` apart.
template <typename V, typename T, typename Round>
__device__ __forceinline__ void store_columns(T* y, long long pitch, int rows, const Sums<V>& acc, int part, Round round) {
#pragma unroll
  for (int g = 0; g < V::kGroups; ++g) {
    const int c0 = V::kGroup * (g * kParts + part);
    if (c0 >= rows) break;
    T* at = y + c0 * pitch;
    if (c0 + V::kGroup <= rows) {
#pragma unroll
      for (int c = 0; c < V::kGroup; ++c, at += pitch) *at = round(acc.get(0, g, c));
    } else {
#pragma unroll
      for (int c = 0; c < V::kGroup; ++c, at += pitch)
        if (c0 + c < rows) *at = round(acc.get(0, g, c));
    }
  }
}

// gate/up: h = silu(gate) up, quantised here.  A tile's 128 columns are one block
// of h: a token's largest magnitude is a reduction over the lanes and the share's
// four warps.  meet(): waits for those (false: given up).
template <typename V, typename Meet>
__device__ __forceinline__ bool epilogue(const BlkExpertArgs& a, const Item& m, Sums<V>& acc, int quarter, int part, int lane,
                                         uint32_t (*maxima)[kMaxTile], Meet meet) {
  if constexpr (V::kMode == kGateUp) {
    const int I = m.shared ? a.I_shared : a.I;
    const int n0 = m.mt * kBlk + 32 * quarter;
#pragma unroll
    for (int g = 0; g < V::kGroups; ++g) {
      const int c0 = V::kGroup * (g * kParts + part);
      if (c0 >= m.rows) break;
      uint32_t most = 0;
#pragma unroll
      for (int c = 0; c < V::kGroup; c += 2) {  // h takes gate's place
        const uint32_t h0 = __float_as_uint(blk_swiglu(acc.get(0, g, c), acc.get(V::kMats - 1, g, c)));
        const uint32_t h1 = __float_as_uint(blk_swiglu(acc.get(0, g, c + 1), acc.get(V::kMats - 1, g, c + 1)));
        acc.v[0][g][c >> 1] = pack2(h0, h1);
        const uint32_t x0 = __reduce_max_sync(0xffffffffu, h0 & 0x7FFFFFFFu), x1 = __reduce_max_sync(0xffffffffu, h1 & 0x7FFFFFFFu);
        if (lane == c) most = x0;
        if (lane == c + 1) most = x1;
      }
      if (lane < V::kGroup) maxima[quarter][c0 + lane] = most;
    }
    if (!meet()) return false;
    uint8_t* hq = (m.shared ? a.h_s : a.h_r) + static_cast<size_t>(m.row0) * I + n0 + 4 * (lane >> 2);
    float* hs = (m.shared ? a.sh_s : a.sh_r) + (static_cast<size_t>(m.slot) * blk_count(I) + m.mt) * a.pitch;
    const bool valid = n0 + 4 * (lane >> 2) < I;
#pragma unroll
    for (int g = 0; g < V::kGroups; ++g) {
      const int c0 = V::kGroup * (g * kParts + part);
      if (c0 >= m.rows) break;
      float inv = 0.0f;  // of token c0 + lane
      if (lane < V::kGroup) {
        const int c = c0 + lane;
        const float s = blk_scale(max(max(maxima[0][c], maxima[1][c]), max(maxima[2][c], maxima[3][c])));
        inv = blk_inverse(s);
        if (quarter == 0 && c < m.rows) hs[c] = s;
      }
#pragma unroll
      for (int c = 0; c < V::kGroup; c += 4) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = acc.get(0, g, c + i) * __shfl_sync(0xffffffffu, inv, c + i);
        const uint32_t code = transpose_bytes(f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]), lane);
        const int r = c0 + c + (lane & 3);
        if (r < m.rows && valid) *reinterpret_cast<uint32_t*>(hq + static_cast<size_t>(r) * I) = code;
      }
    }
  } else {
    // fp32 rows of the experts' outputs, routed ones in permuted order, then the shared expert's in token order
    const int n = m.mt * kBlk + 32 * quarter + lane;
    if (n >= a.d) return true;
    store_columns<V>(a.ypart + (static_cast<size_t>(m.shared ? a.T * a.k : 0) + m.row0) * a.d + n, a.d, m.rows, acc, part,
                     [](float x) { return x; });
  }
  return true;
}
template <typename V, typename Meet>
__device__ __forceinline__ bool epilogue(const BlkLinearArgs& a, const Item& m, Sums<V>& acc, int quarter, int part, int lane,
                                         uint32_t (*)[kMaxTile], Meet) {
  const int n = m.row_m + 32 * quarter + lane;
  if (n >= a.N) return true;
  const size_t at = static_cast<size_t>(m.row_n) * a.N + n;
  if (a.y_type == kFp32)
    store_columns<V>(static_cast<float*>(a.y) + at, a.N, m.rows, acc, part, [](float x) { return x; });
  else if (a.y_type == kFp16)
    store_columns<V>(static_cast<__half*>(a.y) + at, a.N, m.rows, acc, part, [](float x) { return __float2half_rn(x); });
  else
    store_columns<V>(static_cast<__nv_bfloat16*>(a.y) + at, a.N, m.rows, acc, part, [](float x) { return __float2bfloat16_rn(x); });
  return true;
}

// A tile whose blocks a cluster's CTAs share: a warp's sums to shared memory, [token][kBlk rows], and the CTAs' sums of
// every a.split-th token, added up in the CTAs' order, to Y.
template <typename V>
__device__ __forceinline__ void put_sums(float* to, int rows, const Sums<V>& acc, int quarter, int part, int lane) {
#pragma unroll
  for (int g = 0; g < V::kGroups; ++g) {
    const int c0 = V::kGroup * (g * kParts + part);
#pragma unroll
    for (int c = 0; c < V::kGroup; ++c)
      if (c0 + c < rows) to[(c0 + c) * kBlk + 32 * quarter + lane] = acc.get(0, g, c);
  }
}
__device__ __forceinline__ void join_sums(const BlkLinearArgs& a, const Item& m, const float* sums, int warp, int lane) {
  const int rank = static_cast<int>(cluster_ctarank()), n = m.row_m + 4 * lane;
  for (int t = rank + a.split * warp; t < m.rows; t += a.split * kSumWarps) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < a.split; ++p) {
      const float4 f = ld_shared_cluster_f4(mapa_shared(sums + t * kBlk + 4 * lane, p));
      v[0] += f.x;
      v[1] += f.y;
      v[2] += f.z;
      v[3] += f.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < a.N) store1(a.y_type, a.y, static_cast<size_t>(m.row_n + t) * a.N + n + j, v[j]);
  }
}

__device__ __forceinline__ void prefetch_maps(const BlkLinearMaps& m) {
  tma_prefetch_desc(&m.w);
  tma_prefetch_desc(&m.x);
}
__device__ __forceinline__ void prefetch_maps(const BlkExpertMaps&) {}

template <typename V>
__global__ void __launch_bounds__(kThreads, 1)
    blk_gemm_kernel(const __grid_constant__ typename Args<V::kMode>::maps maps,
                    const __grid_constant__ typename Args<V::kMode>::type a, const Plan p) {
  constexpr int kMats = V::kMats;
  constexpr bool kGU = V::kMode == kGateUp;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(stages + p.stages * p.stage_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + p.scale_slots * p.bn);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_empty = empty + kMaxStages;
  uint64_t* part_met = acc_empty + kMaxAccs;  // a share's four warps have written their maxima
  uint64_t* finished = part_met + kParts;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(finished + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Entry* entries = reinterpret_cast<Entry*>(reinterpret_cast<uint8_t*>(full) + 1024);
  uint32_t(*maxima)[kMaxTile] = reinterpret_cast<uint32_t(*)[kMaxTile]>(entries + kEntries);  // [2 x 4][tokens]

  // the same in all lanes, so that the roles' branches are known to be uniform
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  // The routing has completed by now (the kernel before this one lets this one
  // start only after its own wait), so only the activations are waited for.
  const Sched s = make_sched<kBlk>(a, p.bn, kGU);
  for (int i = threadIdx.x; i < min(s.n, kEntries); i += kThreads) entries[i] = make_entry(a, s, s.first + i * s.step);
  auto item = [&](int i) {
    return get_item<kBlk>(a, maps, p.bn, i < kEntries ? entries[i] : make_entry(a, s, s.first + i * s.step), kGU);
  };
  if (threadIdx.x == 32) prefetch_maps(maps);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 3);  // the weights', the activations' and the scales' expect_tx; their bytes complete the phase
      mbar_init(&empty[i], 2);  // the MMAs' commit, and their issuer, who has seen the stage's scales land
    }
    for (int i = 0; i < p.accs; ++i) mbar_init(&acc_empty[i], kSumWarps);
    for (int i = 0; i < kParts; ++i) mbar_init(&part_met[i], 4);
    mbar_init(finished, 1);
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

  if (warp < kSumWarp0) {
    if (warp != kMmaWarp) {
      // one thread for the weights, which starts before the wait, one for the activations' codes and one for their scales
      if (lane == 0) {
        const bool weights = warp == kWeightsWarp;
        if (!weights) pdl_wait();
        int stage = 0, slot = 0, filled = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = 0; i < s.n && ok; ++i) {
          const Item m = item(i);
          if (!m.ok) continue;
          const int blocks = blk_count(m.K);
          const float* sn = m.sn;
          for (int kb = 0; kb < blocks; ++kb, ++filled) {
            if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
              fail();
              ok = false;
              break;
            }
            uint8_t* st = stages + stage * p.stage_bytes;
            uint64_t* bar = &full[stage];
            if (weights) {
              mbar_arrive_expect_tx(bar, kMats * kMatBytes);
              tma_load_3d(st, m.m0, bar, (m.kb0 + kb) * kBlk, m.row_m, m.e);
              if (kGU) tma_load_3d(st + kMatBytes, m.m1, bar, (m.kb0 + kb) * kBlk, m.row_m, m.e);
            } else if (warp == kActivationsWarp) {
              mbar_arrive_expect_tx(bar, m.box * 128);
              tma_load_2d(st + kMats * kMatBytes, m.n, bar, (m.kb0 + kb) * kBlk, m.row_n);
            } else {
              mbar_arrive_expect_tx(bar, m.sn_bytes);
              bulk_g2s(scales + slot * p.bn, sn, m.sn_bytes, bar);
              sn += m.sn_step;
              if (++slot == p.scale_slots) slot = 0;
            }
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
    } else {
      pdl_wait();
      pdl_launch_dependents();
      // One thread issues everything; what it issues is computed by the whole warp
      // from values that are the same in all lanes, which lets the compiler keep
      // descriptors and addresses in uniform registers.
      const uint32_t stage0 = smem_u32(stages);
      const uint64_t ad0 = smem_desc_sw128_kmajor(stage0);
      const uint64_t bd0 = smem_desc_sw128_kmajor(stage0 + kMats * kMatBytes);
      const uint32_t stage_step = static_cast<uint32_t>(p.stage_bytes) >> 4;  // in the descriptors' address fields
      int stage = 0, accb = 0;
      uint32_t phase = 0, accphase = 0, at = 0;
      const bool leader = elect_one();
      for (int i = 0; i < s.n; ++i) {
        const Item m = item(i);
        const int rows = __shfl_sync(0xffffffffu, m.ok ? m.rows : 0, 0);
        if (rows == 0) continue;
        const int n32 = (__shfl_sync(0xffffffffu, m.K, 0) + 31) / 32;
        const uint32_t idesc = idesc_e4m3_f32(kBlk, tile_n(rows));
        for (int k = 0; k < n32; k += 4) {
          mbar_wait_issue(&acc_empty[accb], accphase ^ 1, abort_flag, a.status);
          mbar_wait_issue(&full[stage], phase, abort_flag, a.status);
          tc_fence_after();
          const uint64_t ad = ad0 + at, bd = bd0 + at;
          const uint32_t d = tmem + accb * kMats * p.bn;
          if (leader) {
#pragma unroll
            for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if (kk > 0 && k + kk >= n32) break;
                tc_mma_f8(d + mat * p.bn, ad + mat * (kMatBytes >> 4) + 2 * kk, bd + 2 * kk, idesc, kk > 0 ? 1u : 0u);
              }
            tc_commit(&empty[stage]);
            mbar_arrive(&empty[stage]);
          }
          at += stage_step;
          if (++stage == p.stages) {
            stage = 0;
            at = 0;
            phase ^= 1;
          }
          if (++accb == p.accs) {
            accb = 0;
            accphase ^= 1;
          }
        }
      }
      // every MMA has completed before tensor memory is released
      __syncwarp();
      if (leader) {
        tc_commit(finished);
        if (!mbar_wait(finished, 0, nullptr)) record_status(a.status, MOE_ERR_TIMEOUT);
      }
      __syncwarp();
    }
  } else {
    pdl_wait();
    pdl_launch_dependents();
    const int quarter = warp & 3, part = (warp - kSumWarp0) >> 2;
    int accb = 0, slot = 0, stage = 0;
    uint32_t phase = 0, parity = 0;
    bool ok = true;
    for (int i = 0; i < s.n && ok; ++i) {
      const Item m = item(i);
      if (!m.ok) {
        if (lane == 0) record_status(a.status, MOE_ERR_INVALID_ARG);
        continue;
      }
      const int blocks = blk_count(m.K);
      Sums<V> acc;
#pragma unroll
      for (int mat = 0; mat < kMats; ++mat)
#pragma unroll
        for (int g = 0; g < V::kGroups; ++g)
#pragma unroll
          for (int c = 0; c < V::kGroup / 2; ++c) acc.v[mat][g][c] = 0;
      float sw0 = 0.0f, sw1 = 0.0f;  // the weights' scales of 32 blocks, one a lane
      for (int kb = 0; kb < blocks; ++kb) {
        if ((kb & 31) == 0) {
          sw0 = kb + lane < blocks ? __ldg(m.s0 + kb + lane) : 0.0f;
          if (kGU) sw1 = kb + lane < blocks ? __ldg(m.s1 + kb + lane) : 0.0f;
        }
        // the stage's barrier tells that its MMAs have completed, to the loads that take its place and to the sums: it
        // cannot be a phase further before these have released the accumulator (there are no more of them than stages)
        // (where the wait gives up the warp goes on with what is there: its lanes stay together, and it meets the flag again)
        mbar_wait_issue(&empty[stage], phase, abort_flag, a.status);
        __syncwarp();
        tc_fence_after();
        const uint32_t tbase = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + accb * kMats * p.bn;
        const float* sn = scales + slot * p.bn;
        uint64_t w[2];
        {
          const uint32_t b0 = __float_as_uint(__shfl_sync(0xffffffffu, sw0, kb & 31));
          w[0] = pack2(b0, b0);
          const uint32_t b1 = kGU ? __float_as_uint(__shfl_sync(0xffffffffu, sw1, kb & 31)) : 0u;
          w[1] = pack2(b1, b1);
        }
        // all groups, whether the tile has rows for them or not (a branch for each costs more: 64 x 8192 -> 8192 27.5
        // instead of 21.6 us; accumulators and scales end inside what is allocated), the scales beside the loads
        uint32_t d[V::kGroups][kMats][V::kGroup];
        uint64_t f[V::kGroups][V::kGroup / 2];
#pragma unroll
        for (int g = 0; g < V::kGroups; ++g) {
          const int c0 = V::kGroup * (g * kParts + part);
#pragma unroll
          for (int mat = 0; mat < kMats; ++mat) tmem_ld<V::kGroup>(tbase + mat * p.bn + c0, d[g][mat]);
#pragma unroll
          for (int c = 0; c < V::kGroup / 4; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(sn + c0 + 4 * c);
            f[g][2 * c] = pack2(v.x, v.y);
            f[g][2 * c + 1] = pack2(v.z, v.w);
            if (kMats == 1) {
              f[g][2 * c] = mul2(f[g][2 * c], w[0]);
              f[g][2 * c + 1] = mul2(f[g][2 * c + 1], w[0]);
            }
          }
        }
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[accb]);
#pragma unroll
        for (int g = 0; g < V::kGroups; ++g)
#pragma unroll
          for (int c = 0; c < V::kGroup / 2; ++c)
#pragma unroll
            for (int mat = 0; mat < kMats; ++mat)
              fma2(acc.v[mat][g][c], pack2(d[g][mat][2 * c], d[g][mat][2 * c + 1]), kMats == 1 ? f[g][c] : mul2(f[g][c], w[mat]));
        if (++slot == p.scale_slots) slot = 0;
        if (++accb == p.accs) accb = 0;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if constexpr (V::kMode == kLinear) {
        if (a.split > 1) {  // every MMA of the item has completed: the stages' memory is free
          put_sums<V>(reinterpret_cast<float*>(stages), m.rows, acc, quarter, part, lane);
          continue;
        }
      }
      ok = epilogue<V>(a, m, acc, quarter, part, lane, maxima + 4 * parity, [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&part_met[part]);
        const bool met = mbar_wait_warp(&part_met[part], parity, abort_flag);
        if (!met && lane == 0) fail();
        return met;
      });
      parity ^= 1;  // a warp two items ahead has met all the others in between: two sets of maxima are enough
    }
  }

  if constexpr (V::kMode == kLinear) {
    if (a.split > 1) {
      cluster_arrive_release();
      cluster_wait();
      if (warp >= kSumWarp0) join_sums(a, item(0), reinterpret_cast<const float*>(stages), warp - kSumWarp0, lane);
      cluster_arrive_release();  // (the others' shared memory has been read)
      cluster_wait();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <typename V>
cudaError_t launch(int kind, const typename Args<V::kMode>::maps& maps, const typename Args<V::kMode>::type& a, int bn,
                   int grid, int cluster, cudaStream_t stream, bool pdl) {
  const Plan p = make_plan(V::kMats, bn);
  const int smem = plan_smem(p);
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(blk_gemm_kernel<V>), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  timer_begin(kind, stream);
  e = cudaLaunchKernelEx(&cfg, blk_gemm_kernel<V>, maps, a, p);
  timer_end(kind, stream);
  return e;
}

// The variant for tiles of bn tokens.
template <int kMode>
cudaError_t launch_for(int kind, const typename Args<kMode>::maps& maps, const typename Args<kMode>::type& a, int bn,
                       int grid, int cluster, cudaStream_t stream, bool pdl) {
  if (bn <= 16) return launch<Variant<kMode, 16>>(kind, maps, a, bn, grid, cluster, stream, pdl);
  if (bn <= 32) return launch<Variant<kMode, 32>>(kind, maps, a, bn, grid, cluster, stream, pdl);
  return launch<Variant<kMode, 64>>(kind, maps, a, bn, grid, cluster, stream, pdl);
}

}  // namespace

cudaError_t launch_blk_linear(const BlkLinearArgs& a, const BlkLinearMaps& maps, cudaStream_t stream, bool pdl) {
  const long long items = static_cast<long long>(blk_count(a.N)) * ((a.M + a.bn - 1) / a.bn);
  if (items > (1ll << 30)) return cudaErrorInvalidValue;
  const int grid = static_cast<int>(a.split > 1 ? items * a.split : items < a.num_sms ? items : a.num_sms);
  return launch_for<kLinear>(kKBlkGemm, maps, a, a.bn, grid, a.split, stream, pdl);
}

cudaError_t launch_blk_experts(const BlkExpertArgs& a, const BlkExpertMaps& maps, cudaStream_t stream, bool pdl) {
  cudaError_t e = launch_for<kGateUp>(kKBlkGateUp, maps, a, a.pitch, a.num_sms, 1, stream, pdl);
  if (e != cudaSuccess) return e;
  e = launch_for<kDown>(kKBlkDown, maps, a, a.pitch, a.num_sms, 1, stream, pdl);
  if (e != cudaSuccess) return e;
  return launch_mx_combine(a.ypart, a.inv_perm, a.w, a.T, a.d, a.k, a.I_shared > 0, a.y, a.status, a.num_sms, stream);
}

}  // namespace bm
