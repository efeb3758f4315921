// Block-scaled 8-bit products for tiles of many tokens: the tokens are the M = 128
// side, so a scale is one number a lane, and 256 weight rows the N side: both
// matrices' 128 (gate/up), or 256 rows of one (down, dense).
//
// As in blk_gemm.cu a block of 128 columns multiplies into an accumulator of its
// own (two of 256 columns in turn) and warps with the running sums in registers add
// it, scaled, while the next block multiplies.  Here that is one fused multiply-add
// a value: 128 x 256 of them a stage, against 512 clocks of MMA.
//
// Roles (one persistent CTA per SM): warps 0 and 1 the weights' and the
// activations' loads, warp 2 the MMAs' issue, warps 4 to 11 the sums: two per
// quarter of the tensor-memory lanes (32 tokens), 128 columns each.  Rows of
// results leave through shared memory as TMA stores, 32 x 32 at a time (a lane's
// own stores would touch a line each); the last, partial 32 rows of an expert by
// plain stores.  Every wait is bounded and records MOE_ERR_TIMEOUT.
#include <cuda_runtime.h>

#include "blk_items.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace bm {
namespace {

constexpr int kWeightsWarp = 0;
constexpr int kActivationsWarp = 1;
constexpr int kMmaWarp = 2;
constexpr int kSumWarp0 = 4;
constexpr int kSumWarps = 8;
constexpr int kParts = kSumWarps / 4;  // shares of the columns
constexpr int kThreads = (kSumWarp0 + kSumWarps) * 32;
constexpr int kCols = 2 * kBlk;        // weight rows of a tile
constexpr uint32_t kTmemCols = 512;
constexpr int kAccs = 2;
constexpr int kHalfBytes = kBlk * 128;  // 128 rows' codes of a stage
constexpr int kStageBytes = 3 * kHalfBytes;
constexpr int kBoxBytes = 32 * 32 * 4;  // a 32 x 32 box of a result on its way out
constexpr int kEntries = 64;            // items of a CTA, from its first, whose Entry is in shared memory
template <int kMode>
struct Variant {
  // with results staged in two boxes a warp, three stages are left
  static constexpr int kStages = kMode == kGateUp ? 4 : 3;
  static constexpr int kBoxes = kMode == kGateUp ? 0 : 2;
  static constexpr int kSmem = kStages * kStageBytes + kSumWarps * kBoxes * kBoxBytes + 2 * kParts * kBlk * 4 /* maxima */ +
                               512 /* barriers */ + 16 * kEntries + 1024 /* alignment */;
};
static_assert(Variant<kGateUp>::kSmem <= 227 * 1024 && Variant<kDown>::kSmem <= 227 * 1024, "shared memory of a CTA");

// A warp's sums: 128 columns of each lane's token, two to a register pair; gate/up: 64 of gate, then 64 of up.
struct Sums {
  uint64_t v[4][16];
  __device__ __forceinline__ float get(int c) const {
    float lo, hi;
    unpack2(v[c >> 5][(c & 31) >> 1], lo, hi);
    return c & 1 ? hi : lo;
  }
};

// 32 columns of the warp's 32 tokens as a box of the result: a lane's row in 16-byte chunks, in the order the store's
// swizzle takes (128-byte rows: chunk ^ row % 8; 64-byte rows: chunk ^ row / 2 % 4).
template <bool kWideType>
__device__ __forceinline__ void put_box(uint8_t* box, const Sums& acc, int g, int lane, int type) {
  if constexpr (kWideType) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<float4*>(box + 128 * lane + 16 * (j ^ (lane & 7))) =
          make_float4(acc.get(32 * g + 4 * j), acc.get(32 * g + 4 * j + 1), acc.get(32 * g + 4 * j + 2), acc.get(32 * g + 4 * j + 3));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = acc.get(32 * g + 8 * j + 2 * i), b = acc.get(32 * g + 8 * j + 2 * i + 1);
        if (type == kFp16) {
          o[i] = f32x2_to_f16x2(a, b);
        } else {
          const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
          o[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
      *reinterpret_cast<uint4*>(box + 64 * lane + 16 * (j ^ ((lane >> 1) & 3))) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// The warp's 128 columns of its 32 tokens, of which `rows` exist, from column n0 on: by boxes where `boxed`, else by
// each lane.  `first`: the first token's row of the result, whose rows are N elements long; `turn`: the warp's next box.
__device__ __forceinline__ void store_rows(const Sums& acc, const CUtensorMap* map, uint8_t* boxes, int& turn, bool boxed, int type,
                                           void* y, long long first, int rows, int n0, int N, int lane) {
  if (boxed) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (n0 + 32 * g >= N) break;
      uint8_t* box = boxes + turn * kBoxBytes;
      turn ^= 1;
      if (lane == 0) bulk_wait_group_read<1>();  // the box two turns back, this one, has been read
      __syncwarp();
      if (type == kFp32) put_box<true>(box, acc, g, lane, type); else put_box<false>(box, acc, g, lane, type);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(map, box, n0 + 32 * g, static_cast<int>(first));
        bulk_commit_group();
      }
    }
  } else if (lane < rows) {
    const size_t at = static_cast<size_t>(first + lane) * N + n0;
#pragma unroll
    for (int c = 0; c < 128; ++c)
      if (n0 + c < N) store1(type, y, at + c, acc.get(c));
  }
}

__device__ __forceinline__ void epilogue_rows(const BlkLinearArgs& a, const BlkLinearMaps& maps, const Item& m, const Sums& acc,
                                              uint8_t* boxes, int& turn, int quarter, int part, int lane) {
  // (rows and columns past the result's end are not written by a box)
  store_rows(acc, &maps.y, boxes, turn, a.y_boxed, a.y_type, a.y, static_cast<long long>(m.row_n) + 32 * quarter, m.rows - 32 * quarter,
             m.row_m + kBlk * part, a.N, lane);
}
__device__ __forceinline__ void epilogue_rows(const BlkExpertArgs& a, const BlkExpertMaps& maps, const Item& m, const Sums& acc,
                                              uint8_t* boxes, int& turn, int quarter, int part, int lane) {
  // fp32 rows of the experts' outputs, routed ones in permuted order, then the shared expert's in token order: what
  // follows an item's last row is another item's
  const int rows = m.rows - 32 * quarter;
  store_rows(acc, &maps.ypart, boxes, turn, rows >= 32, kFp32, a.ypart, (m.shared ? static_cast<long long>(a.T) * a.k : 0) + m.row0 + 32 * quarter,
             rows, m.row_m + kBlk * part, a.d, lane);
}

// gate/up: h = silu(gate) up of 64 columns of a lane's token, quantised with the other share's 64 (a block of h).
// meet(): waits until the other share's maxima have been written (false: given up).
template <typename Meet>
__device__ __forceinline__ bool epilogue_gate_up(const BlkExpertArgs& a, const Item& m, Sums& acc, int quarter, int part, int lane,
                                                 uint32_t (*maxima)[kBlk], Meet meet) {
  const int I = m.shared ? a.I_shared : a.I;
  float most = 0.0f;
#pragma unroll
  for (int c = 0; c < 64; c += 2) {  // h takes gate's place
    const float h0 = blk_swiglu(acc.get(c), acc.get(64 + c)), h1 = blk_swiglu(acc.get(c + 1), acc.get(64 + c + 1));
    most = max_nan(most, max_nan(fabsf(h0), fabsf(h1)));
    acc.v[c >> 5][(c & 31) >> 1] = pack2(__float_as_uint(h0), __float_as_uint(h1));
  }
  const int r = 32 * quarter + lane;
  maxima[part][r] = __float_as_uint(most);
  if (!meet()) return false;
  const float s = blk_scale(max(maxima[0][r], maxima[1][r])), inv = blk_inverse(s);
  if (r >= m.rows) return true;
  if (part == 0)
    (m.shared ? a.sh_s : a.sh_r)[(static_cast<size_t>(m.slot) * blk_count(I) + m.mt) * a.pitch + r] = s;
  const int n0 = m.mt * kBlk + 64 * part;
  uint8_t* hq = (m.shared ? a.h_s : a.h_r) + static_cast<size_t>(m.row0 + r) * I + n0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (n0 + 16 * j >= I) break;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 16 * j + 4 * i;
      o[i] = f32x4_to_e4m3x4(acc.get(c) * inv, acc.get(c + 1) * inv, acc.get(c + 2) * inv, acc.get(c + 3) * inv);
    }
    *reinterpret_cast<uint4*>(hq + 16 * j) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  return true;
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    blk_wide_kernel(const __grid_constant__ typename Args<kMode>::maps maps, const __grid_constant__ typename Args<kMode>::type a) {
  using V = Variant<kMode>;
  constexpr bool kGU = kMode == kGateUp;
  constexpr int kStages = V::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* boxes = stages + kStages * kStageBytes;
  uint32_t(*maxima)[kBlk] = reinterpret_cast<uint32_t(*)[kBlk]>(boxes + kSumWarps * V::kBoxes * kBoxBytes);  // [2 x parts][tokens]
  uint64_t* full = reinterpret_cast<uint64_t*>(maxima + 2 * kParts);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + kAccs;
  uint64_t* met = acc_empty + kAccs;  // a quarter's two warps have written their maxima
  uint64_t* finished = met + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(finished + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Entry* entries = reinterpret_cast<Entry*>(reinterpret_cast<uint8_t*>(full) + 512);

  // the same in all lanes, so that the roles' branches are known to be uniform
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  // The routing has completed by now (the kernel before this one lets this one
  // start only after its own wait), so only the activations are waited for.
  const Sched s = make_sched<kCols>(a, kMaxTile, kGU);
  for (int i = threadIdx.x; i < min(s.n, kEntries); i += kThreads) entries[i] = make_entry(a, s, s.first + i * s.step);
  auto item = [&](int i) {
    return get_item<kCols>(a, maps, kMaxTile, i < kEntries ? entries[i] : make_entry(a, s, s.first + i * s.step), kGU);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 2);  // the weights' and the activations' expect_tx; their bytes complete the phase
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kSumWarps);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&met[i], kParts);
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
    // 128 sums take more than 384 threads' equal share of the registers: 128 x 72 + 256 x 216 = 384 x 168
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
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
          const int blocks = blk_count(m.K);
          for (int kb = 0; kb < blocks; ++kb, ++filled) {
            if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
              fail();
              ok = false;
              break;
            }
            uint8_t* st = stages + stage * kStageBytes;
            uint64_t* bar = &full[stage];
            if (weights) {
              mbar_arrive_expect_tx(bar, 2 * kHalfBytes);
              tma_load_3d(st + kHalfBytes, m.m0, bar, kb * kBlk, m.row_m, m.e);
              if (kGU)
                tma_load_3d(st + 2 * kHalfBytes, m.m1, bar, kb * kBlk, m.row_m, m.e);
              else
                tma_load_3d(st + 2 * kHalfBytes, m.m0, bar, kb * kBlk, m.row_m + kBlk, m.e);
            } else {
              mbar_arrive_expect_tx(bar, m.box * 128);
              tma_load_2d(st, m.n, bar, kb * kBlk, m.row_n);
            }
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        // never leave while a load into this CTA's shared memory may be in flight
        for (int i = 0; i < min(filled, kStages); ++i) {
          stage = stage == 0 ? kStages - 1 : stage - 1;
          if (stage == kStages - 1) phase ^= 1;
          if (!mbar_wait(&full[stage], phase, nullptr)) record_status(a.status, MOE_ERR_TIMEOUT);
        }
        if (weights) pdl_wait();
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      pdl_wait();
      pdl_launch_dependents();
      // One thread issues everything; what it issues is computed by the whole warp
      // from values that are the same in all lanes, which lets the compiler keep
      // descriptors and addresses in uniform registers.
      const uint32_t stage0 = smem_u32(stages);
      const uint64_t ad0 = smem_desc_sw128_kmajor(stage0), bd0 = smem_desc_sw128_kmajor(stage0 + kHalfBytes);
      constexpr uint32_t idesc = idesc_e4m3_f32(kBlk, kCols);
      int stage = 0;
      uint32_t phase = 0, acc = 0, accphase = 0, at = 0;
      const bool leader = elect_one();
      for (int i = 0; i < s.n; ++i) {
        const Item m = item(i);
        if (__shfl_sync(0xffffffffu, m.ok ? 1 : 0, 0) == 0) continue;
        const int n32 = (__shfl_sync(0xffffffffu, m.K, 0) + 31) / 32;
        for (int k = 0; k < n32; k += 4) {
          mbar_wait_issue(&acc_empty[acc], accphase ^ 1, abort_flag, a.status);
          mbar_wait_issue(&full[stage], phase, abort_flag, a.status);
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk > 0 && k + kk >= n32) break;
              tc_mma_f8(tmem + acc * kCols, ad0 + at + 2 * kk, bd0 + at + 2 * kk, idesc, kk > 0 ? 1u : 0u);
            }
            tc_commit(&empty[stage]);
            tc_commit(&acc_full[acc]);
          }
          at += kStageBytes >> 4;
          if (++stage == kStages) {
            stage = 0;
            at = 0;
            phase ^= 1;
          }
          acc ^= 1;
          accphase ^= acc ^ 1;
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    pdl_wait();
    pdl_launch_dependents();
    const int quarter = warp & 3, part = (warp - kSumWarp0) >> 2;
    uint32_t acc = 0, accphase = 0, parity = 0;
    int turn = 0;
    bool ok = true;
    // columns of group g in the accumulator
    auto column = [&](int g) { return kGU ? (g >> 1) * kBlk + 64 * part + 32 * (g & 1) : kBlk * part + 32 * g; };
    auto wait_full = [&]() {
      if (mbar_wait(&acc_full[acc], accphase, abort_flag)) return true;
      if (lane == 0) fail();
      return false;
    };
    for (int i = 0; i < s.n && ok; ++i) {
      const Item m = item(i);
      if (!m.ok) {
        if (lane == 0) record_status(a.status, MOE_ERR_INVALID_ARG);
        continue;
      }
      const int blocks = blk_count(m.K);
      const bool some = 32 * quarter < m.rows;  // of this quarter's tokens
      Sums sum;
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int c = 0; c < 16; ++c) sum.v[g][c] = 0;
      // the scales two blocks ahead
      const float* sn = m.sn + min(32 * quarter + lane, static_cast<int>(m.sn_bytes / 4) - 1);
      const float *s0 = kGU || part == 0 ? m.s0 : m.s1, *s1 = m.s1;
      float sx[3], sw0[3], sw1[3];
      auto scales = [&](int kb, int to) {
        sx[to] = kb < blocks ? __ldg(sn + kb * m.sn_step) : 0.0f;
        sw0[to] = kb < blocks ? __ldg(s0 + kb) : 0.0f;
        sw1[to] = kGU && kb < blocks ? __ldg(s1 + kb) : 0.0f;
      };
      scales(0, 0);
      scales(1, 1);
      uint32_t d[2][32];
      ok = wait_full();
      if (!ok) break;
      __syncwarp();
      tc_fence_after();
      const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
      if (some) tmem_ld32(tmem + lanes + acc * kCols + column(0), d[0]);
      for (int kb = 0; kb < blocks; ++kb) {
        scales(kb + 2, 2);
        uint64_t w[2];
        {
          const uint32_t f0 = __float_as_uint(sx[0] * sw0[0]), f1 = __float_as_uint(sx[0] * sw1[0]);
          w[0] = pack2(f0, f0);
          w[1] = pack2(f1, f1);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          tc_wait_ld();
          if (g < 3) {
            if (some) tmem_ld32(tmem + lanes + acc * kCols + column(g + 1), d[(g + 1) & 1]);
          } else {
            // this accumulator has been read: on to the next block's, whose load runs beside the last sums of this one
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
            acc ^= 1;
            accphase ^= acc ^ 1;
            if (kb + 1 < blocks) {
              ok = wait_full();
              if (!ok) break;
              __syncwarp();
              tc_fence_after();
              if (some) tmem_ld32(tmem + lanes + acc * kCols + column(0), d[0]);
            }
          }
          if (some) {
#pragma unroll
            for (int c = 0; c < 16; ++c) fma2(sum.v[g][c], pack2(d[g & 1][2 * c], d[g & 1][2 * c + 1]), w[kGU ? g >> 1 : 0]);
          }
        }
        if (!ok) break;
        sx[0] = sx[1];
        sx[1] = sx[2];
        sw0[0] = sw0[1];
        sw0[1] = sw0[2];
        sw1[0] = sw1[1];
        sw1[1] = sw1[2];
      }
      if (!ok) break;
      if constexpr (kGU) {
        ok = epilogue_gate_up(a, m, sum, quarter, part, lane, maxima + kParts * parity, [&]() {
          __syncwarp();
          if (lane == 0) mbar_arrive(&met[quarter]);
          const bool m2 = mbar_wait(&met[quarter], parity, abort_flag);
          if (!m2 && lane == 0) fail();
          __syncwarp();
          return m2;
        });
        parity ^= 1;  // a warp two items ahead has met the other one in between: two sets of maxima are enough
      } else if (some) {
        epilogue_rows(a, maps, m, sum, boxes + (warp - kSumWarp0) * V::kBoxes * kBoxBytes, turn, quarter, part, lane);
      }
    }
    if (!kGU && lane == 0) bulk_wait_group_all();  // nothing of this CTA's shared memory is read after its end
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int kMode>
cudaError_t launch(int kind, const typename Args<kMode>::maps& maps, const typename Args<kMode>::type& a, int grid,
                   cudaStream_t stream, bool pdl) {
  constexpr int smem = Variant<kMode>::kSmem;
  cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(blk_wide_kernel<kMode>), smem);
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
  e = cudaLaunchKernelEx(&cfg, blk_wide_kernel<kMode>, maps, a);
  timer_end(kind, stream);
  return e;
}

}  // namespace

cudaError_t launch_blk_wide_linear(const BlkLinearArgs& a, const BlkLinearMaps& maps, cudaStream_t stream, bool pdl) {
  const long long items = static_cast<long long>((a.N + kCols - 1) / kCols) * ((a.M + kMaxTile - 1) / kMaxTile);
  if (items > (1ll << 30)) return cudaErrorInvalidValue;
  return launch<kLinear>(kKBlkGemm, maps, a, static_cast<int>(items < a.num_sms ? items : a.num_sms), stream, pdl);
}

cudaError_t launch_blk_wide_experts(const BlkExpertArgs& a, const BlkExpertMaps& maps, cudaStream_t stream, bool pdl) {
  cudaError_t e = launch<kGateUp>(kKBlkGateUp, maps, a, a.num_sms, stream, pdl);
  if (e != cudaSuccess) return e;
  e = launch<kDown>(kKBlkDown, maps, a, a.num_sms, stream, pdl);
  if (e != cudaSuccess) return e;
  return launch_mx_combine(a.ypart, a.inv_perm, a.w, a.T, a.d, a.k, a.I_shared > 0, a.y, a.status, a.num_sms, stream);
}

}  // namespace bm
