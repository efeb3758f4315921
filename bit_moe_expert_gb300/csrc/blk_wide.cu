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
// results leave through shared memory as TMA stores, 64 bytes of 32 rows at a time
// (a lane's own stores would touch a line each); the last, partial 32 rows of an
// expert, and rows that are not 16-byte aligned, by plain stores from there.  Every wait is bounded and records MOE_ERR_TIMEOUT.
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
constexpr int kBoxBytes = 32 * 64;      // 64 bytes of 32 rows of a result on their way out
constexpr int kBoxes = 4;               // of a warp
constexpr int kEntries = 64;            // items of a CTA, from its first, whose Entry is in shared memory
template <int kMode>
struct Variant {
  // with results staged in boxes, three stages are left
  static constexpr int kStages = kMode == kGateUp ? 4 : 3;
  // the tokens' scales of a block are read until its accumulator is free again, which may be kAccs stages after the
  // stage's codes: a ring of their own
  static constexpr int kSlots = kStages + kAccs;
  static constexpr int kSmem = kStages * kStageBytes + (kMode == kGateUp ? 0 : kSumWarps * kBoxes * kBoxBytes) + 2 * kParts * kBlk * 4 /* maxima */ + kSlots * kBlk * 4 /* scales */ +
                               512 /* barriers */ + 16 * kEntries + 1024 /* alignment */;
};
static_assert(Variant<kGateUp>::kSmem <= 227 * 1024 && Variant<kDown>::kSmem <= 227 * 1024, "shared memory of a CTA");

constexpr int kOwn = kCols / kParts;  // columns of a warp; gate/up: half of them gate's, then as many of up's
constexpr int kPiece = 8;            // columns of an accumulator that a warp takes at a time

// A warp's sums: kOwn columns of each lane's token, two to a register pair.
struct Sums {
  uint64_t v[kOwn / 2];
  __device__ __forceinline__ float get(int c) const {
    float lo, hi;
    unpack2(v[c >> 1], lo, hi);
    return c & 1 ? hi : lo;
  }
};

// A box of the result from column c of the warp's on: a lane's row of 64 bytes, its four 16-byte chunks in the order that
// the store's swizzle takes (chunk ^ row / 2 % 4).
template <int kType>
__device__ __forceinline__ void put_box(uint8_t* box, const Sums& acc, int c, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kType == kFp32) {
        o[i] = __float_as_uint(acc.get(c + 4 * j + i));
      } else {
        const float a = acc.get(c + 8 * j + 2 * i), b = acc.get(c + 8 * j + 2 * i + 1);
        if constexpr (kType == kFp16) {
          o[i] = f32x2_to_f16x2(a, b);
        } else {
          const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
          o[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
    }
    *reinterpret_cast<uint4*>(box + 64 * lane + 16 * (j ^ ((lane >> 1) & 3))) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// The warp's columns of its 32 tokens, of which `rows` exist, from column n0 of the result on, through boxes: by TMA stores
// where `boxed`, by 16-byte stores where the result's rows are `aligned` to them, else by a word or a 16-bit value a lane,
// 64 bytes of a row at a time (4000 x 2048 -> 4000 / 4002 / 4001 of bf16: 37 / 42 / 48 us by the three; 187 where each lane
// wrote its token's elements).  `first`:
// the first token's row of the result, whose rows are N elements long; `turn`: the warp's next box.
template <int kType>
__device__ __forceinline__ void store_rows(const Sums& acc, const CUtensorMap* map, uint8_t* boxes, int& turn, bool boxed, bool aligned,
                                           void* y, long long first, int rows, int n0, int N, int lane) {
  constexpr int kBytes = kType == kFp32 ? 4 : 2, kWide = 64 / kBytes;  // columns of a box
#pragma unroll
  for (int c = 0; c < kOwn; c += kWide) {
    if (n0 + c >= N) break;
    uint8_t* box = boxes + turn * kBoxBytes;
    turn = turn + 1 == kBoxes ? 0 : turn + 1;
    if (lane == 0) bulk_wait_group_read<kBoxes - 1>();  // this box has been read
    __syncwarp();
    put_box<kType>(box, acc, c, lane);
    if (boxed) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(map, box, n0 + c, static_cast<int>(first));
        bulk_commit_group();
      }
      continue;
    }
    __syncwarp();
    if (aligned) {
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 8) {  // four lanes a row
        const int r = r0 + (lane >> 2), col = n0 + c + (lane & 3) * (16 / kBytes);
        const uint4 v = *reinterpret_cast<const uint4*>(box + 64 * r + 16 * ((lane & 3) ^ ((r >> 1) & 3)));
        if (r < rows && col < N) *reinterpret_cast<uint4*>(static_cast<char*>(y) + ((first + r) * N + col) * kBytes) = v;
      }
    } else {
      // words of the box's rows, two rows at a time, or 16-bit values of odd N
      auto store = [&](auto element) {
        using Element = decltype(element);
        constexpr int kSize = sizeof(Element), kRow = 64 / kSize;
        const int at = lane % kRow * kSize, col = n0 + c + at / kBytes;
        char* to = static_cast<char*>(y) + ((first + lane / kRow) * N + col) * kBytes;
#pragma unroll 8
        for (int i = 0; i < kRow; ++i, to += static_cast<size_t>(32 / kRow) * N * kBytes) {
          const int r = lane / kRow + i * (32 / kRow);
          const Element v = *reinterpret_cast<const Element*>(box + 64 * r + 16 * ((at >> 4) ^ ((r >> 1) & 3)) + (at & 15));
          if (r < rows && col < N) *reinterpret_cast<Element*>(to) = v;
        }
      };
      if (kBytes == 4 || N % 2 == 0) store(uint32_t{}); else store(uint16_t{});
    }
    __syncwarp();
    if (lane == 0) bulk_commit_group();  // an empty one: a box's turn is a group's
  }
}

__device__ __forceinline__ void epilogue_rows(const BlkLinearArgs& a, const BlkLinearMaps& maps, const Item& m, const Sums& acc,
                                              uint8_t* boxes, int& turn, int quarter, int part, int lane) {
  // (rows and columns past the result's end are not written by a box)
  const long long first = static_cast<long long>(m.row_n) + 32 * quarter;
  const int rows = m.rows - 32 * quarter, n0 = m.row_m + kOwn * part;
  if (a.y_type == kFp32)
    store_rows<kFp32>(acc, &maps.y, boxes, turn, a.y_boxed, a.y_boxed, a.y, first, rows, n0, a.N, lane);
  else if (a.y_type == kFp16)
    store_rows<kFp16>(acc, &maps.y, boxes, turn, a.y_boxed, a.y_boxed, a.y, first, rows, n0, a.N, lane);
  else
    store_rows<kBf16>(acc, &maps.y, boxes, turn, a.y_boxed, a.y_boxed, a.y, first, rows, n0, a.N, lane);
}
__device__ __forceinline__ void epilogue_rows(const BlkExpertArgs& a, const BlkExpertMaps& maps, const Item& m, const Sums& acc,
                                              uint8_t* boxes, int& turn, int quarter, int part, int lane) {
  // fp32 rows of the experts' outputs, routed ones in permuted order, then the shared expert's in token order: what
  // follows an item's last row is another item's
  const int rows = m.rows - 32 * quarter;
  store_rows<kFp32>(acc, &maps.ypart, boxes, turn, rows >= 32, true, a.ypart,
                    (m.shared ? static_cast<long long>(a.T) * a.k : 0) + m.row0 + 32 * quarter, rows, m.row_m + kOwn * part, a.d,
                    lane);
}

// gate/up: h = silu(gate) up of kOwn / 2 columns of a lane's token, quantised with the other shares' (a block of h).
// meet(): waits until their maxima have been written (false: given up).
template <typename Meet>
__device__ __forceinline__ bool epilogue_gate_up(const BlkExpertArgs& a, const Item& m, Sums& acc, int quarter, int part, int lane,
                                                 uint32_t (*maxima)[kBlk], Meet meet) {
  constexpr int kHalf = kOwn / 2;
  const int I = m.shared ? a.I_shared : a.I;
  float most = 0.0f;
#pragma unroll
  for (int c = 0; c < kHalf; c += 2) {  // h takes gate's place
    const float h0 = blk_swiglu(acc.get(c), acc.get(kHalf + c)), h1 = blk_swiglu(acc.get(c + 1), acc.get(kHalf + c + 1));
    most = max_nan(most, max_nan(fabsf(h0), fabsf(h1)));
    acc.v[c >> 1] = pack2(__float_as_uint(h0), __float_as_uint(h1));
  }
  const int r = 32 * quarter + lane;
  maxima[part][r] = __float_as_uint(most);
  if (!meet()) return false;
  const float s = blk_scale(max(maxima[0][r], maxima[1][r])), inv = blk_inverse(s);
  if (r >= m.rows) return true;
  if (part == 0)
    (m.shared ? a.sh_s : a.sh_r)[(static_cast<size_t>(m.slot) * blk_count(I) + m.mt) * a.pitch + r] = s;
  const int n0 = m.mt * kBlk + kHalf * part;
  uint8_t* hq = (m.shared ? a.h_s : a.h_r) + static_cast<size_t>(m.row0 + r) * I + n0;
#pragma unroll
  for (int j = 0; j < kHalf / 16; ++j) {
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
  uint32_t(*maxima)[kBlk] = reinterpret_cast<uint32_t(*)[kBlk]>(boxes + (kGU ? 0 : kSumWarps * kBoxes * kBoxBytes));  // [2 x parts][tokens]
  float* scales = reinterpret_cast<float*>(maxima + 2 * kParts);  // [slots][tokens]
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + V::kSlots * kBlk);
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
      mbar_init(&acc_full[i], 2);  // the MMAs' commit, and their issuer, who has seen the stage's scales land
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
    // 128 sums take more than 384 threads' equal share of the registers: 128 x 40 + 256 x 232 = 384 x 168
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == kWeightsWarp || warp == kActivationsWarp) {
      // one thread for the weights, which starts before the wait, and one for the activations
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
              mbar_arrive_expect_tx(bar, m.box * 128 + m.sn_bytes);
              tma_load_2d(st, m.n, bar, kb * kBlk, m.row_n);
              bulk_g2s(scales + slot * kBlk, sn, m.sn_bytes, bar);
              sn += m.sn_step;
              if (++slot == V::kSlots) slot = 0;
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
            mbar_arrive(&acc_full[acc]);
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    pdl_wait();
    pdl_launch_dependents();
    const int quarter = warp & 3, part = (warp - kSumWarp0) >> 2;
    uint32_t acc = 0, accphase = 0, parity = 0;
    int turn = 0, slot = 0;
    bool ok = true;
    // first column of piece u in the accumulator
    auto column = [&](int u) {
      const int c = u * kPiece;
      return kGU ? c / (kOwn / 2) * kBlk + kOwn / 2 * part + c % (kOwn / 2) : kOwn * part + c;
    };
    auto wait_full = [&]() {
      if (mbar_wait_warp(&acc_full[acc], accphase, abort_flag)) return true;
      if (lane == 0) fail();
      return false;
    };
    for (int i = 0; i < s.n && ok; ++i) {
      // what the loop below needs of the item; the rest is taken again after it, and the weights' scales every 32 blocks,
      // so that their registers are free in between
      int blocks;
      bool some;        // of this quarter's tokens
      {
        const Item m = item(i);
        if (!m.ok) {
          if (lane == 0) record_status(a.status, MOE_ERR_INVALID_ARG);
          continue;
        }
        blocks = blk_count(m.K);
        some = 32 * quarter < m.rows;
      }
      Sums sum;
#pragma unroll
      for (int c = 0; c < kOwn / 2; ++c) sum.v[c] = 0;
      float sw0 = 0.0f, sw1 = 0.0f;  // the weights' scales of 32 blocks, one a lane
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      for (int kb = 0; kb < blocks; ++kb) {
        if ((kb & 31) == 0) {
          const Item m = item(i);
          sw0 = sw1 = 0.0f;
          if (kb + lane < blocks) {
            sw0 = __ldg((kGU || part < kParts / 2 ? m.s0 : m.s1) + kb + lane);
            if (kGU) sw1 = __ldg(m.s1 + kb + lane);
          }
        }
        if (!wait_full()) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint64_t w[2];
        {
          const float sx = scales[slot * kBlk + 32 * quarter + lane];
          if (++slot == V::kSlots) slot = 0;
          const uint32_t f0 = __float_as_uint(sx * __shfl_sync(0xffffffffu, sw0, kb & 31));
          const uint32_t f1 = kGU ? __float_as_uint(sx * __shfl_sync(0xffffffffu, sw1, kb & 31)) : 0u;
          w[0] = pack2(f0, f0);
          w[1] = pack2(f1, f1);
        }
#pragma unroll
        for (int u = 0; u < kOwn / kPiece; ++u) {
          uint32_t d[kPiece];
          tmem_ld<kPiece>(lanes + acc * kCols + column(u), d);
          tc_wait_ld();
          if (u + 1 == kOwn / kPiece) {  // this accumulator has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
          }
#pragma unroll
          for (int c = 0; c < kPiece / 2; ++c)
            fma2(sum.v[u * kPiece / 2 + c], pack2(d[2 * c], d[2 * c + 1]), w[kGU ? 2 * u * kPiece / kOwn : 0]);
        }
        acc ^= 1;
        accphase ^= acc ^ 1;
      }
      if (!ok) break;
      const Item m = item(i);
      if constexpr (kGU) {
        ok = epilogue_gate_up(a, m, sum, quarter, part, lane, maxima + kParts * parity, [&]() {
          __syncwarp();
          if (lane == 0) mbar_arrive(&met[quarter]);
          const bool m2 = mbar_wait_warp(&met[quarter], parity, abort_flag);
          if (!m2 && lane == 0) fail();
          return m2;
        });
        parity ^= 1;  // a warp two items ahead has met the other one in between: two sets of maxima are enough
      } else if (some) {
        epilogue_rows(a, maps, m, sum, boxes + (warp - kSumWarp0) * kBoxes * kBoxBytes, turn, quarter, part, lane);
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
