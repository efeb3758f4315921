// How the tensor-core products of block-scaled 8-bit weights divide their work into
// items: a tile of tokens times 128 weight rows of both matrices (gate/up), or kRows
// weight rows (down, dense).
#pragma once

#include "blk.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace bm {
namespace {

enum Mode { kLinear, kGateUp, kDown };
constexpr int kMaxTile = 128;  // tokens of a tile

struct Item {
  const CUtensorMap *m0, *m1, *n;  // codes of the weights (one or two matrices) and of the tokens
  // scales: of the weight tile (a block after another), of the other matrix's tile (gate/up) or of the tile's second
  // 128 rows, of the tokens' first block
  const float *s0, *s1, *sn;
  long long sn_step;               // from a block's scales of the tokens to the next one's
  uint32_t sn_bytes;
  int e, row_m, row_n;             // matrix of the M side; first rows of the codes
  int mt, rows, K, box;            // M tile, valid tokens, depth, tokens that the TMA box brings
  int kb0;                         // first block of columns
  int row0, slot;                  // experts: first row among the assignments (or tokens), tile slot
  bool shared, ok;
};

// This CTA's items: local index i stands for item first + i * step.
struct Sched {
  int mt_r, mt_s;  // M tiles of a routed and of a shared tile
  int n_routed;    // expert products: items below are routed
  int first, n, step;
};
struct Entry {
  int e, row0;    // expert (-1: malformed) and first row; dense: 0 and the M tile
  int slot;       // entry of the block map, the shared expert's tile of tokens, or the dense product's N tile
  uint32_t what;  // experts: M tile + 2^16 rows + 2^31 for the shared expert
};
constexpr uint32_t kEntryShared = 1u << 31;
static_assert(kBlkMaxCols / kBlk <= 1 << 16 && kMaxTile < 1 << 15, "an Entry's M tile and rows");

template <int kMode>
struct Args {
  using type = BlkExpertArgs;
  using maps = BlkExpertMaps;
};
template <>
struct Args<kLinear> {
  using type = BlkLinearArgs;
  using maps = BlkLinearMaps;
};

template <int kRows>
__device__ __forceinline__ Sched make_sched(const BlkLinearArgs& a, int bn, bool) {
  Sched s{};
  s.mt_r = (a.N + kRows - 1) / kRows;
  const int total = s.mt_r * ((a.M + bn - 1) / bn);
  const unsigned split = kRows == kBlk ? a.split : 1;
  s.first = blockIdx.x / split;
  s.step = gridDim.x / split;
  s.n = (total - s.first + s.step - 1) / s.step;
  return s;
}
__device__ __forceinline__ Entry make_entry(const BlkLinearArgs&, const Sched& s, int it) {
  return Entry{0, it % s.mt_r, it / s.mt_r, 0};
}
template <int kRows>
__device__ __forceinline__ Item get_item(const BlkLinearArgs& a, const BlkLinearMaps& maps, int bn, const Entry& en,
                                         bool) {
  Item m{};
  m.mt = en.row0;
  m.m0 = &maps.w;
  m.n = &maps.x;
  m.row_m = m.mt * kRows;
  m.row_n = en.slot * bn;
  m.rows = min(bn, a.M - m.row_n);
  m.K = a.K;
  m.box = bn;
  m.s0 = a.sw + static_cast<size_t>(m.row_m / kBlk) * blk_count(a.K);
  m.s1 = m.row_m + kBlk < a.N ? m.s0 + blk_count(a.K) : m.s0;
  m.sn = a.sx + m.row_n;
  m.sn_step = a.sx_pitch;
  m.sn_bytes = 4 * static_cast<uint32_t>(min(static_cast<long long>(bn), a.sx_pitch - m.row_n));
  if (kRows == kBlk && a.split > 1) {  // this CTA's share of the blocks
    const int blocks = blk_count(a.K), rank = blockIdx.x % static_cast<unsigned>(a.split);
    m.kb0 = blocks * rank / a.split;
    m.K = min(a.K, blocks * (rank + 1) / a.split * kBlk) - m.kb0 * kBlk;
    m.s0 += m.kb0;
    m.sn += m.kb0 * m.sn_step;
  }
  m.ok = true;
  return m;
}

template <int kRows>
__device__ __forceinline__ Sched make_sched(const BlkExpertArgs& a, int, bool gate_up) {
  Sched s{};
  int nb = *reinterpret_cast<const volatile int32_t*>(a.num_blocks);
  if (nb < 1 || nb > min(a.max_blocks, a.T * a.k)) {  // every tile holds an assignment
    if (threadIdx.x == 0) record_status(a.status, MOE_ERR_INVALID_ARG);
    nb = 0;
  }
  s.mt_r = gate_up ? blk_count(a.I) : (a.d + kRows - 1) / kRows;
  s.mt_s = gate_up ? blk_count(a.I_shared) : s.mt_r;
  s.n_routed = nb * s.mt_r;
  const int total = s.n_routed + (a.I_shared > 0 ? (a.T + a.bn_s - 1) / a.bn_s * s.mt_s : 0);
  s.first = blockIdx.x;
  s.step = gridDim.x;
  s.n = (total - s.first + s.step - 1) / s.step;
  return s;
}
__device__ __forceinline__ Entry make_entry(const BlkExpertArgs& a, const Sched& s, int it) {
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
template <int kRows>
__device__ __forceinline__ Item get_item(const BlkExpertArgs& a, const BlkExpertMaps& maps, int, const Entry& en,
                                         bool gate_up) {
  Item m{};
  m.ok = en.e >= 0;
  if (!m.ok) return m;
  m.e = en.e;
  m.row0 = en.row0;
  m.rows = static_cast<int>(en.what >> 16 & 0x7FFFu);
  m.shared = (en.what & kEntryShared) != 0;
  m.mt = static_cast<int>(en.what & 0xFFFFu);
  m.slot = en.slot;
  const int I = m.shared ? a.I_shared : a.I;
  const int N = gate_up ? I : a.d;
  m.K = gate_up ? a.d : I;
  m.box = m.shared ? a.bn_s : a.bn_r;
  const BlkWeights& w = m.shared ? a.shared : a.routed;
  if (m.shared) {
    m.m0 = gate_up ? &maps.gate_s : &maps.down_s;
    m.m1 = &maps.up_s;
    m.n = gate_up ? &maps.x_s : &maps.h_s;
    m.row_n = gate_up ? a.T * a.k + m.row0 : m.row0;
  } else {
    m.m0 = gate_up ? &maps.gate_r : &maps.down_r;
    m.m1 = &maps.up_r;
    m.n = gate_up ? &maps.x_r : &maps.h_r;
    m.row_n = m.row0;
  }
  const int blocks = blk_count(m.K);
  m.row_m = m.mt * (gate_up ? kBlk : kRows);
  const size_t tile = (static_cast<size_t>(m.e) * blk_count(N) + m.row_m / kBlk) * blocks;
  m.s0 = (gate_up ? w.s_gate : w.s_down) + tile;
  m.s1 = gate_up ? w.s_up + tile : m.row_m + kBlk < N ? m.s0 + blocks : m.s0;
  const float* sn = gate_up ? a.sx : (m.shared ? a.sh_s : a.sh_r);
  m.sn = sn + static_cast<size_t>(gate_up && m.shared ? a.max_blocks + m.slot : m.slot) * blocks * a.pitch;
  m.sn_step = a.pitch;
  m.sn_bytes = 4 * static_cast<uint32_t>(m.box);
  return m;
}

}  // namespace
}  // namespace bm
