// Block-scaled 8-bit products for few tokens: the weights' stream and the number
// of dependent launches bound them.
//
// Y[t][n] = sum_kb sa[t][kb] sw[n/128][kb] sum_{k in kb} a[t][k] w[n][k].  A CTA
// takes 16 weight rows over all of K, its warps the blocks of 128 columns in
// turn.  A lane loads 32 consecutive bytes of each of two rows straight from
// global memory into the A fragments of four warp-level MMAs (m16n8k32, E4M3,
// fp32 accumulate): which columns an MMA takes together is free as long as both
// operands agree, so no byte is moved between lanes.  Eight tokens are an MMA's N.
// Linear products: one token is quantised in the warp that needs the block (its 32
// lanes' four values each), up to 32 tokens come as codes, in groups of eight, a
// lane's bytes of its column's token being the B fragments.  Experts: up to eight
// tokens, bf16 or codes, and h, quantised likewise in the warp that needs them.  The
// blocks' sums are scaled and added in fp32, the warps' at the end through shared
// memory in a fixed order.
#include <cuda_runtime.h>

#include "blk.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace bm {
namespace {

constexpr int kRows = kBlkFewRows;  // weight rows of a CTA
constexpr int kTokens = 8;    // an MMA's N
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// A warp's blocks whose weights are in flight together.  Two CTAs an SM hold 128
// KB of them: with 16 warps of one block each (and one CTA's registers an SM) one
// token's expert layer took 13.6 us, 1 x 8192 -> 8192 21.8.
constexpr int kDepth = 4;       // linear
constexpr int kDepthGU = 2;     // gate/up: of both matrices
// The down product has fewer CTAs than there are SMs and as many (expert, block)
// pairs in each as one token has: 16 warps of three at a time.
constexpr int kWarpsDown = 16;
constexpr int kDepthDown = 3;

// D += A B, m16n8k32, E4M3 operands four to a register (lowest index in the
// lowest byte), fp32 accumulators; g = lane/4, q = lane%4:
//   a0 (row g, k 4q..)  a1 (row g+8, k 4q..)  a2 (row g, k 16+4q..)  a3 (row g+8, k 16+4q..)
//   b0 (k 4q.., col g)  b1 (k 16+4q.., col g)
//   d0, d1 (row g, cols 2q, 2q+1)  d2, d3 (row g+8, ...)
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 bytes of one row: what a lane takes of a block of 128 columns.
struct Piece {
  uint4 v[2];
  __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0, 0, 0, 0); }
  // byte `c` of a row of K bytes, 16 bytes at a time
  __device__ __forceinline__ void load(const uint8_t* row, int c, int K) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (c + 16 * i < K) {
        const uint4* p = reinterpret_cast<const uint4*>(row + c + 16 * i);
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                     : "l"(p));
      }
    }
  }
  __device__ __forceinline__ uint32_t word(int j) const {
    const uint4& u = v[j >> 2];
    return (j & 3) == 0 ? u.x : (j & 3) == 1 ? u.y : (j & 3) == 2 ? u.z : u.w;
  }
};
// A lane's share of 16 weight rows x 128 columns.
struct ABlock {
  Piece r0, r8;
  // rows n0 + g and n0 + g + 8 of w [N][K]
  __device__ __forceinline__ void load(const uint8_t* w, int n0, int N, int K, int kb, int lane) {
    const int n = n0 + (lane >> 2), c = kb * kBlk + 32 * (lane & 3);
    if (n < N) r0.load(w + static_cast<size_t>(n) * K, c, K); else r0.zero();
    if (n + 8 < N) r8.load(w + static_cast<size_t>(n + 8) * K, c, K); else r8.zero();
  }
};
__device__ __forceinline__ void multiply(float (&d)[4], const ABlock& a, const Piece& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    mma_e4m3(d, a.r0.word(2 * j), a.r8.word(2 * j), a.r0.word(2 * j + 1), a.r8.word(2 * j + 1), b.word(2 * j),
             b.word(2 * j + 1));
}

// A lane's four values (4 lane ..) of a block: the block's scale, and the codes.
__device__ __forceinline__ uint32_t quantize4(const float (&f)[4], float& scale) {
  scale = blk_scale(__reduce_max_sync(0xffffffffu, largest_bits(f)));
  const float inv = blk_inverse(scale);
  return f32x4_to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
}

// A lane's share of a block of 128 columns of one row of activations: as loaded, and as codes and the block's scale.
template <int kType>
struct XBlock {
  uint32_t v[kType == kFp32 ? 4 : kType == kBlkCodes ? 1 : 2];
  float s;  // codes: their scale
  __device__ __forceinline__ void load(const BlkX& x, long long row, int kb, int K, int lane) {
    const int c = kb * kBlk + 4 * lane;
    const char* p = static_cast<const char*>(x.x) + (row * x.ldx + c) * (kType == kFp32 ? 4 : kType == kBlkCodes ? 1 : 2);
    const bool in = c < K;
    if constexpr (kType == kFp32) {
      const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else if constexpr (kType == kBlkCodes) {
      v[0] = in ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
      s = __ldg(x.s + kb * x.pitch + row);
    } else {
      const uint2 u = in ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
      v[0] = u.x; v[1] = u.y;
    }
  }
  __device__ __forceinline__ uint32_t codes(float& scale) const {
    if constexpr (kType == kBlkCodes) {
      scale = s;
      return v[0];
    } else if constexpr (kType == kFp32) {
      const float f[4] = {__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3])};
      return quantize4(f, scale);
    } else if constexpr (kType == kFp16) {
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v[0])), b = __half22float2(*reinterpret_cast<const __half2*>(&v[1]));
      const float f[4] = {a.x, a.y, b.x, b.y};
      return quantize4(f, scale);
    } else {
      const float f[4] = {__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u), __uint_as_float(v[1] << 16),
                          __uint_as_float(v[1] & 0xFFFF0000u)};
      return quantize4(f, scale);
    }
  }
};

// A warp's B fragments of a block of up to eight tokens, a column each: put() for
// the columns that there are, then take().  A column that is put again (the same
// codes: an expert that a token takes twice) adds its scale.  `buf`: 8 x 128 bytes of the warp's own.
struct Columns {
  uint32_t* buf;
  int lane;
  uint32_t there = 0;            // columns put
  float sa[2] = {0.0f, 0.0f};    // scales of the lane's two accumulator columns, 2 (lane % 4) and the next
  __device__ __forceinline__ Columns(uint32_t* b, int l) : buf(b), lane(l) { __syncwarp(); }
  __device__ __forceinline__ void put(int column, uint32_t codes, float scale) {
    buf[32 * column + lane] = codes;
    there |= 1u << column;
    if (column == 2 * (lane & 3)) sa[0] += scale;
    if (column == 2 * (lane & 3) + 1) sa[1] += scale;
  }
  __device__ __forceinline__ void take(Piece& b) const {
    __syncwarp();
    b.zero();
    if (there >> (lane >> 2) & 1) {
      const uint4* p = reinterpret_cast<const uint4*>(buf + 32 * (lane >> 2) + 8 * (lane & 3));
      b.v[0] = p[0];
      b.v[1] = p[1];
    }
  }
};

template <int kW, int kSums>
struct Shared {
  uint32_t codes[kW][kTokens * 32];
  float sums[kSums][kW][kRows * kTokens];
};

// A warp's accumulators to its place; element (row, token) at 8 row + token.
__device__ __forceinline__ void put_sums(float* to, const float (&acc)[4], int lane) {
  const int g = lane >> 2, q = lane & 3;
  *reinterpret_cast<float2*>(to + kTokens * g + 2 * q) = make_float2(acc[0], acc[1]);
  *reinterpret_cast<float2*>(to + kTokens * (g + 8) + 2 * q) = make_float2(acc[2], acc[3]);
}
template <int kW>
__device__ __forceinline__ float take_sum(const float (&sums)[kW][kRows * kTokens], int i) {
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < kW; ++w) v += sums[w][i];
  return v;
}
__device__ __forceinline__ void add(float (&acc)[4], const float (&d)[4], float s0, float s1) {
  acc[0] = fmaf(d[0], s0, acc[0]);
  acc[1] = fmaf(d[1], s1, acc[1]);
  acc[2] = fmaf(d[2], s0, acc[2]);
  acc[3] = fmaf(d[3], s1, acc[3]);
}

// One token whose activations are quantised here, each block by the warp that
// needs it.  (For more tokens every CTA would do that again: 4 x 8192 -> 8192 took
// 26.7 us, quantised by a kernel of its own 16.)
template <int kType>
__global__ void __launch_bounds__(kThreads, 2) blk_one_linear_kernel(const BlkFewLinearArgs a) {
  __shared__ Shared<kWarps, 1> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kRows, blocks = blk_count(a.K);
  const float* sw = a.sw + static_cast<size_t>(n0 / kBlk) * blocks;
  ABlock w[kDepth];
  float s[kDepth];
  auto load = [&](int kb, int to) {
    if (kb >= blocks) return;
    w[to].load(a.w, n0, a.N, a.K, kb, lane);
    s[to] = __ldg(sw + kb);
  };
#pragma unroll
  for (int j = 0; j < kDepth; ++j) load(warp + j * kWarps, j);
  pdl_wait();
  pdl_launch_dependents();
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb0 = warp; kb0 < blocks; kb0 += kDepth * kWarps) {
#pragma unroll
    for (int j = 0; j < kDepth; ++j) {
      const int kb = kb0 + j * kWarps;
      if (kb >= blocks) break;
      XBlock<kType> x;
      x.load(a.x, 0, kb, a.K, lane);
      Columns c(sm.codes[warp], lane);
      float sx;
      const uint32_t q = x.codes(sx);
      c.put(0, q, sx);
      Piece b;
      float d[4];
      c.take(b);
      multiply(d, w[j], b);
      add(acc, d, c.sa[0] * s[j], c.sa[1] * s[j]);
      load(kb + kDepth * kWarps, j);
    }
  }
  put_sums(sm.sums[0][warp], acc, lane);
  __syncthreads();
  if (threadIdx.x < kRows && n0 + threadIdx.x < a.N)
    store1(a.y_type, a.y, static_cast<size_t>(n0) + threadIdx.x, take_sum(sm.sums[0], kTokens * threadIdx.x));
}

// Up to 8 kGroups tokens that are quantised already: a lane's 32 bytes of its
// column's token are the B fragments, as its bytes of two rows are the A fragments.
// (Four groups do not quite fit the 128 registers of two CTAs an SM: 108 bytes go through the stack.)
template <int kGroups>
__global__ void __launch_bounds__(kThreads, 2) blk_few_linear_kernel(const BlkFewLinearArgs a) {
  __shared__ float sums[kGroups][kWarps][kRows * kTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kRows, blocks = blk_count(a.K);
  const float* sw = a.sw + static_cast<size_t>(n0 / kBlk) * blocks;
  constexpr int kHere = kGroups > 1 ? kDepth / 2 : kDepth;  // the tokens' registers take the place of weights
  ABlock w[kHere];
  float s[kHere];
  auto load = [&](int kb, int to) {
    if (kb >= blocks) return;
    w[to].load(a.w, n0, a.N, a.K, kb, lane);
    s[to] = __ldg(sw + kb);
  };
#pragma unroll
  for (int j = 0; j < kHere; ++j) load(warp + j * kWarps, j);
  pdl_wait();
  pdl_launch_dependents();
  float acc[kGroups][4];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.0f;
  const int g8 = lane >> 2, q2 = 2 * (lane & 3);
  const uint8_t* x = static_cast<const uint8_t*>(a.x.x);
  for (int kb0 = warp; kb0 < blocks; kb0 += kHere * kWarps) {
#pragma unroll
    for (int j = 0; j < kHere; ++j) {
      const int kb = kb0 + j * kWarps;
      if (kb >= blocks) break;
      Piece b[kGroups];
      float2 sa[kGroups];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int t = kTokens * g + g8;
        if (t < a.T) b[g].load(x + static_cast<size_t>(t) * a.K, kb * kBlk + 32 * (lane & 3), a.K); else b[g].zero();
        // (the scales' rows are padded to a multiple of four: a pair that starts at a token is there)
        const int t2 = kTokens * g + q2;
        sa[g] = t2 < a.T ? __ldg(reinterpret_cast<const float2*>(a.x.s + kb * a.x.pitch + t2)) : make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        float d[4];
        multiply(d, w[j], b[g]);
        add(acc[g], d, sa[g].x * s[j], sa[g].y * s[j]);
      }
      load(kb + kHere * kWarps, j);
    }
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) put_sums(sums[g][warp], acc[g], lane);
  __syncthreads();
  const int r = threadIdx.x & 15;
  if (n0 + r < a.N)
    for (int t = threadIdx.x >> 4; t < min(a.T, kTokens * kGroups); t += kThreads / kRows)
      store1(a.y_type, a.y, static_cast<size_t>(t) * a.N + n0 + r, take_sum(sums[t / kTokens], kTokens * r + t % kTokens));
}

// ------------------------------------------------------------------ experts
// Two launches after the routing.  gate/up: a CTA 16 columns of h of one tile (at
// most eight rows), fp32 h to memory.  down: a CTA
// 16 columns of Y over all experts: its warps take the (expert, block of h) pairs
// in turn, quantise h, and add each token's column with its routing weight, so that
// nothing is added up between CTAs (but those of a cluster, which share the pairs
// where d alone makes few CTAs: one token, d = 320, 8 experts 7.6 -> 7.0 us).  The gate/up kernel lets the down kernel start
// after its own wait, when the routing has completed: the down kernel asks for its
// first weights before it waits for h.

struct Tile {
  int e, row0, rows;
  bool shared, ok, some;
};
__device__ __forceinline__ int routed_tiles(const BlkFewArgs& a) {
  const int nb = *reinterpret_cast<const volatile int32_t*>(a.num_blocks);
  return nb < 1 || nb > a.tiles ? 0 : nb;
}
// i: the shared expert's first (where there is one), then the block map's
__device__ __forceinline__ Tile get_tile(const BlkFewArgs& a, int i) {
  Tile t{};
  if (a.I_shared > 0 && i == 0) {
    t.shared = t.ok = t.some = true;
    t.rows = a.T;
    return t;
  }
  if (a.I_shared > 0) --i;
  const volatile int32_t* b = a.block_map + 3 * i;
  t.e = b[0];
  t.row0 = b[1];
  t.rows = b[2];
  t.some = i < routed_tiles(a);
  t.ok = t.some && t.e >= 0 && t.e < a.E && t.rows >= 1 && t.rows <= kTokens && t.row0 >= 0 && t.row0 <= a.T * a.k - t.rows;
  return t;
}

template <int kType>
__global__ void __launch_bounds__(kThreads, 2) blk_few_gate_up_kernel(const BlkFewArgs a) {
  __shared__ Shared<kWarps, 2> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kRows, blocks = blk_count(a.d);
  const bool early = a.I_shared > 0 && blockIdx.y == 0;  // the shared expert's weights are known before the wait
  if (!early) pdl_wait();
  const Tile tile = get_tile(a, blockIdx.y);
  if (!tile.ok) {
    pdl_launch_dependents();
    if (threadIdx.x == 0 && (tile.some || (blockIdx.x == 0 && routed_tiles(a) == 0))) record_status(a.status, MOE_ERR_INVALID_ARG);
    return;
  }
  const int N = tile.shared ? a.I_shared : a.I;
  if (n0 >= N) {
    if (early) pdl_wait();
    pdl_launch_dependents();
    return;
  }
  const BlkWeights& m = tile.shared ? a.shared : a.routed;
  const size_t matrix = static_cast<size_t>(tile.e) * N * a.d;
  const size_t sat = (static_cast<size_t>(tile.e) * blk_count(N) + n0 / kBlk) * blocks;
  const size_t first = tile.shared ? static_cast<size_t>(a.T) * a.k : tile.row0;
  const int pitch = max(a.I, a.I_shared);
  ABlock wg[kDepthGU], wu[kDepthGU];
  float sg[kDepthGU], su[kDepthGU];
  auto load = [&](int kb, int to) {
    if (kb >= blocks) return;
    wg[to].load(m.gate + matrix, n0, N, a.d, kb, lane);
    wu[to].load(m.up + matrix, n0, N, a.d, kb, lane);
    sg[to] = __ldg(m.s_gate + sat + kb);
    su[to] = __ldg(m.s_up + sat + kb);
  };
#pragma unroll
  for (int j = 0; j < kDepthGU; ++j) load(warp + j * kWarps, j);
  if (early) pdl_wait();
  pdl_launch_dependents();
  int mine = lane;  // the token of row `lane`
  if (!tile.shared) {
    mine = lane < tile.rows ? __ldg(a.perm + tile.row0 + lane) / a.k : 0;
    if (mine < 0 || mine >= a.T) {  // a malformed permutation
      record_status(a.status, MOE_ERR_INVALID_ARG);
      mine = 0;
    }
  }
  float accg[4] = {0.0f, 0.0f, 0.0f, 0.0f}, accu[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb0 = warp; kb0 < blocks; kb0 += kDepthGU * kWarps) {
#pragma unroll
    for (int j = 0; j < kDepthGU; ++j) {
      const int kb = kb0 + j * kWarps;
      if (kb >= blocks) break;
      Columns c(sm.codes[warp], lane);
      for (int i0 = 0; i0 < tile.rows; i0 += 2) {  // two rows' loads in flight
        XBlock<kType> x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (i0 + i < tile.rows) x[i].load(a.x, __shfl_sync(0xffffffffu, mine, i0 + i), kb, a.d, lane);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i0 + i >= tile.rows) break;
          float sx;
          const uint32_t q = x[i].codes(sx);
          c.put(i0 + i, q, sx);
        }
      }
      Piece b;
      float d[4];
      c.take(b);
      multiply(d, wg[j], b);
      add(accg, d, c.sa[0] * sg[j], c.sa[1] * sg[j]);
      multiply(d, wu[j], b);
      add(accu, d, c.sa[0] * su[j], c.sa[1] * su[j]);
      load(kb + kDepthGU * kWarps, j);
    }
  }
  put_sums(sm.sums[0][warp], accg, lane);
  put_sums(sm.sums[1][warp], accu, lane);
  __syncthreads();
  if (threadIdx.x < kRows * kTokens) {
    const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
    if (t < tile.rows && n0 + r < N)
      a.h[(first + t) * pitch + n0 + r] = blk_swiglu(take_sum(sm.sums[0], kTokens * r + t), take_sum(sm.sums[1], kTokens * r + t));
  }
}

constexpr int kMaxRouted = kTokens * kMaxK;  // tiles and assignments of the routed experts at most
struct SharedDown {
  Shared<kWarpsDown, 1> p;
  int e[kMaxRouted], row0[kMaxRouted], rows[kMaxRouted];  // of a routed tile; no rows: malformed
  int token[kMaxRouted];                                  // of an assignment's row; -1: malformed
  float w[kMaxRouted];
  float sums[kRows * kTokens];                            // of the CTA, for the cluster's first
};
__global__ void __launch_bounds__(32 * kWarpsDown) blk_few_down_kernel(const BlkFewArgs a) {
  __shared__ SharedDown sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.split));
  const int n0 = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.split)) * kRows, A = a.T * a.k;
  const int u_first = rank * kWarpsDown + warp, u_step = a.split * kWarpsDown;  // this warp's units
  const int blocks_r = blk_count(a.I), blocks_s = a.I_shared > 0 ? blk_count(a.I_shared) : 0;
  // (the routing has completed: see above)
  const int nb = routed_tiles(a);
  for (int i = threadIdx.x; i < max(nb, A); i += 32 * kWarpsDown) {
    if (i < nb) {
      const Tile t = get_tile(a, i + (a.I_shared > 0 ? 1 : 0));
      sm.e[i] = t.e;
      sm.row0[i] = t.row0;
      sm.rows[i] = t.ok ? t.rows : 0;
    }
    if (i < A) {
      const int at = __ldg(a.perm + i);
      const bool ok = at >= 0 && at < A;
      sm.token[i] = ok ? at / a.k : -1;
      sm.w[i] = ok ? __ldg(a.w + at) : 0.0f;
      if (!ok) record_status(a.status, MOE_ERR_INVALID_ARG);
    }
  }
  __syncthreads();
  const int units = blocks_s + nb * blocks_r;
  ABlock w[kDepthDown];
  float sw[kDepthDown];
  auto load = [&](int u, ABlock& to, float& s) {
    if (u >= units) return;
    const bool shared = u < blocks_s;
    const int i = shared ? 0 : (u - blocks_s) / blocks_r, kb = shared ? u : u - blocks_s - i * blocks_r;
    const int e = shared ? 0 : sm.e[i], K = shared ? a.I_shared : a.I;
    if (!shared && sm.rows[i] == 0) return;
    const BlkWeights& m = shared ? a.shared : a.routed;
    to.load(m.down + static_cast<size_t>(e) * a.d * K, n0, a.d, K, kb, lane);
    s = __ldg(m.s_down + (static_cast<size_t>(e) * blk_count(a.d) + n0 / kBlk) * blk_count(K) + kb);
  };
#pragma unroll
  for (int j = 0; j < kDepthDown; ++j) load(u_first + j * u_step, w[j], sw[j]);
  pdl_wait();
  pdl_launch_dependents();
  const int pitch = max(a.I, a.I_shared);
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  // h's values of row r of unit u
  auto ask = [&](int u, int r) {
    if (u >= units) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const bool shared = u < blocks_s;
    const int i = shared ? 0 : (u - blocks_s) / blocks_r, kb = shared ? u : u - blocks_s - i * blocks_r;
    const int K = shared ? a.I_shared : a.I, rows = shared ? a.T : sm.rows[i], row0 = shared ? A : sm.row0[i];
    const int c = kb * kBlk + 4 * lane;
    if (r >= rows || c >= K) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    return __ldcg(reinterpret_cast<const float4*>(a.h + (row0 + r) * static_cast<size_t>(pitch) + c));
  };
  auto take = [&](int u, const ABlock& m, float s, float4 v) {  // v: the first row's
    const bool shared = u < blocks_s;
    const int i = shared ? 0 : (u - blocks_s) / blocks_r;
    const int rows = shared ? a.T : sm.rows[i];
    if (rows == 0) return;
    Columns c(sm.p.codes[warp], lane);
    for (int r = 0; r < rows; ++r) {
      const float4 next = r + 1 < rows ? ask(u, r + 1) : v;
      const int at = shared ? 0 : sm.row0[i] + r;
      const int t = shared ? r : sm.token[at];
      const float f[4] = {v.x, v.y, v.z, v.w};
      float sx;
      const uint32_t q = quantize4(f, sx);
      if (t >= 0) c.put(t, q, sx * s * (shared ? 1.0f : sm.w[at]));
      v = next;
    }
    Piece b;
    float d[4];
    c.take(b);
    multiply(d, m, b);
    add(acc, d, c.sa[0], c.sa[1]);
  };
  for (int u0 = u_first; u0 < units; u0 += kDepthDown * u_step) {
    float4 v[kDepthDown];
#pragma unroll
    for (int j = 0; j < kDepthDown; ++j) v[j] = ask(u0 + j * u_step, 0);
#pragma unroll
    for (int j = 0; j < kDepthDown; ++j) {
      const int u = u0 + j * u_step;
      if (u >= units) break;
      take(u, w[j], sw[j], v[j]);
      load(u + kDepthDown * u_step, w[j], sw[j]);
    }
  }
  put_sums(sm.p.sums[0][warp], acc, lane);
  __syncthreads();
  const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
  const bool mine = threadIdx.x < kRows * kTokens;
  float v = mine ? take_sum(sm.p.sums[0], kTokens * r + t) : 0.0f;
  if (a.split > 1) {  // the CTAs' sums, in their order
    if (mine) sm.sums[threadIdx.x] = v;
    cluster_arrive_release();
    cluster_wait();
    if (mine && rank == 0)
      for (int p = 1; p < a.split; ++p) v += ld_shared_cluster_f1(mapa_shared(&sm.sums[threadIdx.x], p));
    cluster_arrive_release();  // (the others' shared memory has been read)
    cluster_wait();
  }
  if (mine && rank == 0 && t < a.T && n0 + r < a.d)
    a.y[static_cast<size_t>(t) * a.d + n0 + r] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <typename A>
cudaError_t launch(int kind, void (*kernel)(A), dim3 grid, int threads, int cluster, cudaStream_t stream, bool pdl, const A& a) {
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  timer_begin(kind, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  timer_end(kind, stream);
  return e;
}

}  // namespace

cudaError_t launch_blk_few_linear(const BlkFewLinearArgs& a, cudaStream_t stream, bool pdl) {
  const auto kernel = a.x.type == kBf16   ? blk_one_linear_kernel<kBf16>
                      : a.x.type == kFp16 ? blk_one_linear_kernel<kFp16>
                      : a.x.type == kFp32 ? blk_one_linear_kernel<kFp32>
                      : a.T <= kTokens    ? blk_few_linear_kernel<1>
                      : a.T <= 2 * kTokens ? blk_few_linear_kernel<2>
                                           : blk_few_linear_kernel<4>;
  return launch(kKBlkGemm, kernel, dim3((a.N + kRows - 1) / kRows), kThreads, 1, stream, pdl, a);
}

cudaError_t launch_blk_few_experts(const BlkFewArgs& a, cudaStream_t stream, bool pdl) {
  const int tiles = a.tiles + (a.I_shared > 0 ? 1 : 0), I = a.I > a.I_shared ? a.I : a.I_shared;
  const auto gate_up = a.x.type == kBlkCodes ? blk_few_gate_up_kernel<kBlkCodes> : blk_few_gate_up_kernel<kBf16>;
  const cudaError_t e = launch(kKBlkGateUp, gate_up, dim3((I + kRows - 1) / kRows, tiles), kThreads, 1, stream, pdl, a);
  if (e != cudaSuccess) return e;
  return launch(kKBlkDown, blk_few_down_kernel, dim3((a.d + kRows - 1) / kRows * a.split), 32 * kWarpsDown, a.split, stream, pdl, a);
}

}  // namespace bm
