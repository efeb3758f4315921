// Block-scaled 8-bit products for few tokens: the weights' stream and the number
// of dependent launches bound them.
//
// Y[t][n] = sum_kb sa[t][kb] sw[n/128][kb] sum_{k in kb} a[t][k] w[n][k].  A CTA
// takes 16 weight rows over all of K, its warps the blocks of 128 columns in
// turn.  A lane loads 32 consecutive bytes of each of two rows straight from
// global memory into the A fragments of four warp-level MMAs (m16n8k32, E4M3,
// fp32 accumulate): which columns an MMA takes together is free as long as both
// operands agree, so no byte is moved between lanes.  Eight tokens are the MMA's
// N.  The activations are quantised in the warp that needs them, a block is its
// 32 lanes' four values each.  The blocks' sums are scaled and added in fp32, the
// warps' at the end through shared memory in a fixed order.
#include <cuda_runtime.h>

#include "blk.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace bm {
namespace {

constexpr int kRows = 16;     // weight rows of a CTA
constexpr int kTokens = 8;    // an MMA's N
constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;

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

// Block kb of row `row` of the activations: codes and scale, as quantize4.
__device__ __forceinline__ uint32_t x_block(const BlkX& x, long long row, int kb, int K, int lane, float& scale) {
  const int c = kb * kBlk + 4 * lane;
  if (x.type == kBlkCodes) {
    scale = __ldg(x.s + kb * x.pitch + row);
    return c < K ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(x.x) + row * x.ldx + c)) : 0u;
  }
  float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < K) {
    if (x.type == kFp32) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(x.x) + row * x.ldx + c));
      f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(x.x) + row * x.ldx + c));
      if (x.type == kFp16) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
        f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
      } else {
        f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xFFFF0000u);
        f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xFFFF0000u);
      }
    }
  }
  return quantize4(f, scale);
}

// The B fragments of a block of up to eight tokens: token i's codes by
// code_of(i, scale), for i < n; the others are zeros.  `buf`: 8 x 128 bytes of the
// warp's own.  sa: the scales of the lane's two accumulator columns, tokens
// 2 (lane % 4) and the next.
template <typename CodeOf>
__device__ __forceinline__ void b_fragments(uint32_t* buf, int n, int lane, Piece& b, float (&sa)[2], CodeOf code_of) {
  sa[0] = sa[1] = 0.0f;
  __syncwarp();
  for (int i = 0; i < n; ++i) {
    float s;
    buf[32 * i + lane] = code_of(i, s);
    if (i == 2 * (lane & 3)) sa[0] = s;
    if (i == 2 * (lane & 3) + 1) sa[1] = s;
  }
  __syncwarp();
  b.zero();
  if ((lane >> 2) < n) {
    const uint4* p = reinterpret_cast<const uint4*>(buf + 32 * (lane >> 2) + 8 * (lane & 3));
    b.v[0] = p[0];
    b.v[1] = p[1];
  }
}

struct Shared {
  uint32_t codes[kWarps][kTokens * 32];
  float sums[2][kWarps][kRows * kTokens];
};

// A warp's accumulators to its place; element (row, token) at 8 row + token.
__device__ __forceinline__ void put_sums(float* to, const float (&acc)[4], int lane) {
  const int g = lane >> 2, q = lane & 3;
  *reinterpret_cast<float2*>(to + kTokens * g + 2 * q) = make_float2(acc[0], acc[1]);
  *reinterpret_cast<float2*>(to + kTokens * (g + 8) + 2 * q) = make_float2(acc[2], acc[3]);
}
__device__ __forceinline__ float take_sum(const float (&sums)[kWarps][kRows * kTokens], int i) {
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += sums[w][i];
  return v;
}

__global__ void __launch_bounds__(kThreads) blk_few_linear_kernel(const BlkFewLinearArgs a) {
  __shared__ Shared sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kRows, blocks = blk_count(a.K);
  const float* sw = a.sw + static_cast<size_t>(n0 / kBlk) * blocks;
  ABlock w;
  if (warp < blocks) w.load(a.w, n0, a.N, a.K, warp, lane);
  pdl_wait();
  pdl_launch_dependents();
  for (int t0 = blockIdx.y * kTokens; t0 < a.T; t0 += gridDim.y * kTokens) {
    const int n = min(kTokens, a.T - t0);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = warp; kb < blocks; kb += kWarps) {
      Piece b;
      float sa[2], d[4];
      b_fragments(sm.codes[warp], n, lane, b, sa, [&](int i, float& s) { return x_block(a.x, t0 + i, kb, a.K, lane, s); });
      multiply(d, w, b);
      const float s = __ldg(sw + kb);
      if (kb + kWarps < blocks) w.load(a.w, n0, a.N, a.K, kb + kWarps, lane);
      acc[0] = fmaf(d[0], sa[0] * s, acc[0]);
      acc[1] = fmaf(d[1], sa[1] * s, acc[1]);
      acc[2] = fmaf(d[2], sa[0] * s, acc[2]);
      acc[3] = fmaf(d[3], sa[1] * s, acc[3]);
    }
    put_sums(sm.sums[0][warp], acc, lane);
    __syncthreads();
    if (threadIdx.x < kRows * kTokens) {
      const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
      if (t < n && n0 + r < a.N) store1(a.y_type, a.y, static_cast<size_t>(t0 + t) * a.N + n0 + r, take_sum(sm.sums[0], kTokens * r + t));
    }
    __syncthreads();
    if (t0 + static_cast<int>(gridDim.y) * kTokens < a.T && warp < blocks) w.load(a.w, n0, a.N, a.K, warp, lane);
  }
}

// A tile of the experts' rows.
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
  t.ok = t.some && t.e >= 0 && t.e < a.E && t.rows >= 1 && t.rows <= a.rows && t.row0 >= 0 && t.row0 <= a.T * a.k - t.rows;
  return t;
}

// h = silu(gate) up of 16 columns of a tile's rows, in fp32.
__global__ void __launch_bounds__(kThreads) blk_few_gate_up_kernel(const BlkFewArgs a) {
  __shared__ Shared sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kRows, blocks = blk_count(a.d);
  pdl_wait();
  pdl_launch_dependents();
  const Tile tile = get_tile(a, blockIdx.y);
  if (!tile.ok) {
    if (threadIdx.x == 0 && (tile.some || (blockIdx.x == 0 && routed_tiles(a) == 0))) record_status(a.status, MOE_ERR_INVALID_ARG);
    return;
  }
  const int N = tile.shared ? a.I_shared : a.I;
  if (n0 >= N) return;
  const BlkWeights& m = tile.shared ? a.shared : a.routed;
  const size_t matrix = static_cast<size_t>(tile.e) * N * a.d;
  const size_t sat = (static_cast<size_t>(tile.e) * blk_count(N) + n0 / kBlk) * blocks;
  const size_t first = tile.shared ? static_cast<size_t>(a.T) * a.k : tile.row0;
  const int pitch = max(a.I, a.I_shared);
  for (int r0 = 0; r0 < tile.rows; r0 += kTokens) {
    const int n = min(kTokens, tile.rows - r0);
    float accg[4] = {0.0f, 0.0f, 0.0f, 0.0f}, accu[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = warp; kb < blocks; kb += kWarps) {
      ABlock wg, wu;
      wg.load(m.gate + matrix, n0, N, a.d, kb, lane);
      wu.load(m.up + matrix, n0, N, a.d, kb, lane);
      const float sg = __ldg(m.s_gate + sat + kb), su = __ldg(m.s_up + sat + kb);
      Piece b;
      float sa[2], d[4];
      b_fragments(sm.codes[warp], n, lane, b, sa, [&](int i, float& s) {
        int t = tile.shared ? r0 + i : __ldg(a.perm + tile.row0 + r0 + i) / a.k;
        if (t < 0 || t >= a.T) {  // a malformed permutation
          record_status(a.status, MOE_ERR_INVALID_ARG);
          t = 0;
        }
        return x_block(a.x, t, kb, a.d, lane, s);
      });
      multiply(d, wg, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) accg[i] = fmaf(d[i], sa[i & 1] * sg, accg[i]);
      multiply(d, wu, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) accu[i] = fmaf(d[i], sa[i & 1] * su, accu[i]);
    }
    put_sums(sm.sums[0][warp], accg, lane);
    put_sums(sm.sums[1][warp], accu, lane);
    __syncthreads();
    if (threadIdx.x < kRows * kTokens) {
      const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
      if (t < n && n0 + r < N)
        a.h[(first + r0 + t) * pitch + n0 + r] = blk_swiglu(take_sum(sm.sums[0], kTokens * r + t), take_sum(sm.sums[1], kTokens * r + t));
    }
    __syncthreads();
  }
}

// 16 columns of the experts' outputs, in fp32 rows.
__global__ void __launch_bounds__(kThreads) blk_few_down_kernel(const BlkFewArgs a) {
  __shared__ Shared sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kRows;
  pdl_wait();
  pdl_launch_dependents();
  const Tile tile = get_tile(a, blockIdx.y);
  if (!tile.ok) return;
  const int K = tile.shared ? a.I_shared : a.I, blocks = blk_count(K);
  const BlkWeights& m = tile.shared ? a.shared : a.routed;
  const uint8_t* w = m.down + static_cast<size_t>(tile.e) * a.d * K;
  const float* sw = m.s_down + (static_cast<size_t>(tile.e) * blk_count(a.d) + n0 / kBlk) * blocks;
  const size_t first = tile.shared ? static_cast<size_t>(a.T) * a.k : tile.row0;
  const int pitch = max(a.I, a.I_shared);
  for (int r0 = 0; r0 < tile.rows; r0 += kTokens) {
    const int n = min(kTokens, tile.rows - r0);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = warp; kb < blocks; kb += kWarps) {
      ABlock wd;
      wd.load(w, n0, a.d, K, kb, lane);
      const float s = __ldg(sw + kb);
      Piece b;
      float sa[2], d[4];
      b_fragments(sm.codes[warp], n, lane, b, sa, [&](int i, float& scale) {
        const int c = kb * kBlk + 4 * lane;
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (c < K) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(a.h + (first + r0 + i) * pitch + c));
          f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
        }
        return quantize4(f, scale);
      });
      multiply(d, wd, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[i], sa[i & 1] * s, acc[i]);
    }
    put_sums(sm.sums[0][warp], acc, lane);
    __syncthreads();
    if (threadIdx.x < kRows * kTokens) {
      const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
      if (t < n && n0 + r < a.d) a.ypart[(first + r0 + t) * a.d + n0 + r] = take_sum(sm.sums[0], kTokens * r + t);
    }
    __syncthreads();
  }
}

template <typename A>
cudaError_t launch(int kind, void (*kernel)(A), dim3 grid, cudaStream_t stream, bool pdl, const A& a) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  timer_begin(kind, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  timer_end(kind, stream);
  return e;
}

}  // namespace

cudaError_t launch_blk_few_linear(const BlkFewLinearArgs& a, cudaStream_t stream, bool pdl) {
  const int groups = (a.T + kTokens - 1) / kTokens;
  return launch(kKBlkGemm, blk_few_linear_kernel, dim3((a.N + kRows - 1) / kRows, groups < 65535 ? groups : 65535), stream, pdl, a);
}

cudaError_t launch_blk_few_experts(const BlkFewArgs& a, cudaStream_t stream, bool pdl) {
  const int tiles = a.tiles + (a.I_shared > 0 ? 1 : 0), I = a.I > a.I_shared ? a.I : a.I_shared;
  cudaError_t e = launch(kKBlkGateUp, blk_few_gate_up_kernel, dim3((I + kRows - 1) / kRows, tiles), stream, pdl, a);
  if (e != cudaSuccess) return e;
  e = launch(kKBlkDown, blk_few_down_kernel, dim3((a.d + kRows - 1) / kRows, tiles), stream, pdl, a);
  if (e != cudaSuccess) return e;
  return launch_mx_combine(a.ypart, a.inv_perm, a.w, a.T, a.d, a.k, a.I_shared > 0, a.y, a.status, a.num_sms, stream);
}

}  // namespace bm
