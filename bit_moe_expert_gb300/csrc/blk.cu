// Block-scaled 8-bit floating point: quantisation, its inverse, and the RMS norm
// with the residual's addition (include/moe_blk.h).
#include <cuda_runtime.h>

#include <type_traits>

#include "blk.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace bm {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ activations
// A warp takes 256 columns (eight a lane, a block in either half) of four
// neighbouring rows, whose scales of a block are neighbours too: one 16-byte
// store.  Bound by memory.
//
// The products read weights before they wait for the kernel before them, so what
// may write weights lets no kernel start before it has completed; this one writes
// activations and starts its successor at once.
constexpr int kRowsAWarp = 4;
struct Patch {
  int row, col;
  __device__ __forceinline__ Patch(int K) {
    const int segs = (K + 255) / 256;
    const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    row = unit / segs * kRowsAWarp;
    col = unit % segs * 256 + 8 * (threadIdx.x & 31);
  }
};

template <int kType>
__global__ void __launch_bounds__(kThreads)
    blk_quantize_kernel(const void* __restrict__ X, int rows, int K, long long ldx, uint8_t* __restrict__ q,
                        float* __restrict__ s) {
  const Patch at(K);
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  if (at.row >= rows) return;
  Load8<kType> x[kRowsAWarp];
#pragma unroll
  for (int i = 0; i < kRowsAWarp; ++i) {
    if (at.row + i < rows && at.col < K)
      x[i].load(static_cast<const char*>(X) + (at.row + i) * static_cast<size_t>(ldx) * (kType == kFp32 ? 4 : 2), at.col);
    else
      x[i].zero();
  }
  float scale[kRowsAWarp];
#pragma unroll
  for (int i = 0; i < kRowsAWarp; ++i) {
    float f[8];
    x[i].floats(f);
    scale[i] = blk_scale(half_warp_max(largest_bits(f)));
    if (at.row + i < rows && at.col < K)
      *reinterpret_cast<uint2*>(q + static_cast<size_t>(at.row + i) * K + at.col) = blk_codes8(f, blk_inverse(scale[i]));
  }
  if ((lane & 15) == 0 && at.col < K)
    *reinterpret_cast<float4*>(s + static_cast<size_t>(at.col / kBlk) * blk_scale_rows(rows) + at.row) =
        make_float4(scale[0], scale[1], scale[2], scale[3]);
}

template <int kType>
__global__ void __launch_bounds__(kThreads)
    blk_dequant_kernel(const uint8_t* __restrict__ q, const float* __restrict__ s, int rows, int K, void* __restrict__ X) {
  const Patch at(K);
  pdl_wait();
  if (at.row >= rows || at.col >= K) return;
  uint2 code[kRowsAWarp];
#pragma unroll
  for (int i = 0; i < kRowsAWarp; ++i)
    code[i] = at.row + i < rows ? __ldg(reinterpret_cast<const uint2*>(q + static_cast<size_t>(at.row + i) * K + at.col))
                                : make_uint2(0, 0);
  const float4 s4 = __ldg(reinterpret_cast<const float4*>(s + static_cast<size_t>(at.col / kBlk) * blk_scale_rows(rows) + at.row));
  const float scale[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
  for (int i = 0; i < kRowsAWarp; ++i) {
    if (at.row + i >= rows) break;
    float f[8], lo[4], hi[4];
    e4m3x4_to_f32(code[i].x, lo);
    e4m3x4_to_f32(code[i].y, hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = lo[j] * scale[i];
      f[4 + j] = hi[j] * scale[i];
    }
    store8(kType, X, static_cast<size_t>(at.row + i) * K + at.col, f);
  }
}

// ------------------------------------------------------------------ weights
// One CTA per block of 128 x 128, all of it in registers between the maximum and
// the codes: a half warp per row and pass, eight passes of 16 rows.  Lets no
// kernel start early (its result may be weights).
constexpr int kPasses = 128 / (kThreads / 16);
struct Block {
  int row0, r, col;   // first row of the block, this thread's first row in it, its first column
  size_t matrix;      // rows before the matrix
  size_t scale;       // place of the scale
  __device__ __forceinline__ Block(int N, int K) {
    const int kb = (K + kBlk - 1) / kBlk, nb = (N + kBlk - 1) / kBlk;
    const unsigned b = blockIdx.x;
    const int e = b / (static_cast<unsigned>(nb) * kb), i = b - static_cast<unsigned>(e) * nb * kb;
    row0 = i / kb * kBlk;
    r = threadIdx.x >> 4;
    col = i % kb * kBlk + 8 * (threadIdx.x & 15);
    matrix = static_cast<size_t>(e) * N;
    scale = b;
  }
};

template <int kType>
__global__ void __launch_bounds__(kThreads)
    blk_quantize_weights_kernel(const void* __restrict__ W, int N, int K, uint8_t* __restrict__ q, float* __restrict__ s) {
  __shared__ uint32_t s_max[kThreads / 32];
  const Block at(N, K);
  pdl_wait();
  Load8<kType> x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int n = at.row0 + at.r + i * (kThreads / 16);
    if (n < N && at.col < K)
      x[i].load(static_cast<const char*>(W) + (at.matrix + n) * K * (kType == kFp32 ? 4 : 2), at.col);
    else
      x[i].zero();
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    float f[8];
    x[i].floats(f);
    a = max(a, largest_bits(f));
  }
  a = __reduce_max_sync(0xffffffffu, a);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) a = max(a, s_max[i]);
  const float scale = blk_scale(a), inv = blk_inverse(scale);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int n = at.row0 + at.r + i * (kThreads / 16);
    float f[8];
    x[i].floats(f);
    if (n < N && at.col < K) *reinterpret_cast<uint2*>(q + (at.matrix + n) * K + at.col) = blk_codes8(f, inv);
  }
  if (threadIdx.x == 0) s[at.scale] = scale;
}

template <int kType>
__global__ void __launch_bounds__(kThreads)
    blk_dequant_weights_kernel(const uint8_t* __restrict__ q, const float* __restrict__ s, int N, int K, void* __restrict__ W) {
  const Block at(N, K);
  pdl_wait();
  const float scale = __ldg(s + at.scale);
  uint2 code[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int n = at.row0 + at.r + i * (kThreads / 16);
    code[i] = n < N && at.col < K ? __ldg(reinterpret_cast<const uint2*>(q + (at.matrix + n) * K + at.col)) : make_uint2(0, 0);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int n = at.row0 + at.r + i * (kThreads / 16);
    if (n >= N || at.col >= K) continue;
    float f[8], lo[4], hi[4];
    e4m3x4_to_f32(code[i].x, lo);
    e4m3x4_to_f32(code[i].y, hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = lo[j] * scale;
      f[4 + j] = hi[j] * scale;
    }
    store8(kType, W, (at.matrix + n) * K + at.col, f);
  }
}

// ------------------------------------------------------------------ RMS norm
// One CTA per row, the row in registers (eight columns a thread and chunk: a
// block of 128 columns is a half warp).  Everything is fp32; what has to be more
// exact is a pair (hi, lo) of fp32 numbers whose sum is the value:
//   the sum of squares   eight at a time in fp32, the sums of eight added as
//                        pairs (the addition's error by Knuth's two-sum): the
//                        errors of about 2^-24 of each sum of eight average
//                        out, to some 2^-28 of a row of 2048;
//   1 / sqrt(mean + eps) the hardware's estimate y0 and one Newton step, y0 (1 +
//                        (1 - v y0^2) / 2), whose residual is formed with fused
//                        multiply-adds.
// y = r hi gamma is then off by less than 2^-21 of itself.  Where the codes of y
// (1 - 2^-21) and y (1 + 2^-21) differ, one value in some 10^5, the thread's
// values are evaluated in 64 bits; the block's scale likewise.  (fp64 for all
// would bound the kernel: an SM does two operations a clock.)
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return Pair{s.hi, s.lo + (a.lo + b.lo)};
}
// over n neighbouring lanes, n a power of two; the same bits in all of them (the error of an addition is exact)
__device__ __forceinline__ Pair lanes_sum(Pair a, int n) {
#pragma unroll
  for (int i = 1; i < 32; i *= 2) {
    if (i == n) break;
    a = add(a, Pair{__shfl_xor_sync(0xffffffffu, a.hi, i), __shfl_xor_sync(0xffffffffu, a.lo, i)});
  }
  return a;
}
// 1 / sqrt(sum / d + eps)
__device__ __forceinline__ Pair inverse_root(Pair sum, float d, float eps) {
  const float q = __fdiv_rn(sum.hi, d);
  const float q2 = (fmaf(-q, d, sum.hi) + sum.lo) / d;
  Pair v = two_sum(q, eps);
  v.lo += q2;
  const float y = rsqrtf(v.hi);
  const float p = __fmul_rn(y, y), pe = fmaf(y, y, -p);
  float t = fmaf(-v.hi, p, 1.0f);  // 1 - v y^2, small
  t = fmaf(-v.hi, pe, t);
  t = fmaf(-v.lo, p, t);
  const float c = 0.5f * y * t;
  const float hi = y + c;
  return Pair{hi, c - (hi - y)};
}

// The float nearest to x that rounds to fewer bits as x does: cut towards zero, the last bit set where that cut something.
__device__ __forceinline__ float odd_float(double x) {
  const float f = __double2float_rz(x);
  return static_cast<double>(f) == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// The sums of eight bf16 or fp16 values each.
template <int kType>
__device__ __forceinline__ uint4 add_packed(uint4 a, uint4 b) {
  auto add2 = [](uint32_t x, uint32_t y) {
    uint32_t r;
    if constexpr (kType == kBf16)
      asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    else
      asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
  };
  return make_uint4(add2(a.x, b.x), add2(a.y, b.y), add2(a.z, b.z), add2(a.w, b.w));
}

enum Residual { kNone, kSame, kWide };
struct NormArgs {
  const void* x;
  const void* residual;
  void* residual_out;
  const void* gamma;
  void* y;
  uint8_t* q;
  float* s;
  long long ldx;
  float eps;
  int T, d, gamma_fp32, y_type;
};

constexpr float kNormError = 4.76837158e-7f;  // 2^-21

// y in 64 bits.
__device__ __forceinline__ double exact_value(float r, float g, Pair inv) {
  return static_cast<double>(r) * (static_cast<double>(inv.hi) + static_cast<double>(inv.lo)) * static_cast<double>(g);
}

// A warp has 256 kChunks neighbouring columns, a chunk of 256 after another: from a
// lane's first column on all places are constants apart.
template <int kType, int kResidual, int kChunks>
__global__ void __launch_bounds__(1024)
    rmsnorm_kernel(const NormArgs a) {
  constexpr int kRType = kResidual == kWide ? kFp32 : kType;
  constexpr int kStep = 256;
  __shared__ Pair s_sum[32];
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  const int c = (threadIdx.x >> 5) * kChunks * kStep + 8 * lane;
  const size_t at = blockIdx.x * static_cast<size_t>(a.d) + c;  // of the lane's first column in what has d columns
  constexpr bool kGammaEarly = kChunks == 1;  // registers: an SM holds more rows without (16384 rows of 2048: 59.5 / 57.7 us with the inverse)
  float g[kGammaEarly ? kChunks : 1][8], r[kChunks][8];
  auto load_gamma = [&](int i, float (&to)[8]) {
    if (a.gamma_fp32) {
      Load8<kFp32> v;
      if (c + i * kStep < a.d) v.load(a.gamma, c + i * kStep); else v.zero();
      v.floats(to);
    } else {
      Load8<kBf16> v;
      if (c + i * kStep < a.d) v.load(a.gamma, c + i * kStep); else v.zero();
      v.floats(to);
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  // (the residual, and X where Y is in its place, are read and written by each of several such kernels in a row, whose
  // CTAs share SMs: no read-only loads)
  {
    const char* x = static_cast<const char*>(a.x) + (blockIdx.x * static_cast<size_t>(a.ldx) + c) * (kType == kFp32 ? 4 : 2);
    const char* res = static_cast<const char*>(a.residual) + at * (kRType == kFp32 ? 4 : 2);
    char* out = static_cast<char*>(a.residual_out) + at * (kRType == kFp32 ? 4 : 2);
    Load8<kType> v[kChunks];
    Load8<kRType> w[kResidual == kNone ? 1 : kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const bool in = c + i * kStep < a.d;
      if (in) v[i].load_l2(x, i * kStep); else v[i].zero();
      if constexpr (kResidual != kNone) {
        if (in) w[i].load_l2(res, i * kStep); else w[i].zero();
      }
    }
    if constexpr (kGammaEarly) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) load_gamma(i, g[i]);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if constexpr (kResidual == kSame && kType != kFp32) {  // packed additions, each rounded once
        v[i].v[0] = add_packed<kType>(v[i].v[0], w[i].v[0]);
        if (c + i * kStep < a.d) *reinterpret_cast<uint4*>(out + 2 * i * kStep) = v[i].v[0];
      }
      v[i].floats(r[i]);
      if constexpr (kRType == kFp32 && kResidual != kNone) {
        float f[8];
        w[i].floats(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] += f[j];
        if (c + i * kStep < a.d) store8<kFp32>(out + 4 * i * kStep, r[i]);
      }
    }
  }
  Pair sum{0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    uint64_t q2 = 0;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint64_t v = pack2(__float_as_uint(r[i][j]), __float_as_uint(r[i][j + 1]));
      if (j == 0) q2 = mul2(v, v); else fma2(q2, v, v);
    }
    float q, p;
    unpack2(q2, q, p);
    sum = add(sum, Pair{q + p, 0.0f});
  }
  sum = lanes_sum(sum, 32);
  if (warps > 1) {
    if (lane == 0) s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    int group = 2;  // lanes that add up the warps' sums, each group for itself
    while (group < warps) group *= 2;
    const int l = lane & (group - 1);
    sum = lanes_sum(l < warps ? s_sum[l] : Pair{0.0f, 0.0f}, group);
  }
  const Pair inv = inverse_root(sum, static_cast<float>(a.d), a.eps);
  const size_t pitch = blk_scale_rows(a.T);
  float* s_at = a.s + (c / kBlk) * pitch + blockIdx.x;  // used where a.q is there
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int col = c + i * kStep;
    if (col - 8 * lane >= a.d) break;  // the same for the whole warp
    const int gi = kGammaEarly ? i : 0;
    if constexpr (!kGammaEarly) load_gamma(i, g[0]);
    float y[8];
    const uint64_t inv2 = pack2(__float_as_uint(inv.hi), __float_as_uint(inv.hi));
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      unpack2(mul2(mul2(pack2(__float_as_uint(r[i][j]), __float_as_uint(r[i][j + 1])), inv2),
                   pack2(__float_as_uint(g[gi][j]), __float_as_uint(g[gi][j + 1]))), y[j], y[j + 1]);
    if (a.y && col < a.d) store8(a.y_type, a.y, at + i * kStep, y);
    if (!a.q) continue;
    const uint32_t m = half_warp_max(largest_bits(y));
    float s = blk_scale(m);
    // a largest magnitude within 8 last places (more than 2^-21 of it) of where the scale steps up
    if (__any_sync(0xffffffffu, ((m + 0x1FFFFFu + 8u) & 0x7FFFFFu) <= 16u)) {
      double most = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmax(most, fabs(exact_value(r[i][j], g[gi][j], inv)));
#pragma unroll
      for (int k = 1; k < 16; k *= 2) most = fmax(most, __shfl_xor_sync(0xffffffffu, most, k));
      // (a y past fp32's range is infinite whatever the warp's other block asks for)
      if (m < 0x7F800000u) s = blk_scale(__float_as_uint(odd_float(most)));
    }
    const float t = blk_inverse(s);
    uint2 code = blk_codes8(y, t * (1.0f - kNormError));
    const uint2 other = blk_codes8(y, t * (1.0f + kNormError));
    if (code.x != other.x || code.y != other.y) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = odd_float(exact_value(r[i][j], g[gi][j], inv) * static_cast<double>(t));
      code = blk_codes8(y, 1.0f);
    }
    if (col < a.d) {
      *reinterpret_cast<uint2*>(a.q + at + i * kStep) = code;
      if ((lane & 15) == 0) s_at[2 * i * pitch] = s;
    }
  }
}

// ------------------------------------------------------------------ scatter to the routing's rows
// X's rows quantised once (or taken as they are) and written to the rows of their
// assignments: one CTA per token, a warp per 256 columns.  Where the kernel before
// this one is the routing, which let this one start after its own wait, X is there
// already and is read while the routing runs.
template <bool kCodes>
__global__ void __launch_bounds__(kThreads)
    blk_scatter_kernel(const BlkX x, int d, const MxScatter s, int pitch, uint8_t* __restrict__ q, float* __restrict__ sx) {
  __shared__ long long s_row[kMaxK + 1];    // destination rows of the codes, -1: none
  __shared__ long long s_scale[kMaxK + 1];  // place of the first block's scale
  if (!s.x_ready) pdl_wait();
  const int lane = threadIdx.x & 31;
  const int blocks = blk_count(d);
  const int t = blockIdx.x;
  const int n = s.k + (s.shared_rows > 0 ? 1 : 0);
  int c = (threadIdx.x >> 5) * 256 + 8 * lane;
  uint2 code;
  float scale;
  auto take = [&]() {
    if constexpr (kCodes) {
      code = c < d ? __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(x.x) + static_cast<size_t>(t) * d + c))
                   : make_uint2(0, 0);
      scale = c < d ? __ldg(x.s + static_cast<size_t>(c / kBlk) * x.pitch + t) : 0.0f;
    } else {
      Load8<kBf16> v;
      if (c < d) v.load(static_cast<const uint16_t*>(x.x) + static_cast<size_t>(t) * d, c); else v.zero();
      float f[8];
      v.floats(f);
      scale = blk_scale(half_warp_max(largest_bits(f)));
      code = blk_codes8(f, blk_inverse(scale));
    }
  };
  take();
  pdl_wait();
  pdl_launch_dependents();
  for (int j = threadIdx.x >> 5; j < n; j += kThreads / 32) {
    long long to = -1, at = 0;
    if (j == s.k) {
      to = static_cast<long long>(s.T) * s.k + t;
      at = static_cast<long long>(s.max_blocks + t / s.shared_rows) * blocks * pitch + t % s.shared_rows;
    } else {
      // the last tile that starts at or before p, 32 places at a time
      const int p = __ldg(s.inv_perm + static_cast<size_t>(t) * s.k + j);
      int lo = 0, n_left = min(max(*s.num_blocks, 0), s.max_blocks);  // among lo .. lo + n_left - 1
      int first = -1;
      while (n_left > 0) {
        const int step = (n_left + 31) / 32;
        const int i = lane * step;
        const int v = i < n_left ? __ldg(s.block_map + 3 * static_cast<size_t>(lo + i) + 1) : 0x7FFFFFFF;
        const int before = __popc(__ballot_sync(0xffffffffu, v <= p));  // the tiles' starts ascend
        if (before == 0) break;
        first = __shfl_sync(0xffffffffu, v, before - 1);
        lo += (before - 1) * step;
        n_left = step == 1 ? 0 : min(step, n_left - (before - 1) * step);
      }
      const int r = first >= 0 ? p - first : -1;
      if (p >= 0 && p < s.T * s.k && r >= 0 && r < pitch && lo < s.max_blocks) {
        to = p;
        at = static_cast<long long>(lo) * blocks * pitch + r;
      } else if (lane == 0) {
        record_status(s.status, MOE_ERR_INVALID_ARG);
      }
    }
    if (lane == 0) {
      s_row[j] = to;
      s_scale[j] = at;
    }
  }
  __syncthreads();
  for (int base = 0; base < d; base += 8 * kThreads) {
    if (base > 0) {
      c += 8 * kThreads;
      take();
    }
    if (c - 8 * lane >= d) break;  // the same for the whole warp
    if (c >= d) continue;
    for (int j = 0; j < n; ++j) {
      if (s_row[j] < 0) continue;
      *reinterpret_cast<uint2*>(q + static_cast<size_t>(s_row[j]) * d + c) = code;
      if ((lane & 15) == 0) sx[s_scale[j] + static_cast<size_t>(c / kBlk) * pitch] = scale;
    }
  }
}

template <typename... P, typename... A>
cudaError_t launch(int kind, void (*kernel)(P...), unsigned grid, int threads, cudaStream_t stream, bool pdl, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  timer_begin(kind, stream);
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  timer_end(kind, stream);
  return err;
}

// CTAs of Patch: units of four rows x 256 columns, a warp each.
size_t patches(int rows, int K) {
  const size_t units = static_cast<size_t>((rows + kRowsAWarp - 1) / kRowsAWarp) * ((K + 255) / 256);
  return (units + kThreads / 32 - 1) / (kThreads / 32);
}
constexpr size_t kMaxUnits = 0x7FFFFFFFu / (kThreads / 32);  // a unit's number is an int

template <int kType>
cudaError_t launch_norm(const NormArgs& a, int residual, cudaStream_t stream, bool pdl) {
  // one chunk a thread for few rows, where latency counts; more of them where there are many, so that an SM has more
  // CTAs, which wait for their sums at different times (8192 rows of 8192 with the residual, 1 / 2 / 4 chunks: 160 / 107
  // / 84 us; 4096 of 2048, with the inverse, 22.3 / 20.8 / 23.3; 16 of 4096, with the inverse, 4.0 / 4.6 / 5.4)
  int chunks = a.T < 512 ? 1 : a.d <= 2048 ? 2 : 4;
  while (a.d > 8 * 1024 * chunks) chunks *= 2;
  const int threads = ((a.d + 8 * chunks - 1) / (8 * chunks) + 31) / 32 * 32;
  auto pick = [&](auto r) {
    constexpr int R = decltype(r)::value;
    return chunks == 1 ? rmsnorm_kernel<kType, R, 1> : chunks == 2 ? rmsnorm_kernel<kType, R, 2> : rmsnorm_kernel<kType, R, 4>;
  };
  const auto kernel = residual == kNone   ? pick(std::integral_constant<int, kNone>{})
                      : residual == kSame ? pick(std::integral_constant<int, kSame>{})
                                          : pick(std::integral_constant<int, kWide>{});
  return launch(kKNorm, kernel, static_cast<unsigned>(a.T), threads, stream, pdl, a);
}

}  // namespace

cudaError_t launch_blk_quantize(const void* X, int type, int rows, int K, long long ldx, uint8_t* q, float* s,
                                cudaStream_t stream, bool pdl) {
  const size_t grid = patches(rows, K);
  if (grid > kMaxUnits) return cudaErrorInvalidValue;
  const auto kernel = type == kBf16 ? blk_quantize_kernel<kBf16> : type == kFp16 ? blk_quantize_kernel<kFp16> : blk_quantize_kernel<kFp32>;
  return launch(kKBlkQuantize, kernel, static_cast<unsigned>(grid), kThreads, stream, pdl, X, rows, K, ldx, q, s);
}

cudaError_t launch_blk_dequant(const uint8_t* q, const float* s, int rows, int K, int type, void* X, cudaStream_t stream,
                               bool pdl) {
  const size_t grid = patches(rows, K);
  if (grid > kMaxUnits) return cudaErrorInvalidValue;
  const auto kernel = type == kBf16 ? blk_dequant_kernel<kBf16> : type == kFp16 ? blk_dequant_kernel<kFp16> : blk_dequant_kernel<kFp32>;
  return launch(kKBlkQuantize, kernel, static_cast<unsigned>(grid), kThreads, stream, pdl, q, s, rows, K, X);
}

cudaError_t launch_blk_quantize_weights(const void* W, int type, int E, int N, int K, uint8_t* q, float* s,
                                        cudaStream_t stream, bool pdl) {
  const size_t grid = E * blk_weight_scales(N, K);
  if (grid > 0x7FFFFFFFu) return cudaErrorInvalidValue;
  const auto kernel = type == kBf16   ? blk_quantize_weights_kernel<kBf16>
                      : type == kFp16 ? blk_quantize_weights_kernel<kFp16>
                                      : blk_quantize_weights_kernel<kFp32>;
  return launch(kKBlkQuantize, kernel, static_cast<unsigned>(grid), kThreads, stream, pdl, W, N, K, q, s);
}

cudaError_t launch_blk_dequant_weights(const uint8_t* q, const float* s, int E, int N, int K, int type, void* W,
                                       cudaStream_t stream, bool pdl) {
  const size_t grid = E * blk_weight_scales(N, K);
  if (grid > 0x7FFFFFFFu) return cudaErrorInvalidValue;
  const auto kernel = type == kBf16   ? blk_dequant_weights_kernel<kBf16>
                      : type == kFp16 ? blk_dequant_weights_kernel<kFp16>
                                      : blk_dequant_weights_kernel<kFp32>;
  return launch(kKBlkQuantize, kernel, static_cast<unsigned>(grid), kThreads, stream, pdl, q, s, N, K, W);
}

cudaError_t launch_blk_scatter(const BlkX& x, int d, const MxScatter& s, int pitch, uint8_t* q, float* sx,
                               cudaStream_t stream, bool pdl) {
  return launch(kKBlkQuantize, x.type == kBlkCodes ? blk_scatter_kernel<true> : blk_scatter_kernel<false>,
                static_cast<unsigned>(s.T), kThreads, stream, pdl, x, d, s, pitch, q, sx);
}

cudaError_t launch_rmsnorm(const RmsNorm& n, cudaStream_t stream, bool pdl) {
  const NormArgs a{n.x, n.residual, n.residual_out, n.gamma, n.y, n.q, n.s, n.ldx, n.eps, n.T, n.d, n.gamma_fp32, n.y_type};
  const int residual = !n.residual ? kNone : n.residual_type == n.x_type ? kSame : kWide;
  return n.x_type == kBf16   ? launch_norm<kBf16>(a, residual, stream, pdl)
         : n.x_type == kFp16 ? launch_norm<kFp16>(a, residual, stream, pdl)
                             : launch_norm<kFp32>(a, residual, stream, pdl);
}

}  // namespace bm
