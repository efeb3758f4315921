// MXFP4 quantisation and its inverse: 32 consecutive values along K share a
// power-of-two scale, every value is an E2M1 code (include/moe_mx.h).
//
// The scale needs no logarithm: floor(log2 a) of an fp32 magnitude is its
// exponent field, so the E8M0 byte is that field minus 2 (2 = the exponent of
// E2M1's largest power of two), and 2^-e is the float whose exponent field is
// 254 minus the byte.  The multiplication by it is exact (a power of two), so
// the only rounding is the conversion to E2M1.  Both directions are bound by
// memory: 8192 x 8192 bf16 27.0 us to codes and 26.0 back (25.0 for the bytes at
// the rate of a copy), 512 x 2048 1.6 and 1.3 us (a launch).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "mx.cuh"
#include "ptx.cuh"

namespace bm {
namespace {

// One CTA per 256 columns of 32 rows: those of a 128-row tile whose number mod
// 32 is one of eight, warp w the rows w mod 8, + 32, + 64 and + 96.  The packed
// scales of these four rows are neighbours, so a warp writes (or reads) its
// scales of 128 columns as one 16-byte word (four 4-byte words cost 7 of 38 us
// at 8192 x 8192), and consecutive CTAs read along the rows.
//
// The products read weights before they wait for the kernel before them, so a
// kernel whose result may be weights lets no other start before it has completed:
// the quantisation starts its successor early only inside a linear layer, where
// its result is the activations (`early`), and the inverse never does.
constexpr int kQuantThreads = 256;
constexpr int kUnits = 4;
struct Patch {
  int row, col;       // first row and column of this lane
  long long scales;   // byte offset of the 16 bytes of this lane's 128 columns
  __device__ __forceinline__ explicit Patch(int K) {
    const int segs = (K + 255) / 256, pieces = (K + kMxPieceK - 1) / kMxPieceK;
    const int lane = threadIdx.x & 31;
    const int seg = blockIdx.x % segs, part = blockIdx.x / segs;  // part: 4 a tile
    const int r = (part & 3) * 8 + (threadIdx.x >> 5);
    row = (part >> 2) * kMxPieceRows + r;
    col = seg * 256 + 8 * lane;
    scales = (static_cast<long long>(part >> 2) * pieces + col / kMxPieceK) * kMxPieceBytes + r * 16;
  }
};

template <int kType>
__global__ void __launch_bounds__(kQuantThreads)
    mx_quantize_kernel(const void* __restrict__ X, int rows, int K, long long ldx, uint8_t* __restrict__ q,
                       uint8_t* __restrict__ sp, int early) {
  const Patch at(K);
  const int lane = threadIdx.x & 31;
  const int esize = kType == kFp32 ? 4 : 2;
  pdl_wait();
  if (early) pdl_launch_dependents();
  Load8<kType> x[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (at.row + 32 * i < rows && at.col < K)
      x[i].load(static_cast<const char*>(X) + static_cast<size_t>(at.row + 32 * i) * ldx * esize, at.col);
    else
      x[i].zero();
  }
  uint32_t scales[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t code = quantize8(x[i], scales[i], lane);
    if (at.row + 32 * i < rows && at.col < K)
      *reinterpret_cast<uint32_t*>(q + static_cast<size_t>(at.row + 32 * i) * (K / 2) + at.col / 2) = code;
  }
  if ((lane & 15) == 0 && at.row < rows && at.col < K)
    *reinterpret_cast<uint4*>(sp + at.scales) = make_uint4(scales[0], scales[1], scales[2], scales[3]);
}

// The same division of work within each matrix (blockIdx.y).
template <int kType>
__global__ void __launch_bounds__(kQuantThreads)
    mx_dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sp, int N, int K, void* __restrict__ W) {
  const Patch at(K);
  const int lane = threadIdx.x & 31;
  const int pieces = (K + kMxPieceK - 1) / kMxPieceK;
  const size_t matrix = static_cast<size_t>(blockIdx.y) * N;
  sp += blockIdx.y * static_cast<size_t>((N + kMxPieceRows - 1) / kMxPieceRows) * pieces * kMxPieceBytes;
  pdl_wait();
  if (at.row >= N || at.col >= K) return;
  uint32_t code[kUnits];
  const size_t first = (matrix + at.row) * (K / 8) + at.col / 8;  // in words of eight codes
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
    code[i] = at.row + 32 * i < N ? __ldg(reinterpret_cast<const uint32_t*>(q) + first + static_cast<size_t>(32 * i) * (K / 8)) : 0u;
  const uint4 sw = __ldg(reinterpret_cast<const uint4*>(sp + at.scales));
  const uint32_t scales[kUnits] = {sw.x, sw.y, sw.z, sw.w};
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (at.row + 32 * i >= N) break;
    const size_t to = first + static_cast<size_t>(32 * i) * (K / 8);
    const float s = mx_scale((scales[i] >> (8 * ((lane >> 2) & 3))) & 255u);
    float2 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = e2m1x2_to_float2(code[i] >> (8 * j));
      f[j].x *= s;
      f[j].y *= s;
    }
    if constexpr (kType == kFp32) {
      float4* p = reinterpret_cast<float4*>(W) + 2 * to;
      p[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      p[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    } else {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __float22bfloat162_rn(f[j]);
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      reinterpret_cast<uint4*>(W)[to] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// X's rows quantised once and written to the rows of their assignments: one CTA
// per token, one warp per 256 values.  Where the kernel before this one is the
// routing, which let this one start after its own wait, X is there already: it is
// read and quantised while the routing runs (512 tokens' layer 82.9 -> 82.5 us).
constexpr int kScatterThreads = 256;
__global__ void __launch_bounds__(kScatterThreads)
    mx_scatter_kernel(const uint16_t* __restrict__ X, int d, MxScatter s, uint8_t* __restrict__ q,
                      uint8_t* __restrict__ sp) {
  __shared__ long long s_row[kMaxK + 1];    // destination rows of the codes, -1: none
  __shared__ long long s_scale[kMaxK + 1];  // byte offset of piece 0 of the row's scales
  if (!s.x_ready) pdl_wait();
  const int lane = threadIdx.x & 31;
  const int pieces = (d + kMxPieceK - 1) / kMxPieceK;
  const int t = blockIdx.x;
  const int n = s.k + (s.shared_rows > 0 ? 1 : 0);
  Load8<kBf16> x;
  int c = (threadIdx.x >> 5) * 256 + 8 * lane;
  const uint16_t* row = X + static_cast<size_t>(t) * d;
  if (c < d) x.load(row, c); else x.zero();
  uint32_t scales, code = quantize8(x, scales, lane);
  pdl_wait();
  pdl_launch_dependents();
  for (int j = threadIdx.x >> 5; j < n; j += kScatterThreads / 32) {
    long long to = -1, at = 0;
    if (j == s.k) {
      to = static_cast<long long>(s.T) * s.k + t;
      at = mx_scale_offset(t % s.shared_rows, 0, pieces) +
           static_cast<long long>(s.max_blocks + t / s.shared_rows) * pieces * kMxPieceBytes;
    } else {
      // the last tile that starts at or before p, 32 places at a time: two or
      // three round trips instead of one for each halving
      const int p = __ldg(s.inv_perm + static_cast<size_t>(t) * s.k + j);
      int lo = 0, n_left = min(max(*s.num_blocks, 0), s.max_blocks);  // among lo .. lo + n_left - 1
      int first = -1;
      while (n_left > 0) {
        const int step = (n_left + 31) / 32;
        const int i = lane * step;
        const int v = i < n_left ? __ldg(s.block_map + 3 * (lo + i) + 1) : 0x7FFFFFFF;
        const int before = __popc(__ballot_sync(0xffffffffu, v <= p));  // the tiles' starts ascend
        if (before == 0) break;
        first = __shfl_sync(0xffffffffu, v, before - 1);
        lo += (before - 1) * step;
        n_left = step == 1 ? 0 : min(step, n_left - (before - 1) * step);
      }
      const int r = first >= 0 ? p - first : -1;
      if (p >= 0 && p < s.T * s.k && r >= 0 && r < kMxMaxBN && lo < s.max_blocks) {
        to = p;
        at = mx_scale_offset(r, 0, pieces) + static_cast<long long>(lo) * pieces * kMxPieceBytes;
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
  for (int base = 0; base < d; base += 8 * kScatterThreads) {
    if (base > 0) {
      c += 8 * kScatterThreads;
      if (c < d) x.load(row, c); else x.zero();
      code = quantize8(x, scales, lane);
    }
    if (c - 8 * lane >= d) break;  // the same for the whole warp
    for (int j = 0; j < n; ++j) {
      if (s_row[j] < 0) continue;
      if (c < d) *reinterpret_cast<uint32_t*>(q + static_cast<size_t>(s_row[j]) * (d / 2) + c / 2) = code;
      if ((lane & 15) == 0 && c < d)
        *reinterpret_cast<uint32_t*>(sp + s_scale[j] + static_cast<size_t>(c / kMxPieceK) * kMxPieceBytes) = scales;
    }
  }
}

// One thread per 32-bit word of the packed scales: four blocks of one row.
__global__ void mx_prepack_kernel(const uint8_t* __restrict__ scale, int E, int N, int G, uint8_t* __restrict__ sp) {
  const int pieces = (G + 3) / 4;
  const int tiles = (N + kMxPieceRows - 1) / kMxPieceRows;
  const size_t total = static_cast<size_t>(E) * tiles * pieces * (kMxPieceBytes / 4);
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const int w = static_cast<int>(i % (kMxPieceBytes / 4));  // word 4 (r % 32) + r / 32 of the piece
    size_t p = i / (kMxPieceBytes / 4);
    const int piece = static_cast<int>(p % pieces);
    p /= pieces;
    const int tile = static_cast<int>(p % tiles);
    const int e = static_cast<int>(p / tiles);
    const int n = tile * kMxPieceRows + (w >> 2) + 32 * (w & 3);
    uint32_t v = 0;
    for (int b = 0; b < 4; ++b)
      if (n < N && 4 * piece + b < G)
        v |= static_cast<uint32_t>(scale[(static_cast<size_t>(e) * N + n) * G + 4 * piece + b]) << (8 * b);
    reinterpret_cast<uint32_t*>(sp)[i] = v;
  }
}

// The sum over a token's experts: a thread per four columns of a token, the rows
// of four slots in flight together (eight take registers that other warps' loads
// need: 4096 tokens of 8 + 1 experts, d = 2048, 226 instead of 219 us for the whole
// layer), added in slot order, the shared expert's last.
//
// Bound by memory: the rows are read once and never again, so the loads say so,
// and what of the down product's writes is still in L2 is discarded instead of
// written to memory: 60 -> 51 us of the above (302 MB), 512 tokens' layer 87.7 ->
// 84.3 us, where none of the rows leaves L2.  A token's places and weights are read
// one turn ahead, a slot a lane: 218 -> 212 us of the above.
constexpr int kCombineThreads = 128;
constexpr int kCombineSlots = 4;
__global__ void __launch_bounds__(kCombineThreads)
    mx_combine_kernel(float* __restrict__ ypart, const int32_t* __restrict__ inv_perm, const float* __restrict__ w,
                      int T, int d, int k, int has_shared, uint16_t* __restrict__ Y, uint32_t* status) {
  const int warps = (d + 127) / 128;  // of a token
  const int A = T * k;
  const int lane = threadIdx.x & 31;
  const long long total = static_cast<long long>(T) * warps, step = static_cast<long long>(gridDim.x) * (kCombineThreads / 32);
  long long i = static_cast<long long>(blockIdx.x) * (kCombineThreads / 32) + (threadIdx.x >> 5);
  // slot `lane` of the warp's token, read ahead (before the wait the first time: the routing completed kernels ago)
  int next_row = 0;
  float next_w = 0.0f;
  auto read_slot = [&]() {
    if (i < total && lane < k) {
      const size_t at = static_cast<size_t>(i / warps) * k + lane;
      next_row = __ldg(inv_perm + at);
      next_w = __ldg(w + at);
    }
  };
  read_slot();
  pdl_wait();
  pdl_launch_dependents();
  bool ok = true;
  while (i < total) {
    const int t = static_cast<int>(i / warps);
    const int c0 = 128 * static_cast<int>(i - static_cast<long long>(t) * warps), c = c0 + 4 * lane;
    const bool valid = next_row >= 0 && next_row < A;
    const int row = valid ? next_row : -1;
    const float wt = valid ? next_w : 0.0f;
    if (lane < k && !valid) ok = false;
    i += step;
    read_slot();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f), sh = acc;
    if (has_shared && c < d) sh = __ldlu(reinterpret_cast<const float4*>(ypart + (static_cast<size_t>(A) + t) * d + c));
    for (int j0 = 0; j0 < k; j0 += kCombineSlots) {
      float4 v[kCombineSlots];
      float wj[kCombineSlots];
#pragma unroll
      for (int u = 0; u < kCombineSlots; ++u) {
        const int p = __shfl_sync(0xffffffffu, row, j0 + u);  // past the last slot: a lane without one
        wj[u] = __shfl_sync(0xffffffffu, wt, j0 + u);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j0 + u < k && p >= 0 && c < d) v[u] = __ldlu(reinterpret_cast<const float4*>(ypart + static_cast<size_t>(p) * d + c));
      }
#pragma unroll
      for (int u = 0; u < kCombineSlots; ++u) {
        if (j0 + u >= k) continue;
        acc.x = fmaf(wj[u], v[u].x, acc.x);
        acc.y = fmaf(wj[u], v[u].y, acc.y);
        acc.z = fmaf(wj[u], v[u].z, acc.z);
        acc.w = fmaf(wj[u], v[u].w, acc.w);
      }
    }
    if (c < d) {
      if (has_shared) acc = make_float4(acc.x + sh.x, acc.y + sh.y, acc.z + sh.z, acc.w + sh.w);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
      *reinterpret_cast<uint2*>(Y + static_cast<size_t>(t) * d + c) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    // the warp's 512 bytes of each row, a line of 128 bytes (32 columns: d is a multiple) a lane
    __syncwarp();
    const int line = c0 + 32 * (lane & 3);
    for (int j0 = 0; j0 < k; j0 += 8) {
      const int j = j0 + (lane >> 2), p = __shfl_sync(0xffffffffu, row, j);
      if (j < k && p >= 0 && line < d) discard_line(ypart + static_cast<size_t>(p) * d + line);
    }
    if (has_shared && lane < 4 && line < d) discard_line(ypart + (static_cast<size_t>(A) + t) * d + line);
  }
  if (!ok) record_status(status, MOE_ERR_INVALID_ARG);
}

// Programmatic dependent launch of `kernel` where `pdl` allows it.
template <typename... P, typename... A>
cudaError_t launch(int kind, void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, bool pdl, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  timer_begin(kind, stream);
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  timer_end(kind, stream);
  return err;
}

int blocks_for(size_t threads, int per_block, int most) {
  const size_t n = (threads + per_block - 1) / per_block;
  return static_cast<int>(n < 1 ? 1 : n < static_cast<size_t>(most) ? n : most);
}

// CTAs of a matrix's quantisation: 256 columns of 32 rows each.
size_t patches(int rows, int K) {
  return static_cast<size_t>((rows + kMxPieceRows - 1) / kMxPieceRows) * 4 * ((K + 255) / 256);
}

}  // namespace

cudaError_t launch_mx_prepack(const uint8_t* scale, int E, int N, int K, uint8_t* sp, cudaStream_t stream) {
  const size_t words = static_cast<size_t>(E) * mx_pieces(N, K) * (kMxPieceBytes / 4);
  return launch(kKPrepack, mx_prepack_kernel, blocks_for(words, 256, 65536), 256, stream, false, scale, E, N,
                K / kMxBlock, sp);
}

cudaError_t launch_mx_quantize(const void* X, int type, int rows, int K, long long ldx, uint8_t* q, uint8_t* sp,
                               bool early, cudaStream_t stream, bool pdl) {
  const size_t grid = patches(rows, K);
  if (grid > 0x7FFFFFFFu) return cudaErrorInvalidValue;
  const auto kernel = type == kBf16 ? mx_quantize_kernel<kBf16>
                                    : (type == kFp16 ? mx_quantize_kernel<kFp16> : mx_quantize_kernel<kFp32>);
  return launch(kKMxQuantize, kernel, dim3(static_cast<unsigned>(grid)), kQuantThreads, stream, pdl, X, rows, K, ldx, q, sp,
                early ? 1 : 0);
}

cudaError_t launch_mx_dequant(const uint8_t* q, const uint8_t* sp, int E, int N, int K, int type, void* W,
                              cudaStream_t stream, bool pdl) {
  const size_t grid = patches(N, K);
  if (grid > 0x7FFFFFFFu) return cudaErrorInvalidValue;
  return launch(kKMxQuantize, type == kFp32 ? mx_dequant_kernel<kFp32> : mx_dequant_kernel<kBf16>, dim3(static_cast<unsigned>(grid), E),
                kQuantThreads, stream, pdl, q, sp, N, K, W);
}

cudaError_t launch_mx_combine(float* ypart, const int32_t* inv_perm, const float* w, int T, int d, int k,
                              bool has_shared, uint16_t* Y, uint32_t* status, int num_sms, cudaStream_t stream) {
  const int grid = blocks_for(static_cast<size_t>(T) * ((d + 127) / 128), kCombineThreads / 32, num_sms * 16);
  return launch(kKCombine, mx_combine_kernel, grid, kCombineThreads, stream, true, ypart, inv_perm, w, T, d, k,
                has_shared ? 1 : 0, Y, status);
}

cudaError_t launch_mx_scatter(const uint16_t* X, int d, const MxScatter& s, uint8_t* q, uint8_t* sp,
                              cudaStream_t stream, bool pdl) {
  return launch(kKMxQuantize, mx_scatter_kernel, s.T, kScatterThreads, stream, pdl, X, d, s, q, sp);
}

}  // namespace bm
