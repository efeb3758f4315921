// Device pieces of the MXFP4 format shared by its kernels (include/moe_mx.h).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace bm {

// E8M0 byte of a block whose largest magnitude has the fp32 bits `amax` (sign
// bit clear): 2^(byte - 127) = 2^(floor(log2 a) - 2), at least 2^-127; 255 for
// an infinity or a NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^-(byte - 127), for bytes that mx_scale_byte gives (at most 252, or 255,
// whose codes mean nothing).
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) { return __uint_as_float(((254u - byte) & 255u) << 23); }

// 2^(byte - 127): subnormal for byte 0, NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// Byte offset of the four scales of row r, 128-column piece `piece`, in packed
// scales with `pieces` pieces a row.
__device__ __forceinline__ long long mx_scale_offset(int r, int piece, int pieces) {
  return (static_cast<long long>(r / kMxPieceRows) * pieces + piece) * kMxPieceBytes + (r % 32) * 16 +
         ((r % kMxPieceRows) / 32) * 4;
}

enum { kBf16 = 0, kFp16 = 1, kFp32 = 2 };

// Eight consecutive values of a row, as loaded and as fp32.
template <int kType>
struct Load8 {
  uint4 v[kType == kFp32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* row, int c) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + static_cast<size_t>(c) * (kType == kFp32 ? 4 : 2));
    v[0] = __ldg(p);
    if constexpr (kType == kFp32) v[1] = __ldg(p + 1);
  }
  // the same of memory that is written while this kernel may already be resident and that its SM may hold an older line
  // of: past L1
  __device__ __forceinline__ void load_l2(const void* row, int c) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + static_cast<size_t>(c) * (kType == kFp32 ? 4 : 2));
    v[0] = __ldcg(p);
    if constexpr (kType == kFp32) v[1] = __ldcg(p + 1);
  }
  __device__ __forceinline__ void zero() {
    v[0] = make_uint4(0, 0, 0, 0);
    if constexpr (kType == kFp32) v[1] = v[0];
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
    if constexpr (kType == kBf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else if constexpr (kType == kFp16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        f[2 * j] = p.x;
        f[2 * j + 1] = p.y;
      }
    } else {
      const uint32_t u[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = __uint_as_float(w[j]);
        f[4 + j] = __uint_as_float(u[j]);
      }
    }
  }
};

// The warp's 256 values, eight a lane (a block is four lanes): the lane's eight
// codes, and the scale bytes of the lane's half of the warp (four blocks, one
// 32-bit word).  Lanes past the row's end hold zeros and get the byte 0.
template <int kType>
__device__ __forceinline__ uint32_t quantize8(const Load8<kType>& x, uint32_t& scales, int lane) {
  float f[8];
  x.floats(f);
  float m = fabsf(f[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) m = max_nan(m, fabsf(f[j]));
  uint32_t a = __float_as_uint(m);  // a NaN's bits are above infinity's
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
  const uint32_t byte = mx_scale_byte(a);
  const float inv = mx_inverse_scale(byte);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] *= inv;
  const uint32_t code = f32x8_to_e2m1x8(f);
  scales = byte << (8 * ((lane >> 2) & 3));
  scales |= __shfl_xor_sync(0xffffffffu, scales, 4);
  scales |= __shfl_xor_sync(0xffffffffu, scales, 8);
  return code;
}

// silu(g) u = g / (1 + 2^(-g log2 e)) u, the same bits in every kernel that forms
// h.  Flushing subnormals saves their scaling (ten instructions).  The quotient is
// 0 where the denominator passes 2^126, for g below -87.3: what that drops of
// silu(g) is at most 88 x 2^-126, 1e-36, times u.
__device__ __forceinline__ float mx_swiglu(float g, float u) {
  return div_approx(g, 1.0f + exp2_approx(g * -1.44269504f)) * u;
}

// Scale byte of one value a lane: a block across the warp.
__device__ __forceinline__ uint32_t mx_warp_scale_byte(float v) {
  return mx_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu));
}

}  // namespace bm
