// Device pieces of the MXFP4 format shared by its kernels (include/moe_mx.h).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"

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

// Value of the E2M1 code in bits 0..3.
__device__ __forceinline__ float mx_code_value(uint32_t code) {
  // the two exponent bits and the mantissa bit at fp32's exponent and top
  // mantissa bits stand for the value times 2^-126; code 1 (0.5) is subnormal there
  return __uint_as_float(((code & 8u) << 28) | ((code & 7u) << 22)) * 0x1p126f;
}

// Byte offset of the four scales of row r, 128-column piece `piece`, in packed
// scales with `pieces` pieces a row.
__device__ __forceinline__ long long mx_scale_offset(long long r, int piece, int pieces) {
  return ((r / kMxPieceRows) * pieces + piece) * kMxPieceBytes + (r % 32) * 16 + ((r % kMxPieceRows) / 32) * 4;
}

}  // namespace bm
