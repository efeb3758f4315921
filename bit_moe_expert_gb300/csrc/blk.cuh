// Device pieces of the block-scaled 8-bit format shared by its kernels
// (include/moe_blk.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "mx.cuh"  // Load8
#include "ptx.cuh"

namespace bm {

// The scale of a block whose largest magnitude has the fp32 bits `amax` (sign
// bit clear): the least power of two, at least 2^-126, with a <= 448 s.  448 is
// 1.75 x 2^8: the exponent field minus 8, one more where the mantissa is above
// .75 (the addition carries).  NaN for an infinity or a NaN.
__device__ __forceinline__ float blk_scale(uint32_t amax) {
  const int e = static_cast<int>((amax + 0x1FFFFFu) >> 23) - 8;
  return __uint_as_float(amax >= 0x7F800000u ? 0x7FC00000u : static_cast<uint32_t>(max(e, 1)) << 23);
}
// 1 / s of such a scale (exact); NaN for NaN
__device__ __forceinline__ float blk_inverse(float s) {
  const uint32_t b = __float_as_uint(s);
  return __uint_as_float(b >= 0x7F800000u ? 0x7FC00000u : (254u << 23) - b);
}

// Four fp32 values -> E4M3 codes (round to nearest even, magnitudes above 448 to
// 448), the first in the lowest byte.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// The values of four codes (exact).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t q, float (&f)[4]) {
  uint32_t l, h;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(l), "=r"(h)
      : "r"(q));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&l));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h));
  f[0] = x.x;
  f[1] = x.y;
  f[2] = y.x;
  f[3] = y.y;
}

// silu(g) u = g / (1 + e^-g) u.  A quotient by the approximate division, whose
// error is 2 units in the last place; 0 for g below -87.3, which drops at most
// 88 x 2^-126 of silu(g).
__device__ __forceinline__ float blk_swiglu(float g, float u) {
  return div_approx(g, 1.0f + exp2_approx(g * -1.44269504f)) * u;
}

// Two fp32 numbers in one 64-bit register.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void fma2(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

// n (8 or 16) columns of each lane's own row of tensor memory.
template <int n>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[n]) {
  if constexpr (n == 8) tmem_ld8(taddr, v); else tmem_ld16(taddr, v);
}

// |x| of the largest of the lane's values, as bits; a NaN's are above infinity's.
template <int n>
__device__ __forceinline__ uint32_t largest_bits(const float (&f)[n]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int j = 1; j < n; ++j) m = max_nan(m, fabsf(f[j]));
  return __float_as_uint(m);
}

// The same over the lane's half of the warp: a block of 128 columns, eight a lane.
__device__ __forceinline__ uint32_t half_warp_max(uint32_t a) {
#pragma unroll
  for (int i = 1; i < 16; i *= 2) a = max(a, __shfl_xor_sync(0xffffffffu, a, i));
  return a;
}

// Eight codes of values times inv.
__device__ __forceinline__ uint2 blk_codes8(const float (&f)[8], float inv) {
  float v[8];
  const uint64_t i2 = pack2(__float_as_uint(inv), __float_as_uint(inv));
#pragma unroll
  for (int j = 0; j < 8; j += 2) unpack2(mul2(pack2(__float_as_uint(f[j]), __float_as_uint(f[j + 1])), i2), v[j], v[j + 1]);
  return make_uint2(f32x4_to_e4m3x4(v[0], v[1], v[2], v[3]), f32x4_to_e4m3x4(v[4], v[5], v[6], v[7]));
}

// Eight values to consecutive places of a row of type kType (16-byte aligned).
template <int kType>
__device__ __forceinline__ void store8(void* p, const float (&f)[8]) {
  if constexpr (kType == kFp32) {
    float4* o = static_cast<float4*>(p);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kType == kBf16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        o[j] = f32x2_to_f16x2(f[2 * j], f[2 * j + 1]);
      }
    }
    *static_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}
__device__ __forceinline__ void store8(int type, void* base, size_t at, const float (&f)[8]) {
  if (type == kFp32)
    store8<kFp32>(static_cast<float*>(base) + at, f);
  else if (type == kFp16)
    store8<kFp16>(static_cast<uint16_t*>(base) + at, f);
  else
    store8<kBf16>(static_cast<uint16_t*>(base) + at, f);
}
// One value.
__device__ __forceinline__ void store1(int type, void* base, size_t at, float f) {
  if (type == kFp32)
    static_cast<float*>(base)[at] = f;
  else if (type == kFp16)
    static_cast<__half*>(base)[at] = __float2half_rn(f);
  else
    static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(f);
}

}  // namespace bm
