// Device building blocks of the 8-bit (e4m3) kernels: conversions, the block
// scale, and the 16 x 16 x 128 matrix product.
#pragma once

#include "esg_device.hpp"

namespace esg {

constexpr int kQB = 128;                              // elements of a scale block
constexpr float kE4m3Max = 448.0f;                    // largest e4m3 value
constexpr uint32_t kAmaxFloorBits = 0x0d800000u;      // 2^-100: smallest block magnitude a scale is taken from

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Block scale from the largest |x| of a block, given as float bits.  Integer
// order on the bits is the order of the magnitudes with infinities and NaN
// above every number, so a block that holds one gets an infinite or NaN scale
// (and its products are NaN) instead of losing it in a float maximum.
__device__ __forceinline__ void block_scale(uint32_t amax_bits, float& scale, float& inv) {
  const float a = __uint_as_float(amax_bits > kAmaxFloorBits ? amax_bits : kAmaxFloorBits);
  scale = a / kE4m3Max;
  inv = kE4m3Max / a;
}

// Four floats -> four e4m3 bytes (low byte first), round to nearest even.
// |v| <= 448 * (1 + 2^-23) here, which rounds to at most 448: no overflow.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// 16 x 16 x 128 product of e4m3 operands on zero: lane l gives 32 bytes of row
// l % 16 of each operand (any 128 K positions, split alike on both sides over
// the four lane groups and their bytes); the result sits as for the bf16
// product: rows (l / 16) * 4 + i of column l % 16.  This form runs at twice
// the rate per K of the 32-wide 8-bit product.
__device__ __forceinline__ f32x4 mma_e4m3_k128(const uint4& a0, const uint4& a1, const uint4& b0, const uint4& b1) {
  const i32x8_t a = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
  const i32x8_t b = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// Eight e4m3 bytes -> eight bf16 (exact: 4 significant bits, exponents inside bf16's).
__device__ __forceinline__ uint4 e4m3x8_to_bf16(uint32_t lo, uint32_t hi) {
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  return r;
}

}  // namespace esg
