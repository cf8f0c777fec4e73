// Device building blocks of the 4-bit kernels: e2m1 elements (0, 0.5, 1, 1.5, 2,
// 3, 4, 6 and their negatives) in blocks of 32 with one power of two each, held
// as a biased exponent byte (e8m0: 2^(byte - 127), 255 is NaN).
#pragma once

#include "esg_fp8.hpp"

namespace esg {

constexpr int kMxBlock = 32;

// Exponent byte of a block from its largest |x|'s bits: two below the exponent
// of that value, so it lies in [4, 8) of the block's unit (and what rounds above 6
// is 6); at least 0.  255 for a block that holds an infinity or NaN.
__device__ __forceinline__ uint32_t mx_exponent(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// 2^(127 - e), by which an element is multiplied (exactly) before its rounding; e <= 252.
__device__ __forceinline__ float mx_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// 2^(e - 127), NaN for 255.
__device__ __forceinline__ float mx_value(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : e == 255u ? 0x7fc00000u : e << 23);
}

// Eight elements times inv -> eight codes, the first in the low half of the low
// byte; to nearest even, at most 6.
__device__ __forceinline__ uint32_t mx_pack8(const float (&v)[8], float inv) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * inv, v[1] * inv, 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * inv, v[3] * inv, 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * inv, v[5] * inv, 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * inv, v[7] * inv, 1.0f, 3);
  return r;
}

// Maximum over the 4 lanes that hold a block, left in all of them.
__device__ __forceinline__ uint32_t max_lanes4(uint32_t m) {
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));
  return m;
}

// Codes and exponent of the block of 32 that four neighbouring lanes hold, eight elements each.
__device__ __forceinline__ uint32_t mx_block(const float (&v)[8], uint32_t& e) {
  e = mx_exponent(max_lanes4(max8(v)));
  return e == 255u ? 0u : mx_pack8(v, mx_inverse(e));
}

// Eight codes -> their eight values.
__device__ __forceinline__ void mx_unpack8(uint32_t q, float (&v)[8]) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0);
  const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
  const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2);
  const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
  v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
  v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
}

}  // namespace esg
