// Device building blocks of the 8-bit (e4m3) kernels: reads of eight elements,
// conversions, the block scale, and the 16 x 16 x 128 matrix product.
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

// Eight consecutive elements as floats, and the largest magnitude's bits.
template <typename T>
struct Oct;
template <>
struct Oct<bf16_t> {
  uint4 w;
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const bf16_t* p) { w = *(const uint4*)p; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Oct<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = *(const float4*)p;
    b = *(const float4*)(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<bf16_t>(bf16_t* p, const float (&v)[8]) {
  *(uint4*)p = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7]));
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t max8(const float (&v)[8]) {
  uint32_t m = mag(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = umax(m, mag(v[i]));
  return m;
}

// Maximum over the 16 lanes of a row group (lanes 16g .. 16g + 15), left in all
// of them: exchanges inside quads (xor 1, xor 2), then mirrored half rows and
// rows, all in the vector unit's data-parallel moves.
__device__ __forceinline__ uint32_t max_lanes16(uint32_t m) {
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xf, 0xf, true));
  m = umax(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xf, 0xf, true));
  return m;
}

__device__ __forceinline__ uint2 scale_pack8(const float (&v)[8], float inv) {
  return make_uint2(pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    pack_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
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
