// Quantisation to 4-bit floating point (e2m1) in blocks of 32 with a power of two
// each, and the values that codes and exponents stand for.
//
// For a block with largest magnitude a:
//   e = max(exponent of a - 2, -127),  q = e2m1(x 2^-e), to nearest even, at most 6.
// The scale is a power of two, so nothing but the last rounding rounds: a plain
// program gives the same codes whatever its precision.
//
// Both directions are bound by memory.  A lane takes eight elements (16 or 32
// bytes in, 4 out), four lanes a block; kUnroll of them in flight per lane.
// 32768 x 2048 in bf16: 32.7 us to 4 bits (5.2 TB/s), 25.5 back (6.6, with caches).
#include <algorithm>

#include "esg_internal.hpp"
#include "esg_mx.hpp"

namespace esg {
namespace {

constexpr int kUnroll = 4;

template <typename T>
__global__ __launch_bounds__(256) void mx_quant_kernel(const T* __restrict__ x, int64_t octs, uint32_t* __restrict__ q,
                                                       uint8_t* __restrict__ scale) {
  // octs is a multiple of 4: the four lanes of a block are in or out together
  for (int64_t o0 = (int64_t)blockIdx.x * 256 * kUnroll + threadIdx.x; o0 < octs;
       o0 += (int64_t)gridDim.x * 256 * kUnroll) {
    Oct<T> o[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = o0 + u * 256;
      o[u].zero();
      if (at < octs) o[u].load(x + at * 8);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = o0 + u * 256;
      float v[8];
      uint32_t e;
      o[u].get(v);
      const uint32_t c = mx_block(v, e);
      if (at < octs) {
        q[at] = c;
        if ((threadIdx.x & 3) == 0) scale[at >> 2] = (uint8_t)e;
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint32_t* __restrict__ q,
                                                         const uint8_t* __restrict__ scale, int64_t octs,
                                                         T* __restrict__ y) {
  for (int64_t o0 = (int64_t)blockIdx.x * 256 * kUnroll + threadIdx.x; o0 < octs;
       o0 += (int64_t)gridDim.x * 256 * kUnroll) {
    uint32_t c[kUnroll], e[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = o0 + u * 256;
      c[u] = at < octs ? q[at] : 0;
      e[u] = at < octs ? scale[at >> 2] : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = o0 + u * 256;
      float v[8];
      mx_unpack8(c[u], v);
      const float s = mx_value(e[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= s;
      if (at < octs) store8<T>(y + at * 8, v);
    }
  }
}

unsigned grid_of(int64_t octs) {
  return (unsigned)std::min<int64_t>((octs + 256 * kUnroll - 1) / (256 * kUnroll), (int64_t)compute_units() * 16);
}

}  // namespace

hipError_t launch_mx_quant(int dtype, const void* x, int64_t blocks, void* q, void* scale, hipStream_t stream) {
  if (blocks == 0) return hipSuccess;
  const int64_t octs = blocks * 4;
  LaunchTimer timer("mx_quant", stream);
  if (dtype == 0)
    hipLaunchKernelGGL(mx_quant_kernel<float>, dim3(grid_of(octs)), dim3(256), 0, stream, (const float*)x, octs,
                       (uint32_t*)q, (uint8_t*)scale);
  else
    hipLaunchKernelGGL(mx_quant_kernel<bf16_t>, dim3(grid_of(octs)), dim3(256), 0, stream, (const bf16_t*)x, octs,
                       (uint32_t*)q, (uint8_t*)scale);
  return hipGetLastError();
}

hipError_t launch_mx_dequant(int dtype, const void* q, const void* scale, int64_t blocks, void* y,
                             hipStream_t stream) {
  if (blocks == 0) return hipSuccess;
  const int64_t octs = blocks * 4;
  LaunchTimer timer("mx_dequant", stream);
  if (dtype == 0)
    hipLaunchKernelGGL(mx_dequant_kernel<float>, dim3(grid_of(octs)), dim3(256), 0, stream, (const uint32_t*)q,
                       (const uint8_t*)scale, octs, (float*)y);
  else
    hipLaunchKernelGGL(mx_dequant_kernel<bf16_t>, dim3(grid_of(octs)), dim3(256), 0, stream, (const uint32_t*)q,
                       (const uint8_t*)scale, octs, (bf16_t*)y);
  return hipGetLastError();
}

}  // namespace esg
