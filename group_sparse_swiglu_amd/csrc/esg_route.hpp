// Scores and ordered keys of the sigmoid top-k selection, shared by the routing
// kernel and the whole expert layer.
#pragma once

#include "esg_device.hpp"

namespace esg {

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float exact_sigmoid(float z) { return (float)(1.0 / (1.0 + exp(-(double)z))); }

}  // namespace esg
