// Wavefront pieces of the sigmoid top-k selection, shared by the routing kernel
// and the whole expert layer: ordered keys, the k-th largest by a radix
// descent, and the slots of the selected experts.  One wavefront works on one
// token row; lane l holds C experts in ascending order.
#pragma once

#include "esg_device.hpp"

namespace esg {

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float exact_sigmoid(float z) { return (float)(1.0 / (1.0 + exp(-(double)z))); }

__device__ __forceinline__ uint32_t wave_min_u32(uint32_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, off);
    v = o < v ? o : v;
  }
  return v;
}

// Radix descent over the top NB key bits of the C keys per lane: returns the
// k-th largest key of the valid ones (its top NB bits; the rest zero) and
// leaves in `need` how many keys equal to it the row takes.  With NB = 32 the
// descent stops as soon as the class of keys sharing the prefix holds exactly
// `need` keys: they are all taken, the k-th largest is their minimum, and
// `need` is recounted against it.
template <int C, int NB>
__device__ __forceinline__ uint32_t kth_largest(const uint32_t (&u)[C], const bool (&valid)[C], int nvalid, int k,
                                                int& need) {
  uint32_t prefix = 0;
  int cls = nvalid;  // keys matching the prefix so far
  need = k;
  for (int bit = 31; bit >= 32 - NB; --bit) {
    const uint32_t m = ~0u << bit;
    const uint32_t cand = prefix | (1u << bit);
    int cnt = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) cnt += __popcll(__ballot(valid[c] && (u[c] & m) == cand));
    if (cnt >= need) {
      prefix = cand;
      cls = cnt;
    } else {
      need -= cnt;
      cls -= cnt;
    }
    if (NB == 32 && cls == need && bit > 0) {
      uint32_t mn = 0xffffffffu;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (valid[c] && (u[c] & m) == prefix && u[c] < mn) mn = u[c];
      prefix = wave_min_u32(mn);
      int above = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) above += __popcll(__ballot(valid[c] && u[c] > prefix));
      need = k - above;
      break;
    }
  }
  return prefix;
}

// Slots of the selected keys (C per lane, lanes in ascending expert order):
// keys above tau fill slots [0, k - need) in order, then the first `need` keys
// equal to tau fill the rest.  Writes score and expert of each to the row's
// LDS lists.
template <int C>
__device__ __forceinline__ void place(const uint32_t (&u)[C], const bool (&valid)[C], const float (&sc)[C],
                                      const int (&ex)[C], uint32_t tau, int k, int need, int lane, float* s_row,
                                      int* e_row) {
  const uint64_t lower = (1ull << lane) - 1ull;
  int ia = 0, ie = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    ia += __popcll(__ballot(valid[c] && u[c] > tau) & lower);
    ie += __popcll(__ballot(valid[c] && u[c] == tau) & lower);
  }
  const int n_above = k - need;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    int slot = -1;
    if (valid[c] && u[c] > tau) {
      slot = ia++;
    } else if (valid[c] && u[c] == tau) {
      if (ie < need) slot = n_above + ie;
      ++ie;
    }
    if (slot >= 0) {
      s_row[slot] = sc[c];
      e_row[slot] = ex[c];
    }
  }
}

__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace esg
