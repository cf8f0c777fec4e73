// Root-mean-square norm after the residual's addition, forward and backward.
//   h = x + residual (rounded to their type: the new residual), r = (mean h^2 + eps)^-1/2, y = h r w
//   backward, g = dy w:  dx = dresidual = dh + r (g - h r mean(g h r)),  dw = sum over the rows of dy h r
// y leaves in the type of x, or in 8 bits (e4m3, a float32 scale per 1 x 128
// block) or 4 bits (e2m1, a power of two per 32) from its float32 value.  Sums
// and r are float32, every output is rounded once.
//
// Bound by memory.  A row stays in registers: 64 lanes take one of up to 1024
// elements (four rows per workgroup, no barrier), a workgroup of 256 threads one
// of up to 16384, eight consecutive elements at a time per lane, so that blocks
// of 128 and 32 are 16 and 4 neighbouring lanes and their maxima need no LDS.
// The split depends on the width alone: a row's result does not depend on the
// batch.  Workgroups go through the rows in strides with the weights in registers.
// 32768 x 2048 with residual, bf16: forward 91 to 103 us (5.2 TB/s; 8-bit output
// 93, 4-bit 85), backward 97 to 108 (5.0 to 5.6 TB/s).  64 x 2048: 3.4 us, a launch.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "esg_internal.hpp"
#include "esg_mx.hpp"

namespace esg {
namespace {

enum { Y_SAME = 0, Y_E4M3 = 1, Y_MX = 2 };

struct NormArgs {
  const void* x;
  const void* residual;  // NULL: none
  const void* w;
  int w_f32;
  int rows, d;
  float eps;
  void* y;
  void* scale;
  void* h;               // with residual
  float* rstd;           // or NULL
};

// Sum over the TPR threads of a row, in all of them.  lds: one float per wave;
// TPR == 256 takes a barrier, so two calls in a row need different lds.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* lds) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  if constexpr (TPR == 256) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  }
  return v;
}

template <int TPR, int NV>
__device__ __forceinline__ void load_weights(const void* w, int w_f32, int l, int d, float (&v)[NV][8]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + l) * 8;
    if (w_f32) {
      Oct<float> o;
      o.zero();
      if (c < d) o.load((const float*)w + c);
      o.get(v[i]);
    } else {
      Oct<bf16_t> o;
      o.zero();
      if (c < d) o.load((const bf16_t*)w + c);
      o.get(v[i]);
    }
  }
}

// v rounded to T, as floats
__device__ __forceinline__ void round8(float (&)[8], float) {}
__device__ __forceinline__ void round8(float (&v)[8], bf16_t) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint32_t p = pack_bf16x2(v[j], v[j + 1]);
    v[j] = __uint_as_float(p << 16);
    v[j + 1] = __uint_as_float(p & 0xffff0000u);
  }
}

template <typename T, int TPR, int NV, int Y>
__global__ __launch_bounds__(256) void rms_norm_kernel(NormArgs g) {
  __shared__ float lds[3][4];  // the third: a row's second sum, which the next row's barrier parts from its like
  const int l = threadIdx.x % TPR;
  constexpr int RPW = 256 / TPR;
  float w[NV][8];
  load_weights<TPR, NV>(g.w, g.w_f32, l, g.d, w);
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR; row < g.rows; row += (int64_t)gridDim.x * RPW) {
    const int64_t at = row * g.d;
    Oct<T> x[NV], s[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + l) * 8;
      x[i].zero();
      s[i].zero();
      if (c < g.d) {
        x[i].load((const T*)g.x + at + c);
        if (g.residual != nullptr) s[i].load((const T*)g.residual + at + c);
      }
    }
    float v[NV][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + l) * 8;
      x[i].get(v[i]);
      if (g.residual != nullptr) {
        float t[8];
        s[i].get(t);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += t[j];
        round8(v[i], T{});
        if (c < g.d) store8<T>((T*)g.h + at + c, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
    }
    sum = row_sum<TPR>(sum, lds[turn]);
    turn ^= 1;
    float r = 1.0f / sqrtf(sum / (float)g.d + g.eps);
    float rstd = r;
    if (!(sum <= FLT_MAX)) {  // the squares leave the range: again from 2^-80 h (the whole row branches alike)
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j] * 0x1p-80f, v[i][j] * 0x1p-80f, sum);
      rstd = r = 0x1p-80f / sqrtf(row_sum<TPR>(sum, lds[2]) / (float)g.d + g.eps * 0x1p-80f * 0x1p-80f);
    } else if (sum < 0x1p-100f && fabsf(g.eps) < 0x1p-100f) {  // at its other end, and eps does not cover what they lose
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] *= 0x1p100f;
          sum = fmaf(v[i][j], v[i][j], sum);
        }
      r = 1.0f / sqrtf(row_sum<TPR>(sum, lds[2]) / (float)g.d + g.eps * 0x1p100f * 0x1p100f);
      rstd = r * 0x1p100f;
    }
    if (g.rstd != nullptr && l == 0) g.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + l) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r * w[i][j];
      if constexpr (Y == Y_SAME) {
        if (c < g.d) store8<T>((T*)g.y + at + c, v[i]);
      } else if constexpr (Y == Y_E4M3) {
        float sc, inv;
        block_scale(max_lanes16(max8(v[i])), sc, inv);
        if (c < g.d) {
          *(uint2*)((uint8_t*)g.y + at + c) = scale_pack8(v[i], inv);
          if (c % kQB == 0) ((float*)g.scale)[row * ((g.d + kQB - 1) / kQB) + c / kQB] = sc;
        }
      } else {
        uint32_t e;
        const uint32_t q = mx_block(v[i], e);
        if (c < g.d) {
          *(uint32_t*)((uint8_t*)g.y + (at + c) / 2) = q;
          if (c % kMxBlock == 0) ((uint8_t*)g.scale)[(at + c) / kMxBlock] = (uint8_t)e;
        }
      }
    }
  }
}

struct NormBwdArgs {
  const void* dy;
  const void* dh;  // or NULL
  const void* h;
  const void* w;
  int w_f32;
  const float* rstd;
  int rows, d;
  void* dx;
  float* part;     // [row_wgs][d], or NULL: no weight gradient, or by the workgroups from row_wgs on
  void* dw;        // theirs
  int row_wgs;
};

// The weight gradient of 32 columns, straight from dy and h: eight threads take them, 32 row groups.
template <typename T>
__device__ __forceinline__ void dw_columns(const NormBwdArgs& g, int wg) {
  __shared__ float4 lds[4][8];
  const int cl = threadIdx.x & 7, rg = threadIdx.x >> 3, c = wg * 32 + cl * 4;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < g.d) {
#pragma unroll 8
    for (int row = rg; row < g.rows; row += 32) {
      float dy[4], h[4];
      Quad<T>::load((const T*)g.dy + (int64_t)row * g.d + c, dy);
      Quad<T>::load((const T*)g.h + (int64_t)row * g.d + c, h);
      const float r = g.rstd[row];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = fmaf(dy[j], h[j] * r, s[j]);
    }
  }
#pragma unroll
  for (int off = 8; off < 64; off *= 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] += __shfl_xor(s[j], off);
  if ((threadIdx.x & 63) < 8) lds[threadIdx.x >> 6][cl] = make_float4(s[0], s[1], s[2], s[3]);
  __syncthreads();
  if (threadIdx.x < 8 && c < g.d) {
    const float4 a = lds[0][cl], b = lds[1][cl], e = lds[2][cl], f = lds[3][cl];
    const float o[4] = {(a.x + b.x) + (e.x + f.x), (a.y + b.y) + (e.y + f.y), (a.z + b.z) + (e.z + f.z),
                        (a.w + b.w) + (e.w + f.w)};
    if (g.w_f32)
      Quad<float>::store((float*)g.dw + c, o);
    else
      Quad<bf16_t>::store((bf16_t*)g.dw + c, o);
  }
}

// The weight gradient's sum stays in registers over the rows of a workgroup and leaves once as a float32 row (or, of few
// rows, is the business of other workgroups).
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(256) void rms_norm_bwd_kernel(NormBwdArgs g) {
  if ((int)blockIdx.x >= g.row_wgs) return dw_columns<T>(g, blockIdx.x - g.row_wgs);
  constexpr int RPW = 256 / TPR;
  __shared__ float lds[2][4];
  __shared__ float dw_lds[RPW > 1 ? RPW : 1][RPW > 1 ? TPR * NV * 8 : 1];
  const int l = threadIdx.x % TPR;
  float w[NV][8], acc[NV][8];
  load_weights<TPR, NV>(g.w, g.w_f32, l, g.d, w);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  int turn = 0;
  const int64_t stride = (int64_t)g.row_wgs * RPW;
  int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
  Oct<T> hn[NV], yn[NV], nn[NV];  // the next row's values
  float rn = 0.f;
  auto load = [&](int64_t row) __attribute__((always_inline)) {
    const int64_t at = row * g.d;
    rn = g.rstd[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + l) * 8;
      hn[i].zero();
      yn[i].zero();
      nn[i].zero();
      if (c < g.d) {
        hn[i].load((const T*)g.h + at + c);
        yn[i].load((const T*)g.dy + at + c);
        if (g.dh != nullptr) nn[i].load((const T*)g.dh + at + c);
      }
    }
  };
  // rows of up to 4096 are requested one ahead of the sums (118 -> 108 us at 32768 x 2048, with what follows); wider
  // ones keep memory busy with the loads of one
  constexpr bool AHEAD = NV <= 2;
  if (AHEAD && row < g.rows) load(row);
  for (; row < g.rows; row += stride) {
    const int64_t at = row * g.d;
    if (!AHEAD) load(row);
    Oct<T> ho[NV], yo[NV], no[NV];
    const float r = rn;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      ho[i] = hn[i];
      yo[i] = yn[i];
      no[i] = nn[i];
    }
    if (AHEAD && row + stride < g.rows) load(row + stride);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float h[8], dy[8];
      ho[i].get(h);
      yo[i].get(dy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hr = h[j] * r;  // not h alone: its products with g may leave the range
        sum = fmaf(dy[j] * w[i][j], hr, sum);
        acc[i][j] = fmaf(dy[j], hr, acc[i][j]);
      }
    }
    const float mean = row_sum<TPR>(sum, lds[turn]) / (float)g.d;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + l) * 8;
      float h[8], dy[8], o[8];
      ho[i].get(h);
      yo[i].get(dy);
      no[i].get(o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += r * (dy[j] * w[i][j] - h[j] * r * mean);
      if (c < g.d) store8<T>((T*)g.dx + at + c, o);
    }
  }
  if (g.part == nullptr) return;
  float* out = g.part + (size_t)blockIdx.x * g.d;
  if constexpr (RPW > 1) {
    const int u = threadIdx.x / TPR;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) dw_lds[u][(i * TPR + l) * 8 + j] = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < g.d; c += 256) {
      float s = dw_lds[0][c];
#pragma unroll
      for (int k = 1; k < RPW; ++k) s += dw_lds[k][c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + l) * 8;
      if (c < g.d) store8<float>(out + c, acc[i]);
    }
  }
}

// dw = sum of `parts` rows, in a fixed order: a workgroup takes 64 columns, 16 threads four of them, 16 row ranges
template <typename T>
__global__ __launch_bounds__(256) void rms_norm_dw_kernel(const float* __restrict__ part, int parts, int d,
                                                          T* __restrict__ dw) {
  __shared__ float4 lds[16][16];
  const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const int c = blockIdx.x * 64 + cl * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < d) {
#pragma unroll 8
    for (int p = rg; p < parts; p += 16) {
      const float4 v = *(const float4*)(part + (size_t)p * d + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  lds[rg][cl] = s;
  __syncthreads();
  if (rg == 0 && c < d) {
    for (int k = 1; k < 16; ++k) {
      const float4 v = lds[k][cl];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const float o[4] = {s.x, s.y, s.z, s.w};
    Quad<T>::store(dw + c, o);
  }
}

// Lanes of a row and eights of a lane, by the width alone.
template <typename F>
hipError_t by_width(int d, F&& f) {
  if (d <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (d <= 1024) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (d <= 2048) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (d <= 4096) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (d <= 8192) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 8>{});
}
int rows_per_wg(int d) { return d <= 1024 ? 4 : 1; }

template <typename T, int Y>
hipError_t fwd_t(const NormArgs& g, hipStream_t stream) {
  return by_width(g.d, [&](auto tpr, auto nv) {
    const int64_t units = ((int64_t)g.rows + rows_per_wg(g.d) - 1) / rows_per_wg(g.d);
    const unsigned wgs = (unsigned)std::min<int64_t>(units, (int64_t)compute_units() * 8);
    LaunchTimer timer("rms_norm", stream);
    hipLaunchKernelGGL((rms_norm_kernel<T, tpr.value, nv.value, Y>), dim3(wgs), dim3(256), 0, stream, g);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t bwd_t(const NormBwdArgs& g, int wgs, hipStream_t stream) {
  return by_width(g.d, [&](auto tpr, auto nv) {
    LaunchTimer timer("rms_norm_bwd", stream);
    hipLaunchKernelGGL((rms_norm_bwd_kernel<T, tpr.value, nv.value>), dim3(wgs), dim3(256), 0, stream, g);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_rms_norm(int dtype, int w_dtype, const void* x, const void* residual, const void* w, int rows, int d,
                           float eps, int y_format, void* y, void* scale, void* h, float* rstd, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const NormArgs g{x, residual, w, w_dtype == 0, rows, d, eps, y, scale, h, rstd};
  if (y_format == kNormSame) return dtype == 0 ? fwd_t<float, Y_SAME>(g, stream) : fwd_t<bf16_t, Y_SAME>(g, stream);
  if (y_format == kNormE4m3) return dtype == 0 ? fwd_t<float, Y_E4M3>(g, stream) : fwd_t<bf16_t, Y_E4M3>(g, stream);
  return dtype == 0 ? fwd_t<float, Y_MX>(g, stream) : fwd_t<bf16_t, Y_MX>(g, stream);
}

// Workgroups of the backward, each leaving one float32 row of the weight gradient: two for each CU (us at 32768 x 2048,
// two / four: 99 / 108), as many as the registers of rows up to 8192 allow anyway; wider rows take a CU's.
static int bwd_parts(int rows, int d) {
  return std::min((int)(((int64_t)rows + rows_per_wg(d) - 1) / rows_per_wg(d)), kNominalCUs * (d > 8192 ? 1 : 2));
}

// Few rows: the weight gradient needs no second kernel, workgroups beside those of the rows read dy and h again, out of
// the caches (us, bf16, one / two kernels: 64 x 2048 2.8 / 6.1, 333 x 768 3.4 / 7.0, 1024 x 2048
// 5.7 / 10.1, 512 x 8192 12.5 / 17.6; 1024 x 8192 22.5 / 17.8, 2048 x 2048 13.5 / 11.9).
static bool direct_dw(int rows, int d) { return rows <= 1024 && (int64_t)rows * d <= 1024 * 4096; }

size_t rms_norm_bwd_bytes(int rows, int d) { return direct_dw(rows, d) ? 0 : (size_t)bwd_parts(rows, d) * d * 4; }

hipError_t launch_rms_norm_bwd(int dtype, int w_dtype, const void* dy, const void* dh, const void* h, const void* w,
                               const float* rstd, int rows, int d, void* dx, void* dw, void* workspace,
                               hipStream_t stream) {
  const int parts = bwd_parts(rows, d);
  const bool direct = direct_dw(rows, d);
  const NormBwdArgs g{dy, dh, h, w, w_dtype == 0, rstd, rows, d, dx, dw != nullptr && !direct ? (float*)workspace : nullptr,
                      dw, parts};
  const int wgs = parts + (dw != nullptr && direct ? (d + 31) / 32 : 0);
  if (wgs > 0) {  // (without rows the weight gradient is zeros)
    const hipError_t e = dtype == 0 ? bwd_t<float>(g, wgs, stream) : bwd_t<bf16_t>(g, wgs, stream);
    if (e != hipSuccess) return e;
  }
  if (dw == nullptr || direct) return hipSuccess;
  LaunchTimer timer("rms_norm_dw", stream);
  if (w_dtype == 0)
    hipLaunchKernelGGL(rms_norm_dw_kernel<float>, dim3((d + 63) / 64), dim3(256), 0, stream, (const float*)workspace,
                       parts, d, (float*)dw);
  else
    hipLaunchKernelGGL(rms_norm_dw_kernel<bf16_t>, dim3((d + 63) / 64), dim3(256), 0, stream, (const float*)workspace,
                       parts, d, (bf16_t*)dw);
  return hipGetLastError();
}

}  // namespace esg
