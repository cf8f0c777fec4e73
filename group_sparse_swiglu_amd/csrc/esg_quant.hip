// Quantisation to 8-bit floating point (e4m3) with a float32 scale per block
// of 128.  For a block with largest magnitude a (at least 2^-100):
//   scale = a / 448,  q = e4m3(x * (448 / a)),
// every operation rounded once to float32, the last one to nearest even.
// Blocks are 1 x 128 (rows), 128 x 1 written transposed (columns), or
// 128 x 128 (tiles, whose transpose has the same bytes and scales).
//
// All forms are bound by memory: 2 or 4 bytes are read per element, 1 or 2
// written, and about 8 vector instructions spent.  The quotient 448 / a and the
// scale are computed once per block, in float32, and one product rounds each
// element before its conversion, so a plain float32 program gives the same bytes.
#include <algorithm>
#include <type_traits>

#include "esg_fp8.hpp"
#include "esg_internal.hpp"

namespace esg {
namespace {

// Row blocks only.  16 lanes take one block (8 elements each), kUnroll blocks
// per lane group in flight.  A call of 64 x 2048 takes 2.8 us on the device, which
// is about what an empty launch takes; its 0.4 MB would need 0.1.
constexpr int kUnroll = 2;

template <typename T>
__global__ __launch_bounds__(256) void quant_rows_kernel(const T* __restrict__ x, int64_t blocks, int cols, int kb,
                                                         uint8_t* __restrict__ q, float* __restrict__ scale) {
  const int g = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t stride = (int64_t)gridDim.x * 16 * kUnroll;
  for (int64_t b0 = ((int64_t)blockIdx.x * 16 + g) * kUnroll; b0 < blocks; b0 += stride) {
    Oct<T> o[kUnroll];
    int64_t at[kUnroll];
    bool in[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t b = b0 + u;
      const int64_t r = b / kb;
      const int c = (int)(b - r * kb) * kQB + l * 8;
      in[u] = b < blocks && c < cols;
      at[u] = r * cols + c;
      o[u].zero();
      if (in[u]) o[u].load(x + at[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float v[8], s, inv;
      o[u].get(v);
      block_scale(max_lanes16(max8(v)), s, inv);
      if (in[u]) *(uint2*)(q + at[u]) = scale_pack8(v, inv);
      if (l == 0 && b0 + u < blocks) scale[b0 + u] = s;
    }
  }
}

// One 128 x 128 tile per workgroup, held in registers: thread t has rows
// (t / 16) * 8 + 0..7 and columns (t % 16) * 8 + 0..7, so both the row and the
// column blocks' maxima and both outputs come from one read.  The transposed
// bytes go through LDS so that 128 bytes of an output row are written together.
// Both directions of 32768 x 2048 in bf16 (273 MB): 53 to 59 us, 4.6 to 5.1 TB/s, as
// fast as a plain copy of 256 MB (5.07 TB/s); two passes would read the input twice
// (half as many bytes again).
enum { Q_BOTH = 0, Q_TILE = 1, Q_TILE_T = 2 };

// position of the 16-byte chunk c of transposed row r in its 128-byte LDS row
__device__ __forceinline__ int tchunk(int r, int c) { return r * 128 + ((c ^ (r >> 3) ^ r) & 7) * 16; }

template <int MODE>
struct TileLds {
  uint32_t part[4][kQB];
  __attribute__((aligned(16))) char tr[MODE == Q_TILE ? 16 : kQB * kQB];
};

template <typename T>
struct TileArgs {
  const T* x;
  int rows, cols, rows_pad;
  uint8_t* q;
  float* scale;
  uint8_t* qt;
  float* scale_t;
};

template <typename T, int MODE, typename Lds>
__device__ __forceinline__ void quant_tile(const TileArgs<T>& g, unsigned block, Lds& lds) {
  uint32_t(&part)[4][kQB] = lds.part;
  char* tr = lds.tr;
  const int rows = g.rows, cols = g.cols, rows_pad = g.rows_pad;
  const T* __restrict__ x = g.x;
  uint8_t* __restrict__ q = g.q;
  float* __restrict__ scale = g.scale;
  uint8_t* __restrict__ qt = g.qt;
  float* __restrict__ scale_t = g.scale_t;
  const int nb = (rows + kQB - 1) / kQB, kb = (cols + kQB - 1) / kQB;
  // column tiles vary fastest: neighbouring workgroups read neighbouring parts of the same rows
  const int64_t tiles = (int64_t)nb * kb;
  const int64_t z = block / tiles;
  const int64_t rest = block - z * tiles;
  const int ti = (int)(rest / kb), tj = (int)(rest % kb);
  x += z * rows * cols;
  q += z * rows * cols;
  scale += z * (MODE == Q_BOTH ? (int64_t)rows * kb : tiles);
  if constexpr (MODE != Q_TILE) {
    qt += z * rows_pad * cols;
    scale_t += z * (MODE == Q_BOTH ? (int64_t)cols * nb : tiles);
  }
  const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
  const int r0 = ti * kQB + rg * 8, c0 = tj * kQB + cg * 8;
  Oct<T> o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o[i].zero();
    if (r0 + i < rows && c0 < cols) o[i].load(x + (int64_t)(r0 + i) * cols + c0);
  }
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i].get(v[i]);

  float inv_r[8], inv_c[8];
  if constexpr (MODE == Q_BOTH) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s;
      block_scale(max_lanes16(max8(v[i])), s, inv_r[i]);
      if (cg == 0 && r0 + i < rows) scale[(int64_t)(r0 + i) * kb + tj] = s;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = mag(v[0][j]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = umax(m, mag(v[i][j]));
      m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
      m = umax(m, (uint32_t)__shfl_xor((int)m, 32));
      if ((tid & 48) == 0) part[tid >> 6][cg * 8 + j] = m;
    }
    __syncthreads();
    const int cc = tid & 127;
    const uint32_t m = umax(umax(part[0][cc], part[1][cc]), umax(part[2][cc], part[3][cc]));
    float s, inv;
    block_scale(m, s, inv);
    __syncthreads();
    if (tid < kQB) {
      part[0][cc] = __float_as_uint(inv);
      if (tj * kQB + cc < cols) scale_t[(int64_t)(tj * kQB + cc) * nb + ti] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) inv_c[j] = __uint_as_float(part[0][cg * 8 + j]);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, max8(v[i]));
    m = max_lanes16(m);
    m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
    m = umax(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((tid & 63) == 0) part[tid >> 6][0] = m;
    __syncthreads();
    m = umax(umax(part[0][0], part[1][0]), umax(part[2][0], part[3][0]));
    float s;
    block_scale(m, s, inv_r[0]);
    if (tid == 0) {
      scale[(int64_t)ti * kb + tj] = s;
      if constexpr (MODE == Q_TILE_T) scale_t[(int64_t)tj * nb + ti] = s;
    }
#pragma unroll
    for (int i = 1; i < 8; ++i) inv_r[i] = inv_r[0];
#pragma unroll
    for (int j = 0; j < 8; ++j) inv_c[j] = inv_r[0];
  }

#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + i < rows && c0 < cols) *(uint2*)(q + (int64_t)(r0 + i) * cols + c0) = scale_pack8(v[i], inv_r[i]);

  if constexpr (MODE != Q_TILE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = v[i][j];
      *(uint2*)(tr + tchunk(cg * 8 + j, rg >> 1) + (rg & 1) * 8) = scale_pack8(w, inv_c[j]);
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int r = p * 32 + (tid >> 3), c = tid & 7;  // transposed row, 16-byte chunk
      const int col = tj * kQB + r, row = ti * kQB + c * 16;
      // rows_pad is a multiple of 16: a chunk lies inside or outside as a whole; rows past the input are zeros
      if (col < cols && row < rows_pad) *(uint4*)(qt + (int64_t)col * rows_pad + row) = *(const uint4*)(tr + tchunk(r, c));
    }
  }
}

template <typename T, int MODE>
__global__ __launch_bounds__(256) void quant_tile_kernel(TileArgs<T> g) {
  __shared__ TileLds<MODE> lds;
  quant_tile<T, MODE>(g, blockIdx.x, lds);
}

// Weights in tiles and rows in both directions, side by side: for a linear layer of a few hundred tokens each alone is
// a few dozen workgroups, as long as its memory latency (333 x 768 and 2048 x 768: 5.0 and 6.4 us one after the other).
template <typename TW, int MODE, typename TX>
__global__ __launch_bounds__(256) void quant_pair_kernel(TileArgs<TW> w, TileArgs<TX> x, unsigned wtiles) {
  __shared__ TileLds<Q_BOTH> lds;
  if (blockIdx.x < wtiles)
    quant_tile<TW, MODE>(w, blockIdx.x, lds);
  else
    quant_tile<TX, Q_BOTH>(x, blockIdx.x - wtiles, lds);
}

int64_t tiles_of(int rows, int cols) { return (int64_t)((rows + kQB - 1) / kQB) * ((cols + kQB - 1) / kQB); }

template <typename TW, typename TX>
hipError_t pair_t(const TileArgs<TW>& w, const TileArgs<TX>& x, hipStream_t stream) {
  const unsigned wt = (unsigned)tiles_of(w.rows, w.cols), all = wt + (unsigned)tiles_of(x.rows, x.cols);
  LaunchTimer timer("quant_pair", stream);
  if (w.qt != nullptr)
    hipLaunchKernelGGL((quant_pair_kernel<TW, Q_TILE_T, TX>), dim3(all), dim3(256), 0, stream, w, x, wt);
  else
    hipLaunchKernelGGL((quant_pair_kernel<TW, Q_TILE, TX>), dim3(all), dim3(256), 0, stream, w, x, wt);
  return hipGetLastError();
}

template <typename T>
hipError_t rows_t(const T* x, int rows, int cols, uint8_t* q, float* scale, uint8_t* qt, float* scale_t,
                  hipStream_t stream) {
  const int kb = (cols + kQB - 1) / kQB;
  if (qt != nullptr) {
    LaunchTimer timer("quant_both", stream);
    hipLaunchKernelGGL((quant_tile_kernel<T, Q_BOTH>), dim3((unsigned)tiles_of(rows, cols)), dim3(256), 0, stream,
                       (TileArgs<T>{x, rows, cols, (rows + 15) / 16 * 16, q, scale, qt, scale_t}));
    return hipGetLastError();
  }
  const int64_t blocks = (int64_t)rows * kb;
  const int64_t wgs = std::min<int64_t>((blocks + 16 * kUnroll - 1) / (16 * kUnroll), (int64_t)compute_units() * 8);
  LaunchTimer timer("quant_rows", stream);
  hipLaunchKernelGGL(quant_rows_kernel<T>, dim3((unsigned)wgs), dim3(256), 0, stream, x, blocks, cols, kb, q, scale);
  return hipGetLastError();
}

template <typename T>
hipError_t tiles_t(const T* w, int batch, int rows, int cols, uint8_t* q, float* scale, uint8_t* qt, float* scale_t,
                   hipStream_t stream) {
  const unsigned tiles = (unsigned)(batch * tiles_of(rows, cols));
  const TileArgs<T> g{w, rows, cols, (rows + 15) / 16 * 16, q, scale, qt, scale_t};
  LaunchTimer timer("quant_tiles", stream);
  if (qt != nullptr)
    hipLaunchKernelGGL((quant_tile_kernel<T, Q_TILE_T>), dim3(tiles), dim3(256), 0, stream, g);
  else
    hipLaunchKernelGGL((quant_tile_kernel<T, Q_TILE>), dim3(tiles), dim3(256), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_rows(int dtype, const void* x, int rows, int cols, void* q, float* scale, void* qt,
                             float* scale_t, hipStream_t stream) {
  return dtype == 0 ? rows_t((const float*)x, rows, cols, (uint8_t*)q, scale, (uint8_t*)qt, scale_t, stream)
                    : rows_t((const bf16_t*)x, rows, cols, (uint8_t*)q, scale, (uint8_t*)qt, scale_t, stream);
}

hipError_t launch_quant_tiles(int dtype, const void* w, int batch, int rows, int cols, void* q, float* scale, void* qt,
                              float* scale_t, hipStream_t stream) {
  return dtype == 0 ? tiles_t((const float*)w, batch, rows, cols, (uint8_t*)q, scale, (uint8_t*)qt, scale_t, stream)
                    : tiles_t((const bf16_t*)w, batch, rows, cols, (uint8_t*)q, scale, (uint8_t*)qt, scale_t, stream);
}

hipError_t launch_quant_pair(int w_dtype, const void* w, int w_rows, void* wq, float* w_scale, void* wqt,
                             float* w_scale_t, int x_dtype, const void* x, int x_rows, void* xq, float* x_scale,
                             void* xqt, float* x_scale_t, int cols, hipStream_t stream) {
  if (tiles_of(w_rows, cols) + tiles_of(x_rows, cols) >= 1 << 24) {  // a launch's threads within 2^32
    const hipError_t e = launch_quant_tiles(w_dtype, w, 1, w_rows, cols, wq, w_scale, wqt, w_scale_t, stream);
    return e != hipSuccess ? e : launch_quant_rows(x_dtype, x, x_rows, cols, xq, x_scale, xqt, x_scale_t, stream);
  }
  auto args = [&](auto* p, int rows, void* q, float* scale, void* qt, float* scale_t) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    return TileArgs<T>{p, rows, cols, (rows + 15) / 16 * 16, (uint8_t*)q, scale, (uint8_t*)qt, scale_t};
  };
  auto with_w = [&](const auto& gw) {
    return x_dtype == 0 ? pair_t(gw, args((const float*)x, x_rows, xq, x_scale, xqt, x_scale_t), stream)
                        : pair_t(gw, args((const bf16_t*)x, x_rows, xq, x_scale, xqt, x_scale_t), stream);
  };
  return w_dtype == 0 ? with_w(args((const float*)w, w_rows, wq, w_scale, wqt, w_scale_t))
                      : with_w(args((const bf16_t*)w, w_rows, wq, w_scale, wqt, w_scale_t));
}

}  // namespace esg
