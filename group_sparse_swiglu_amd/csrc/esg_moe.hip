// A whole mixture-of-experts layer for a few tokens (at most 64):
//   s[t,e] = sigmoid(x_t . r_e), the chosen experts by the sigmoid top-k rule
//   with an expert bias, p[t,j] their normalised (and scaled) scores, and
//   y[t] = sum over the chosen experts j of
//          p[t,j] (SiLU(x_t W_gate[e]^T) * (x_t W_up[e]^T)) W_down[e]^T.
// Weights are bf16, or e4m3 with a float32 scale per 128 x 128 block.
//
// The layer is a read of the chosen experts' weights: with few tokens the
// matrix cores are idle nearly all the time, so every product is a 16 x 16 x 32
// bf16 one with 16 weight rows on its row side, loaded straight from memory
// into the operand registers, and up to 16 tokens on its column side.  8-bit
// weights are widened to bf16 (exactly) in registers; x stays bf16.
#include <algorithm>

#include "esg_fp8.hpp"
#include "esg_internal.hpp"
#include "esg_pipe.hpp"
#include "esg_route.hpp"

namespace esg {
namespace {

enum { W_BF16 = 0, W_E4M3 = 1 };
constexpr int kChunk = 128;  // K elements a wave takes at a time: one scale block
constexpr int kMoeWaves = 8;

struct MoeArgs {
  const bf16_t* x;        // [T][d]
  const bf16_t* router;   // [E][d]
  const float* bias;      // [E], stride bias_stride
  const void* wg;         // [E][ff][d]
  const void* wu;
  const void* wd;         // [E][d][ff]
  const float* sg;        // scales (8-bit weights): [E][ceil(ff/128)][ceil(d/128)]
  const float* su;
  const float* sd;        // [E][ceil(d/128)][ceil(ff/128)]
  float* scores;          // [T][E]
  bf16_t* h;              // [2][T*k][ff]: p * SiLU(gate) * up of each (token, expert) pair, pairs in expert
                          // order, as the sum of two bf16 values (see gate_up_unit)
  bf16_t* y;              // [T][d]
  float* probs;           // [T][k]
  int64_t* indices;       // [T][k]
  int T, E, k, d, ff, bias_stride, apply_scaling;
  float scaling;
};

// One wave's share of 16 weight rows: kChunk consecutive K of each, four MFMA
// steps of 32.  Lane l holds row l % 16; step s of lane group g = l / 16 covers
// K elements koff(s, g) .. + 7, the same on the other operand.
template <int WT>
struct Rows16;
template <>
struct Rows16<W_BF16> {
  uint4 w[4];
  static __device__ __forceinline__ int koff(int s, int g) { return s * 32 + g * 8; }
  __device__ __forceinline__ void load(const void* row, int k0, int K, bool on, int g) {
    const bf16_t* p = (const bf16_t*)row + k0;
#pragma unroll
    for (int s = 0; s < 4; ++s)
      w[s] = on && k0 + koff(s, g) < K ? *(const uint4*)(p + koff(s, g)) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint4 frag(int s) const { return w[s]; }
};
template <>
struct Rows16<W_E4M3> {
  uint4 w[2];
  static __device__ __forceinline__ int koff(int s, int g) { return (s >> 1) * 64 + g * 16 + (s & 1) * 8; }
  __device__ __forceinline__ void load(const void* row, int k0, int K, bool on, int g) {
    const uint8_t* p = (const uint8_t*)row + k0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = on && k0 + koff(2 * i, g) < K ? *(const uint4*)(p + koff(2 * i, g)) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint4 frag(int s) const {
    const uint4& v = w[s >> 1];
    return (s & 1) ? e4m3x8_to_bf16(v.z, v.w) : e4m3x8_to_bf16(v.x, v.y);
  }
};

// The matching chunk of a column operand (bf16 rows; `on` false: zeros).
template <int WT>
struct Cols16 {
  uint4 v[4];
  __device__ __forceinline__ void load(const bf16_t* row, int k0, int K, bool on, int g) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = k0 + Rows16<WT>::koff(s, g);
      v[s] = on && k < K ? *(const uint4*)(row + k) : make_uint4(0, 0, 0, 0);
    }
  }
};

// acc += (16 rows x 128) . (128 x 16 columns) [* scale]
template <int WT>
__device__ __forceinline__ void mma_chunk128(f32x4& acc, const Rows16<WT>& a, const Cols16<WT>& b, float scale) {
  if constexpr (WT == W_BF16) {
#pragma unroll
    for (int s = 0; s < 4; ++s) mma_bf16(acc, a.frag(s), b.v[s]);
  } else {
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) mma_bf16(t, a.frag(s), b.v[s]);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(t[e], scale, acc[e]);
  }
}

// The same with the columns given as a sum of two, added only in lanes with
// `in`: the other columns' operand is zero, but zero times an infinite or NaN
// weight of an expert that their token did not choose is not.
template <int WT>
__device__ __forceinline__ void mma_chunk128_masked(f32x4& acc, const Rows16<WT>& a, const Cols16<WT> (&b)[2],
                                                    float scale, bool in) {
  f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint4 f = a.frag(s);
    mma_bf16(t, f, b[0].v[s]);
    mma_bf16(t, f, b[1].v[s]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v = WT == W_BF16 ? acc[e] + t[e] : fmaf(t[e], scale, acc[e]);
    acc[e] = in ? v : acc[e];
  }
}

template <int WT>
__device__ __forceinline__ const void* row_ptr(const void* w, size_t row, int K) {
  return (const char*)w + row * K * (WT == W_BF16 ? 2 : 1);
}

// ---------------------------------------------------------------------------
// Scores: 16 experts per workgroup, all tokens; the waves split d.
// ---------------------------------------------------------------------------
template <int MT>
__global__ __launch_bounds__(kMoeWaves * 64) void moe_scores_kernel(MoeArgs g) {
  __shared__ f32x4 red[kMoeWaves][MT][64];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int lr = lane & 15, lg = lane >> 4;
  const int e0 = blockIdx.x * 16;
  const void* row = row_ptr<W_BF16>(g.router, min(e0 + lr, g.E - 1), g.d);
  f32x4 acc[MT];
  zero_acc(acc);
  for (int k0 = w * kChunk; k0 < g.d; k0 += kMoeWaves * kChunk) {
    Rows16<W_BF16> a;
    a.load(row, k0, g.d, true, lg);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int t = j * 16 + lr;
      Cols16<W_BF16> b;
      b.load(g.x + (size_t)t * g.d, k0, g.d, t < g.T, lg);
      mma_chunk128<W_BF16>(acc[j], a, b, 1.0f);
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) red[w][j][lane] = acc[j];
  __syncthreads();
  const float* rf = (const float*)red;
  for (int o = threadIdx.x; o < MT * 256; o += kMoeWaves * 64) {
    const int e = o & 15, t = o >> 4;
    const int at = ((t >> 4) * 64 + (e >> 2) * 16 + (t & 15)) * 4 + (e & 3);
    float s = rf[at];
#pragma unroll
    for (int v = 1; v < kMoeWaves; ++v) s += rf[v * MT * 256 + at];
    if (t < g.T && e0 + e < g.E) g.scores[(size_t)t * g.E + e0 + e] = exact_sigmoid(s);
  }
}

// ---------------------------------------------------------------------------
// Routing of all tokens, repeated by every workgroup (the scores are a few KB):
// which tokens each expert has, and the (token, expert) pairs in expert order.
// ---------------------------------------------------------------------------
template <int EMAX, int TMAX>
struct RouteLds {
  unsigned long long mask[EMAX];         // tokens of each expert
  float sel_s[TMAX][kRouteMaxK];
  int sel_e[TMAX][kRouteMaxK];
  float prob[TMAX * kRouteMaxK];         // of each pair
  uint16_t base[EMAX];                   // first pair of each expert
  uint16_t list[EMAX];                   // experts with tokens, ascending
  uint8_t tok[TMAX * kRouteMaxK];        // token of each pair
  int active;
};

template <int EMAX, int TMAX>
__device__ __forceinline__ void route_all(const MoeArgs& g, RouteLds<EMAX, TMAX>& R, bool write) {
#pragma clang fp contract(off)
  constexpr int C = EMAX / 64;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < g.E; e += kMoeWaves * 64) R.mask[e] = 0;
  __syncthreads();
  for (int t = w; t < g.T; t += kMoeWaves) {
    const float* row = g.scores + (size_t)t * g.E;
    bool valid[C];
    int ex[C];
    float sc[C];
    uint32_t u[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      ex[c] = lane * C + c;
      valid[c] = ex[c] < g.E;
      sc[c] = valid[c] ? row[ex[c]] : 0.f;
      u[c] = order_key(sc[c] + (valid[c] ? g.bias[(size_t)ex[c] * g.bias_stride] : 0.f));
    }
    int need;
    const uint32_t tau = kth_largest<C, 32>(u, valid, g.E, g.k, need);
    place<C>(u, valid, sc, ex, tau, g.k, need, lane, R.sel_s[t], R.sel_e[t]);
    wave_lds_sync();
    float total = 0.0f;
    for (int i = 0; i < g.k; ++i) total = total + R.sel_s[t][i];
    wave_lds_sync();
    if (lane < g.k) {
      float p = R.sel_s[t][lane] / (total + 1e-20f);
      if (g.apply_scaling) p = p * g.scaling;
      const int e = R.sel_e[t][lane];
      R.sel_s[t][lane] = p;
      atomicOr(&R.mask[e], 1ull << t);
      if (write) {
        g.probs[(size_t)t * g.k + lane] = p;
        g.indices[(size_t)t * g.k + lane] = e;
      }
    }
  }
  __syncthreads();
  if (w == 0) {  // active experts and the first pair of each, 64 experts at a time
    int n = 0, pos = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
      const int e = e0 + lane;
      const int cnt = e < g.E ? __popcll(R.mask[e]) : 0;
      const uint64_t on = __ballot(cnt > 0);
      int incl = cnt;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int up = __shfl_up(incl, off);
        if (lane >= off) incl += up;
      }
      if (e < g.E) R.base[e] = (uint16_t)(pos + incl - cnt);
      if (cnt > 0) R.list[n + __popcll(on & ((1ull << lane) - 1ull))] = (uint16_t)e;
      n += __popcll(on);
      pos += __shfl(incl, 63);
    }
    if (lane == 0) R.active = n;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < g.T * g.k; i += kMoeWaves * 64) {
    const int t = i / g.k, j = i - t * g.k;
    const int e = R.sel_e[t][j];
    const int pos = R.base[e] + __popcll(R.mask[e] & ((1ull << t) - 1ull));
    R.prob[pos] = R.sel_s[t][j];
    R.tok[pos] = (uint8_t)t;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Gate and up: 16 neurons of one expert for all its tokens.
// ---------------------------------------------------------------------------
template <int WT, int MT, int EMAX>
__device__ __forceinline__ void gate_up_unit(const MoeArgs& g, const RouteLds<EMAX, MT * 16>& R, f32x4* red, int e,
                                             int n0, int lane, int w) {
  const int lr = lane & 15, lg = lane >> 4;
  const int cnt = __popcll(R.mask[e]), base = R.base[e];
  const int tiles = (cnt + 15) >> 4;
  const size_t wrow = (size_t)e * g.ff + n0 + lr;
  const void* rg = row_ptr<WT>(g.wg, wrow, g.d);
  const void* ru = row_ptr<WT>(g.wu, wrow, g.d);
  const int kb = (g.d + kChunk - 1) / kChunk;
  const size_t srow = WT == W_BF16 ? 0 : ((size_t)e * ((g.ff + kQB - 1) / kQB) + n0 / kQB) * kb;
  const bf16_t* xr[MT];
  bool in[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    in[j] = j * 16 + lr < cnt;
    xr[j] = g.x + (size_t)(in[j] ? R.tok[base + j * 16 + lr] : 0) * g.d;
  }
  f32x4 acc[2][MT];
  zero_acc(acc);
  constexpr int U = 2;
  for (int c0 = w; c0 < kb; c0 += kMoeWaves * U) {
    Rows16<WT> ag[U], au[U];
    float sg[U], su[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * kMoeWaves;
      ag[u].load(rg, c * kChunk, g.d, c < kb, lg);
      au[u].load(ru, c * kChunk, g.d, c < kb, lg);
      sg[u] = WT != W_BF16 && c < kb ? g.sg[srow + c] : 0.f;
      su[u] = WT != W_BF16 && c < kb ? g.su[srow + c] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      if (j < tiles) {
        Cols16<WT> b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) b[u].load(xr[j], (c0 + u * kMoeWaves) * kChunk, g.d, in[j], lg);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          mma_chunk128<WT>(acc[0][j], ag[u], b[u], sg[u]);
          mma_chunk128<WT>(acc[1][j], au[u], b[u], su[u]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j)
    if (j < tiles) {
      red[((w * MT + j) * 2 + 0) * 64 + lane] = acc[0][j];
      red[((w * MT + j) * 2 + 1) * 64 + lane] = acc[1][j];
    }
  __syncthreads();
  const float* rf = (const float*)red;
  for (int o = threadIdx.x; o < tiles * 256; o += kMoeWaves * 64) {
    const int n = o & 15, c = o >> 4;  // neuron, column
    const int at = (c >> 4) * 512 + ((n >> 2) * 16 + (c & 15)) * 4 + (n & 3);
    float hg = rf[at], hu = rf[at + 256];
#pragma unroll
    for (int v = 1; v < kMoeWaves; ++v) {
      hg += rf[v * MT * 512 + at];
      hu += rf[v * MT * 512 + at + 256];
    }
    if (c < cnt) {
      // Rounding h to bf16 alone would add an error as large as that of rounding y (together 1.41 times
      // it); as bf16(h) + bf16(rest) it keeps 16 bits, for one more product per step of the down kernel,
      // whose matrix cores are idle.
      const float a = hg / (1.0f + __expf(-hg)) * hu * R.prob[base + c];
      bf16_t* const at_h = g.h + (size_t)(base + c) * g.ff + n0 + n;
      const uint32_t hi = f32_to_bf16(a);
      const float rest = a - bf16_to_f32(hi);
      at_h->bits = (uint16_t)hi;
      store_elem<bf16_t>(at_h + (size_t)g.T * g.k * g.ff, fabsf(a) < __builtin_inff() ? rest : 0.f);
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Down: 16 columns of y for all tokens; the waves take (expert, K chunk) items
// in turn and sum over the experts in the products' accumulators.
// ---------------------------------------------------------------------------
template <int WT, int MT, int EMAX>
__device__ __forceinline__ void down_unit(const MoeArgs& g, const RouteLds<EMAX, MT * 16>& R, f32x4* red, int d0,
                                          int lane, int w) {
  const int lr = lane & 15, lg = lane >> 4;
  const int kb = (g.ff + kChunk - 1) / kChunk, db = (g.d + kQB - 1) / kQB;
  const int items = R.active * kb;
  f32x4 acc[MT];
  zero_acc(acc);
  constexpr int U = 4;
  for (int i0 = w; i0 < items; i0 += kMoeWaves * U) {
    Rows16<WT> a[U];
    float s[U];
    int ex[U], kc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u * kMoeWaves, items - 1);
      ex[u] = __builtin_amdgcn_readfirstlane((int)R.list[i / kb]);
      kc[u] = i % kb;
      a[u].load(row_ptr<WT>(g.wd, (size_t)ex[u] * g.d + d0 + lr, g.ff), kc[u] * kChunk, g.ff,
                i0 + u * kMoeWaves < items, lg);
      s[u] = WT != W_BF16 ? g.sd[((size_t)ex[u] * db + d0 / kQB) * kb + kc[u]] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * kMoeWaves >= items) continue;
      const unsigned long long mask = R.mask[ex[u]];
      const int base = R.base[ex[u]];
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        if (((mask >> (j * 16)) & 0xffffull) == 0) continue;
        const int t = j * 16 + lr;
        const bool in = (mask >> t) & 1;
        const int pos = base + __popcll(mask & ((1ull << t) - 1ull));
        Cols16<WT> b[2];
        b[0].load(g.h + (size_t)pos * g.ff, kc[u] * kChunk, g.ff, in, lg);
        b[1].load(g.h + ((size_t)g.T * g.k + pos) * g.ff, kc[u] * kChunk, g.ff, in, lg);
        mma_chunk128_masked<WT>(acc[j], a[u], b, s[u], in);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) red[(w * MT + j) * 64 + lane] = acc[j];
  __syncthreads();
  const float* rf = (const float*)red;
  for (int o = threadIdx.x; o < MT * 256; o += kMoeWaves * 64) {
    const int n = o & 15, t = o >> 4;
    const int at = ((t >> 4) * 64 + (n >> 2) * 16 + (t & 15)) * 4 + (n & 3);
    float v = rf[at];
#pragma unroll
    for (int q = 1; q < kMoeWaves; ++q) v += rf[q * MT * 256 + at];
    if (t < g.T) store_elem<bf16_t>(g.y + (size_t)t * g.d + d0 + n, v);
  }
  __syncthreads();
}

template <int WT, int MT, int EMAX>
__global__ __launch_bounds__(kMoeWaves * 64) void moe_gate_up_kernel(MoeArgs g) {
  __shared__ RouteLds<EMAX, MT * 16> R;
  __shared__ f32x4 red[kMoeWaves * MT * 2 * 64];
  route_all<EMAX, MT * 16>(g, R, blockIdx.x == 0);
  const int lane = threadIdx.x & 63, w = wave_id();
  const int nt = g.ff / 16, units = R.active * nt;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int a = u / nt;
    gate_up_unit<WT, MT, EMAX>(g, R, red, R.list[a], (u - a * nt) * 16, lane, w);
  }
}

template <int WT, int MT, int EMAX>
__global__ __launch_bounds__(kMoeWaves * 64) void moe_down_kernel(MoeArgs g) {
  __shared__ RouteLds<EMAX, MT * 16> R;
  __shared__ f32x4 red[kMoeWaves * MT * 64];
  route_all<EMAX, MT * 16>(g, R, false);
  const int lane = threadIdx.x & 63, w = wave_id();
  for (int u = blockIdx.x; u < g.d / 16; u += gridDim.x) down_unit<WT, MT, EMAX>(g, R, red, u * 16, lane, w);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int WT, int MT, int EMAX>
hipError_t launch_t(const MoeArgs& g, hipStream_t stream) {
  const dim3 block(kMoeWaves * 64);
  {
    LaunchTimer timer("moe_scores", stream);
    hipLaunchKernelGGL(moe_scores_kernel<MT>, dim3((g.E + 15) / 16), block, 0, stream, g);
  }
  const int cus = compute_units();
  {
    LaunchTimer timer("moe_gate_up", stream);
    const long long most = (long long)std::min(g.E, g.T * g.k) * (g.ff / 16);
    hipLaunchKernelGGL((moe_gate_up_kernel<WT, MT, EMAX>), dim3((unsigned)std::min<long long>(most, 2 * cus)), block,
                       0, stream, g);
  }
  LaunchTimer timer("moe_down", stream);
  hipLaunchKernelGGL((moe_down_kernel<WT, MT, EMAX>), dim3(std::min(g.d / 16, 2 * cus)), block, 0, stream, g);
  return hipGetLastError();
}

template <int WT, int MT>
hipError_t launch_e(const MoeArgs& g, hipStream_t stream) {
  return g.E <= 256 ? launch_t<WT, MT, 256>(g, stream) : launch_t<WT, MT, kMoeMaxExperts>(g, stream);
}

template <int WT>
hipError_t launch_m(const MoeArgs& g, hipStream_t stream) {
  if (g.T <= 16) return launch_e<WT, 1>(g, stream);
  return g.T <= 32 ? launch_e<WT, 2>(g, stream) : launch_e<WT, 4>(g, stream);
}

}  // namespace

size_t moe_decode_workspace_bytes(int tokens, int experts, int topk, int d_ff) {
  return align256((size_t)tokens * experts * 4) + align256((size_t)tokens * topk * d_ff * 4);
}

hipError_t launch_moe_decode(const MoeCall& c, void* workspace, hipStream_t stream) {
  MoeArgs g{};
  g.x = (const bf16_t*)c.x;
  g.router = (const bf16_t*)c.w_router;
  g.bias = c.expert_bias;
  g.wg = c.w_gate;
  g.wu = c.w_up;
  g.wd = c.w_down;
  g.sg = c.s_gate;
  g.su = c.s_up;
  g.sd = c.s_down;
  g.scores = (float*)workspace;
  g.h = (bf16_t*)((char*)workspace + align256((size_t)c.tokens * c.experts * 4));
  g.y = (bf16_t*)c.y;
  g.probs = c.probs;
  g.indices = c.indices;
  g.T = c.tokens;
  g.E = c.experts;
  g.k = c.topk;
  g.d = c.d_model;
  g.ff = c.d_ff;
  g.bias_stride = c.bias_stride;
  g.scaling = c.scaling;
  g.apply_scaling = c.apply_scaling;
  return c.w_dtype == 1 ? launch_m<W_BF16>(g, stream) : launch_m<W_E4M3>(g, stream);
}

}  // namespace esg
