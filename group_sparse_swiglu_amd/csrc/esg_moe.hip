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
//
// Two launches: the scores, and everything else.  Measured (both, bytes of the
// chosen experts' weights over the whole time): one token, 8 of 256 experts, d =
// 2048, d_ff = 1024, bf16: 37.4 us, 2.7 TB/s; five tokens, d_ff = 1008, 8-bit: 70 us,
// 3.4 TB/s; 64 tokens, 6 of 64 experts, d_ff = 1408, 8-bit: 152 us, 3.6 TB/s.  The gate
// and up products themselves read at 5.2 TB/s; the rest is the way between the
// parts: scores 5 us, start and routing 4 to 12, waiting for the last h 3 to 10.
#include <algorithm>
#include <type_traits>

#include "esg_fp8.hpp"
#include "esg_internal.hpp"
#include "esg_pipe.hpp"
#include "esg_route.hpp"

namespace esg {
namespace {

enum { W_BF16 = 0, W_E4M3 = 1 };
constexpr int kChunk = 128;  // K elements a wave takes at a time: one scale block
constexpr int kMoeWaves = 8;
constexpr int kMoeMaxGrid = 1024;  // workgroups of the experts' launch
constexpr int kMaxSplits = 8;      // parts of the down items
// 16-row tiles of a down unit: they share the loads of h, which go past the L2 (64 tokens, 6 of 64 experts, d = 2048,
// d_ff = 1408, 8-bit: down part 62 us with one tile, 44 with two).  One where h is small beside the weights (up to 16
// tokens), and with 16-bit weights, where two tiles in flight do not fit the registers.
__host__ __device__ constexpr int down_tiles(bool e4m3, bool many) { return e4m3 && many ? 2 : 1; }

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
  float* part;            // [splits][d/16][T][16]: the parts of y where the down items are split
  int* flags;             // [kMoeMaxGrid]: workgroups whose gate/up units are done
  int* tickets;           // [kMoeMaxGrid]: units taken, of each team
  int* arrived;           // [d/16]: workgroups done with a tile of y
  int T, E, k, d, ff, bias_stride, apply_scaling;
  int splits;             // parts of the down items
  int teams;              // workgroups that run on CUs of their own
  int patience;           // polls before a workgroup does others' gate/up units itself
  float scaling;
};

// One wave's share of 16 weight rows: kChunk consecutive K of each, four MFMA
// steps of 32.  Lane l holds row l % 16; step s of lane group g = l / 16 covers
// K elements koff(s, g) .. + 7, the same on the other operand.  Buffer loads:
// what lies past K, or belongs to no row, is an offset past the buffer and
// reads zeros, without a branch.
constexpr int kDevice = 16;  // sc1 bit of a buffer access: device scope (past the caches that XCDs do not share)
template <int CPOL = 0>
__device__ __forceinline__ uint4 load16(rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(uint4, (i32x4_t)__builtin_amdgcn_raw_buffer_load_b128(r, off, 0, CPOL));
}

template <int WT>
struct Rows16;
template <>
struct Rows16<W_BF16> {
  uint4 w[4];
  static __device__ __forceinline__ int koff(int s, int g) { return s * 32 + g * 8; }
  // r: the 16 rows of K elements; row: this lane's
  __device__ __forceinline__ void load(rsrc_t r, int row, int k0, int K, int g) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = k0 + koff(s, g);
      w[s] = load16(r, k < K ? (uint32_t)(row * K + k) * 2 : kOOB);
    }
  }
  __device__ __forceinline__ uint4 frag(int s) const { return w[s]; }
};
template <>
struct Rows16<W_E4M3> {
  uint4 w[2];
  static __device__ __forceinline__ int koff(int s, int g) { return (s >> 1) * 64 + g * 16 + (s & 1) * 8; }
  __device__ __forceinline__ void load(rsrc_t r, int row, int k0, int K, int g) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = k0 + koff(2 * i, g);
      w[i] = load16(r, k < K ? (uint32_t)(row * K + k) : kOOB);
    }
  }
  __device__ __forceinline__ uint4 frag(int s) const {
    const uint4& v = w[s >> 1];
    return (s & 1) ? e4m3x8_to_bf16(v.z, v.w) : e4m3x8_to_bf16(v.x, v.y);
  }
};

// Buffer over 16 weight rows of K elements from row `row` (uniform).
template <int WT>
__device__ __forceinline__ rsrc_t rows_rsrc(const void* w, size_t row, int K, int rows = 16) {
  constexpr int B = WT == W_BF16 ? 2 : 1;
  return make_rsrc((const char*)w + row * K * B, (uint32_t)(rows * K * B));
}

// The matching chunk of a column operand: bf16 elements `at` (32-bit, of the
// buffer's start) and on (`on` false: zeros).
template <int WT, int CPOL = 0>
struct Cols16 {
  uint4 v[4];
  __device__ __forceinline__ void load(rsrc_t r, uint32_t at, int k0, int K, bool on, int g) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = k0 + Rows16<WT>::koff(s, g);
      v[s] = load16<CPOL>(r, on && k < K ? (at + k) * 2 : kOOB);
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

// ---------------------------------------------------------------------------
// Scores: 4 experts and 16 tokens per workgroup (the other rows of the products
// are zeros); the waves split d.  Also clears the counters of the launch that
// follows.  Bound by latency: 5.3 us for one token and 256 experts (1 MB), 5.5 for
// 64 tokens and 64 experts (6.3 with 16 experts per workgroup, whose few CUs read
// too much each).
// ---------------------------------------------------------------------------
constexpr int kScoreWaves = 16, kScoreRows = 4;

__global__ __launch_bounds__(kScoreWaves * 64) void moe_scores_kernel(MoeArgs g) {
  __shared__ f32x4 red[kScoreWaves][64];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int lr = lane & 15, lg = lane >> 4;
  const int e0 = blockIdx.x * kScoreRows, t0 = blockIdx.y * 16;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < 2 * kMoeMaxGrid + g.d / 16; i += kScoreWaves * 64) g.flags[i] = 0;
  const rsrc_t rr = rows_rsrc<W_BF16>(g.router, e0, g.d, min(kScoreRows, g.E - e0));  // the other rows read zeros
  const rsrc_t rx = make_rsrc(g.x, (uint32_t)(g.T * g.d * 2));
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = w * kChunk; k0 < g.d; k0 += kScoreWaves * kChunk) {
    Rows16<W_BF16> a;
    Cols16<W_BF16> b;
    a.load(rr, lr, k0, g.d, lg);
    b.load(rx, (t0 + lr) * g.d, k0, g.d, t0 + lr < g.T, lg);
    mma_chunk128<W_BF16>(acc, a, b, 1.0f);
  }
  red[w][lane] = acc;
  __syncthreads();
  if (threadIdx.x >= kScoreRows * 16) return;
  const int e = threadIdx.x % kScoreRows, t = threadIdx.x / kScoreRows;
  if (t0 + t >= g.T || e0 + e >= g.E) return;
  const float* rf = (const float*)red;
  const int at = ((e >> 2) * 16 + t) * 4 + (e & 3);
  float s = rf[at];
#pragma unroll
  for (int v = 1; v < kScoreWaves; ++v) s += rf[v * 256 + at];
  g.scores[(size_t)(t0 + t) * g.E + e0 + e] = exact_sigmoid(s);
}

// ---------------------------------------------------------------------------
// Routing of all tokens, repeated by every workgroup (the scores are a few KB):
// which tokens each expert has, and the (token, expert) pairs in expert order.
// ---------------------------------------------------------------------------
template <int EMAX, int TMAX>
struct RouteLds {
  float prob[TMAX * kRouteMaxK];         // of each pair
  uint32_t act[EMAX];                    // experts with tokens, ascending: expert | first pair << 10 | pairs << 21
  uint8_t tok[TMAX * kRouteMaxK];        // token of each pair
  int active;
};
template <int EMAX, int TMAX>
struct RouteScratch {                    // during the routing only
  unsigned long long mask[EMAX];         // tokens of each expert
  float sel_s[TMAX][kRouteMaxK];
  int sel_e[TMAX][kRouteMaxK];
  uint16_t base[EMAX];                   // first pair of each expert with tokens
};
static_assert(kMoeMaxExperts <= 1 << 10 && 64 * kRouteMaxK <= 1 << 11, "fields of act");

// One data-parallel move inside the vector unit: the value of another lane of
// the wavefront (ctrl), zero where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, true);
}
// lanes 1, 2, 4, 8 below inside a row of 16; then lane 15 of a row to the next row, lane 31 to the upper half
template <class Op>
__device__ __forceinline__ uint32_t wave_scan_u32(uint32_t v, Op op) {
  v = op(v, dpp_u32<0x111, 0xf>(v));
  v = op(v, dpp_u32<0x112, 0xf>(v));
  v = op(v, dpp_u32<0x114, 0xf>(v));
  v = op(v, dpp_u32<0x118, 0xf>(v));
  v = op(v, dpp_u32<0x142, 0xa>(v));
  v = op(v, dpp_u32<0x143, 0xc>(v));
  return v;
}
// largest value of the wavefront, as a scalar, of each of N rows
template <int N>
__device__ __forceinline__ void wave_max_rows(uint32_t (&v)[N]) {
  auto step = [&](auto ctrl, auto rows) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t o = dpp_u32<decltype(ctrl)::value, decltype(rows)::value>(v[i]);
      v[i] = o > v[i] ? o : v[i];
    }
  };
  using std::integral_constant;
  step(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});
  step(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (uint32_t)__builtin_amdgcn_readlane((int)v[i], 63);
}
// sums of the lanes up to each
__device__ __forceinline__ int wave_prefix_sum(int v) {
  return (int)wave_scan_u32((uint32_t)v, [](uint32_t a, uint32_t b) { return a + b; });
}

// Top-k of one token row (the rule of esg_sigmoid_topk_routing).  With the small
// k of an expert layer, k maxima over the wavefront are quicker than a radix
// descent over the key bits: each lane keeps its C keys in descending order, so
// a pick is a maximum over the lanes' first keys (about 150 cycles) and a shift
// in the lane that held it.  The picks come by descending key, equal keys by
// ascending expert; lane i keeps the i-th.  Outputs, in lane i < k: the expert
// and score of the i-th in output order (keys above the k-th largest by
// ascending expert, then the ones equal to it).
// RW rows at a time: their chains of dependent instructions fill each other's waits.
template <int C, int RW>
__device__ __forceinline__ void topk_rows(const float (&sc)[RW][C], const uint32_t (&key)[RW][C], int k, int lane,
                                          int (&expert)[RW], float (&score)[RW]) {
  uint32_t u[RW][C];
  int c_of[RW][C];
#pragma unroll
  for (int r = 0; r < RW; ++r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      u[r][c] = key[r][c];
      c_of[r][c] = c;
    }
#pragma unroll
    for (int i = 1; i < C; ++i)  // insertion: equal keys keep their order
#pragma unroll
      for (int j = i; j > 0; --j) {
        const bool up = u[r][j] > u[r][j - 1];
        const uint32_t a = u[r][j - 1];
        const int b = c_of[r][j - 1];
        u[r][j - 1] = up ? u[r][j] : a;
        u[r][j] = up ? a : u[r][j];
        c_of[r][j - 1] = up ? c_of[r][j] : b;
        c_of[r][j] = up ? b : c_of[r][j];
      }
  }
  int my_e[RW] = {};
  uint32_t my_key[RW] = {}, kth[RW] = {};
  for (int i = 0; i < k; ++i) {
    uint32_t best[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) best[r] = u[r][0];
    wave_max_rows(best);
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      kth[r] = best[r];
      const int from = __ffsll((unsigned long long)__ballot(u[r][0] == kth[r])) - 1;
      const int e = from * C + __builtin_amdgcn_readlane(c_of[r][0], from);
      my_e[r] = lane == i ? e : my_e[r];
      my_key[r] = lane == i ? kth[r] : my_key[r];
      const bool pop = lane == from;
#pragma unroll
      for (int c = 0; c + 1 < C; ++c) {
        u[r][c] = pop ? u[r][c + 1] : u[r][c];
        c_of[r][c] = pop ? c_of[r][c + 1] : c_of[r][c];
      }
      u[r][C - 1] = pop ? 0u : u[r][C - 1];  // candidates' keys are at least 1
    }
  }
  int id[RW], slot[RW] = {};
  float my_s[RW] = {};
#pragma unroll
  for (int r = 0; r < RW; ++r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float v = __shfl(sc[r][c], my_e[r] / C);
      my_s[r] = my_e[r] % C == c ? v : my_s[r];
    }
    // output order: rank of (equal to the k-th, expert) among the k picks
    id[r] = (my_key[r] == kth[r] ? 1 << 16 : 0) | my_e[r];
  }
  for (int i = 0; i < k; ++i)
#pragma unroll
    for (int r = 0; r < RW; ++r) slot[r] += __builtin_amdgcn_readlane(id[r], i) < id[r] ? 1 : 0;
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int to = (lane < k ? slot[r] : lane) * 4;
    expert[r] = __builtin_amdgcn_ds_permute(to, my_e[r]);
    score[r] = __uint_as_float((uint32_t)__builtin_amdgcn_ds_permute(to, (int)__float_as_uint(my_s[r])));
  }
}

// Selection and weights of every token; probabilities and token sets into LDS.
template <int C, int EMAX, int TMAX>
__device__ __forceinline__ void select_tokens(const MoeArgs& g, RouteScratch<EMAX, TMAX>& S, bool write) {
#pragma clang fp contract(off)
  constexpr int RW = TMAX == 16 || C > 4 ? 1 : C > 1 ? 2 : 4;  // tokens of a wave at a time (registers)
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float bias[C], nxt[RW][C];
  bool valid[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = lane * C + c;
    valid[c] = e < g.E;
    bias[c] = valid[c] ? g.bias[(size_t)e * g.bias_stride] : 0.f;
  }
  auto load = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int t = t0 + r * kMoeWaves;
        nxt[r][c] = valid[c] && t < g.T ? g.scores[(size_t)t * g.E + lane * C + c] : 0.f;
      }
  };
  load(w);
  for (int t0 = w; t0 < g.T; t0 += RW * kMoeWaves) {
    float sc[RW][C];
    uint32_t key[RW][C];
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        sc[r][c] = nxt[r][c];
        const uint32_t o = order_key(sc[r][c] + bias[c]);
        key[r][c] = valid[c] ? (o > 1u ? o : 1u) : 0u;
      }
    load(t0 + RW * kMoeWaves);
    int e[RW];
    float s[RW], total[RW] = {};
    topk_rows<C, RW>(sc, key, g.k, lane, e, s);
    for (int i = 0; i < g.k; ++i)
#pragma unroll
      for (int r = 0; r < RW; ++r)
        total[r] = total[r] + __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(s[r]), i));
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int t = t0 + r * kMoeWaves;
      if (lane < g.k && t < g.T) {
        float p = s[r] / (total[r] + 1e-20f);
        if (g.apply_scaling) p = p * g.scaling;
        S.sel_s[t][lane] = p;
        S.sel_e[t][lane] = e[r];
        atomicOr(&S.mask[e[r]], 1ull << t);
        if (write) {
          g.probs[(size_t)t * g.k + lane] = p;
          g.indices[(size_t)t * g.k + lane] = e[r];
        }
      }
    }
  }
}

struct Active {
  int e, base, cnt;  // an expert with tokens, its first pair, its pairs (all wave-uniform)
};
template <int EMAX, int TMAX>
__device__ __forceinline__ Active active(const RouteLds<EMAX, TMAX>& R, int a) {
  const uint32_t v = (uint32_t)__builtin_amdgcn_readfirstlane((int)R.act[a]);
  return {(int)(v & 0x3ffu), (int)(v >> 10 & 0x7ffu), (int)(v >> 21)};
}

template <int EMAX, int TMAX>
__device__ __forceinline__ void route_all(const MoeArgs& g, RouteLds<EMAX, TMAX>& R,
                                           RouteScratch<EMAX, TMAX>& S, bool write) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < EMAX; e += kMoeWaves * 64) S.mask[e] = 0;
  __syncthreads();
  if (EMAX > 256)
    select_tokens<EMAX / 64>(g, S, write);
  else if (g.E <= 64)
    select_tokens<1>(g, S, write);
  else
    select_tokens<4>(g, S, write);
  __syncthreads();
  if (w == 0) {  // experts with tokens, ascending, and the first pair of each: 64 experts at a time
    int n = 0, pos = 0;
#pragma unroll
    for (int c = 0; c < EMAX / 64; ++c) {
      const int e = c * 64 + lane;
      const int cnt = __popcll(S.mask[e]);
      const uint64_t on = __ballot(cnt > 0);
      const int incl = wave_prefix_sum(cnt);
      if (cnt > 0) {
        S.base[e] = (uint16_t)(pos + incl - cnt);
        R.act[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(on >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)on, 0))] =
            (uint32_t)e | (uint32_t)(pos + incl - cnt) << 10 | (uint32_t)cnt << 21;
      }
      n += __popcll(on);
      pos += __builtin_amdgcn_readlane(incl, 63);
    }
    if (lane == 0) R.active = n;
  }
  __syncthreads();
  for (int t = w; t < g.T; t += kMoeWaves) {
    if (lane < g.k) {
      const int e = S.sel_e[t][lane];
      const int pos = S.base[e] + __popcll(S.mask[e] & ((1ull << t) - 1ull));
      R.prob[pos] = S.sel_s[t][lane];
      R.tok[pos] = (uint8_t)t;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// The experts, in one launch.  Gate/up units (16 neurons of one expert for all
// its tokens), then down units (16 columns of y for all tokens over one part of
// the (expert, K chunk) items), each kind dealt out in turn: the gate/up units to
// teams of the workgroups that share a CU (b and b + teams), which take them
// from a counter of the team.  (With every workgroup's units fixed, the second
// workgroup of a CU, which gets less of it, ended at 45 us and the first at 30
// us of a 70 us launch; with one counter for all, 512 workgroups on one address,
// a ticket took 13000 to 84000 cycles.)  A workgroup raises a flag when the h of
// all gate/up units that it took is stored and its team has no more, and polls
// the flags of all before its down units.
//
// That wait always ends, also when some workgroups cannot start because others
// wait (launches on several streams that share the device): a workgroup that
// has polled `patience` times computes the missing units itself, one team after
// another.  They give the same bits whoever computes them, so it does no harm if
// their owner does so too.
//
// What a workgroup hands to others in the same launch (h, parts of y) is
// written through to memory (device-scope stores) and waited for before the
// flag or count that announces it, and read at device scope.  (Fences by every
// workgroup work on whole caches instead: 22 us for the release, 27 us for the
// acquire over 512 workgroups.)
// ---------------------------------------------------------------------------
template <int WT, int MT, int EMAX>
__global__ __launch_bounds__(kMoeWaves * 64, 4) void moe_experts_kernel(MoeArgs g) {
  constexpr int TMAX = MT * 16, DT = down_tiles(WT == W_E4M3, MT > 1), DN = DT * 16;
  __shared__ RouteLds<EMAX, TMAX> R;
  __shared__ union {
    RouteScratch<EMAX, TMAX> route;
    f32x4 red[2][kMoeWaves][2][64];      // gate/up: sums of the waves
    f32x4 sums[kMoeWaves][TMAX][DT * 4];  // down: [token][DN] sums, by wave
  } L;
  __shared__ int shared_int;
  __shared__ int ticket[2];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int lr = lane & 15, lg = lane >> 4;
  const int team = blockIdx.x % g.teams;
  auto take = [&]() __attribute__((always_inline)) {
    return __hip_atomic_fetch_add(g.tickets + team, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  if (threadIdx.x == 0) ticket[0] = take();
  route_all<EMAX, TMAX>(g, R, L.route, blockIdx.x == 0);
  int ahead = 0;  // thread 0: the ticket after the next
  if (threadIdx.x == 0) ahead = take();

  const int nt = g.ff / 16, dtiles = (g.d + DN - 1) / DN, grid = gridDim.x;
  const int gu_units = R.active * nt, d_units = dtiles * g.splits;
  const int kb = (g.d + kChunk - 1) / kChunk, fb = (g.ff + kQB - 1) / kQB;
  const size_t plane = (size_t)g.T * g.k * g.ff;
  const rsrc_t rh = make_rsrc(g.h, (uint32_t)(plane * 4));
  const rsrc_t rx = make_rsrc(g.x, (uint32_t)(g.T * g.d * 2));

  // ---- down, first half.  A unit's items are (expert, K chunk) pairs; each wave
  // takes a run of them.  P are on their way or in use, each with its weights and
  // its columns: h of up to 8 pairs, the upper bf16 values in columns 0..7 and the
  // rest in columns 8..15 (one product for both; their sums are added below). ----
  constexpr int P = WT == W_BF16 || DT > 1 ? 2 : 3;
  const int items = R.active * fb;
  struct Item {
    Rows16<WT> w[DT];
    Cols16<WT, kDevice> h;
    float scale;
    int cnt, base, kc, tok;  // tok: of this lane's column (-1: none)
  } q[P];
  int d0 = 0, lo = 0, hi = 0;
  int at_a = 0, at_kc = 0;  // the next item to request
  Active at = {0, 0, 0};
  auto weights = [&](int i, Item& t) __attribute__((always_inline)) {
    const bool on = i < hi;
    t.cnt = on ? at.cnt : 0;
    t.base = at.base;
    t.kc = at_kc;
    const rsrc_t rw = rows_rsrc<WT>(g.wd, (size_t)at.e * g.d + d0, g.ff, min(DN, g.d - d0));
#pragma unroll
    for (int v = 0; v < DT; ++v) t.w[v].load(rw, v * 16 + lr, on ? at_kc * kChunk : g.ff, g.ff, lg);
    t.scale = WT != W_BF16 ? g.sd[((size_t)at.e * kb + d0 / kQB) * fb + at_kc] : 1.f;
    if (++at_kc == fb) {
      at_kc = 0;
      at_a = min(at_a + 1, R.active - 1);
      at = active(R, at_a);
    }
  };
  auto columns = [&](int j, Item& t) __attribute__((always_inline)) {
    const int col = j * 8 + (lr & 7);
    const bool in = col < t.cnt;
    const int pair = t.base + (in ? col : 0);
    t.tok = in ? R.tok[pair] : -1;
    t.h.load(rh, (uint32_t)(lr < 8 ? 0 : plane) + pair * g.ff, t.kc * kChunk, g.ff, in, lg);
  };
  auto begin_down = [&](int unit) __attribute__((always_inline)) {
    const int part = unit / dtiles;
    d0 = (unit - part * dtiles) * DN;
    lo = (int)((long long)items * (part * kMoeWaves + w) / (g.splits * kMoeWaves));
    hi = (int)((long long)items * (part * kMoeWaves + w + 1) / (g.splits * kMoeWaves));
    at_a = min(lo / fb, R.active - 1);
    at_kc = lo - lo / fb * fb;
    at = active(R, at_a);
#pragma unroll
    for (int u = 0; u < P; ++u) weights(lo + u, q[u]);
  };

  bool own = true;  // this workgroup's share of its team's units; else all units of a team that is missed
  for (int owner = team, polls = 0; owner >= 0; own = false) {
    // ---- gate and up units of team `owner`: the waves split d and add their sums in
    // LDS.  The weights of the next step (the rest of d, or the next unit) are
    // requested as soon as the products have taken the current ones, so they are
    // on the way during the reduction. ----
    constexpr int U = WT == W_BF16 && MT > 1 ? 1 : 2;  // K chunks in flight per wave (registers)
    const int steps = (kb + kMoeWaves * U - 1) / (kMoeWaves * U);
    Rows16<WT> ag[U], au[U];
    float sg[U], su[U];
    // unit t of the team: number owner + t * teams, by active expert, then 16-neuron tile
    auto load = [&](int t, int step) __attribute__((always_inline)) {
      const int unit = owner + t * g.teams;
      const int d = unit < gu_units ? g.d : 0;  // no such unit: zeros, without a branch
      const int a = d ? unit / nt : 0, n0 = d ? (unit - a * nt) * 16 : 0;
      const int e = active(R, d ? a : 0).e;
      const rsrc_t rg = rows_rsrc<WT>(g.wg, (size_t)e * g.ff + n0, g.d);
      const rsrc_t ru = rows_rsrc<WT>(g.wu, (size_t)e * g.ff + n0, g.d);
      const size_t srow = ((size_t)e * fb + n0 / kQB) * kb;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = (step * U + u) * kMoeWaves + w;
        ag[u].load(rg, lr, c * kChunk, d, lg);
        au[u].load(ru, lr, c * kChunk, d, lg);
        if (WT != W_BF16) {
          sg[u] = c < kb ? g.sg[srow + c] : 0.f;
          su[u] = c < kb ? g.su[srow + c] : 0.f;
        }
      }
    };
    int buf = 0, turn = 0;
    int cur = own ? ticket[0] : 0;
    load(cur, 0);
    if (own && threadIdx.x == 0) ticket[1] = ahead;
    __syncthreads();
    int nxt = own ? ticket[1] : 1;
    while (owner + cur * g.teams < gu_units) {
      const int unit = owner + cur * g.teams, a = unit / nt, n0 = (unit - a * nt) * 16;
      const Active act = active(R, a);
      const int cnt = act.cnt, base = act.base;
      const int tiles = (cnt + 15) >> 4;
      if (own && threadIdx.x == 0) ahead = take();
      f32x4 acc[2][MT];
      zero_acc(acc);
      for (int step = 0; step < steps; ++step) {
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          if (j < tiles) {
            const bool in = j * 16 + lr < cnt;
            const uint32_t xr = (in ? R.tok[base + j * 16 + lr] : 0) * g.d;
#pragma unroll
            for (int u = 0; u < U; ++u) {
              Cols16<WT> b;
              b.load(rx, xr, ((step * U + u) * kMoeWaves + w) * kChunk, g.d, in, lg);
              mma_chunk128<WT>(acc[0][j], ag[u], b, sg[u]);
              mma_chunk128<WT>(acc[1][j], au[u], b, su[u]);
            }
          }
        }
        const bool more = step + 1 < steps;
        load(more ? cur : nxt, more ? step + 1 : 0);
      }
      if (own && threadIdx.x == 0) ticket[turn] = ahead;
      int after = nxt + 1;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        if (j >= tiles) break;
        // two buffers by turns: a buffer is written again only after the barrier in between
        L.red[buf][w][0][lane] = acc[0][j];
        L.red[buf][w][1][lane] = acc[1][j];
        wait_lgkm0();
        barrier();  // not __syncthreads: that would wait for the weights on their way
        if (j == 0 && own) after = ticket[turn];
        const float* rf = (const float*)L.red[buf];
        buf ^= 1;
        const int o = threadIdx.x;  // two neurons of one column
        if (o < min(cnt - j * 16, 16) * 8) {
          const int n = (o & 7) * 2, c = o >> 3;
          const int at = ((n >> 2) * 16 + c) * 4 + (n & 3);
          float hv[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float hg = rf[at + r], hu = rf[at + r + 256];
#pragma unroll
            for (int v = 1; v < kMoeWaves; ++v) {
              hg += rf[v * 512 + at + r];
              hu += rf[v * 512 + at + r + 256];
            }
            hv[r] = hg / (1.0f + __expf(-hg)) * hu * R.prob[base + j * 16 + c];
          }
          // Rounding h to bf16 alone would add an error as large as that of rounding y (together 1.41 times
          // it); as bf16(h) + bf16(rest) it keeps 16 bits, for one more product per step of the down part,
          // whose matrix cores are idle.
          const uint32_t hh = pack_bf16x2(hv[0], hv[1]);
          const float r0 = (hh & 0x7f80u) != 0x7f80u ? hv[0] - __uint_as_float(hh << 16) : 0.f;
          const float r1 = (hh & 0x7f800000u) != 0x7f800000u ? hv[1] - __uint_as_float(hh & 0xffff0000u) : 0.f;
          const uint32_t at_h = (uint32_t)(base + j * 16 + c) * g.ff + n0 + n;
          __builtin_amdgcn_raw_buffer_store_b32(hh, rh, at_h * 2, 0, kDevice);
          __builtin_amdgcn_raw_buffer_store_b32(pack_bf16x2(r0, r1), rh, ((uint32_t)plane + at_h) * 2, 0,
                                                kDevice);
        }
      }
      cur = nxt;
      nxt = after;
      turn ^= 1;
    }
    wait_vmcnt<0>();
    barrier();  // every wave's h is stored
    // this workgroup has done its share of the team's units, or all of them for the whole team
    if (threadIdx.x == 0)
      for (int b = own ? blockIdx.x : owner; b < grid; b += own ? grid : g.teams)
        __hip_atomic_store(g.flags + b, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if ((int)blockIdx.x >= d_units) return;
    begin_down(blockIdx.x);
    for (;; ++polls) {  // threads watch different flags
      int missing = -1;
      for (int b = threadIdx.x; b < grid; b += kMoeWaves * 64)
        if (__hip_atomic_load(g.flags + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 0) missing = b % g.teams;
      owner = -1;
      if (!__syncthreads_or(missing >= 0)) break;
      if (polls >= g.patience) {  // uniform: help one of the teams that some thread misses
        if (missing >= 0) shared_int = missing;
        __syncthreads();
        owner = __builtin_amdgcn_readfirstlane(shared_int);
        __syncthreads();
        break;
      }
      __builtin_amdgcn_s_sleep(2);
    }
  }

  // ---- down, second half: a wave takes a run of consecutive items and adds into
  // sums of its own; where the items are split over several workgroups, each
  // writes its sums and the last to arrive adds them in part order. ----
  for (int unit = blockIdx.x; unit < d_units; unit += grid) {
    if (unit != (int)blockIdx.x) begin_down(unit);
    const int part = unit / dtiles, dt = unit - part * dtiles;
    for (int i = lane; i < g.T * DT * 4; i += 64) ((f32x4*)L.sums[w])[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto add = [&](const Item& t) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < DT; ++c) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s) mma_bf16(v, t.w[c].frag(s), t.h.v[s]);
#pragma unroll
        for (int r = 0; r < 4; ++r)  // columns c and c + 8
          v[r] += __uint_as_float(dpp_u32<0x128, 0xf>(__float_as_uint(v[r])));
        if (t.tok >= 0 && lr < 8) {
          f32x4& sum = L.sums[w][t.tok][c * 4 + lg];
          f32x4 y = sum;
#pragma unroll
          for (int r = 0; r < 4; ++r) y[r] = fmaf(v[r], t.scale, y[r]);
          sum = y;
        }
      }
    };
#pragma unroll
    for (int u = 0; u < P; ++u) columns(0, q[u]);
    // registers by turns, not moved: a move would wait for the load on its way
    for (int i0 = lo; i0 < hi; i0 += P) {
#pragma unroll
      for (int u = 0; u < P; ++u) {
        if (i0 + u < hi) {
          add(q[u]);
          for (int j = 1; j * 8 < q[u].cnt; ++j) {
            columns(j, q[u]);
            add(q[u]);
          }
          weights(i0 + u + P, q[u]);
          columns(0, q[u]);
        }
      }
    }
    __syncthreads();
    // four columns of a token at a time
    const int quads = g.T * (DN / 4);
    auto sum = [&](int o) __attribute__((always_inline)) {
      f32x4 v = (&L.sums[0][0][0])[o];
#pragma unroll
      for (int r = 1; r < kMoeWaves; ++r) v += (&L.sums[r][0][0])[o];
      return v;
    };
    auto store = [&](int o, const f32x4& v) __attribute__((always_inline)) {
      const int t = o / (DN / 4), n = d0 + o % (DN / 4) * 4;
      const float out[4] = {v[0], v[1], v[2], v[3]};
      if (n < g.d) Quad<bf16_t>::store(g.y + (size_t)t * g.d + n, out);
    };
    if (g.splits == 1) {
      for (int o = threadIdx.x; o < quads; o += kMoeWaves * 64) store(o, sum(o));
    } else {
      const uint32_t tile = quads * 16, pstride = dtiles * tile;  // bytes
      const rsrc_t rp = make_rsrc((const char*)g.part + (size_t)dt * tile, (g.splits - 1) * pstride + tile);
      for (int o = threadIdx.x; o < quads; o += kMoeWaves * 64)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4_t, sum(o)), rp, part * pstride + o * 16, 0,
                                               kDevice);
      wait_vmcnt<0>();
      __syncthreads();  // every wave's stores are done
      if (threadIdx.x == 0)
        shared_int =
            __hip_atomic_fetch_add(g.arrived + dt, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == g.splits - 1;
      __syncthreads();
      if (shared_int) {
        for (int o = threadIdx.x; o < quads; o += kMoeWaves * 64) {
          f32x4 v[kMaxSplits];
#pragma unroll
          for (int r = 0; r < kMaxSplits; ++r)  // all on their way together; past the last part: zeros
            v[r] = __builtin_bit_cast(f32x4, load16<kDevice>(rp, r < g.splits ? r * pstride + o * 16 : kOOB));
#pragma unroll
          for (int r = 1; r < kMaxSplits; ++r) v[0] += v[r];
          store(o, v[0]);
        }
      }
    }
    __syncthreads();
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Parts of the down items: the tiles of y alone would leave workgroup slots (two
// per CU) empty.  A part is worth its adding (2 to 4 us) where each wave has an
// item, counted as one token's experts, or four, counted as every expert that
// the tokens can choose (us, without / with the second: 32 tokens, 8 of 256
// experts, d = 1024, d_ff = 512, 8-bit, 88.6 / 80.3; with one item in place of four,
// 4 tokens, 11 of 43 experts, d = 2048, d_ff = 128, 26.5 / 30.8).  By shape alone, so a
// shape rounds alike everywhere.
int down_splits(int tokens, int experts, int topk, int d_model, int d_ff, int dt) {
  const int tiles = (d_model + dt * 16 - 1) / (dt * 16);
  const int chunks = (d_ff + kChunk - 1) / kChunk, all = std::min(experts, tokens * topk);
  const int worth = std::max(topk * chunks / kMoeWaves, all * chunks / (4 * kMoeWaves));
  return std::max(1, std::min({2 * kNominalCUs / tiles, worth, kMaxSplits}));
}

struct MoeLayout {
  size_t scores = 0, h = 0, part = 0, flags = 0, bytes = 0;
};
MoeLayout layout(int tokens, int experts, int topk, int d_model, int d_ff) {
  MoeLayout L;
  // the parts of y, with either type of weights
  size_t part = 0;
  for (const int dt : {down_tiles(false, tokens > 16), down_tiles(true, tokens > 16)}) {
    const int splits = down_splits(tokens, experts, topk, d_model, d_ff, dt);
    if (splits > 1) part = std::max(part, (size_t)splits * tokens * ((d_model + dt * 16 - 1) / (dt * 16) * dt * 16) * 4);
  }
  L.h = align256((size_t)tokens * experts * 4);
  L.part = L.h + align256((size_t)tokens * topk * d_ff * 4);
  L.flags = L.part + align256(part);
  L.bytes = L.flags + align256((size_t)(2 * kMoeMaxGrid + d_model / 16) * 4);
  return L;
}

template <int WT, int MT, int EMAX>
hipError_t launch_t(MoeArgs g, hipStream_t stream) {
  constexpr int DT = down_tiles(WT == W_E4M3, MT > 1);
  g.splits = down_splits(g.T, g.E, g.k, g.d, g.ff, DT);
  {
    LaunchTimer timer("moe_scores", stream);
    hipLaunchKernelGGL(moe_scores_kernel, dim3((g.E + kScoreRows - 1) / kScoreRows, (g.T + 15) / 16), dim3(kScoreWaves * 64), 0, stream,
                       g);
  }
  // two workgroups per CU; more than there can be units of either kind would find none
  const int slots = std::min(2 * compute_units(), kMoeMaxGrid);
  const long long most = std::max<long long>((long long)std::min(g.E, g.T * g.k) * (g.ff / 16), (g.d + DT * 16 - 1) / (DT * 16) * g.splits);
  const int grid = (int)std::min<long long>(most, slots);
  g.teams = std::min(grid, slots / 2);
  LaunchTimer timer("moe_experts", stream);
  hipLaunchKernelGGL((moe_experts_kernel<WT, MT, EMAX>), dim3(grid), dim3(kMoeWaves * 64), 0, stream, g);
  return hipGetLastError();
}

template <int WT, int MT>
hipError_t launch_e(const MoeArgs& g, hipStream_t stream) {
  return g.E <= 256 ? launch_t<WT, MT, 256>(g, stream) : launch_t<WT, MT, kMoeMaxExperts>(g, stream);
}

template <int WT>
hipError_t launch_m(const MoeArgs& g, hipStream_t stream) {
  return g.T <= 16 ? launch_e<WT, 1>(g, stream) : launch_e<WT, 4>(g, stream);
}

}  // namespace

size_t moe_decode_workspace_bytes(int tokens, int experts, int topk, int d_model, int d_ff) {
  return layout(tokens, experts, topk, d_model, d_ff).bytes;
}

hipError_t launch_moe_decode(const MoeCall& c, void* workspace, hipStream_t stream) {
  const MoeLayout L = layout(c.tokens, c.experts, c.topk, c.d_model, c.d_ff);
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
  g.h = (bf16_t*)((char*)workspace + L.h);
  g.part = (float*)((char*)workspace + L.part);
  g.flags = (int*)((char*)workspace + L.flags);
  g.tickets = g.flags + kMoeMaxGrid;
  g.arrived = g.tickets + kMoeMaxGrid;
  g.patience = c.patience;
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
