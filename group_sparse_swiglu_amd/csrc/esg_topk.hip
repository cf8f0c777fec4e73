// Routing to experts, forward and backward: softmax or sigmoid scores, a bias for
// the choice, groups of experts, the k largest keys, their weights.
//   score s_e   sigmoid(z_e) or softmax(z)_e, the fp64 value rounded once to float32
//   key         s_e + bias_e, one float32 addition
//   groups      ranked by the sum of their two largest keys (one float32 addition);
//               the best topk_groups stay (equal ones: the lower group)
//   choice      the k largest keys of these, equal ones by lower expert, written in
//               ascending expert order
//   weights     s / (sum of the chosen s + 1e-20) * scaling, or s * scaling
//   backward    of the weights, with ds_j the gradient of a chosen score:
//               sigmoid  dz_j = ds_j s_j (1 - s_j);  softmax  dz_e = s_e (ds_e - sum_i s_i ds_i)
//
// LPR lanes take a token row, C experts each: 16 lanes (four rows per wave) while a
// row fits 16 x 16, else the whole wave.  A group owns a power of two of lanes, so
// ascending lanes are ascending experts and a group's maxima are moves between
// neighbouring lanes.  The forward works on float32 estimates of the keys, off by a few
// units in the last place: each lane sorts its C keys, and the row's largest head is
// taken k + 1 times.  Equal estimates on both sides of the border are settled by their
// experts where they come from equal logits and biases.  Where else the k-th and the next
// key, or the last group that stays and the first that goes, are nearer to each other
// than the estimates are to the keys, the row is done again with exact keys in 64 bits
// beside their slots.  Which experts are chosen is thus that of the exact keys; the
// weights are float32 either way.
//
// Bound by the vector unit, not by memory: about 1400 instructions for four rows of 256
// (the unit is busy for 94 % of the cycles), 28 us for 32768 x 256, k = 8 in bf16, whose
// bytes take 4; the exact keys of all rows would take 94.  A decode batch is as long as
// its launch and one row's chain of steps, 6.7 us.
#include <algorithm>
#include <type_traits>

#include "esg_internal.hpp"
#include "esg_route.hpp"

namespace esg {
namespace {

constexpr int kThreads = 256;

// ---- exchanges between the N (a power of two) neighbouring lanes of a segment ----
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
template <int CTRL, typename V>
__device__ __forceinline__ V dpp8(V v) {  // 8-byte values
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t r = (uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32 | dpp<CTRL>((uint32_t)b);
  return __builtin_bit_cast(V, r);
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp(uint64_t v) { return dpp8<CTRL>(v); }
template <int CTRL>
__device__ __forceinline__ double dpp(double v) { return dpp8<CTRL>(v); }

// f over a segment of n lanes, left in all of them: the partner of a step lies in the
// other half of the next larger segment, whose lanes all hold the same by then.
template <typename V, typename F>
__device__ __forceinline__ V seg_reduce(V v, int n, F f) {
  if (n > 1) v = f(v, dpp<0xB1>(v));    // lane ^ 1
  if (n > 2) v = f(v, dpp<0x4E>(v));    // lane ^ 2
  if (n > 4) v = f(v, dpp<0x141>(v));   // mirrored in 8
  if (n > 8) v = f(v, dpp<0x140>(v));   // mirrored in 16
  if (n > 16) v = f(v, __shfl_xor(v, 16));
  if (n > 32) v = f(v, __shfl_xor(v, 32));
  return v;
}
template <int LPR, typename V, typename F>
__device__ __forceinline__ V row_reduce(V v, F f) {
  return seg_reduce(v, LPR, f);
}
struct Max {
  template <typename V>
  __device__ __forceinline__ V operator()(V a, V b) const { return a > b ? a : b; }
};
struct Min {
  template <typename V>
  __device__ __forceinline__ V operator()(V a, V b) const { return a < b ? a : b; }
};
struct Add {
  template <typename V>
  __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct Or {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a | b; }
};

// Sum over the lanes up to and with this one of its row.
template <int LPR>
__device__ __forceinline__ uint32_t row_scan(uint32_t v) {
  v += dpp<0x111>(v);  // from 1, 2, 4, 8 lanes below, 0 past the lower end of 16
  v += dpp<0x112>(v);
  v += dpp<0x114>(v);
  v += dpp<0x118>(v);
  if constexpr (LPR == 64) {
    const int lane = threadIdx.x & 63;
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 15), b = (uint32_t)__builtin_amdgcn_readlane((int)v, 31),
                   c = (uint32_t)__builtin_amdgcn_readlane((int)v, 47);
    v += (lane >= 16 ? a : 0u) + (lane >= 32 ? b : 0u) + (lane >= 48 ? c : 0u);
  }
  return v;
}

// ---- scores ----
// e^(x + rest) to about 2 units in the last place, |rest| at most half a unit of x: the
// exponent's product with log2(e) in two parts.  x is taken into [-150, 88], whose
// ends give 0 and, still finite, 2^126.96.
__device__ __forceinline__ float fast_exp(float x, float rest = 0.f) {
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-8f, kLn2 = 0.693147182464599609375f;
  x = __builtin_amdgcn_fmed3f(x, -150.f, 88.f);
  const float t = x * kHi;
  const float lo = fmaf(x, kLo, fmaf(x, kHi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, fmaf(lo, kLn2, rest), e);
}
// e^(z - top), the difference with what its rounding loses (half a unit of a difference of 64 is 2^-18 of the result)
__device__ __forceinline__ float exp_below(float z, float top) {
  const float d = z - top, b = d - z;
  const float rest = (z - (d - b)) - (top + b);
  return fast_exp(d, d >= -150.f ? rest : 0.f);  // z may be -infinity
}
__device__ __forceinline__ float fast_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + fast_exp(-z)); }

enum { SIGMOID = 0, SOFTMAX = 1 };

struct RouteArgs {
  const void* logits;
  const float* bias;  // or NULL
  int bias_stride;
  int tokens, experts, topk;
  int per;            // experts of a group
  int groups, keep;   // keep == groups: every group stays, and groups is 1
  int lanes;          // lanes of a group
  int vec, bias_vec;  // a lane's logits, and biases, are whole 16-byte pieces, if they are any
  int normalize;
  float scaling;
  float* probs;
  int32_t* idx;
};

// n consecutive logits from p (zeros past them) as floats; vec: n is 0 or C, p is 16-byte aligned.
template <int C>
__device__ __forceinline__ void load_logits(const float* p, int n, int vec, float (&z)[C]) {
  if constexpr (C % 4 == 0) {
    if (vec) {
#pragma unroll
      for (int q = 0; q < C / 4; ++q) {
        const float4 v = n > 0 ? *(const float4*)(p + 4 * q) : make_float4(0.f, 0.f, 0.f, 0.f);
        z[4 * q] = v.x; z[4 * q + 1] = v.y; z[4 * q + 2] = v.z; z[4 * q + 3] = v.w;
      }
      return;
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) z[c] = c < n ? p[c] : 0.f;
}
template <int C>
__device__ __forceinline__ void load_logits(const bf16_t* p, int n, int vec, float (&z)[C]) {
  if constexpr (C % 8 == 0) {
    if (vec) {
#pragma unroll
      for (int q = 0; q < C / 8; ++q) {
        const uint4 v = n > 0 ? *(const uint4*)(p + 8 * q) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[8 * q + 2 * i] = __uint_as_float(u[i] << 16);
          z[8 * q + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
      }
      return;
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) z[c] = c < n ? load_elem<bf16_t>(p + c) : 0.f;
}

// ---- ordered keys, exact ones above what is left of the row behind their slot; 0 is no key ----
__device__ __forceinline__ float key_float(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}
template <bool EXACT>
struct Key;
template <>
struct Key<false> {
  using type = uint32_t;
  __device__ static __forceinline__ type make(float f, int) { return order_key(f); }
  __device__ static __forceinline__ float value(type k) { return key_float(k); }
};
template <>
struct Key<true> {
  using type = uint64_t;
  __device__ static __forceinline__ type make(float f, int slot) {
    return (uint64_t)order_key(f) << 32 | (uint32_t)(kRouteMaxExperts - slot);
  }
  __device__ static __forceinline__ float value(type k) { return key_float((uint32_t)(k >> 32)); }
};

// by value: a condition between two elements of an array becomes an index into it
template <typename V>
__device__ __forceinline__ V choose(bool c, V a, V b) { return c ? a : b; }

// descending, a bitonic network
template <int C, typename V>
__device__ __forceinline__ void sort_desc(V (&v)[C]) {
#pragma unroll
  for (int k = 2; k <= C; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int o = i ^ j;
        if (o > i) {
          const V a = v[i], b = v[o];
          const V hi = a > b ? a : b, lo = a > b ? b : a;
          v[i] = (i & k) ? lo : hi;
          v[o] = (i & k) ? hi : lo;
        }
      }
}

// A score's estimate is off by at most this of itself: two to three units in its last place from exponential and
// reciprocal, and with softmax up to 20 additions of the row's sum.
constexpr float kEstimate = 0x1p-19f;

// The k-th largest key of the row's best groups from keys u (0: none) and, of estimates, the one after it; sure:
// whether they decide which groups stay (always, for exact keys).  An estimate is off by at most kEstimate of itself
// and abs_err.
template <int LPR, int C, bool EXACT>
__device__ __forceinline__ typename Key<EXACT>::type threshold(const typename Key<EXACT>::type (&u)[C],
                                                               const RouteArgs& g, int l, float abs_err,
                                                               uint32_t& in_group, bool& sure,
                                                               typename Key<EXACT>::type& next) {
  using K = Key<EXACT>;
  using V = typename K::type;
  V s[C];
#pragma unroll
  for (int c = 0; c < C; ++c) s[c] = u[c];
  sort_desc<C>(s);
  sure = true;
  in_group = 1;
  if (g.keep < g.groups) {
    struct Two {
      V a, b;
    };
    Two t{s[0], C > 1 ? s[C > 1 ? 1 : 0] : V(0)};
    // two largest of the segment, step by step as in seg_reduce
    auto step = [&](V a, V b) __attribute__((always_inline)) {
      const V lo = t.a < a ? t.a : a;
      t.a = t.a < a ? a : t.a;
      t.b = t.b < b ? b : t.b;
      t.b = t.b < lo ? lo : t.b;
    };
    if (g.lanes > 1) step(dpp<0xB1>(t.a), dpp<0xB1>(t.b));
    if (g.lanes > 2) step(dpp<0x4E>(t.a), dpp<0x4E>(t.b));
    if (g.lanes > 4) step(dpp<0x141>(t.a), dpp<0x141>(t.b));
    if (g.lanes > 8) step(dpp<0x140>(t.a), dpp<0x140>(t.b));
    if (g.lanes > 16) step(__shfl_xor(t.a, 16), __shfl_xor(t.b, 16));
    if (g.lanes > 32) step(__shfl_xor(t.a, 32), __shfl_xor(t.b, 32));
    float score = t.a == 0 ? -INFINITY : K::value(t.a);
    float size = fabsf(score);
    if (t.b != 0) {
      const float second = K::value(t.b);
      score = score + second;
      score = score == score ? score : INFINITY;  // +infinity (of the first) and -infinity: an expert that has to be there
      size += fabsf(second);
    }
    // rank of this lane's group: groups with a larger score, or an equal one and a lower number
    const int row0 = (int)(threadIdx.x & 63) - l;
    int rank = 0;
    for (int o = g.lanes; o < LPR; o += g.lanes) {
      const int from = (l + o) & (LPR - 1);
      const float other = __shfl(score, row0 + from);
      rank += other > score || (other == score && from < l);
    }
    in_group = rank < g.keep;
    if constexpr (!EXACT) {
      const float kept = row_reduce<LPR>(in_group ? score : INFINITY, Min{});
      const float gone = row_reduce<LPR>(in_group ? -INFINITY : score, Max{});
      const float most = row_reduce<LPR>(t.a == 0 ? 0.f : size, Max{});
      sure = kept - gone > most * (2.f * kEstimate) + 4.f * abs_err;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = in_group ? s[c] : V(0);
  }
  V thr = 0, m = 0;
  const int lane = threadIdx.x & 63;
  const uint64_t below = ((1ull << l) - 1ull) << (lane - l);  // the row's lanes below this one
  for (int j = 0; j < g.topk + (EXACT ? 0 : 1); ++j) {
    thr = m;
    m = row_reduce<LPR>(s[0], Max{});
    bool mine = s[0] == m;
    if constexpr (!EXACT) mine = mine && (__ballot(mine) & below) == 0;  // of equal heads the lowest lane's
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = choose(mine, c + 1 < C ? s[c + 1 < C ? c + 1 : c] : V(0), s[c]);
  }
  next = m;
  return EXACT ? m : thr;
}

// whether estimates a >= b are further apart than they may be off
__device__ __forceinline__ bool apart(float a, float b, float abs_err) {
  return a - b > (fabsf(a) + fabsf(b)) * kEstimate + 2.f * abs_err;
}

template <typename T, int LPR, int C>
__global__ __launch_bounds__(kThreads) void topk_routing_kernel(RouteArgs g, int scoring) {
  constexpr int ROWS = kThreads / LPR;
  const int l = threadIdx.x & (LPR - 1);
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
  const bool live = row < g.tokens;  // a wave goes on while one of its rows is one
  const int grp = l / g.lanes, e_in = (l - grp * g.lanes) * C;
  const int n = live && grp < g.groups ? min(max(g.per - e_in, 0), C) : 0;  // experts of this lane
  const int e0 = grp * g.per + e_in;
  float z[C], b[C];
  load_logits<C>((const T*)g.logits + (live ? row : 0) * g.experts + (n > 0 ? e0 : 0), n, g.vec, z);
  if (g.bias != nullptr && g.bias_stride == 1) {
    load_logits<C>(g.bias + (n > 0 ? e0 : 0), n, g.bias_vec, b);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) b[c] = g.bias != nullptr && c < n ? g.bias[(int64_t)(e0 + c) * g.bias_stride] : 0.f;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) b[c] = b[c] == b[c] ? b[c] : -INFINITY;  // no key is NaN
  uint32_t bad = 0;  // a NaN, or an infinity that softmax divides by: the row's weights are NaN
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool nan = z[c] != z[c] || (scoring == SOFTMAX && z[c] == INFINITY);
    bad |= nan;
    z[c] = nan ? -INFINITY : z[c];
  }
  float s[C], top = 0.f, most = 1.f;  // most: no score of the row is larger
  if (scoring == SIGMOID) {
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = fast_sigmoid(z[c]);
  } else {
    top = -INFINITY;
#pragma unroll
    for (int c = 0; c < C; ++c) top = c < n ? fmaxf(top, z[c]) : top;
    top = row_reduce<LPR>(top, Max{});
    top = top == -INFINITY ? 0.f : top;  // nothing but -inf: all scores are 0
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s[c] = c < n ? exp_below(z[c], top) : 0.f;
      sum += s[c];
    }
    sum = row_reduce<LPR>(sum, Add{});
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    most = inv;
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] *= inv;
  }
  // beside a bias the error of the score counts whole; scores below the normal range are off by themselves
  const float abs_err = (g.bias != nullptr ? most * kEstimate : 0.f) + 0x1p-125f;
  using Fast = Key<false>;
  using Exact = Key<true>;
  uint32_t flags = 0;  // bit c: chosen
  bool sure = true;
  uint32_t in_group;
  {
    uint32_t u[C];
#pragma unroll
    for (int c = 0; c < C; ++c) u[c] = c < n ? Fast::make(s[c] + b[c], l * C + c) : 0u;
    uint32_t next;
    const uint32_t thr = threshold<LPR, C, false>(u, g, l, abs_err, in_group, sure, next);
    uint32_t equal = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      u[c] = in_group ? u[c] : 0u;
      flags |= (uint32_t)(u[c] >= thr) << c;
      equal |= (uint32_t)(u[c] == thr) << c;
    }
    const bool tie = next == thr;
    const float ft = Fast::value(thr);
    if (!tie && next != 0) sure = sure && apart(ft, Fast::value(next), abs_err);
    if (__ballot(live && tie) != 0) {
      // equal estimates on both sides of the border (logits of 16 bits have many equals): the lower ones are taken, if
      // all of them come from equal logits and biases and no other estimate is near
      uint32_t over = 0xffffffffu, under = 0, zlo = 0xffffffffu, zhi = 0, blo = 0xffffffffu, bhi = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool eq = u[c] == thr;
        const uint32_t kz = order_key(z[c]), kb = order_key(b[c]);
        over = u[c] > thr ? Min{}(over, u[c]) : over;
        under = u[c] < thr ? Max{}(under, u[c]) : under;
        zlo = eq ? Min{}(zlo, kz) : zlo;
        zhi = eq ? Max{}(zhi, kz) : zhi;
        blo = eq ? Min{}(blo, kb) : blo;
        bhi = eq ? Max{}(bhi, kb) : bhi;
      }
      over = row_reduce<LPR>(over, Min{});
      under = row_reduce<LPR>(under, Max{});
      const bool same = row_reduce<LPR>(zlo, Min{}) == row_reduce<LPR>(zhi, Max{}) &&
                        row_reduce<LPR>(blo, Min{}) == row_reduce<LPR>(bhi, Max{});
      const bool alone = (over == 0xffffffffu || apart(Fast::value(over), ft, abs_err)) &&
                         (under == 0 || apart(ft, Fast::value(under), abs_err));
      const uint32_t above = row_reduce<LPR>((uint32_t)__popc(flags & ~equal), Add{});
      const int before = (int)(row_scan<LPR>((uint32_t)__popc(equal)) - __popc(equal));
      int need = g.topk - (int)above - before;
      uint32_t kept = flags & ~equal;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool take = (equal >> c & 1) && need > 0;
        kept |= (uint32_t)take << c;
        need -= take;
      }
      flags = tie ? kept : flags;
      sure = tie ? sure && same && alone : sure;
    }
  }
  if (__ballot(live && !sure) != 0) {
    // for the unsure rows alone: what a row gives does not depend on the others of its wave
    const bool redo = !sure;
    float x[C];
    uint64_t u[C];
    if (scoring == SIGMOID) {
#pragma unroll
      for (int c = 0; c < C; ++c) x[c] = exact_sigmoid(z[c]);
    } else {
      double sum = 0.0;
#pragma unroll
      for (int c = 0; c < C; ++c) sum += c < n ? exp((double)z[c] - (double)top) : 0.0;
      sum = row_reduce<LPR>(sum, Add{});
      const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
      for (int c = 0; c < C; ++c) x[c] = (float)(exp((double)z[c] - (double)top) * inv);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) u[c] = c < n ? Exact::make(x[c] + b[c], l * C + c) : 0ull;
    uint64_t next;
    const uint64_t thr = threshold<LPR, C, true>(u, g, l, 0.f, in_group, sure, next);
    uint32_t exact = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      exact |= (uint32_t)(c < n && in_group && u[c] >= thr) << c;
      s[c] = redo ? x[c] : s[c];
    }
    flags = redo ? exact : flags;
  }
  // place of this lane's first chosen expert: chosen ones of the lanes below it
  int place = (int)(row_scan<LPR>((uint32_t)__popc(flags)) - __popc(flags));
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) sum += (flags >> c & 1) ? s[c] : 0.f;
  sum = row_reduce<LPR>(sum, Add{});
  bad = row_reduce<LPR>(bad, Or{});
  float f = g.normalize ? g.scaling / (sum + 1e-20f) : g.scaling;
  f = bad ? NAN : f;
  if (!live) return;
  float* const p = g.probs + row * g.topk;
  int32_t* const ix = g.idx + row * g.topk;
#pragma unroll
  for (int c = 0; c < C; ++c)
    if ((flags >> c & 1) && place < g.topk) {
      p[place] = s[c] * f;
      ix[place] = e0 + c;
      ++place;
    }
}

// ---------------------------------------------------------------------------
// Backward.  Lanes hold the chosen experts (two per lane where LPR is 16 and k
// above that), their sums are exchanged, and the row of gradients is laid out in
// LDS and written in whole 16-byte pieces.
// ---------------------------------------------------------------------------
struct RouteBwdArgs {
  const float* dp;
  const void* logits;
  const int32_t* idx;
  int tokens, experts, topk;
  int vec;  // rows of logits and gradients are whole 16-byte pieces
  int normalize;
  float scaling;
  void* dz;
};

__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename T, int LPR, int C>
__global__ __launch_bounds__(kThreads) void topk_routing_bwd_kernel(RouteBwdArgs g, int scoring) {
  constexpr int ROWS = kThreads / LPR, SLOTS = LPR * C, PER = (kRouteMaxK + LPR - 1) / LPR;
  __shared__ __attribute__((aligned(16))) float rows_[ROWS][SLOTS];
  const int l = threadIdx.x & (LPR - 1);
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
  const bool live = row < g.tokens;
  float* const buf = rows_[threadIdx.x / LPR];
  const T* const lrow = (const T*)g.logits + (live ? row : 0) * g.experts;
  const int n = live ? min(max(g.experts - l * C, 0), C) : 0;
  float base[C], top = 0.f, inv = 0.f;
  // both kinds of scores read the whole row: a logit that made its weights NaN makes its gradient NaN
  load_logits<C>(lrow + (n > 0 ? l * C : 0), n, g.vec && n == C, base);
  uint32_t bad = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) bad |= base[c] != base[c] || (scoring == SOFTMAX && base[c] == INFINITY);
  bad = row_reduce<LPR>(bad, Or{});
  if (scoring == SOFTMAX) {
    top = -INFINITY;
#pragma unroll
    for (int c = 0; c < C; ++c) top = c < n ? fmaxf(top, base[c]) : top;
    top = row_reduce<LPR>(top, Max{});
    top = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      base[c] = c < n ? exp_below(base[c], top) : 0.f;
      sum += base[c];
    }
    sum = row_reduce<LPR>(sum, Add{});
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }
  int e[PER];
  float s[PER], sn[PER], dp[PER], sum = 0.f, gs = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = i * LPR + l;
    e[i] = live && j < g.topk ? g.idx[row * g.topk + j] : -1;
    const bool in = (unsigned)e[i] < (unsigned)g.experts;
    e[i] = in ? e[i] : -1;
    dp[i] = in ? g.dp[row * g.topk + j] : 0.f;
    const float z = in ? load_elem<T>(lrow + e[i]) : 0.f;
    s[i] = scoring == SIGMOID ? fast_sigmoid(z) : exp_below(z, top) * inv;
    sn[i] = scoring == SIGMOID ? fast_sigmoid(-z) : 1.f;  // 1 - s without cancellation
    s[i] = in ? s[i] : 0.f;
    sum += s[i];
    gs = fmaf(dp[i], s[i], gs);
  }
  sum = row_reduce<LPR>(sum, Add{});
  gs = row_reduce<LPR>(gs, Add{});
  const float total = sum + 1e-20f;
  // gradient of a chosen score: a (dp - m); dot = sum of s ds
  const float a = bad ? NAN : g.normalize ? g.scaling / total : g.scaling;
  const float m = g.normalize ? gs / total : 0.f;
  float dot = 0.f;  // with the weights normalised, total - sum being 1e-20, what that leaves of it
  if (scoring == SOFTMAX) dot = g.normalize ? a * m * 1e-20f : a * gs;
#pragma unroll
  for (int c = 0; c < C; ++c) base[c] = bad ? NAN : scoring == SOFTMAX ? -(base[c] * inv) * dot : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) buf[l * C + c] = base[c];
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (e[i] >= 0) buf[e[i]] = s[i] * sn[i] * (a * (dp[i] - m) - dot);
  wave_lds_sync();
  if (!live) return;
  T* const out = (T*)g.dz + row * g.experts;
  constexpr int V = 16 / Elem<T>::BYTES;
  if (g.vec) {
    for (int c = l * V; c < g.experts; c += LPR * V) {
      if constexpr (V == 4) {
        *(float4*)(out + c) = *(const float4*)(buf + c);
      } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = buf[c + i];
        *(uint4*)(out + c) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                        pack_bf16x2(v[6], v[7]));
      }
    }
  } else {
    for (int c = l; c < g.experts; c += LPR) store_elem<T>(out + c, buf[c]);
  }
}

// Lanes of a row and experts of a lane for `groups` groups of `per` experts; slots 0: not supported.
struct RouteShape {
  int lpr = 0, c = 0, lanes = 0;
};
RouteShape route_shape(int groups, int per) {
  int g2 = 1;
  while (g2 < groups) g2 *= 2;
  for (int lpr : {16, 64}) {
    if (g2 > lpr) continue;
    const int lanes = lpr / g2, need = (per + lanes - 1) / lanes;
    int c = 1;
    while (c < need) c *= 2;
    if (c <= 16) return RouteShape{lpr, c, lanes};
  }
  return RouteShape{};
}

template <typename F>
hipError_t by_shape(const RouteShape& s, F&& f) {
  auto with = [&](auto lpr) {
    switch (s.c) {
      case 1: return f(lpr, std::integral_constant<int, 1>{});
      case 2: return f(lpr, std::integral_constant<int, 2>{});
      case 4: return f(lpr, std::integral_constant<int, 4>{});
      case 8: return f(lpr, std::integral_constant<int, 8>{});
      default: return f(lpr, std::integral_constant<int, 16>{});
    }
  };
  return s.lpr == 16 ? with(std::integral_constant<int, 16>{}) : with(std::integral_constant<int, 64>{});
}

template <typename T>
hipError_t fwd_t(const RouteArgs& g, const RouteShape& s, int scoring, hipStream_t stream) {
  return by_shape(s, [&](auto lpr, auto c) {
    const unsigned wgs = (unsigned)(((int64_t)g.tokens * s.lpr + kThreads - 1) / kThreads);
    LaunchTimer timer("topk_routing", stream);
    hipLaunchKernelGGL((topk_routing_kernel<T, lpr.value, c.value>), dim3(wgs), dim3(kThreads), 0, stream, g, scoring);
    return hipGetLastError();
  });
}
template <typename T>
hipError_t bwd_t(const RouteBwdArgs& g, const RouteShape& s, int scoring, hipStream_t stream) {
  return by_shape(s, [&](auto lpr, auto c) {
    const unsigned wgs = (unsigned)(((int64_t)g.tokens * s.lpr + kThreads - 1) / kThreads);
    LaunchTimer timer("topk_routing_bwd", stream);
    hipLaunchKernelGGL((topk_routing_bwd_kernel<T, lpr.value, c.value>), dim3(wgs), dim3(kThreads), 0, stream, g,
                       scoring);
    return hipGetLastError();
  });
}

}  // namespace

bool topk_routing_supported(int experts, int topk, int groups, int topk_groups) {
  if (experts < 1 || groups < 1 || experts % groups != 0 || topk_groups < 1 || topk_groups > groups) return false;
  if (topk < 1 || topk > kRouteMaxK || (int64_t)topk > (int64_t)topk_groups * (experts / groups)) return false;
  if (route_shape(1, experts).lpr == 0) return false;
  return topk_groups == groups || route_shape(groups, experts / groups).lpr != 0;
}

hipError_t launch_topk_routing(int dtype, const void* logits, const float* bias, int bias_stride, int tokens,
                               int experts, int topk, int scoring, int groups, int topk_groups, int normalize,
                               float scaling, float* probs, int32_t* idx, hipStream_t stream) {
  if (tokens == 0) return hipSuccess;
  if (topk_groups == groups) groups = topk_groups = 1;  // every group stays
  const int per = experts / groups, size = dtype == 0 ? 4 : 2;
  const RouteShape s = route_shape(groups, per);
  const int vec = s.c * size >= 16 && per % s.c == 0 && experts * size % 16 == 0 && per * size % 16 == 0 &&
                  (uintptr_t)logits % 16 == 0;
  const int bias_vec = per % s.c == 0 && s.c % 4 == 0 && (uintptr_t)bias % 16 == 0;  // per a multiple of 4
  const RouteArgs g{logits, bias, bias_stride, tokens, experts, topk, per, groups, topk_groups, s.lanes, vec, bias_vec,
                    normalize, scaling, probs, idx};
  return dtype == 0 ? fwd_t<float>(g, s, scoring, stream) : fwd_t<bf16_t>(g, s, scoring, stream);
}

hipError_t launch_topk_routing_bwd(const float* dprobs, int dtype, const void* logits, const int32_t* idx, int tokens,
                                   int experts, int topk, int scoring, int normalize, float scaling, void* dlogits,
                                   hipStream_t stream) {
  if (tokens == 0) return hipSuccess;
  const int size = dtype == 0 ? 4 : 2;
  const RouteShape s = route_shape(1, experts);
  const int vec = experts * size % 16 == 0 && (uintptr_t)logits % 16 == 0 && (uintptr_t)dlogits % 16 == 0;
  const RouteBwdArgs g{dprobs, logits, idx, tokens, experts, topk, vec, normalize, scaling, dlogits};
  return dtype == 0 ? bwd_t<float>(g, s, scoring, stream) : bwd_t<bf16_t>(g, s, scoring, stream);
}

}  // namespace esg
