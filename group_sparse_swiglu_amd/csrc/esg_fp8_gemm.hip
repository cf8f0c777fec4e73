// Matrix product of 8-bit floating point (e4m3) operands with a float32 scale
// per block of 128 K elements:
//   y[m, n] = sum over k of a[m, k] sa[m, k/128] * b[n, k] sb[n or n/128, k/128]
// a: [M, K] (activations), b: [N, K] (weights); the blocks of b are 1 x 128
// (SB_ROWS) or 128 x 128 (SB_TILES).  K is a multiple of 16.
//
// One 16 x 16 x 128 product covers exactly one block of K, so the inner sum of
// a block comes out of the matrix core unscaled and is added to the float32
// result with its scales by vector FMAs, four per product.  b is the products'
// row side: a lane then holds four consecutive n of one m, so it needs one
// a-scale and (128 x 128 blocks) a wave-uniform b-scale per product.
//
// Precision: the 8-bit matrix product adds the terms of a block in groups of
// eight, in which every term is cut, toward zero, 14 bits below the leading bit
// of the group's largest (measured: beside 448 * 448 a term of 4 is lost, one of 8
// kept); the groups are added with about 25 bits.  So a sum is off by at most 7 *
// 2^-14 of the sum of its |terms|, and by 2.1e-5 to 3.0e-5 of the result's norm on
// normal data with channels of unequal size, the same for every 8-bit form; bf16
// products keep float32 accuracy (1.3e-8).  A bf16 result rounds at 1.7e-3, and
// rounding an operand to e4m3 moves a term by up to 2^-4 of it, over a hundred times
// the cut, so it takes the 8-bit products.  Where large terms cancel, the cut can
// exceed the rounding of what they leave, though: a caller whose operands are exact
// and cancel asks for a float32 result.  That one would lose bits it can hold, so
// its operands are widened to bf16 (exactly) on the way into bf16 products, at half
// the matrix rate.
//
// Two kernels: fp8_rows_kernel for few rows and small products, where latency and
// the read of b count, fp8_tile_kernel (128 x 128 or 256 x 256 tiles) for the rest;
// plan() chooses between them.
#include <algorithm>

#include "esg_fp8.hpp"
#include "esg_internal.hpp"
#include "esg_pipe.hpp"

namespace esg {
namespace {

enum { SB_TILES = 0, SB_ROWS = 1 };
// OUT_PART: float32 partial sums of a split K axis (FINE: of a float32 result)
enum { OUT_F32 = 0, OUT_BF16 = 1, OUT_PART = 2, OUT_PART_FINE = 3 };
__host__ __device__ constexpr bool fine(int out) { return out == OUT_F32 || out == OUT_PART_FINE; }

// One K block of a 16-row operand as a lane holds it: 16 bytes of chunk g and
// 16 of chunk g + 4, as they are, or widened to bf16 (four products of 32 K).
template <bool FINE>
struct Frag;
template <>
struct Frag<false> {
  uint4 v[2];
  __device__ __forceinline__ Frag() {}
  __device__ __forceinline__ Frag(const uint4& lo, const uint4& hi) : v{lo, hi} {}
};
template <>
struct Frag<true> {
  uint4 v[4];
  __device__ __forceinline__ Frag() {}
  __device__ __forceinline__ Frag(const uint4& lo, const uint4& hi)
      : v{e4m3x8_to_bf16(lo.x, lo.y), e4m3x8_to_bf16(lo.z, lo.w), e4m3x8_to_bf16(hi.x, hi.y),
          e4m3x8_to_bf16(hi.z, hi.w)} {}
};
__device__ __forceinline__ f32x4 mma_block(const Frag<false>& a, const Frag<false>& b) {
  return mma_e4m3_k128(a.v[0], a.v[1], b.v[0], b.v[1]);
}
__device__ __forceinline__ f32x4 mma_block(const Frag<true>& a, const Frag<true>& b) {
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s) mma_bf16(d, a.v[s], b.v[s]);
  return d;
}

struct Fp8Args {
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  void* y;
  float* part;    // [splits][M][N] float32 partial sums of a split K axis
  int M, N, K, KB;
  int nm, nn;     // tiles along m and n
  int splits, kb_split;  // K splits, blocks of K in one
};

// ---------------------------------------------------------------------------
// Range.  The kernels multiply the two scales of a block with each other before
// they meet its sum, one operation per element.  With both scales below 2^64 that
// product is finite.  Above, it may not be though the block adds nothing (large
// values of one side against zeros of the other) or something finite: those
// blocks are scaled in 64 bits.  (A product below the normal range is off by
// 2^-150 at most, and the sum of a block is below 2^25: 2^-125 of the result.)
// ---------------------------------------------------------------------------
constexpr float kFarScale = 0x1p64f;
__device__ __forceinline__ float top4(float top, float a, float b, float c, float d) {
  return fmaxf(fmaxf(fmaxf(top, fabsf(a)), fabsf(b)), fmaxf(fabsf(c), fabsf(d)));
}
__device__ __forceinline__ float add_far(float acc, float d, float sa, float sb) {
  return acc + (float)((double)d * (double)sa * (double)sb);
}

// A 16 x 16 piece of the product over every kstep-th of the blocks kb0 .. kb1 - 1, straight from memory and scaled in
// 64 bits: element i of lane l is row n0 + (l / 16) * 4 + i of b and row m0 + l % 16 of a.
template <bool FINE, int SB>
__device__ __forceinline__ f32x4 far_piece(const Fp8Args& g, int m0, int n0, int kb0, int kb1, int kstep,
                                           int lr, int lg) {
  const int m = m0 + lr, n = n0 + lr;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int kb = kb0; kb < kb1; kb += kstep) {
    auto chunk = [&](const uint8_t* p, int row, int rows, int k) __attribute__((always_inline)) {
      return row < rows && k < g.K ? *(const uint4*)(p + (size_t)row * g.K + k) : make_uint4(0, 0, 0, 0);
    };
    const int k = kb * kQB + lg * 16;
    const Frag<FINE> a(chunk(g.a, m, g.M, k), chunk(g.a, m, g.M, k + 64));
    const Frag<FINE> b(chunk(g.b, n, g.N, k), chunk(g.b, n, g.N, k + 64));
    const f32x4 d = mma_block(b, a);
    const float sa = g.sa[(size_t)min(m, g.M - 1) * g.KB + kb];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int ne = min(n0 + lg * 4 + e, g.N - 1);
      acc[e] = add_far(acc[e], d[e], sa, g.sb[(size_t)(SB == SB_ROWS ? ne : ne / kQB) * g.KB + kb]);
    }
  }
  return acc;
}

// ---------------------------------------------------------------------------
// Tiles.  BM x BN outputs per workgroup; K in steps of one block (128 bytes per
// row) through two direct-to-LDS stages of K-row tiles.
//
// One step of a wave: FN row fragments of b against FM column fragments of a.
// The products of row fragment i run while the results of fragment i - 1 are
// scaled and added (the last one's in the next step) and fragment i + 1 is read.
// The barrier sits before the last fragment, whose operands are in registers:
// under its products the next step's first fragments are read and the loads of
// the step after that are issued.  (The compiler's own order waited out every
// product's latency.)
//
// The scales of four K blocks at a time go through registers to LDS, [4][BM +
// BN] floats in two alternating slots.  Results go through LDS, so that whole
// lines are written, where the rows of y are whole 16-byte chunks (N a multiple of
// 8, of 4 for float32); else each element is a store (4133 x 4366 x 784 76 us, with
// N = 4368 37).
//
// Bound by issue: the products' and the vector unit's busy times hardly overlap
// (matrix cores and vector unit busy 0.49 and 0.32 of the busy cycles at 32768 x
// 5504 x 2048, 0.42 and 0.45 at 2688 x 1024 x 16400), and each 16 x 16 x 128 product
// (32 cycles) needs four FMAs for its scales.  32768 x 5504 x 2048, 16-bit results:
// 371 to 393 us by box, 1.88 to 1.99 PFLOP/s; side by side on the same operands 374
// us, and 319 for the library's product with one scale per tensor, without these
// FMAs (8192 cubed: 470 and 353 us, 2.34 and 3.11 PFLOP/s).
// Float32 results: 2688 x 1024 x 16400 in 110 to 115 us with its adding of three K
// splits, 0.79 to 0.82 PFLOP/s; widening costs 16 conversions per fragment, and what
// a 256 x 256 tile would save on them it spills (61 registers).
// ---------------------------------------------------------------------------
template <int BM, int BN>
struct Tile {
  static constexpr int NW = BM * BN / (128 * 64) < 4 ? 4 : BM * BN / (128 * 64);  // waves
  static constexpr int NTH = NW * 64;
  static constexpr int WM = 64;                         // m per wave
  static constexpr int WN = BM * BN / (NW * WM);        // n per wave
  static constexpr int NWM = BM / WM;                   // waves along m
  static constexpr int FM = WM / 16, FN = WN / 16;
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int SROWS = BM + BN;
  static constexpr int SLOT = 4 * SROWS;                // floats of one scale slot
  static constexpr int FAR_AT = 2 * STAGE + 2 * SLOT * 4;  // a word per wave: it has met a scale of kFarScale or more
  static constexpr int LDS = FAR_AT + NW * 4;           // one workgroup per CU, or two
  static_assert(SROWS == NTH, "one scale row per thread");
  static_assert(WN <= 128, "the n range of a wave lies in one 128-row block");
};

// One lane's 16-byte direct-to-LDS load (see dma16) at voff + soff, soff scalar.
// The range check compares voff with the buffer's size less soff, so soff must
// not be past the buffer.
__device__ __forceinline__ void dma16_at(const DmaSrc& s, ESG_LDS char* wave_base, uint32_t voff, uint32_t soff) {
  const int m = __builtin_amdgcn_readfirstlane((int)(unsigned)(unsigned long long)wave_base);
  const int so = __builtin_amdgcn_readfirstlane((int)soff);
  asm volatile("buffer_load_dwordx4 %0, %1, %3 offen lds" : : "v"(voff), "s"(s.d), "{m0}"(m), "s"(so) : "memory");
}

template <int ROWS, int NW>
struct RowDma {
  static constexpr int NI = ROWS / 8 / NW;  // 1 KB instructions (8 rows of 128 bytes) per wave and stage
  uint32_t base[NI];
  __device__ __forceinline__ static int koff(int lane) { return ((lane & 7) ^ (lane >> 3)) * 16; }
  __device__ __forceinline__ void init(int w, int lane, int rows, int K) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = (w * NI + i) * 8 + (lane >> 3);
      base[i] = r < rows ? (uint32_t)r * (uint32_t)K + koff(lane) : kOOB;
    }
  }
  // before the block from k0 is issued that K cuts short: chunks at or past K read zeros from here on
  __device__ __forceinline__ void cut(int lane, int k0, int K) {
#pragma unroll
    for (int i = 0; i < NI; ++i) base[i] = k0 + koff(lane) < K ? base[i] : kOOB;
  }
  // k0: first K element of the step, below K
  __device__ __forceinline__ void issue(const DmaSrc& src, ESG_LDS char* st, int w, int k0) {
#pragma unroll
    for (int i = 0; i < NI; ++i) dma16_at(src, st + (w * NI + i) * 1024, base[i], (uint32_t)k0);
  }
};

// Block id -> tile: each XCD (id % 8) takes a contiguous run of an order that
// walks eight m tiles, then the next n tile, so the 32 workgroups of an XCD
// share operand panels in its L2.
__device__ __forceinline__ void tile_of(int id, int total, int nm, int nn, int& tm, int& tn) {
  const int per = total >> 3, extra = total & 7, x = id & 7;
  const int o = x * per + (x < extra ? x : extra) + (id >> 3);
  const int band = 8 * nn;
  const int bi = o / band, in = o - bi * band;
  const int rows = min(8, nm - bi * 8);
  tm = bi * 8 + in % rows;
  tn = in / rows;
}

template <int BM, int BN, int SB, int OUT>
__global__ __launch_bounds__((Tile<BM, BN>::NTH), 2) void fp8_tile_kernel(Fp8Args g) {
  using C = Tile<BM, BN>;
  using F = Frag<fine(OUT)>;
  __shared__ __attribute__((aligned(1024))) char lds_[C::LDS];
  ESG_LDS char* const lds = (ESG_LDS char*)lds_;
  ESG_LDS float* const slots = (ESG_LDS float*)(lds + 2 * C::STAGE);
  const int lane = threadIdx.x & 63, w = wave_id();
  const int wm = w % C::NWM, wn = w / C::NWM;
  const int lr = lane & 15, lg = lane >> 4;
  int tm, tn;
  tile_of(blockIdx.x, g.nm * g.nn, g.nm, g.nn, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int mrows = min(BM, g.M - m0), nrows = min(BN, g.N - n0);
  const int kb0 = blockIdx.y * g.kb_split, kb1 = min(g.KB, kb0 + g.kb_split);
  const int nk = kb1 - kb0;

  const DmaSrc ra = make_dma_src(g.a + (size_t)m0 * g.K, (uint32_t)mrows * (uint32_t)g.K);
  const DmaSrc rb = make_dma_src(g.b + (size_t)n0 * g.K, (uint32_t)nrows * (uint32_t)g.K);
  RowDma<BM, C::NW> da;
  RowDma<BN, C::NW> db;
  da.init(w, lane, mrows, g.K);
  db.init(w, lane, nrows, g.K);
  // loads of step t into stage S; past the last step: its block again (not used)
  auto issue = [&](int t, ESG_LDS char* st) __attribute__((always_inline)) {
    const int k0 = min(kb0 + t, kb1 - 1) * kQB;
    da.issue(ra, st, w, k0);
    db.issue(rb, st + C::A_BYTES, w, k0);
  };
  auto cut = [&](int t) __attribute__((always_inline)) {  // before issue(t)
    const int k0 = (kb0 + t) * kQB;
    if (k0 < g.K && k0 + kQB > g.K) {
      da.cut(lane, k0, g.K);
      db.cut(lane, k0, g.K);
    }
  };

  // this thread's row of scales (rows outside the matrix take the last one; their outputs are not stored)
  const float* srow;
  if ((int)threadIdx.x < BM) {
    srow = g.sa + (size_t)min(m0 + (int)threadIdx.x, g.M - 1) * g.KB;
  } else {
    const int n = min(n0 + (int)threadIdx.x - BM, g.N - 1);
    srow = g.sb + (size_t)(SB == SB_ROWS ? n : n / kQB) * g.KB;
  }
  float sreg[4];
  float top = 0.f;  // largest |scale| of this thread's row so far
  auto load_scales = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sreg[e] = srow[min(kb + e, kb1 - 1)];
  };
  auto put_scales = [&](int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) slots[slot * C::SLOT + e * C::SROWS + threadIdx.x] = sreg[e];
    top = top4(top, sreg[0], sreg[1], sreg[2], sreg[3]);
  };

  f32x4 acc[C::FN][C::FM];
  f32x4 dp[C::FM], sp = {0.f, 0.f, 0.f, 0.f};  // products not added yet, and their scales
  float fp[C::FM];
  F am[C::FM], bn;
  float fm[C::FM];
  f32x4 sn;
  zero_acc(acc);
#pragma unroll
  for (int j = 0; j < C::FM; ++j) {
    dp[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    fp[j] = 0.f;
  }
  auto add_scaled = [](f32x4& to, const f32x4& d, float f, const f32x4& s) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e] = fmaf(d[e], SB == SB_ROWS ? f * s[e] : f, to[e]);
  };
  // This lane's chunks lg and lg + 4 of the first column and row fragment in stage 0 (krow_off); the others lie
  // at constant distances, so the reads need no address arithmetic.
  const ESG_LDS char* const a_lo = lds + krow_off(wm * C::WM + lr, lg);
  const ESG_LDS char* const a_hi = lds + krow_off(wm * C::WM + lr, lg + 4);
  const ESG_LDS char* const b_lo = lds + C::A_BYTES + krow_off(wn * C::WN + lr, lg);
  const ESG_LDS char* const b_hi = lds + C::A_BYTES + krow_off(wn * C::WN + lr, lg + 4);
  struct Raw {
    uint4 v[2];
  };
  auto read16 = [](const ESG_LDS char* p) __attribute__((always_inline)) {
    return __builtin_bit_cast(uint4, *(const ESG_LDS u32x4_t*)p);
  };
  auto raw_a = [&](int st, int j) __attribute__((always_inline)) {
    return Raw{{read16(a_lo + st * C::STAGE + j * 2048), read16(a_hi + st * C::STAGE + j * 2048)}};
  };
  auto raw_b = [&](int st, int i) __attribute__((always_inline)) {
    return Raw{{read16(b_lo + st * C::STAGE + i * 2048), read16(b_hi + st * C::STAGE + i * 2048)}};
  };
  auto read_a = [&](int st, int j) __attribute__((always_inline)) {
    const Raw r = raw_a(st, j);
    am[j] = F(r.v[0], r.v[1]);
  };
  auto read_b = [&](int st, int i) __attribute__((always_inline)) {
    const Raw r = raw_b(st, i);
    return F(r.v[0], r.v[1]);
  };
  // scales of the step whose line is sc
  auto read_fa = [&](const ESG_LDS float* sc, int j) __attribute__((always_inline)) {
    fm[j] = sc[wm * C::WM + j * 16 + lr];
    if constexpr (SB == SB_TILES) fm[j] *= sc[BM + wn * C::WN];
  };
  auto read_sb = [&](const ESG_LDS float* sc, int i) __attribute__((always_inline)) {
    return SB == SB_ROWS ? *(const ESG_LDS f32x4*)(sc + BM + wn * C::WN + i * 16 + lg * 4) : f32x4{1.f, 1.f, 1.f, 1.f};
  };

  load_scales(kb0);
  cut(0);
  issue(0, lds);
  if (nk > 1) cut(1);
  issue(1, lds + C::STAGE);
  put_scales(0);
  wait_vmcnt<0>();
  wait_lgkm0();
  barrier();
  bn = read_b(0, 0);
  sn = read_sb(slots, 0);
#pragma unroll
  for (int j = 0; j < C::FM; ++j) {
    read_a(0, j);
    read_fa(slots, j);
  }
  // step t, in stage S (a constant at each of its two places)
  auto step = [&](int t, int S) __attribute__((always_inline)) {
    if (t + 2 < nk) cut(t + 2);
    // the next four blocks' scales: requested at a group's first step, written two steps later
    if ((t & 3) == 0 && t + 4 < nk) load_scales(kb0 + t + 4);
    if ((t & 3) == 2 && t + 2 < nk) put_scales(((t >> 2) + 1) & 1);
    const int st = S, st2 = S ^ 1;  // st2: the next step's stage (past the last step: read, not used)
    const ESG_LDS float* sc = slots + ((t >> 2) & 1) * C::SLOT + (t & 3) * C::SROWS;
    const ESG_LDS float* sc2 = slots + (((t + 1) >> 2) & 1) * C::SLOT + ((t + 1) & 3) * C::SROWS;
#pragma unroll
    for (int i = 0; i < C::FN && fine(OUT); ++i) {
      // The same order for widened operands: the four products of a block go through all column fragments in
      // turn (each depends on the one before), and what is read for the next fragment is widened under the
      // last of them, when it has arrived.
      Raw braw, araw[C::FM];
      F bnext;
      f32x4 snext;
      if (i + 1 < C::FN) {
        braw = raw_b(st, i + 1);
        snext = read_sb(sc, i + 1);
      } else {
        wait_lgkm0();
        wait_vmcnt<0>();
        barrier();
        issue(t + 2, lds + S * C::STAGE);
        braw = raw_b(st2, 0);
        snext = read_sb(sc2, 0);
#pragma unroll
        for (int j = 0; j < C::FM; ++j) araw[j] = raw_a(st2, j);
      }
      f32x4 d[C::FM];
      static_assert(C::FM == 4, "one of the four products per column fragment's sums");
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < C::FM; ++j) {
          if (s == 0) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
          mma_bf16(d[j], bn.v[s % (fine(OUT) ? 4 : 2)], am[j].v[s % (fine(OUT) ? 4 : 2)]);
        }
        add_scaled(acc[(i + C::FN - 1) % C::FN][s], dp[s], fp[s], sp);
      }
      bnext = F(braw.v[0], braw.v[1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < C::FM; ++j) {
        dp[j] = d[j];
        fp[j] = fm[j];
        if (i + 1 == C::FN) am[j] = F(araw[j].v[0], araw[j].v[1]);
      }
      sp = sn;
      bn = bnext;
      sn = snext;
    }
#pragma unroll
    for (int i = 0; i < C::FN && !fine(OUT); ++i) {
      F bnext;
      f32x4 snext;
      if (i + 1 < C::FN) {
        bnext = read_b(st, i + 1);
        snext = read_sb(sc, i + 1);
      } else {
        // this step's operands are all in registers; the next step's have landed
        wait_lgkm0();
        wait_vmcnt<0>();
        barrier();
        issue(t + 2, lds + S * C::STAGE);
        bnext = read_b(st2, 0);
        snext = read_sb(sc2, 0);
      }
      f32x4 d[C::FM];
#pragma unroll
      for (int j = 0; j < C::FM; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        d[j] = mma_block(bn, am[j]);
        add_scaled(acc[(i + C::FN - 1) % C::FN][j], dp[j], fp[j], sp);
        if (i + 1 == C::FN) read_a(st2, j);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < C::FM; ++j) {
        dp[j] = d[j];
        fp[j] = fm[j];
      }
      sp = sn;
      bn = bnext;
      sn = snext;
    }
#pragma unroll
    for (int j = 0; j < C::FM; ++j) read_fa(sc2, j);
  };
  for (int t = 0; t < nk; t += 2) {
    step(t, 0);
    if (t + 1 < nk) step(t + 1, 1);
  }
#pragma unroll
  for (int j = 0; j < C::FM; ++j) add_scaled(acc[C::FN - 1][j], dp[j], fp[j], sp);
  ESG_LDS int* const met = (ESG_LDS int*)(lds + C::FAR_AT);
  // a row with an infinite scale needs no second look: all of it is NaN in either form
  const bool far = __ballot(top >= kFarScale && top < INFINITY) != 0;
  if (lane == 0) met[w] = far;
  wait_lgkm0();
  wait_vmcnt<0>();
  barrier();  // the stages are free

  // ---- results: a lane holds 4 consecutive n of one m.  A wave takes 16 rows at
  // a time through 8 KB of its own (16 rows of 512 bytes at most), in 16-byte
  // chunks swizzled by row, and stores whole rows of its WN columns. ----
  constexpr int ES = OUT == OUT_BF16 ? 2 : 4;
  constexpr int NCH = C::WN * ES / 16;  // chunks per row
  char* y = OUT == OUT_BF16 || OUT == OUT_F32 ? (char*)g.y : (char*)(g.part + (size_t)blockIdx.y * g.M * g.N);
  const int mw = m0 + wm * C::WM, nw = n0 + wn * C::WN;
  auto store1 = [&](int m, int n, float v) __attribute__((always_inline)) {
    if (m < g.M && n < g.N) {
      if constexpr (ES == 2)
        store_elem<bf16_t>((bf16_t*)y + (size_t)m * g.N + n, v);
      else
        ((float*)y)[(size_t)m * g.N + n] = v;
    }
  };
  if (__ballot(met[lane % C::NW] != 0) != 0) {
    // a scale of kFarScale or more in this tile: all of it again, a piece of 16 x 16 at a time
    for (int f = 0; f < C::FM * C::FN; ++f) {
      const int mp = mw + f % C::FM * 16, np = nw + f / C::FM * 16;
      const f32x4 v = far_piece<fine(OUT), SB>(g, mp, np, kb0, kb1, 1, lr, lg);
#pragma unroll
      for (int e = 0; e < 4; ++e) store1(mp + lr, np + lg * 4 + e, v[e]);
    }
    return;
  }
  if (g.N * ES % 16 == 0) {
    static_assert(16 * NCH * 16 * C::NW <= 2 * C::STAGE, "the pieces lie in the stages");
    ESG_LDS char* out = lds + w * (16 * NCH * 16);
#pragma unroll
    for (int j = 0; j < C::FM; ++j) {
#pragma unroll
      for (int i = 0; i < C::FN; ++i) {
        const f32x4& v = acc[i][j];
        if constexpr (ES == 2)
          lds_write8(out + (lr * NCH + ((i * 2 + (lg >> 1)) ^ (lr & (NCH - 1)))) * 16 + (lg & 1) * 8,
                     pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else
          *(ESG_LDS f32x4*)(out + (lr * NCH + ((i * 4 + lg) ^ (lr & (NCH - 1)))) * 16) = v;
      }
      wait_lgkm0();
#pragma unroll
      for (int h = 0; h < 16 * NCH / 64; ++h) {
        const int r = (h * 64 + lane) / NCH, c = lane % NCH;
        const u32x4_t v = *(const ESG_LDS u32x4_t*)(out + (r * NCH + (c ^ (r & (NCH - 1)))) * 16);
        const int m = mw + j * 16 + r, n = nw + c * (16 / ES);
        if (m < g.M && n < g.N) *(u32x4_t*)(y + ((size_t)m * g.N + n) * ES) = v;
      }
      wait_lgkm0();  // read before the next rows are written
    }
  } else {
#pragma unroll
    for (int j = 0; j < C::FM; ++j) {
      const int m = mw + j * 16 + lr;
#pragma unroll
      for (int i = 0; i < C::FN; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) store1(m, nw + i * 16 + lg * 4 + e, acc[i][j][e]);
    }
  }
}

// y = sum of the K splits' partials, in split order.  Bound by memory and, below a few MB, by its launch (2 us;
// 33 MB of partials, 2688 x 1024 in three splits, 7.1 us).
template <typename T>
__global__ __launch_bounds__(256) void fp8_reduce_kernel(const float* __restrict__ part, int splits, size_t n,
                                                         T* __restrict__ y) {
  for (size_t i = (blockIdx.x * (size_t)256 + threadIdx.x) * 4; i < n; i += (size_t)gridDim.x * 1024) {
    if (i + 4 <= n && (n & 3) == 0) {
      float4 s = *(const float4*)(part + i);
      for (int z = 1; z < splits; ++z) {
        const float4 v = *(const float4*)(part + (size_t)z * n + i);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      const float o[4] = {s.x, s.y, s.z, s.w};
      Quad<T>::store(y + i, o);
    } else {
      for (size_t e = i; e < i + 4 && e < n; ++e) {
        float s = part[e];
        for (int z = 1; z < splits; ++z) s += part[(size_t)z * n + e];
        store_elem<T>(y + e, s);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows: a workgroup takes 16 rows of b and up to 64 rows of a (MT tiles of
// 16); its NW waves take the K blocks in turn and add their sums in LDS in wave
// order.  The read of b bounds it, with a's rows from L2 beside it (each
// workgroup reads them all, so the time grows with M).
//
// Everything goes through LDS: loads into the products' registers touch 16 rows,
// one per lane, in every quarter of a wave and come at about 15 bytes per clock
// and CU; direct-to-LDS loads of whole 128-byte rows come at about 40 (37 rows,
// N = 2048, K = 5504: 11.7 us from registers, 5.8 through LDS).  Each wave has P
// slots of its own, with a block of b, of a and their scales, and waits for its
// own loads only, never for another wave.
//
// Measured (graph of 30 calls on the same operands, 16-bit results): N = 2048, K =
// 5504: 4.0 us for one row, 5.8 for 37, 7.2 for 64; N = 11008, K = 2048: 4.7, 8.6 and
// 9.8 us (3.8 us is the read of b at 6 TB/s); N = K = 8192: 11.9 us for one row (5.6
// TB/s).
// ---------------------------------------------------------------------------
constexpr int kFewRows = 64;

template <int MT, int P>
struct SlotLayout {
  static constexpr int A_AT = 2048, SA_AT = A_AT + MT * 2048, SB_AT = SA_AT + 256, BYTES = SB_AT + 256;
  static constexpr int NI = 2 + 2 * MT + 2;  // load instructions of a block
  static_assert((P - 1) * NI < 64, "vmcnt range");
};

template <int MT, int NW, int P, int SB, int OUT>
__global__ __launch_bounds__(NW * 64) void fp8_rows_kernel(Fp8Args g) {
  using S = SlotLayout<MT, P>;
  constexpr int RED = NW * MT * 1024, RING = NW * P * S::BYTES;
  __shared__ __attribute__((aligned(1024))) char lds_[RED > RING ? RED : RING];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int lr = lane & 15, lg = lane >> 4;
  ESG_LDS char* const ring = (ESG_LDS char*)lds_ + w * P * S::BYTES;
  const int n0 = blockIdx.x * 16, nrows = min(16, g.N - n0);
  const int kb0 = blockIdx.y * g.kb_split, kb1 = min(g.KB, kb0 + g.kb_split);
  const int m0 = blockIdx.z * kFewRows, mrows = min(kFewRows, g.M - m0);
  const DmaSrc rb = make_dma_src(g.b + (size_t)n0 * g.K, (uint32_t)(nrows * g.K));
  const DmaSrc ra = make_dma_src(g.a + (size_t)m0 * g.K, (uint32_t)(mrows * g.K));
  const DmaSrc rsa = make_dma_src(g.sa + (size_t)m0 * g.KB, (uint32_t)(mrows * g.KB * 4));
  const DmaSrc rsb = SB == SB_TILES ? make_dma_src(g.sb + (size_t)(n0 / kQB) * g.KB, (uint32_t)(g.KB * 4))
                                    : make_dma_src(g.sb + (size_t)n0 * g.KB, (uint32_t)(nrows * g.KB * 4));
  // rows of eight, 16-byte chunks in the K-row swizzle; offsets of K block 0
  const int koff = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t ob[2], oa[2 * MT];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = i * 8 + (lane >> 3);
    ob[i] = r < nrows ? (uint32_t)(r * g.K + koff) : kOOB;
  }
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    const int r = i * 8 + (lane >> 3);
    oa[i] = r < mrows ? (uint32_t)(r * g.K + koff) : kOOB;
  }
  const uint32_t osa = lane < mrows ? (uint32_t)(lane * g.KB) * 4 : kOOB;
  const uint32_t osb = SB == SB_TILES ? 0u : lane < nrows ? (uint32_t)(lane * g.KB) * 4 : kOOB;
  // block kb into a slot; past the last block: zeros (so every block is the same number of loads).  kOOB plus an
  // offset below 2^31 stays past every buffer.
  auto request = [&](int kb, ESG_LDS char* slot) __attribute__((always_inline)) {
    const int k0 = kb * kQB;
    const bool in = kb < kb1 && k0 + koff < g.K;
#pragma unroll
    for (int i = 0; i < 2; ++i) dma16(rb, slot + i * 1024, in ? ob[i] + (uint32_t)k0 : kOOB);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) dma16(ra, slot + S::A_AT + i * 1024, in ? oa[i] + (uint32_t)k0 : kOOB);
    dma4(rsa, slot + S::SA_AT, kb < kb1 ? osa + (uint32_t)kb * 4 : kOOB);
    dma4(rsb, slot + S::SB_AT, kb < kb1 ? osb + (uint32_t)kb * 4 : kOOB);
  };
  f32x4 acc[MT];
  float top = 0.f;  // largest |scale| that this wave has met
  zero_acc(acc);
#pragma unroll
  for (int u = 0; u < P; ++u) request(kb0 + w + u * NW, ring + u * S::BYTES);
  int at = 0;
  for (int kb = kb0 + w; kb < kb1; kb += NW) {
    ESG_LDS char* slot = ring + at * S::BYTES;
    at = at + 1 == P ? 0 : at + 1;
    wait_vmcnt<(P - 1) * S::NI>();
    __builtin_amdgcn_sched_barrier(0);
    const Frag<fine(OUT)> bn(frag_krow(slot, lr, lg), frag_krow(slot, lr, lg + 4));
    const ESG_LDS float* fa = (const ESG_LDS float*)(slot + S::SA_AT);
    const ESG_LDS float* fb = (const ESG_LDS float*)(slot + S::SB_AT);
    f32x4 sn;
    if constexpr (SB == SB_ROWS)
      sn = *(const ESG_LDS f32x4*)(fb + lg * 4);
    else
      sn = f32x4{fb[0], fb[0], fb[0], fb[0]};
    top = top4(top, sn[0], sn[1], sn[2], sn[3]);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const ESG_LDS char* a = slot + S::A_AT;
      const Frag<fine(OUT)> am(frag_krow(a, j * 16 + lr, lg), frag_krow(a, j * 16 + lr, lg + 4));
      const f32x4 d = mma_block(bn, am);
      const float f = fa[j * 16 + lr];
      top = fmaxf(top, fabsf(f));
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(d[e], f * sn[e], acc[j][e]);
    }
    wait_lgkm0();  // the slot has been read
    __builtin_amdgcn_sched_barrier(0);
    request(kb + P * NW, slot);
  }
  if (__ballot(top >= kFarScale) != 0) {
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[j] = far_piece<fine(OUT), SB>(g, m0 + j * 16, n0, kb0 + w, kb1, NW, lr, lg);
  }
  wait_vmcnt<0>();
  __syncthreads();  // the slots become the sums of the waves
  f32x4* red = (f32x4*)lds_;
#pragma unroll
  for (int j = 0; j < MT; ++j) red[(w * MT + j) * 64 + lane] = acc[j];
  __syncthreads();
  const float* rf = (const float*)red;
  for (int o = threadIdx.x; o < mrows * 16; o += NW * 64) {
    const int n = o & 15, m = o >> 4;
    const int at_o = ((m >> 4) * 64 + (n >> 2) * 16 + (m & 15)) * 4 + (n & 3);
    float s = rf[at_o];
#pragma unroll
    for (int v = 1; v < NW; ++v) s += rf[v * MT * 256 + at_o];
    if (n < nrows) {
      const size_t out = (size_t)(m0 + m) * g.N + n0 + n;
      if constexpr (OUT == OUT_BF16)
        store_elem<bf16_t>((bf16_t*)g.y + out, s);
      else if constexpr (OUT == OUT_F32)
        ((float*)g.y)[out] = s;
      else
        g.part[(size_t)blockIdx.y * g.M * g.N + out] = s;
    }
  }
}

template <int MT, int NW, int P, int SB, int OUT>
hipError_t launch_rows(const Fp8Args& g, hipStream_t stream) {
  LaunchTimer timer("fp8_rows", stream);
  hipLaunchKernelGGL((fp8_rows_kernel<MT, NW, P, SB, OUT>), dim3((g.N + 15) / 16, g.splits, g.nm),
                     dim3(NW * 64), 0, stream, g);
  return hipGetLastError();
}

// Four waves where there is more than a workgroup for each CU, eight otherwise
// (us, four against eight waves: one row of N = 2048, K = 5504 4.3 / 4.0, of
// N = 11008, K = 2048 4.7 / 5.6; 64 rows: 8.8 / 7.2 and 9.8 / 12.3).  A slot per wave
// where slots are large, or two workgroups of a CU would not fit (64 rows of
// N = 11008: 9.8 us with one slot, 12.3 with two).
template <int SB, int OUT>
hipError_t launch_few_rows(const Fp8Args& g, hipStream_t stream) {
  if ((g.N + 15) / 16 * g.splits * g.nm > kNominalCUs) {
    if (g.M > 48) return launch_rows<4, 4, 1, SB, OUT>(g, stream);
    if (g.M > 32) return launch_rows<3, 4, 2, SB, OUT>(g, stream);
    if (g.M > 16) return launch_rows<2, 4, 2, SB, OUT>(g, stream);
    return launch_rows<1, 4, 2, SB, OUT>(g, stream);
  }
  if (g.M > 48) return launch_rows<4, 8, 1, SB, OUT>(g, stream);
  if (g.M > 32) return launch_rows<3, 8, 1, SB, OUT>(g, stream);
  if (g.M > 16) return launch_rows<2, 8, 2, SB, OUT>(g, stream);
  return launch_rows<1, 8, 2, SB, OUT>(g, stream);
}

template <int BM, int BN, int SB, int OUT>
hipError_t launch_tiles(const Fp8Args& g, hipStream_t stream) {
  LaunchTimer timer("fp8_tile", stream);
  hipLaunchKernelGGL((fp8_tile_kernel<BM, BN, SB, OUT>), dim3(g.nm * g.nn, g.splits), dim3(Tile<BM, BN>::NTH), 0,
                     stream, g);
  return hipGetLastError();
}

// Kernel, tile size and K splits by shape alone (so a shape rounds alike everywhere).
struct Plan {
  bool rows = false, big = false;
  int nm = 0, nn = 0, splits = 1, kb_split = 0;
};

Plan plan(int M, int N, int K, bool f32_out) {
  Plan p;
  const int KB = (K + kQB - 1) / kQB;
  p.kb_split = KB;
  auto split_k = [&](int s) {
    s = std::min(std::max(s, 1), 16);
    p.kb_split = (KB + s - 1) / s;
    p.splits = (KB + p.kb_split - 1) / p.kb_split;
  };
  // The few-rows kernel, in chunks of 64 rows, while its workgroups are one round of the CUs, or two with a short K
  // (us, few rows / 128 x 128 tiles: 128 rows of N = 2048, K = 5504 8.1 / 15.0; 512 rows of N = 512, K = 2048
  // 5.0 / 10.5; 256 rows of N = K = 2048, two rounds, 6.8 / 13.0, of N = 2048, K = 16384 38.8 / 23.2).
  const long long wgs = (long long)((N + 15) / 16) * ((M + kFewRows - 1) / kFewRows);
  if (M <= kFewRows || wgs <= kNominalCUs || (wgs <= 2 * kNominalCUs && KB <= 32)) {
    p.rows = true;
    p.nm = (M + kFewRows - 1) / kFewRows;
    // Few workgroups with much work in each: split K.  The second launch costs 2 us (N = 512, K = 16384, whole / split:
    // one row 6.5 / 5.5 us, 64 rows 15.4 / 8.7; N = 512, K = 7168: 4.3 / 5.0 and 8.6 / 7.0).
    const int work = KB * ((std::min(M, kFewRows) + 15) / 16);
    if (wgs <= kNominalCUs / 2 && work >= (wgs <= kNominalCUs / 4 ? 128 : 256))
      split_k(std::min({std::max(4, work / 64), std::max(4, kNominalCUs / (int)wgs), KB / 8}));
    return p;
  }
  const long long big = (long long)((M + 255) / 256) * ((N + 255) / 256);
  // float32 results: the widened operands of a 256 x 256 tile do not fit the registers (61 spilled)
  p.big = big >= kNominalCUs && !f32_out;
  const int t = p.big ? 256 : 128;
  p.nm = (M + t - 1) / t;
  p.nn = (N + t - 1) / t;
  if (p.big) return p;
  // 128 x 128 tiles: a step of K takes a CU 0.63 us (1.08 with widening), and two workgroups on it twice that; a split
  // costs a launch (2.5 us) and its partials' way to memory and back (5 TB/s).  The number of splits with the least sum
  // (us; M x N x K: splitting to fill two workgroups per CU / this): 2048 x 2048 x 2048 25.1 / 16.6,
  // 333 x 5504 x 2048 18.3 / 14.2, 1024 x 4096 x 4096 33.0 / 28.6.
  const double step = f32_out ? 1.08 : 0.63;
  double best = 1e30;
  int splits = 1;
  for (int s = 1; s <= std::min(16, KB); ++s) {
    const int per = (KB + s - 1) / s, n = (KB + per - 1) / per;
    const long long rounds = ((long long)p.nm * p.nn * n + kNominalCUs - 1) / kNominalCUs;
    const double cost = step * per * (double)rounds + (n > 1 ? 2.5 + n * (double)M * N * 8.0 / 5e6 : 0.0);
    if (cost < best) best = cost, splits = s;
  }
  split_k(splits);
  return p;
}

}  // namespace

size_t fp8_matmul_workspace_bytes(int M, int N, int K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  const int splits = std::max(plan(M, N, K, false).splits, plan(M, N, K, true).splits);
  return splits > 1 ? (size_t)splits * M * N * 4 : 0;
}

template <int SB, int OUT>
static hipError_t launch_products(const Fp8Args& g, const Plan& p, hipStream_t stream) {
  if (p.rows) return launch_few_rows<SB, OUT>(g, stream);
  if constexpr (OUT == OUT_BF16)
    if (p.big) return launch_tiles<256, 256, SB, OUT>(g, stream);
  return launch_tiles<128, 128, SB, OUT>(g, stream);
}

template <int SB>
static hipError_t run(Fp8Args& g, const Plan& p, int out_bf16, hipStream_t stream) {
  if (p.splits == 1)
    return out_bf16 ? launch_products<SB, OUT_BF16>(g, p, stream) : launch_products<SB, OUT_F32>(g, p, stream);
  const hipError_t e = out_bf16 ? launch_products<SB, OUT_PART>(g, p, stream)
                                : launch_products<SB, OUT_PART_FINE>(g, p, stream);
  if (e != hipSuccess) return e;
  const size_t n = (size_t)g.M * g.N;
  const unsigned blocks = (unsigned)std::min<size_t>((n + 1023) / 1024, 2048);
  LaunchTimer timer("fp8_reduce", stream);
  if (out_bf16)
    hipLaunchKernelGGL(fp8_reduce_kernel<bf16_t>, dim3(blocks), dim3(256), 0, stream, g.part, g.splits, n,
                       (bf16_t*)g.y);
  else
    hipLaunchKernelGGL(fp8_reduce_kernel<float>, dim3(blocks), dim3(256), 0, stream, g.part, g.splits, n,
                       (float*)g.y);
  return hipGetLastError();
}

hipError_t launch_fp8_matmul(const void* a, const float* sa, const void* b, const float* sb, int sb_rows, int out_dtype,
                             int M, int N, int K, void* y, void* workspace, hipStream_t stream) {
  const Plan p = plan(M, N, K, out_dtype == 0);
  Fp8Args g{};
  g.a = (const uint8_t*)a;
  g.b = (const uint8_t*)b;
  g.sa = sa;
  g.sb = sb;
  g.y = y;
  g.part = (float*)workspace;
  g.M = M;
  g.N = N;
  g.K = K;
  g.KB = (K + kQB - 1) / kQB;
  g.nm = p.nm;
  g.nn = p.nn;
  g.splits = p.splits;
  g.kb_split = p.kb_split;
  return sb_rows ? run<SB_ROWS>(g, p, out_dtype == 1, stream) : run<SB_TILES>(g, p, out_dtype == 1, stream);
}

}  // namespace esg
