// Matrix product of 4-bit floating point (e2m1) operands with a power of two per 32
// K elements, of one pair or of rows grouped by expert:
//   y[m, n] = sum over k of a[m, k] 2^(sa[m, k/32] - 127) * b[n, k] 2^(sb[n, k/32] - 127)
// a: [M, K] (activations), b: [N, K] or [E, N, K] (weights), two codes a byte, K a
// multiple of 32.  Grouped: rows offsets[e] .. offsets[e+1] - 1 of y take b[e]; row m of
// the left operand is a[rows[m]] where rows is given.
//
// The matrix cores apply the powers of two themselves, one byte per lane and 32
// elements.  Products of codes have 4 significant bits and, inside a block, a range
// of 8, so a block's sum is exact; sums of blocks are float32 (measured: off by at most
// 2^-22.5 of the sum of the |terms| of 128 elements and the accumulator), whatever the
// result's type.  b is the products' row side: a lane then holds four consecutive n of
// one m.
//
// Two kernels: mx_rows_kernel for few rows, bound by the read of b, and mx_tile_kernel
// for many; plan() chooses between them, and cuts a long K into parts where outputs are
// few.
#include <algorithm>

#include "esg_internal.hpp"
#include "esg_mx.hpp"
#include "esg_pipe.hpp"

namespace esg {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

struct MxArgs {
  const uint8_t* a;
  const uint8_t* b;
  const uint8_t* sa;
  const uint8_t* sb;
  const int32_t* offsets;  // [E + 1], or NULL: one b for all rows
  const int32_t* rows;     // [M], or NULL
  void* y;
  const uint32_t* ta;      // exponents as the large tiles take them: [ceil(K/128)][M] and [ceil(K/128)][E N] words
  const uint32_t* tb;
  int a_rows, M, N, K, E, grouped;
  int nm, nn;              // row chunks or tiles (grouped: at most so many), tiles along n
  int parts, per_part;     // K in parts of so many steps (of kFewK or 128 elements); one: y is written, not float32 parts
};

// Type of the result: float32, bfloat16, or float32 sums of parts of K, [parts][M][N].
enum { OUT_F32 = 0, OUT_BF16 = 1, OUT_PARTS = 2 };

// Rows m0 .. m1 - 1 of y with b[e]; none for m1 <= m0.
struct Span {
  int e, m0, m1;
};

// The z-th chunk of up to `chunk` rows: of all rows, or counted expert after expert, without the first `skip` of each.
// Every wave looks for itself: 64 experts at a time, their chunks counted by a prefix sum over the lanes.  Offsets are
// taken into 0 .. M.
__device__ __forceinline__ Span find_span(const MxArgs& g, int z, int chunk, int lane, int skip = 0) {
  if (g.offsets == nullptr) return Span{0, z * chunk, min(g.M, (z + 1) * chunk)};
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < g.E) {
      lo = min(max(g.offsets[e], 0), g.M);
      hi = min(max(g.offsets[e + 1], 0), g.M);
    }
    const int own = hi > lo ? max((hi - lo + chunk - 1) / chunk - skip, 0) : 0;
    int upto = own;
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
      const int v = __shfl_up(upto, off);
      upto += lane >= off ? v : 0;
    }
    const uint64_t has = __ballot(upto > z);
    if (has != 0) {
      const int at = __builtin_ctzll(has);
      const int first = __builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(own, at);
      const int m0 = __builtin_amdgcn_readlane(lo, at) + (z - first + skip) * chunk;
      return Span{e0 + at, m0, min(__builtin_amdgcn_readlane(hi, at), m0 + chunk)};
    }
    z -= __builtin_amdgcn_readlane(upto, 63);
  }
  return Span{0, 0, 0};
}

// Direct-to-LDS loads (see dma16) of 16 bytes per lane at voff + soff, soff scalar and not past the buffer (the range
// check compares voff with the buffer's size less soff), and of 4.  The compiler does not see which scalar registers an
// asm block reads, and one that a vector instruction wrote (a readlane, of a spilled descriptor for one) may be read
// by a load five states later at the earliest: hence the s_nop.
__device__ __forceinline__ void load16(const DmaSrc& s, ESG_LDS char* wave_base, uint32_t voff, uint32_t soff = 0) {
  const int m = __builtin_amdgcn_readfirstlane((int)(unsigned)(unsigned long long)wave_base);
  const int so = __builtin_amdgcn_readfirstlane((int)soff);
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds"
               :
               : "v"(voff), "s"(s.d), "{m0}"(m), "s"(so)
               : "memory");
}
__device__ __forceinline__ void load4(const DmaSrc& s, ESG_LDS char* wave_base, uint32_t voff) {
  const int m = __builtin_amdgcn_readfirstlane((int)(unsigned)(unsigned long long)wave_base);
  asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds" : : "v"(voff), "s"(s.d), "{m0}"(m) : "memory");
}

// The same for the few-row kernel, which asks for as many spans as there are experts and full chunks: the e-th is the
// first chunk of expert e, two loads away and not a search, and those from E on are the other chunks, which only an
// expert of more rows than a chunk has.
__device__ __forceinline__ Span find_few(const MxArgs& g, int z, int chunk, int lane) {
  if (g.offsets == nullptr) return Span{0, z * chunk, min(g.M, (z + 1) * chunk)};
  if (z < g.E) {
    const int lo = min(max(g.offsets[z], 0), g.M), hi = min(max(g.offsets[z + 1], 0), g.M);
    return Span{z, lo, min(hi, lo + chunk)};
  }
  return find_span(g, z - g.E, chunk, lane, 1);
}

// Descriptor of `bytes` exponents from byte `from` of p (at any address), in whole dwords; skew: what they start past
// the descriptor's base.  A dword at either end that holds a wanted byte may hold others beside it.
__device__ __forceinline__ DmaSrc scale_src(const uint8_t* p, size_t from, uint32_t bytes, uint32_t& skew) {
  skew = (uint32_t)((uintptr_t)(p + from) & 3);
  return make_dma_src(p + from - skew, (skew + bytes + 3) & ~3u);
}

// 16 x 16 x 128 and 32 x 32 x 64 products with exponents from byte OP of each side's word
template <int OP>
__device__ __forceinline__ void mma_mx16(f32x4& acc, const uint4& a, const uint4& b, uint32_t sa, uint32_t sb) {
  const i32x8_t x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, OP, (int)sa, OP, (int)sb);
}
template <int OP>
__device__ __forceinline__ void mma_mx32(f32x16_t& acc, const u32x4_t& a, const u32x4_t& b, uint32_t sa, uint32_t sb) {
  const i32x8_t x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 4, 4, OP, (int)sa, OP, (int)sb);
}

// ---------------------------------------------------------------------------
// Few rows: a workgroup takes 16 rows of b and up to 64 rows of a (MT tiles of 16);
// its NW waves take the steps of K in turn and add their sums in LDS in wave order.
// The read of b bounds it.  Everything goes through LDS in whole 128-byte rows, a wave
// into a slot of its own, and it waits for its own loads only: what keeps memory busy is
// many workgroups side by side (64 tokens, 6 of 64 experts, N = 2816, K = 2048: 40 us
// with two or four waves and one slot each, 48 with eight; four waves of two slots, which
// leave room for half as many workgroups, took 51 where one slot each took 36).  The exponents of a step (8 bytes
// of a row that starts at any byte) come as the three dwords that hold them, and the one
// needed is read back as a byte.
// ---------------------------------------------------------------------------
constexpr int kStream = 2;   // store policy: past the caches
constexpr int kFewRows = 64;
constexpr int kFewK = 256;  // K elements of a step: 128 bytes of a row, 8 exponents

template <int MT>
struct Slot {
  static constexpr int A_AT = 2048, SB_AT = A_AT + MT * 2048, SA_AT = SB_AT + 256, BYTES = SA_AT + MT * 256;
};
template <int NW, int MTMAX>
constexpr int rows_lds() {
  int most = 0;
  for (int mt = 1; mt <= MTMAX; ++mt) {
    const int slot = (2048 + 256) * (1 + mt), red = mt * 1024;
    most = most > slot ? most : slot;
    most = most > red ? most : red;
  }
  return NW * most;
}

template <int MT, int NW, int OUT>
__device__ __forceinline__ void few_rows(const MxArgs& g, const Span& s, char* lds_) {
  using S = Slot<MT>;
  const int lane = threadIdx.x & 63, w = wave_id();
  const int lr = lane & 15, lg = lane >> 4;
  ESG_LDS char* const slot = (ESG_LDS char*)lds_ + w * S::BYTES;
  const int n0 = blockIdx.x * 16, nrows = min(16, g.N - n0), mrows = s.m1 - s.m0;
  const int KH = g.K >> 1, KS = g.K >> 5, steps = (g.K + kFewK - 1) / kFewK;
  const size_t b0 = (size_t)s.e * g.N + n0;
  uint32_t b_skew, a_skew;
  const DmaSrc rb = make_dma_src(g.b + b0 * KH, (uint32_t)(nrows * KH));
  const DmaSrc rsb = scale_src(g.sb, b0 * KS, (uint32_t)(nrows * KS), b_skew);
  const bool gather = g.rows != nullptr;
  const DmaSrc ra = gather ? make_dma_src(g.a, (uint32_t)g.a_rows * (uint32_t)KH)
                           : make_dma_src(g.a + (size_t)s.m0 * KH, (uint32_t)(mrows * KH));
  const DmaSrc rsa = gather ? scale_src(g.sa, 0, (uint32_t)g.a_rows * (uint32_t)KS, a_skew)
                            : scale_src(g.sa, (size_t)s.m0 * KS, (uint32_t)(mrows * KS), a_skew);
  // rows of eight, 16-byte chunks in the K-row swizzle; offsets of step 0
  const int koff = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t ob[2], oa[2 * MT], osa[MT], osb;
  // exponents: lane = dword * 16 + row; of row lr the byte for chunk lg of the first and second 128 elements
  int eb[2], ea[MT][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = i * 8 + (lane >> 3);
    ob[i] = r < nrows ? (uint32_t)(r * KH + koff) : kOOB;
  }
  {
    const uint32_t at = b_skew + (uint32_t)(lr * KS);
    osb = lr < nrows && lg < 3 ? (at & ~3u) + lg * 4 : kOOB;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int p = (int)(at & 3) + j * 4 + lg;
      eb[j] = S::SB_AT + (p >> 2) * 64 + lr * 4 + (p & 3);
    }
  }
  // b's and a's part of step t into the slot, chunks at or past K as zeros (kOOB plus an offset below 2^31 stays past
  // every buffer)
  auto request_b = [&](int t) __attribute__((always_inline)) {
    const bool in = t * 128 + koff < KH;
#pragma unroll
    for (int i = 0; i < 2; ++i) load16(rb, slot + i * 1024, in ? ob[i] + (uint32_t)t * 128u : kOOB);
    load4(rsb, slot + S::SB_AT, osb + (uint32_t)t * 8u);
  };
  auto request_a = [&](int t) __attribute__((always_inline)) {
    const bool in = t * 128 + koff < KH;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) load16(ra, slot + S::A_AT + i * 1024, in ? oa[i] + (uint32_t)t * 128u : kOOB);
#pragma unroll
    for (int i = 0; i < MT; ++i) load4(rsa, slot + S::SA_AT + i * 256, osa[i] + (uint32_t)t * 8u);
  };
  const int t0 = OUT == OUT_PARTS ? blockIdx.z * g.per_part : 0;
  const int t1 = OUT == OUT_PARTS ? min(t0 + g.per_part, steps) : steps;
  if (t0 + w < t1) request_b(t0 + w);  // b is on its way before the rows of a are looked up
  // row of a behind row i of the span; -1: none
  auto a_row = [&](int i) __attribute__((always_inline)) {
    if (i >= mrows) return -1;
    if (!gather) return i;
    const int r = g.rows[s.m0 + i];
    return (unsigned)r < (unsigned)g.a_rows ? r : -1;
  };
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    const int r = a_row(i * 8 + (lane >> 3));
    oa[i] = r >= 0 ? (uint32_t)r * (uint32_t)KH + koff : kOOB;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = a_row(i * 16 + lr);
    const uint32_t at = a_skew + (uint32_t)(r >= 0 ? r : 0) * (uint32_t)KS;
    osa[i] = r >= 0 && lg < 3 ? (at & ~3u) + lg * 4 : kOOB;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int p = (int)(at & 3) + j * 4 + lg;
      ea[i][j] = S::SA_AT + i * 256 + (p >> 2) * 64 + lr * 4 + (p & 3);
    }
  }
  if (t0 + w < t1) request_a(t0 + w);
  f32x4 acc[MT];
  zero_acc(acc);
  for (int t = t0 + w; t < t1; t += NW) {
    wait_vmcnt<0>();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // past K the codes are zeros, and the exponents those of other rows: any but 255 will do
      const bool in = t * kFewK + (j * 4 + lg) * 32 < g.K;
      const uint4 bv = frag_krow(slot, lr, j * 4 + lg);
      const uint32_t bs = in ? *(const ESG_LDS uint8_t*)(slot + eb[j]) : 0u;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint4 av = frag_krow(slot + S::A_AT, i * 16 + lr, j * 4 + lg);
        const uint32_t as = in ? *(const ESG_LDS uint8_t*)(slot + ea[i][j]) : 0u;
        mma_mx16<0>(acc[i], bv, av, bs, as);
      }
    }
    wait_lgkm0();  // the slot has been read
    __builtin_amdgcn_sched_barrier(0);
    if (t + NW < t1) {
      request_b(t + NW);
      request_a(t + NW);
    }
  }
  wait_vmcnt<0>();
  __syncthreads();  // the slots become the sums of the waves
  f32x4* red = (f32x4*)lds_;
#pragma unroll
  for (int i = 0; i < MT; ++i) red[(w * MT + i) * 64 + lane] = acc[i];
  __syncthreads();
  const float* rf = (const float*)red;
  float* const part = (float*)g.y + (OUT == OUT_PARTS ? (size_t)blockIdx.z * g.M * g.N : 0);
  for (int o = threadIdx.x; o < mrows * 16; o += NW * 64) {
    const int n = o & 15, m = o >> 4;
    const int at_o = ((m >> 4) * 64 + (n >> 2) * 16 + (m & 15)) * 4 + (n & 3);
    float v = rf[at_o];
#pragma unroll
    for (int u = 1; u < NW; ++u) v += rf[u * MT * 256 + at_o];
    if (n < nrows) {
      const size_t out = (size_t)(s.m0 + m) * g.N + n0 + n;
      if constexpr (OUT == OUT_BF16)
        store_elem<bf16_t>((bf16_t*)g.y + out, v);
      else
        part[out] = v;
    }
  }
}

// MTMAX * 16 rows of a at most: 64, or, for LDS that lets more workgroups stand side by side, 16
template <int NW, int MTMAX, int OUT>
__global__ __launch_bounds__(NW * 64) void mx_rows_kernel(MxArgs g) {
  __shared__ __attribute__((aligned(1024))) char lds[rows_lds<NW, MTMAX>()];
  const Span s = find_few(g, blockIdx.y, MTMAX * 16, threadIdx.x & 63);
  const int mrows = s.m1 - s.m0;
  if (mrows <= 0) return;
  if constexpr (MTMAX > 1) {
    if (mrows > 48) return few_rows<4, NW, OUT>(g, s, lds);
    if (mrows > 32) return few_rows<3, NW, OUT>(g, s, lds);
    if (mrows > 16) return few_rows<2, NW, OUT>(g, s, lds);
  }
  few_rows<1, NW, OUT>(g, s, lds);
}

// ---------------------------------------------------------------------------
// Tiles.  BM x BN outputs per workgroup of waves of 64 x BN/2 each.  K in steps of 128
// (64 bytes per row) through a ring of four direct-to-LDS stages; in a step two slices of
// 64, each FN x FM products of 32 x 32 x 64.
//
// A slice's operands are read under the products of the one before.  The barrier of a step
// sits before the products of its second slice, whose operands are in registers: behind
// it the step's stage is free, and the loads of four steps on go there, spread over the
// next two slices' products.  So three steps' loads are on their way at any time, and the
// only wait is for the oldest.  In large tiles a step's loads all go to the stage that the
// step before has left, and those of a tile's last three steps are the next tile's first:
// the ring runs on from tile to tile (8191 tokens, 6 of 64 experts, 2048 x 1408, eleven
// steps: 136 -> 126 us; 32768 x 5504 x 2048, sixteen: equal, see below).
// The exponents of a step are a word per row and step.  Large tiles take them from arrays in
// which a step's words of neighbouring rows are neighbours (mx_words_kernel lays them out
// first): one load of whole lines per wave and step.  Read where they are, 16 bytes of each
// of 64 rows at a time, they took a quarter of the loop (30000 cycles against 22000 for 16
// steps).  The small tile, whose products are too short for a launch before them, does read
// them there: the five dwords that hold the bytes of four steps (a row starts at any byte)
// go into two slots, and the lanes that use a step's four bytes put them together.
//
// 32768 x 5504 x 2048 to bf16: 211 to 272 us (2.7 to 3.5 PFLOP/s), 8192 cubed 260 to 290 (3.8 to 4.2).  Long loops are
// bound by the power that the products draw (registers alone: 8.1 to 9.1 PFLOP/s on zeros, 5.9 to 6.4 on random codes,
// at a clock of 1.4 to 1.5 GHz): the matrix cores are busy for 69 % of the second's cycles.  Of the first's they are for
// 49 %: a step's reads and loads fill LDS for about as long as its products take, and the way between two tiles comes on
// top (without the results' way 206 for 227, without their stores alone 214 to 223).
// ---------------------------------------------------------------------------
template <int BM, int BN>
struct Tile {
  static constexpr int NWM = BM / 64, NWN = 2, NW = NWM * NWN, NTH = NW * 64;
  static constexpr int WM = 64, WN = BN / NWN;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int A_BYTES = BM * 64, B_BYTES = BN * 64, STAGE = A_BYTES + B_BYTES;
  static constexpr int SROWS = BM + BN;                 // rows of exponents: one per thread
  static constexpr bool WORDS = BM * BN > 128 * 128;    // exponents laid out in words before
  static constexpr int SLOT = SROWS * (WORDS ? 4 : 20); // of a step; or 16 bytes of each row, then 4 of each
  static constexpr int LDS = 4 * STAGE + (WORDS ? 4 : 2) * SLOT;
  static_assert(SROWS == NTH, "a row of exponents per thread");
};

// position of 16-byte chunk c of row r: 16 consecutive rows at one chunk lie in different banks
__device__ __forceinline__ int mx_swz(int r) { return (r >> 2) & 3; }

// Block id -> tile: each XCD (id % 8) takes a contiguous run of an order that walks eight m tiles, then the next n
// tile, so the workgroups of an XCD share operand panels in its L2.
__device__ __forceinline__ void tile_of(int id, int total, int nm, int nn, int& tm, int& tn) {
  const int per = total >> 3, extra = total & 7, x = id & 7;
  const int o = x * per + (x < extra ? x : extra) + (id >> 3);
  const int band = 8 * nn;
  const int bi = o / band, in = o - bi * band;
  const int rows = min(8, nm - bi * 8);
  tm = bi * 8 + in % rows;
  tn = in / rows;
}

// The first `left` elements of v (all if there are more) to y, aligned to an element: rows whose length is no multiple of
// 16 bytes (32768 x 5501 x 2048: 272 us; element by element 598).
template <int OUT>
__device__ __forceinline__ void store_chunk(char* y, const u32x4_t& v, int left) {
  typedef u32x4_t chunk_t __attribute__((aligned(2)));
  constexpr int PER = OUT == OUT_BF16 ? 8 : 4;
  if (left >= PER) {
    *(chunk_t*)y = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < PER - 1; ++e)
    if (e < left) {
      if constexpr (OUT == OUT_BF16)
        *(uint16_t*)(y + e * 2) = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
      else
        *(uint32_t*)(y + e * 4) = v[e];
    }
}

template <int BM, int BN, int OUT>
__global__ __launch_bounds__((Tile<BM, BN>::NTH), 2) void mx_tile_kernel(MxArgs g) {
  using C = Tile<BM, BN>;
  __shared__ __attribute__((aligned(1024))) char lds_[C::LDS];
  ESG_LDS char* const lds = (ESG_LDS char*)lds_;
  ESG_LDS char* const slots = lds + 4 * C::STAGE;
  const int w = wave_id();
  const int wm = w % C::NWM, wn = w / C::NWM;
  int lane, lr, lh;
  const int KH = g.K >> 1, KS = g.K >> 5;
  int steps = (g.K + 127) / 128;
  const bool gather = g.rows != nullptr;
  const bool skewed = (((uintptr_t)g.sa | (uintptr_t)g.sb | KS) & 3) != 0;  // some row of exponents starts inside a dword

  // ---- the tile: its rows and columns, where its loads start ----
  constexpr int NA = BM / 16 / C::NW, NB = BN / 16 / C::NW, NL = NA + NB + C::WORDS;  // loads of a wave and step
  constexpr int PER = C::FM * C::FN, FR = C::FM + C::FN;
  int koff, ra0, rb0;
  // what follows from the lane, each time anew: kept over the tiles, its many addresses would drive out the sums
  auto set_lane = [&]() __attribute__((always_inline)) {
    lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    lr = lane & 31;
    lh = lane >> 5;
    koff = ((lane & 3) ^ mx_swz(lane >> 2)) * 16;  // a load fills sixteen rows of 64 bytes
    ra0 = wm * C::WM + lr;
    rb0 = wn * C::WN + lr;
  };
  auto is_a = [](int f) { return f >= 1 && f <= C::FM; };  // fragments in the order b0, a0 .., b1 ..
  auto frag_row = [&](int f) __attribute__((always_inline)) {  // of the tile's rows, A's then B's
    return is_a(f) ? ra0 + (f - 1) * 32 : BM + rb0 + (f == 0 ? 0 : f - C::FM) * 32;
  };
  Span s, snext;
  int n0, id = blockIdx.x;
  DmaSrc ra, rb, rs;
  uint32_t oa[NA], ob[NB], os, skew[FR];
  constexpr bool PARTS = OUT == OUT_PARTS;
  static_assert(!PARTS || !C::WORDS, "parts of K: small tiles");
  const int tiles = g.nm * g.nn, total = PARTS ? tiles * g.parts : tiles;
  int t0 = 0, kend = KH, part = 0;  // the part's first step, where its bytes of a row end
  // this workgroup's next tile from id on, its rows in snext (grouped rows may fill fewer tiles than are counted)
  auto find_tile = [&]() __attribute__((always_inline)) {
    for (; id < total; id += gridDim.x) {
      int tm, tn;
      tile_of(PARTS ? id % tiles : id, tiles, g.nm, g.nn, tm, tn);
      snext = find_span(g, tm, BM, lane);
      if (snext.m1 > snext.m0) return;
    }
  };
  auto set_tile = [&]() __attribute__((always_inline)) {  // the tile that find_tile found
    int tm, tn;
    tile_of(PARTS ? id % tiles : id, tiles, g.nm, g.nn, tm, tn);
    if constexpr (PARTS) {
      part = id / tiles;
      t0 = part * g.per_part;  // a multiple of four
      steps = min(g.per_part, (g.K + 127) / 128 - t0);
      kend = min(KH, (t0 + steps) * 64);
    }
    s = snext;
    const int mrows = s.m1 - s.m0;
    n0 = tn * BN;
    const int nrows = min(BN, g.N - n0);
    const size_t b0 = (size_t)s.e * g.N + n0;
    rb = make_dma_src(g.b + b0 * KH, (uint32_t)(nrows * KH));
    // (a without rows: the bytes of one, for soff; none is read)
    ra = gather ? make_dma_src(g.a, (uint32_t)max(g.a_rows, 1) * (uint32_t)KH)
                : make_dma_src(g.a + (size_t)s.m0 * KH, (uint32_t)(mrows * KH));
    auto a_row = [&](int i) __attribute__((always_inline)) {
      if (i >= mrows) return -1;
      if (!gather) return i;
      const int r = g.rows[s.m0 + i];
      return (unsigned)r < (unsigned)g.a_rows ? r : -1;
    };
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int r = a_row((w * NA + i) * 16 + (lane >> 2));
      oa[i] = r >= 0 ? (uint32_t)r * (uint32_t)KH + koff : kOOB;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int r = (w * NB + i) * 16 + (lane >> 2);
      ob[i] = r < nrows ? (uint32_t)(r * KH) + koff : kOOB;
    }
    if constexpr (C::WORDS) {
      // a wave's rows lie on one side (BM is a multiple of 64); the step's distance is soff, so no range check: the words
      // of rows past the tile are those of others, or zeros, and meet zeros or results that are not stored
      rs = w * 64 < BM ? make_dma_src(g.ta, (uint32_t)g.M * (uint32_t)steps * 4u)
                       : make_dma_src(g.tb, (uint32_t)(g.E * g.N) * (uint32_t)steps * 4u);
      os = (uint32_t)(w * 64 < BM ? s.m0 + (int)threadIdx.x : (int)b0 + (int)threadIdx.x - BM) * 4u;
    } else {
      // this thread's row of the tile, from the dword that holds its first byte
      uint32_t a_skew, b_skew;
      const DmaSrc rsb = scale_src(g.sb, b0 * KS, (uint32_t)(nrows * KS), b_skew);
      const DmaSrc rsa = gather ? scale_src(g.sa, 0, (uint32_t)g.a_rows * (uint32_t)KS, a_skew)
                                : scale_src(g.sa, (size_t)s.m0 * KS, (uint32_t)(mrows * KS), a_skew);
      if (w * 64 < BM) {
        rs = rsa;
        const int r = a_row((int)threadIdx.x);
        os = r >= 0 ? (a_skew + (uint32_t)r * (uint32_t)KS) & ~3u : kOOB;
      } else {
        rs = rsb;
        const int r = (int)threadIdx.x - BM;
        os = r < nrows ? (b_skew + (uint32_t)(r * KS)) & ~3u : kOOB;
      }
#pragma unroll
      for (int f = 0; f < FR; ++f) {
        const int r = frag_row(f);
        skew[f] = 0;
        if (skewed) {
          const int ar = is_a(f) ? a_row(r) : 0;
          skew[f] = (is_a(f) ? a_skew + (uint32_t)(ar >= 0 ? ar : 0) * (uint32_t)KS
                             : b_skew + (uint32_t)((r - BM) * KS)) & 3;
        }
      }
    }
  };

  // ---- loads ----
  // The wave's i-th load of step t into its stage (the last: its exponents).  Chunks at or past K, and steps past the last, read zeros.  (No
  // branch: one between two slices would draw the products before it behind it.)
  auto issue = [&](int t, int S, int i) __attribute__((always_inline)) {
    ESG_LDS char* const st = lds + S * C::STAGE;
    if (C::WORDS && i == NA + NB) {  // (a step past the last: its last's, not used)
      const uint32_t row = w * 64 < BM ? (uint32_t)g.M : (uint32_t)(g.E * g.N);
      load4(rs, slots + S * C::SLOT + w * 256, os + (uint32_t)min(t, steps - 1) * row * 4u);
      return;
    }
    const int k = (t0 + t) * 64;
    const uint32_t at = i < NA ? oa[i < NA ? i : 0] : ob[i < NA ? 0 : i - NA];
    const uint32_t voff = koff < kend - k ? at : kOOB;
    const uint32_t soff = (uint32_t)min(k, KH);
    if (i < NA)
      load16(ra, st + (w * NA + i) * 1024, voff, soff);
    else
      load16(rb, st + C::A_BYTES + (w * NB + i - NA) * 1024, voff, soff);
  };
  // exponents of the four steps of group u, where they are read as they are
  auto issue_scales = [&](int u, int slot) __attribute__((always_inline)) {
    if constexpr (C::WORDS) return;
    ESG_LDS char* const to = slots + slot * C::SLOT;
    const uint32_t k = u * 4 < steps ? os + (uint32_t)(t0 + u * 4) * 4u : kOOB;
    load16(rs, to + w * 1024, k);
    load4(rs, to + C::SROWS * 16 + w * 256, skewed ? k + 16u : kOOB);
  };
  int ring = 0;  // stage of the tile's step 0 (large tiles: they follow each other around the ring)
  // a tile's first loads: steps 0 to 2, the exponents of steps 0 to 7
  auto first_loads = [&]() __attribute__((always_inline)) {
    issue_scales(0, 0);
#pragma unroll
    for (int t = 0; t < 3; ++t) {
#pragma unroll
      for (int i = 0; i < NL; ++i) issue(t, C::WORDS ? (ring + t) & 3 : t, i);
      if (t == 0) issue_scales(1, 1);
    }
  };
  constexpr int BEHIND_FIRST = (C::WORDS ? 0 : 2) + 2 * NL;  // of them those behind step 0's

  // ---- operands of a slice, and the exponents of a step as this lane's half needs them: bytes 0 and 2 of a word ----
  u32x4_t av[2][C::FM], bv[2][C::FN];
  uint32_t es[2][FR], raw[FR][2];  // of even and odd steps
  // 32 rows further on are 32 * 64 bytes: the swizzle repeats every 16 rows
  auto read_frag = [&](int S, int sl, int to, int f) __attribute__((always_inline)) {
    const ESG_LDS char* const st = lds + S * C::STAGE;
    if (is_a(f)) {
      const ESG_LDS char* p = st + ra0 * 64 + (((sl * 2 + lh) ^ mx_swz(ra0)) << 4);
      av[to][f - 1] = *(const ESG_LDS u32x4_t*)(p + (f - 1) * 2048);
    } else {
      const ESG_LDS char* p = st + C::A_BYTES + rb0 * 64 + (((sl * 2 + lh) ^ mx_swz(rb0)) << 4);
      bv[to][f == 0 ? 0 : f - C::FM] = *(const ESG_LDS u32x4_t*)(p + (f == 0 ? 0 : f - C::FM) * 2048);
    }
  };
  // the two dwords that hold the step's bytes: the fifth dword of a row lies apart
  auto read_raw = [&](int slot, int S, int f) __attribute__((always_inline)) {
    if constexpr (C::WORDS) {
      raw[f][0] = *(const ESG_LDS uint32_t*)(slots + S * C::SLOT + frag_row(f) * 4);
      return;
    }
    const ESG_LDS char* const sc = slots + slot * C::SLOT;
    raw[f][0] = *(const ESG_LDS uint32_t*)(sc + frag_row(f) * 16 + S * 4);
    raw[f][1] = S < 3 ? *(const ESG_LDS uint32_t*)(sc + frag_row(f) * 16 + S * 4 + 4)
                      : *(const ESG_LDS uint32_t*)(sc + C::SROWS * 16 + frag_row(f) * 4);
  };
  auto set_scales = [&](int t, int to) __attribute__((always_inline)) {
    if constexpr (C::WORDS) {
#pragma unroll
      for (int f = 0; f < FR; ++f) es[to][f] = raw[f][0] >> (8 * lh);
      return;
    }
    const int left = KS - (t0 + t) * 4;  // bytes of the row still in K; those past it are other rows'
    const uint32_t mask = left >= 4 ? ~0u : left > 0 ? (1u << (8 * left)) - 1u : 0u;
#pragma unroll
    for (int f = 0; f < FR; ++f) es[to][f] = (__builtin_amdgcn_alignbyte(raw[f][1], raw[f][0], skew[f]) & mask) >> (8 * lh);
  };
  f32x16_t acc[C::FN][C::FM];
  // the products of a slice, with `beside(p)` in the issue order behind the p-th of them
  auto products = [&](int sl, int of, auto&& beside) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < C::FN; ++i)
#pragma unroll
      for (int j = 0; j < C::FM; ++j) {
        const uint32_t eb = es[of][i == 0 ? 0 : C::FM + i], ea = es[of][1 + j];
        if (sl == 1)
          mma_mx32<2>(acc[i][j], bv[sl][i], av[sl][j], eb, ea);
        else
          mma_mx32<0>(acc[i][j], bv[sl][i], av[sl][j], eb, ea);
        beside(i * C::FM + j);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  constexpr int HALF = NL / 2;  // loads of a step issued behind its barrier; the others in the next slice
  // Step t in stage S = t % 4, exponents in slot U = t / 4 % 2 (constants at each place).  What the next slice needs is
  // read behind a slice's first products, two reads at a time, so that it is there when they end: both waves of a SIMD
  // are at the same place, and what one of them waits for nothing covers.  The barrier lies before the last quarter of
  // the first slice's products, which cover some of it.
  auto step = [&](int t, int S, int U) __attribute__((always_inline)) {
    constexpr int WAIT = PER * 3 / 4 - 1;
    products(0, S & 1, [&](int p) __attribute__((always_inline)) {
      if (p < FR / 2) {
        read_frag(S, 1, 1, 2 * p);
        read_frag(S, 1, 1, 2 * p + 1);
      }
      if (p >= PER / 4 - 1 && p < PER / 4 - 1 + NL - HALF) issue(t + 3, (S + 3) & 3, HALF + p - PER / 4 + 1);
      if (p == WAIT) {
        // the second slice's operands are in registers and the next step's have landed: two steps' loads are newer
        wait_lgkm0();
        wait_vmcnt<2 * NL>();
        barrier();
        if (S == 3) issue_scales((t >> 2) + 2, U);  // the slot's last bytes were read before the barrier
      }
    });
    products(1, S & 1, [&](int p) __attribute__((always_inline)) {
      if (p < FR / 2) {
        read_frag((S + 1) & 3, 0, 0, 2 * p);
        read_frag((S + 1) & 3, 0, 0, 2 * p + 1);
      }
      if (p == (FR + 1) / 2 - 1) {
#pragma unroll
        for (int f = 0; f < FR; ++f) read_raw(S == 3 ? U ^ 1 : U, (S + 1) & 3, f);
      }
      if (p >= PER / 4 && p < PER / 4 + HALF) issue(t + 4, S, p - PER / 4);
      if (p == PER - 2) set_scales(t + 1, (S & 1) ^ 1);
    });
  };
  // The same for large tiles: stage and step's parity apart, and the loads are those of three steps on, all of them, so
  // that they pass from one tile to the next between two steps.  `from`: the load's step 0 in steps of this tile.
  auto large_step = [&](int t, int P, int from) __attribute__((always_inline)) {
    constexpr int WAIT = PER * 3 / 4 - 1, FIRST = NL - HALF;
    const int S = (ring + t) & 3, S1 = (ring + t + 1) & 3, S3 = (ring + t + 3) & 3;
    products(0, P, [&](int p) __attribute__((always_inline)) {
      if (p < FR / 2) {
        read_frag(S, 1, 1, 2 * p);
        read_frag(S, 1, 1, 2 * p + 1);
      }
      if (p >= PER / 4 - 1 && p < PER / 4 - 1 + FIRST) issue(t + 3 - from, S3, p - PER / 4 + 1);
      if (p == WAIT) {
        wait_lgkm0();
        wait_vmcnt<NL + FIRST>();  // the next step has landed: newer are one step's loads and a part of another's
        barrier();
      }
    });
    products(1, P, [&](int p) __attribute__((always_inline)) {
      if (p < FR / 2) {
        read_frag(S1, 0, 0, 2 * p);
        read_frag(S1, 0, 0, 2 * p + 1);
      }
      if (p == (FR + 1) / 2 - 1) {
#pragma unroll
        for (int f = 0; f < FR; ++f) read_raw(0, S1, f);
      }
      if (p >= PER / 4 && p < PER / 4 + HALF) issue(t + 3 - from, S3, FIRST + p - PER / 4);
      if (p == PER - 2) set_scales(t + 1, P ^ 1);
    });
  };
  static_assert(FR % 2 == 0 && FR / 2 <= PER * 3 / 4 && PER / 4 - 1 + NL - HALF <= PER * 3 / 4, "reads and loads before the barrier");

  constexpr int ES = OUT == OUT_BF16 ? 2 : 4;
  constexpr int NCH = C::WN * ES / 16;                     // 16-byte chunks of a wave's row
  constexpr int PIECE = C::STAGE / C::NW / (NCH * 16);     // rows of a wave that its share of a stage holds
  static_assert(PIECE <= 32 && 32 % PIECE == 0 && PIECE * NCH % 64 == 0, "whole pieces");
  const bool whole = g.N * ES % 16 == 0;

  set_lane();
  find_tile();
  if (id >= total) return;
  set_tile();
  first_loads();
  bool loaded = false;  // the tile's first loads went out, and its step 0 landed, in the steps of the tile before
  for (;;) {
    set_lane();
#pragma unroll
    for (int i = 0; i < C::FN; ++i)
#pragma unroll
      for (int j = 0; j < C::FM; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    // Loads come back in the order of their issue, but stores not in order with them: with so many of both under way,
    // step 0's loads, which have as many loads behind them, are done.
    if (!C::WORDS || !loaded) wait_vmcnt<BEHIND_FIRST>();
    barrier();  // step 0 has landed, and the last stage is free of the results
    if constexpr (!C::WORDS) {
#pragma unroll
      for (int i = 0; i < HALF; ++i) issue(3, 3, i);
    }
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      read_raw(0, C::WORDS ? ring : 0, f);
      read_frag(C::WORDS ? ring : 0, 0, 0, f);
    }
    set_scales(0, 0);
    const int m0 = s.m0 + wm * C::WM, mend = s.m1, nw = n0 + wn * C::WN;
    char* const y = (char*)g.y + (PARTS ? (size_t)part * g.M * g.N * ES : 0);
    id += gridDim.x;
    find_tile();  // its reads' latency passes here rather than between the tiles
    if constexpr (C::WORDS) {
      // the last three steps load the next tile's first three
      loaded = steps >= 3;
      const int last = steps, own = loaded && id < total ? steps - 3 : steps;
      int from = 0;
      for (int t = 0;; t += 2) {
        if (t == own) {
          set_tile();
          from = last;
        }
        large_step(t, 0, from);
        if (t + 1 >= last) break;
        if (t + 1 == own) {
          set_tile();
          from = last;
        }
        large_step(t + 1, 1, from);
        if (t + 2 >= last) break;
      }
    } else {
      for (int t = 0;; t += 8) {
        step(t, 0, 0);
        if (t + 1 >= steps) break;
        step(t + 1, 1, 0);
        if (t + 2 >= steps) break;
        step(t + 2, 2, 0);
        if (t + 3 >= steps) break;
        step(t + 3, 3, 0);
        if (t + 4 >= steps) break;
        step(t + 4, 0, 1);
        if (t + 5 >= steps) break;
        step(t + 5, 1, 1);
        if (t + 6 >= steps) break;
        step(t + 6, 2, 1);
        if (t + 7 >= steps) break;
        step(t + 7, 3, 1);
        if (t + 8 >= steps) break;
      }
    }
    ring = (ring + steps) & 3;
    wait_lgkm0();
    if (!C::WORDS || !loaded) {
      wait_vmcnt<0>();
      barrier();  // the stages are free
      // the next tile's first loads go out before this one's results
      set_lane();
      if (id < total) {
        set_tile();
        first_loads();
      }
    }
    // ---- results: a lane holds, of one m, four consecutive n out of every eight.  A wave takes PIECE rows at a time
    // through its share of the last stage, in 16-byte chunks swizzled by row, and stores whole rows of its WN columns,
    // past the caches where chunks are aligned: what a product leaves is larger than they are, or read elsewhere. ----
    ESG_LDS char* const out = lds + (C::WORDS ? (ring + 3) & 3 : 3) * C::STAGE + w * (PIECE * NCH * 16);
    const int row = lr % PIECE;
#pragma unroll
    for (int j = 0; j < C::FM; ++j)
#pragma unroll
      for (int h = 0; h < 32 / PIECE; ++h) {
        const int m = m0 + j * 32 + h * PIECE, live = min(max(mend - m, 0), PIECE);
        const rsrc_t to = make_rsrc(y + (size_t)m * g.N * ES, (uint32_t)(live * g.N) * ES);
        if (lr / PIECE == h) {
#pragma unroll
          for (int i = 0; i < C::FN; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x16_t v = acc[i][j];
              if constexpr (ES == 2)
                lds_write8(out + (row * NCH + ((i * 4 + q) ^ (row & (NCH - 1)))) * 16 + lh * 8,
                           pack_bf16x2(v[q * 4], v[q * 4 + 1]), pack_bf16x2(v[q * 4 + 2], v[q * 4 + 3]));
              else
                *(ESG_LDS f32x4*)(out + (row * NCH + ((i * 8 + q * 2 + lh) ^ (row & (NCH - 1)))) * 16) =
                    f32x4{v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]};
            }
        }
        wait_lgkm0();
#pragma unroll
        for (int c0 = 0; c0 < PIECE * NCH / 64; ++c0) {
          const int r = (c0 * 64 + lane) / NCH, c = lane % NCH;
          const u32x4_t v = *(const ESG_LDS u32x4_t*)(out + (r * NCH + (c ^ (r & (NCH - 1)))) * 16);
          const int n = nw + c * (16 / ES);
          if (whole) {
            __builtin_amdgcn_raw_buffer_store_b128(v, to, n < g.N ? (r * g.N + n) * ES : (int)kOOB, 0, kStream);
          } else if (r < live) {
            store_chunk<OUT>(y + ((size_t)(m + r) * g.N + n) * ES, v, g.N - n);
          }
        }
        wait_lgkm0();  // read before the next rows are written
      }
    if (id >= total) {
      wait_vmcnt<0>();  // loads past the last tile, of zeros, have reached this workgroup's LDS
      return;
    }
  }
}

// The exponents of a and b as words, [ceil(K/128)][rows]: word (t, r) holds those of elements 128 t .. 128 t + 127 of row
// r, zeros past K.  A thread takes 64 bytes of a row, from any address on; a's rows in the order of y's (zeros for rows[] outside a).
struct WordsSide {
  const uint8_t* scale;
  const int32_t* index;  // or NULL
  uint32_t* out;
  int rows, src_rows;
};
constexpr int kWordLoads = 4;  // 16 bytes each
__global__ __launch_bounds__(256) void mx_words_kernel(WordsSide a, WordsSide b, unsigned a_blocks, int KS) {
  const bool second = blockIdx.x >= a_blocks;
  const WordsSide& g = second ? b : a;
  const unsigned block = second ? blockIdx.x - a_blocks : blockIdx.x;
  const int words = (KS + 3) / 4, pieces = (words + 4 * kWordLoads - 1) / (4 * kWordLoads);
  const unsigned chunk = block / pieces;
  const int t0 = (int)(block - chunk * pieces) * 4 * kWordLoads;
  const int r = (int)chunk * 256 + (int)threadIdx.x;
  if (r >= g.rows) return;
  const int src = g.index != nullptr ? g.index[r] : r;
  const bool in = (unsigned)src < (unsigned)g.src_rows;
  const uint8_t* p = g.scale + (size_t)(in ? src : 0) * KS + t0 * 4;
  const int left = in ? KS - t0 * 4 : 0;  // bytes of the row from t0 on
  typedef u32x4_t piece_t __attribute__((aligned(1)));
  typedef uint32_t word_t __attribute__((aligned(1)));
  u32x4_t v[kWordLoads];
#pragma unroll
  for (int i = 0; i < kWordLoads; ++i) {
    v[i] = u32x4_t{0, 0, 0, 0};
    if (left >= 16 * (i + 1)) {
      v[i] = *(const piece_t*)(p + 16 * i);
    } else if (left > 16 * i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = 16 * i + 4 * j;
        if (at + 4 <= left) {
          v[i][j] = *(const word_t*)(p + at);
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e) v[i][j] |= at + e < left ? (uint32_t)p[at + e] << (8 * e) : 0u;
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4 * kWordLoads; ++j)
    if (t0 + j < words) g.out[(size_t)(t0 + j) * g.rows + r] = v[j / 4][j % 4];
}

// y = sum of the parts, in their order.  V elements of a thread.
template <int V, int OUT>
__global__ __launch_bounds__(256) void mx_parts_kernel(const float* __restrict__ part, int parts, size_t n,
                                                       void* __restrict__ y) {
  const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (at >= n) return;
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    if constexpr (V == 4) {
      const float4 q = *(const float4*)(part + p * n + at);
      v[0] += q.x;
      v[1] += q.y;
      v[2] += q.z;
      v[3] += q.w;
    } else {
      v[0] += part[p * n + at];
    }
  }
  if constexpr (OUT == OUT_BF16) {
    if constexpr (V == 4)
      *(uint2*)((bf16_t*)y + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else
      store_elem<bf16_t>((bf16_t*)y + at, v[0]);
  } else {
    if constexpr (V == 4)
      *(float4*)((float*)y + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
      ((float*)y)[at] = v[0];
  }
}

// Kernel and tile size by shape alone (so a shape rounds alike everywhere).
struct Plan {
  int tile = 0;   // 0: few rows,
  int few = 0;    // so many at a time
  int nm = 0, nn = 0;
  int parts = 1, per_part = 0;
};
// chunks of `chunk` rows, at most: grouped rows leave up to one short chunk per expert
long long chunks(const MxArgs& g, int chunk) {
  return !g.grouped ? (g.M + chunk - 1) / chunk : (long long)g.M / chunk + std::min(g.E, g.M);
}
Plan plan(const MxArgs& g) {
  Plan p;
  // K in parts of a multiple of `unit` steps where that leaves no more workgroups than CUs and takes `spare` steps or
  // more off each one's chain: a second kernel adds the parts, whose launch and reads cost 5 to 9 us.
  auto split = [&](int steps, int unit, int spare) {
    const long long wgs = (long long)p.nm * p.nn;
    if (g.grouped || wgs * 2 > kNominalCUs) return;
    const int units = (steps + unit - 1) / unit, most = (int)std::min<long long>(units, kNominalCUs / wgs);
    const int per = (units + most - 1) / most * unit;
    if (steps - per < spare) return;
    p.parts = (steps + per - 1) / per;
    p.per_part = per;
  };
  const int per = g.grouped ? (g.M + g.E - 1) / g.E : g.M;  // rows that share a b, on average
  const long long wgs =
      (long long)((g.N + 15) / 16) * (g.grouped ? g.M / kFewRows + std::min(g.E, g.M) : (g.M + kFewRows - 1) / kFewRows);
  // Few rows: by expert up to 16 of each on average (us, few rows / tiles, N = 2816, K = 2048, 64 experts: 9 rows 34 /
  // 42, 15 rows 45 / 47, 18 rows 72 / 47), in chunks of 16, else up to 64; or while the workgroups are no more than three
  // for each CU (256 x 2048 x 5504, 512 of them, 9.8 / 16.9; 100 x 5504 x 2048, 688, 7.4 / 9.7; 128 x 8192 x 2048, 1024,
  // 10.7 / 9.4; 87 tokens, 2 of 5 experts, 232 x 1952, 105, 7.7 / 10.6; 1000, 2 of 8, 512 x 1024, 1248, 11 / 8.5) or,
  // where K is long enough for tiles in parts, one (200 x 2048 x 8192, 512, 15.8 / 15.2; 200 x 3000 x 8192, 752, 22 / 17).
  constexpr int kLongK = 56 * 128;
  const int most = g.grouped || g.K < kLongK ? 3 : 1;
  if (per <= (g.grouped ? 16 : kFewRows) || wgs <= kNominalCUs * most) {
    p.few = per <= 16 ? 16 : kFewRows;
    p.nm = (int)(g.grouped ? g.E + g.M / p.few : (g.M + p.few - 1) / p.few);
    p.nn = (g.N + 15) / 16;
    // a round of the eight waves takes 0.5 us for one row and 1.5 for 64 (us, whole / parts: 64 x 512 x 16384 14.3 / 10.2;
    // 1 x 512 x 16384 6.7 / 10.2, 40 x 256 x 8192 7.3 / 10.5)
    split((g.K + kFewK - 1) / kFewK, 8, 2560 / (16 + std::min(g.M, kFewRows)));
    return p;
  }
  // Tiles, by the microseconds of each size: rounds of a tile for each CU, a round by its steps and the way between tiles
  // (of the small ones, two of which run side by side, half of it; a quarter more where rows of exponents start inside
  // dwords), and the words' launch before the large.  By expert half a tile of rows is expected to stay empty.  Measured,
  // 256 / 128: 4096 x 4096 x 2048, 1 and 4 rounds, 30 / 36; x 512 16.4 / 15; 3000 x 5504 x 2048, 2 and 5, 40 / 35; 4096 x
  // 5504 x 2048, 2 and 6, 42 / 43; 32768 x 5504 x 2048, 11 and 43, 272 / 335; by expert 2500 tokens, 4 of 32, 2048 x 2048,
  // 2 and 6, 59 / 51; 3000, 6 of 64, 2816 x 2048, 5 and 15, 114 / 125; 3006, 5 of 27, 1116 x 3808, 2 and 5, 76 / 98.
  const int steps = (g.K + 127) / 128;
  auto rounds = [&](int tile) {
    const long long m = (g.M + tile - 1) / tile + (g.grouped ? std::min(g.E, g.M) / 2 : 0);
    return (double)((m * ((g.N + tile - 1) / tile) + kNominalCUs - 1) / kNominalCUs);
  };
  const double large = rounds(256) * (3. + steps) + 5., small = rounds(128) * (1.5 + steps * (g.K % 128 != 0 ? 0.45 : 0.36));
  // words of exponents within 32-bit offsets
  const bool near = std::max<long long>(g.M, (long long)g.E * g.N) * ((g.K + 127) / 128) < (1 << 29);
  p.tile = near && large < small ? 256 : 128;
  p.nm = (int)chunks(g, p.tile);
  p.nn = (g.N + p.tile - 1) / p.tile;
  // a step takes 0.28 us (us, whole / parts: 300 x 1024 x 16384 40.7 / 17.2, 1000 x 512 x 8192 23.2 / 17.5; 1024 x 1024 x
  // 4096 14.8 / 18.1)
  if (p.tile == 128) split(steps, 16, 40);
  return p;
}

size_t words_bytes(const MxArgs& g) { return ((size_t)g.M + (size_t)g.E * g.N) * ((g.K + 127) / 128) * 4; }

template <int OUT>
hipError_t run(MxArgs& g, const Plan& p, hipStream_t stream) {
  if (OUT != OUT_PARTS && p.parts > 1) {
    MxArgs to = g;
    to.y = (void*)g.ta;
    const hipError_t e = run<OUT_PARTS>(to, p, stream);
    if (e != hipSuccess) return e;
    LaunchTimer timer("mx_parts", stream);
    const size_t n = (size_t)g.M * g.N;
    if (n % 4 == 0)
      hipLaunchKernelGGL((mx_parts_kernel<4, OUT>), dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream,
                         (const float*)to.y, p.parts, n, g.y);
    else
      hipLaunchKernelGGL((mx_parts_kernel<1, OUT>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream,
                         (const float*)to.y, p.parts, n, g.y);
    return hipGetLastError();
  }
  if (p.tile == 0) {
    // Waves of a workgroup: the fewer the more workgroups there are (us, two / four / eight, in turn on one card: 64
    // tokens, 6 of 64 experts, 2816 x 2048, 15488 of them, 39.9 / 39.7 / 48.5, 2048 x 1408 24.3 / 24.7 / 30.5; one row of
    // N = 11008, K = 2048 6.2 / 6.2 / 6.9, of N = K = 8192 12.6 / 8.5 / 7.0)
    const long long wgs = (long long)p.nn * p.nm;
    auto launch = [&](const char* name, auto* kernel, int waves) {
      LaunchTimer timer(name, stream);
      hipLaunchKernelGGL(kernel, dim3(p.nn, p.nm, p.parts), dim3(waves * 64), 0, stream, g);
      return hipGetLastError();
    };
    if constexpr (OUT != OUT_PARTS) {  // (in parts they are fewer than CUs)
      if (p.few == 16) {
        if (wgs >= 16 * kNominalCUs) return launch("mx_rows_2_16", mx_rows_kernel<2, 1, OUT>, 2);
        if (wgs > 2 * kNominalCUs) return launch("mx_rows_4_16", mx_rows_kernel<4, 1, OUT>, 4);
      } else if (wgs > kNominalCUs) {
        return launch("mx_rows_4_64", mx_rows_kernel<4, 4, OUT>, 4);
      }
    }
    if (p.few == 16) return launch("mx_rows_8_16", mx_rows_kernel<8, 1, OUT>, 8);
    return launch("mx_rows_8_64", mx_rows_kernel<8, 4, OUT>, 8);
  }
  if constexpr (OUT != OUT_PARTS) if (p.tile == 256) {
    const int KS = g.K / 32, pieces = ((g.K + 127) / 128 + 4 * kWordLoads - 1) / (4 * kWordLoads);
    const WordsSide a{g.sa, g.rows, (uint32_t*)g.ta, g.M, g.a_rows}, b{g.sb, nullptr, (uint32_t*)g.tb, g.E * g.N, g.E * g.N};
    const unsigned na = (unsigned)((a.rows + 255) / 256) * pieces, nb = (unsigned)((b.rows + 255) / 256) * pieces;
    LaunchTimer timer("mx_words", stream);
    hipLaunchKernelGGL(mx_words_kernel, dim3(na + nb), dim3(256), 0, stream, a, b, na, KS);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  LaunchTimer timer(p.tile == 256 ? "mx_tile_256" : "mx_tile_128", stream);
  // as many workgroups as the LDS of the CUs holds at once: one, or two of the smaller tile
  if constexpr (OUT != OUT_PARTS) {
    if (p.tile == 256) {
      hipLaunchKernelGGL((mx_tile_kernel<256, 256, OUT>), dim3(std::min(p.nm * p.nn, compute_units())),
                         dim3(Tile<256, 256>::NTH), 0, stream, g);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((mx_tile_kernel<128, 128, OUT>), dim3(std::min(p.nm * p.nn * p.parts, 2 * compute_units())),
                     dim3(Tile<128, 128>::NTH), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

static MxArgs args_of(const MxMatmul& c) {
  MxArgs g{};
  g.a = (const uint8_t*)c.a;
  g.b = (const uint8_t*)c.b;
  g.sa = (const uint8_t*)c.sa;
  g.sb = (const uint8_t*)c.sb;
  g.offsets = c.offsets;
  g.rows = c.rows;
  g.y = c.y;
  g.a_rows = c.a_rows;
  g.M = c.M;
  g.N = c.N;
  g.K = c.K;
  g.E = c.E;
  g.grouped = c.grouped;
  return g;
}

size_t mx_matmul_workspace_bytes(const MxMatmul& c) {
  const MxArgs g = args_of(c);
  if (c.M <= 0 || c.N <= 0) return 0;
  const Plan p = plan(g);
  return p.tile == 256 ? words_bytes(g) : p.parts > 1 ? (size_t)p.parts * c.M * c.N * 4 : 0;
}

hipError_t launch_mx_matmul(const MxMatmul& c, hipStream_t stream) {
  MxArgs g = args_of(c);
  const Plan p = plan(g);
  g.nm = p.nm;
  g.nn = p.nn;
  g.parts = p.parts;
  g.per_part = p.per_part;
  g.ta = (const uint32_t*)c.workspace;
  g.tb = g.ta + (size_t)g.M * ((g.K + 127) / 128);
  return c.out_dtype == 1 ? run<OUT_BF16>(g, p, stream) : run<OUT_F32>(g, p, stream);
}

}  // namespace esg
