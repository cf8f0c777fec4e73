// The C ABI (include/esg.h): argument validation, workspace layout and the
// launch sequence of each entry point.  No device memory is allocated here.
#include "esg.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "esg_internal.hpp"

namespace esg {
void subsample_index(int d_ff, int group_size, int spg, uint64_t seed, int32_t* out);
void timing_set(bool on);
void timing_reset();
int timing_read(const char* name, double* total_ms, int* launches);
}  // namespace esg

using namespace esg;

namespace {

constexpr int kMaxGroups = 1024;
constexpr int kMaxK = 128;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }

// Shape rules of the eugen_sparse README ("Parameters and how to choose
// them"): group_size a power of two >= 16; d_ff a multiple of it with at
// least two groups; d_model a multiple of 16; 1 <= k <= G; tokens*k < 2^31.
int check_shape(int dtype, int tokens, int d_model, int d_ff, int group_size, int k) {
  if (dtype != ESG_F32 && dtype != ESG_BF16) return ESG_ERR_UNSUPPORTED;
  if (tokens < 0 || d_model <= 0 || d_ff <= 0 || group_size <= 0 || k <= 0) return ESG_ERR_INVALID_ARG;
  if (!pow2(group_size) || group_size < 16) return ESG_ERR_UNSUPPORTED;
  if (d_ff % group_size != 0 || d_ff / group_size < 2) return ESG_ERR_UNSUPPORTED;
  if (d_model % 16 != 0) return ESG_ERR_UNSUPPORTED;
  const int groups = d_ff / group_size;
  if (groups > kMaxGroups || k > groups) return ESG_ERR_UNSUPPORTED;
  if ((long long)tokens * k >= (1ll << 31)) return ESG_ERR_UNSUPPORTED;
  return ESG_OK;
}

int hip_status(hipError_t e) { return e == hipSuccess ? ESG_OK : ESG_ERR_HIP; }

struct Layout {
  int mt = 0;            // maximum tiles
  size_t rows = 0;       // padded positions
  size_t offsets = 0, tile_off = 0, tile_group = 0, ptoken = 0, pinv = 0, hg = 0, hu = 0, saved = 0;
  size_t f_bucket = 0, f_part = 0, f_route = 0, f_act = 0, fwd = 0;
  size_t b_dg = 0, b_du = 0, b_act = 0, b_part = 0, b_slots = 0, bwd = 0;
  int cht = 0;           // weight-gradient chunk tiles (dw_chunk_tiles)
};

// train: the layout of a forward that saves for the backward, whose groups are
// padded to tile_pad(s) positions; an inference forward pads to whole tiles only
Layout make_layout(const FfnShape& s, bool train = true) {
  Layout L;
  const int G = s.groups();
  L.mt = max_tiles(s.tokens, s.k, G, kTileRows, train ? tile_pad(s) : kTileRows);
  L.rows = (size_t)L.mt * kTileRows;
  const size_t es = s.elem_bytes();
  const size_t act_bytes = (size_t)s.nsub() * L.rows * s.gsb() * es;
  const size_t part_bytes = (size_t)s.nsub() * L.rows * s.d_model * es;
  size_t o = 0;
  L.offsets = o;    o = align256(o + (size_t)(G + 1) * 4);
  L.tile_off = o;   o = align256(o + (size_t)(G + 1) * 4);
  L.tile_group = o; o = align256(o + (size_t)L.mt * 4);
  L.ptoken = o;     o = align256(o + L.rows * 4);
  L.pinv = o;       o = align256(o + (size_t)s.tokens * s.k * 4);
  L.hg = o;         o = align256(o + act_bytes);
  L.hu = o;         o = align256(o + act_bytes);
  L.saved = o;
  o = 0;
  L.f_bucket = o;   o = align256(o + bucket_scratch_bytes(s.tokens, G));
  L.f_part = o;     o = align256(o + part_bytes);
  L.f_route = o;    o = align256(o + L.hg);  // the routing arrays of `saved`, for saved = NULL (inference)
  L.f_act = o;      o = align256(o + fwd_split_bytes(s, L.mt));  // [hg; hu] partials of a split forward
  L.fwd = o;
  o = 0;
  L.b_dg = o;       o = align256(o + act_bytes);
  L.b_du = o;       o = align256(o + act_bytes);
  L.b_act = o;      o = align256(o + act_bytes);
  L.b_part = o;     o = align256(o + part_bytes);
  L.cht = train ? dw_chunk_tiles(s, L.mt, tile_pad(s)) : 0;
  L.b_slots = o;    o = align256(o + dw_slot_bytes(s, L.rows, L.cht));
  L.bwd = o;
  return L;
}

template <typename P>
P* at(void* base, size_t off) {
  return (P*)((char*)base + off);
}
template <typename P>
const P* at(const void* base, size_t off) {
  return (const P*)((const char*)base + off);
}

hipError_t zero_bytes(void* p, size_t bytes, hipStream_t st) {
  return launch_fill_i32((int32_t*)p, 0, bytes / 4, st);
}

}  // namespace

size_t esg::inference_fwd_scratch_bytes(const FfnShape& s) { return make_layout(s, false).fwd; }

extern "C" {

const char* esg_status_string(int status) {
  switch (status) {
    case ESG_OK: return "ok";
    case ESG_ERR_INVALID_ARG: return "invalid argument";
    case ESG_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case ESG_ERR_WORKSPACE: return "workspace too small";
    case ESG_ERR_HIP: return "HIP runtime error";
    default: return "unknown status";
  }
}

int esg_version(void) { return 10000; }

int esg_make_subsample_index(int d_ff, int group_size, int samples_per_group, uint64_t seed, int32_t* out) {
  if (out == nullptr) return ESG_ERR_INVALID_ARG;
  if (!pow2(group_size) || group_size < 16 || d_ff <= 0 || d_ff % group_size != 0 || d_ff / group_size < 2)
    return ESG_ERR_UNSUPPORTED;
  if (samples_per_group < 1 || samples_per_group > group_size) return ESG_ERR_UNSUPPORTED;
  subsample_index(d_ff, group_size, samples_per_group, seed, out);
  return ESG_OK;
}

int esg_grouped_topk_select_ws(const void* x, const void* w_gate, int dtype, int tokens, int d_model, int d_ff,
                               int group_size, int k, const int32_t* sub, int samples_per_group, const float* bias,
                               int32_t* idx_out, int32_t* counts_out, void* workspace, size_t workspace_bytes,
                               void* stream) {
  int st = check_shape(dtype, tokens, d_model, d_ff, group_size, k);
  if (st != ESG_OK) return st;
  if ((tokens > 0 && (x == nullptr || idx_out == nullptr)) || w_gate == nullptr) return ESG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_gate) || !aligned16(workspace)) return ESG_ERR_INVALID_ARG;
  int rpg = group_size;
  if (sub != nullptr) {
    if (samples_per_group < 1 || samples_per_group > group_size) return ESG_ERR_UNSUPPORTED;
    rpg = samples_per_group;
  }
  const int groups = d_ff / group_size;
  float* ews = workspace != nullptr && workspace_bytes >= select_energy_bytes(tokens, groups) ? (float*)workspace
                                                                                             : nullptr;
  return hip_status(launch_select(dtype, x, w_gate, tokens, d_model, groups, k, sub, rpg, group_size, bias,
                                  idx_out, counts_out, ews, (hipStream_t)stream));
}

int esg_grouped_topk_select(const void* x, const void* w_gate, int dtype, int tokens, int d_model, int d_ff,
                            int group_size, int k, const int32_t* sub, int samples_per_group, const float* bias,
                            int32_t* idx_out, int32_t* counts_out, void* stream) {
  return esg_grouped_topk_select_ws(x, w_gate, dtype, tokens, d_model, d_ff, group_size, k, sub, samples_per_group,
                                    bias, idx_out, counts_out, nullptr, 0, stream);
}

int esg_grouped_topk_select_workspace_size(int tokens, int d_ff, int group_size, size_t* workspace_bytes) {
  if (workspace_bytes == nullptr || tokens < 0 || d_ff <= 0 || group_size <= 0 || d_ff % group_size != 0)
    return ESG_ERR_INVALID_ARG;
  *workspace_bytes = select_energy_bytes(tokens, d_ff / group_size);
  return ESG_OK;
}

int esg_bucket_workspace_size(int tokens, int k, int groups, size_t* scratch_bytes) {
  if (scratch_bytes == nullptr || tokens < 0 || k <= 0 || groups <= 0) return ESG_ERR_INVALID_ARG;
  if (groups > kMaxGroups || k > kMaxK || (long long)tokens * k >= (1ll << 31)) return ESG_ERR_UNSUPPORTED;
  *scratch_bytes = bucket_scratch_bytes(tokens, groups);
  return ESG_OK;
}

int esg_bucket_by_group(const int32_t* idx, int tokens, int k, int groups, int32_t* offsets, int32_t* perm_token,
                        int32_t* inv, int32_t* status_dev, void* scratch, size_t scratch_bytes, void* stream) {
  size_t need = 0;
  int st = esg_bucket_workspace_size(tokens, k, groups, &need);
  if (st != ESG_OK) return st;
  if (offsets == nullptr || scratch == nullptr || (tokens > 0 && (idx == nullptr || perm_token == nullptr ||
                                                                  inv == nullptr)))
    return ESG_ERR_INVALID_ARG;
  if (scratch_bytes < need) return ESG_ERR_WORKSPACE;
  BucketOut out{offsets, perm_token, inv, nullptr, nullptr, nullptr, nullptr, status_dev};
  return hip_status(launch_bucket(idx, tokens, k, groups, kTileRows, out, scratch, (hipStream_t)stream));
}

int esg_sparse_swiglu_workspace_size(int tokens, int d_model, int d_ff, int group_size, int k, int dtype, int dense,
                                     size_t* saved_bytes, size_t* fwd_scratch_bytes, size_t* bwd_scratch_bytes) {
  int st = check_shape(dtype, tokens, d_model, d_ff, group_size, k);
  if (st != ESG_OK) return st;
  if (dense) {
    const FfnShape s{dtype, tokens, d_model, d_ff, group_size, k};
    if (k != s.groups()) return ESG_ERR_INVALID_ARG;
    if (!dense_supported(s)) return ESG_ERR_UNSUPPORTED;
    if (saved_bytes) *saved_bytes = 0;
    if (fwd_scratch_bytes) *fwd_scratch_bytes = 0;
    if (bwd_scratch_bytes) *bwd_scratch_bytes = dense_bwd_layout(tokens, d_model, d_ff).bytes;
    return ESG_OK;
  }
  if (k > kMaxK) return ESG_ERR_UNSUPPORTED;
  const Layout L = make_layout(FfnShape{dtype, tokens, d_model, d_ff, group_size, k});
  if (saved_bytes) *saved_bytes = L.saved;
  if (fwd_scratch_bytes) *fwd_scratch_bytes = L.fwd;
  if (bwd_scratch_bytes) *bwd_scratch_bytes = L.bwd;
  return ESG_OK;
}

int esg_sparse_swiglu_fwd(const void* x, const void* w_gate, const void* w_up, const void* w_down, int dtype,
                          int tokens, int d_model, int d_ff, int group_size, int k, const int32_t* idx, void* y,
                          void* saved, size_t saved_bytes, void* scratch, size_t scratch_bytes, int32_t* status_dev,
                          void* stream) {
  int st = check_shape(dtype, tokens, d_model, d_ff, group_size, k);
  if (st != ESG_OK) return st;
  if (w_gate == nullptr || w_up == nullptr || w_down == nullptr) return ESG_ERR_INVALID_ARG;
  if (tokens == 0) return ESG_OK;  // nothing to route or compute (an empty idx may be NULL)
  if (idx == nullptr) {            // dense limit: every group active, nothing saved
    const FfnShape s{dtype, tokens, d_model, d_ff, group_size, k};
    if (k != s.groups()) return ESG_ERR_INVALID_ARG;
    if (!dense_supported(s)) return ESG_ERR_UNSUPPORTED;
    if (x == nullptr || y == nullptr) return ESG_ERR_INVALID_ARG;
    for (const void* p : {x, w_gate, w_up, w_down, (const void*)y})
      if (!aligned16(p)) return ESG_ERR_INVALID_ARG;
    return hip_status(launch_dense_fwd(s, x, w_gate, w_up, w_down, y, (hipStream_t)stream));
  }
  if (scratch == nullptr) return ESG_ERR_INVALID_ARG;
  if (k > kMaxK) return ESG_ERR_UNSUPPORTED;
  if (tokens > 0 && (x == nullptr || y == nullptr)) return ESG_ERR_INVALID_ARG;
  for (const void* p : {x, w_gate, w_up, w_down, (const void*)y, (const void*)idx, (const void*)saved,
                        (const void*)scratch})
    if (!aligned16(p)) return ESG_ERR_INVALID_ARG;
  const FfnShape s{dtype, tokens, d_model, d_ff, group_size, k};
  const bool train = saved != nullptr;  // NULL: forward only, the routing lives in the scratch
  const Layout L = make_layout(s, train);
  if ((train && saved_bytes < L.saved) || scratch_bytes < L.fwd) return ESG_ERR_WORKSPACE;
  void* route = train ? saved : at<char>(scratch, L.f_route);
  hipStream_t stream_h = (hipStream_t)stream;
  BucketOut out{at<int32_t>(route, L.offsets), nullptr, nullptr, at<int32_t>(route, L.tile_off),
                at<int32_t>(route, L.tile_group), at<int32_t>(route, L.ptoken), at<int32_t>(route, L.pinv),
                status_dev};
  const int pad = train ? tile_pad(s) : kTileRows;
  hipError_t e = launch_bucket(idx, tokens, k, s.groups(), kTileRows, out, at<char>(scratch, L.f_bucket), stream_h,
                               pad);
  if (e != hipSuccess) return ESG_ERR_HIP;
  char* hg = train ? at<char>(saved, L.hg) : nullptr;
  char* hu = train ? at<char>(saved, L.hu) : nullptr;
  e = bf16_pipelined(s, L.mt)
          ? launch_fwd2(s, x, w_gate, w_up, w_down, out.tile_group, out.ptoken, L.mt, pad, hg, hu,
                        at<char>(scratch, L.f_part), at<char>(scratch, L.f_act), stream_h)
          : launch_fwd_grouped(s, x, w_gate, w_up, w_down, out.tile_group, out.ptoken, L.mt, hg, hu,
                               at<char>(scratch, L.f_part), stream_h);
  if (e != hipSuccess) return ESG_ERR_HIP;
  e = launch_rowsum(s, at<char>(scratch, L.f_part), L.rows, out.pinv, y, stream_h);
  return hip_status(e);
}

int esg_sparse_swiglu_bwd(const void* dy, const void* x, const void* w_gate, const void* w_up, const void* w_down,
                          int dtype, int tokens, int d_model, int d_ff, int group_size, int k, const int32_t* idx,
                          const void* saved, size_t saved_bytes, void* dx, void* dw_gate, void* dw_up,
                          void* dw_down, void* scratch, size_t scratch_bytes, void* stream) {
  return esg_sparse_swiglu_bwd_overlap(dy, x, w_gate, w_up, w_down, dtype, tokens, d_model, d_ff, group_size, k, idx,
                                       saved, saved_bytes, dx, dw_gate, dw_up, dw_down, scratch, scratch_bytes, stream,
                                       nullptr);
}

int esg_sparse_swiglu_bwd_overlap(const void* dy, const void* x, const void* w_gate, const void* w_up,
                                  const void* w_down, int dtype, int tokens, int d_model, int d_ff, int group_size,
                                  int k, const int32_t* idx, const void* saved, size_t saved_bytes, void* dx,
                                  void* dw_gate, void* dw_up, void* dw_down, void* scratch, size_t scratch_bytes,
                                  void* stream, void* aux_stream) {
  int st = check_shape(dtype, tokens, d_model, d_ff, group_size, k);
  if (st != ESG_OK) return st;
  if (w_gate == nullptr || w_up == nullptr || w_down == nullptr || scratch == nullptr || dw_gate == nullptr ||
      dw_up == nullptr || dw_down == nullptr)
    return ESG_ERR_INVALID_ARG;
  if (tokens == 0) {  // no token: every weight gradient is zero (an empty idx may be NULL)
    hipStream_t stream_h = (hipStream_t)stream;
    const size_t wbytes = (size_t)d_ff * d_model * (dtype == ESG_BF16 ? 2 : 4);
    hipError_t e = zero_bytes(dw_gate, wbytes, stream_h);
    if (e == hipSuccess) e = zero_bytes(dw_up, wbytes, stream_h);
    if (e == hipSuccess) e = zero_bytes(dw_down, wbytes, stream_h);
    return hip_status(e);
  }
  if (idx == nullptr) {  // dense limit: gate/up recomputed, nothing saved
    const FfnShape s{dtype, tokens, d_model, d_ff, group_size, k};
    if (k != s.groups()) return ESG_ERR_INVALID_ARG;
    if (!dense_supported(s)) return ESG_ERR_UNSUPPORTED;
    hipStream_t stream_h = (hipStream_t)stream;
    if (x == nullptr || dy == nullptr || dx == nullptr) return ESG_ERR_INVALID_ARG;
    for (const void* p : {dy, x, w_gate, w_up, w_down, (const void*)dx, (const void*)dw_gate, (const void*)dw_up,
                          (const void*)dw_down, (const void*)scratch})
      if (!aligned16(p)) return ESG_ERR_INVALID_ARG;
    if (scratch_bytes < dense_bwd_layout(tokens, d_model, d_ff).bytes) return ESG_ERR_WORKSPACE;
    return hip_status(
        launch_dense_bwd(s, dy, x, w_gate, w_up, w_down, dx, dw_gate, dw_up, dw_down, scratch, stream_h));
  }
  if (saved == nullptr) return ESG_ERR_INVALID_ARG;
  if (k > kMaxK) return ESG_ERR_UNSUPPORTED;
  if (tokens > 0 && (x == nullptr || dy == nullptr || dx == nullptr)) return ESG_ERR_INVALID_ARG;
  for (const void* p : {dy, x, w_gate, w_up, w_down, saved, (const void*)dx, (const void*)dw_gate,
                        (const void*)dw_up, (const void*)dw_down, (const void*)scratch})
    if (!aligned16(p)) return ESG_ERR_INVALID_ARG;
  const FfnShape s{dtype, tokens, d_model, d_ff, group_size, k};
  const Layout L = make_layout(s);
  if (saved_bytes < L.saved || scratch_bytes < L.bwd) return ESG_ERR_WORKSPACE;
  hipStream_t stream_h = (hipStream_t)stream;
  const int32_t* tile_group = at<int32_t>(saved, L.tile_group);
  const int32_t* tile_off = at<int32_t>(saved, L.tile_off);
  const int32_t* ptoken = at<int32_t>(saved, L.ptoken);
  const int32_t* pinv = at<int32_t>(saved, L.pinv);
  const bool v2 = bf16_pipelined(s, L.mt);
  hipError_t e = v2 ? launch_dhdx2(s, dy, w_gate, w_up, w_down, tile_group, ptoken, L.mt, at<char>(saved, L.hg),
                                   at<char>(saved, L.hu), at<char>(scratch, L.b_dg), at<char>(scratch, L.b_du),
                                   at<char>(scratch, L.b_act), at<char>(scratch, L.b_part), stream_h)
                    : launch_bwd_dh_dx(s, dy, w_gate, w_up, w_down, tile_group, ptoken, L.mt, at<char>(saved, L.hg),
                                       at<char>(saved, L.hu), at<char>(scratch, L.b_dg), at<char>(scratch, L.b_du),
                                       at<char>(scratch, L.b_act), at<char>(scratch, L.b_part), stream_h);
  if (e != hipSuccess) return ESG_ERR_HIP;
  // The slot-order sum of dx and the weight gradients only read what dh+dx
  // wrote.  With a caller-supplied second stream the weight gradients run on
  // it beside the sum (forked after dh+dx, joined back into `stream` by two
  // events created and destroyed in this call); else one after the other.
  hipStream_t aux = (hipStream_t)aux_stream;
  hipEvent_t forked = nullptr, done = nullptr;
  if (aux != nullptr && aux != stream_h) {
    if (hipEventCreateWithFlags(&forked, hipEventDisableTiming) != hipSuccess) return ESG_ERR_HIP;
    if (hipEventCreateWithFlags(&done, hipEventDisableTiming) != hipSuccess) {
      (void)hipEventDestroy(forked);
      return ESG_ERR_HIP;
    }
    e = hipEventRecord(forked, stream_h);
    if (e == hipSuccess) e = hipStreamWaitEvent(aux, forked, 0);
  } else {
    aux = stream_h;
  }
  if (e == hipSuccess)
    e = v2 ? launch_dw2(s, x, dy, tile_off, ptoken, (int)L.rows, at<char>(scratch, L.b_dg),
                        at<char>(scratch, L.b_du), at<char>(scratch, L.b_act), dw_gate, dw_up, dw_down, L.cht,
                        at<char>(scratch, L.b_slots), aux)
           : launch_bwd_dw(s, x, dy, tile_off, ptoken, (int)L.rows, at<char>(scratch, L.b_dg),
                           at<char>(scratch, L.b_du), at<char>(scratch, L.b_act), dw_gate, dw_up, dw_down, aux);
  if (e == hipSuccess) e = launch_rowsum(s, at<char>(scratch, L.b_part), L.rows, pinv, dx, stream_h);
  if (forked != nullptr) {
    if (e == hipSuccess) e = hipEventRecord(done, aux);
    if (e == hipSuccess) e = hipStreamWaitEvent(stream_h, done, 0);
    (void)hipEventDestroy(forked);
    (void)hipEventDestroy(done);
  }
  return hip_status(e);
}

int esg_update_load_balance_bias(float* bias, float* freq_ema, const float* current_freq, float target_freq,
                                 float gamma, float bias_max, float momentum, int groups, void* stream) {
  if (bias == nullptr || freq_ema == nullptr || current_freq == nullptr || groups < 0) return ESG_ERR_INVALID_ARG;
  return hip_status(launch_bias_update(bias, freq_ema, current_freq, nullptr, nullptr, 1, target_freq, gamma,
                                       bias_max, momentum, groups, (hipStream_t)stream));
}

int esg_update_load_balance_bias_from_counts(float* bias, float* freq_ema, const int32_t* counts, int tokens,
                                             float target_freq, float gamma, float bias_max, float momentum,
                                             int groups, void* stream) {
  if (bias == nullptr || freq_ema == nullptr || counts == nullptr || groups < 0 || tokens <= 0)
    return ESG_ERR_INVALID_ARG;
  return hip_status(launch_bias_update(bias, freq_ema, nullptr, counts, nullptr, tokens, target_freq, gamma,
                                       bias_max, momentum, groups, (hipStream_t)stream));
}

int esg_update_load_balance_bias_from_routing(float* bias, float* freq_ema, const void* saved, size_t saved_bytes,
                                              int tokens, int d_model, int d_ff, int group_size, int k, int dtype,
                                              float target_freq, float gamma, float bias_max, float momentum,
                                              void* stream) {
  int st = check_shape(dtype, tokens, d_model, d_ff, group_size, k);
  if (st != ESG_OK) return st;
  if (bias == nullptr || freq_ema == nullptr || saved == nullptr || tokens <= 0) return ESG_ERR_INVALID_ARG;
  if (k > kMaxK) return ESG_ERR_UNSUPPORTED;
  const FfnShape s{dtype, tokens, d_model, d_ff, group_size, k};
  const Layout L = make_layout(s);
  if (saved_bytes < L.saved) return ESG_ERR_WORKSPACE;
  return hip_status(launch_bias_update(bias, freq_ema, nullptr, nullptr, at<int32_t>(saved, L.offsets), tokens,
                                       target_freq, gamma, bias_max, momentum, s.groups(), (hipStream_t)stream));
}

namespace {
int mlp_shape(int tokens, int d_model, int d_ff) {
  if (tokens < 0 || d_model <= 0 || d_ff <= 0) return ESG_ERR_INVALID_ARG;
  if (d_model % 8 || d_ff % 8) return ESG_ERR_UNSUPPORTED;
  const long long wide = d_model > d_ff ? d_model : d_ff;
  if ((long long)tokens * wide * 2 >= (1ll << 31) || (long long)d_model * d_ff * 2 >= (1ll << 31))
    return ESG_ERR_UNSUPPORTED;
  return ESG_OK;
}
}  // namespace

int esg_leaky_mlp_workspace_size(int tokens, int d_model, int d_ff, size_t* saved_bytes, size_t* scratch_bytes) {
  if (saved_bytes == nullptr || scratch_bytes == nullptr) return ESG_ERR_INVALID_ARG;
  const int e = mlp_shape(tokens, d_model, d_ff);
  if (e != ESG_OK) return e;
  const size_t tf = (size_t)tokens * d_ff * 2;
  *saved_bytes = 2 * align256(tf);
  *scratch_bytes = align256(tf) + align256(mlp_partial_bytes(tokens, d_model, d_ff));
  return ESG_OK;
}

int esg_leaky_mlp_fwd(const void* x, const void* w_up, const void* w_down, int tokens, int d_model, int d_ff,
                      void* y, void* saved, size_t saved_bytes, void* stream) {
  size_t need_saved, need_scratch;
  int e = esg_leaky_mlp_workspace_size(tokens, d_model, d_ff, &need_saved, &need_scratch);
  if (e != ESG_OK) return e;
  if (tokens == 0) return ESG_OK;
  if (x == nullptr || w_up == nullptr || w_down == nullptr || y == nullptr || saved == nullptr)
    return ESG_ERR_INVALID_ARG;
  if (saved_bytes < need_saved) return ESG_ERR_WORKSPACE;
  void* post = saved;
  void* act = (char*)saved + align256((size_t)tokens * d_ff * 2);
  return hip_status(launch_mlp_fwd(x, w_up, w_down, tokens, d_model, d_ff, y, post, act, (hipStream_t)stream));
}

int esg_leaky_mlp_bwd(const void* dy, const void* x, const void* w_up, const void* w_down, int tokens, int d_model,
                      int d_ff, const void* saved, void* dx, void* dw_up, void* dw_down, void* scratch,
                      size_t scratch_bytes, void* stream) {
  size_t need_saved, need_scratch;
  int e = esg_leaky_mlp_workspace_size(tokens, d_model, d_ff, &need_saved, &need_scratch);
  if (e != ESG_OK) return e;
  if (w_up == nullptr || w_down == nullptr || dw_up == nullptr || dw_down == nullptr) return ESG_ERR_INVALID_ARG;
  if (tokens > 0 && (dy == nullptr || x == nullptr || saved == nullptr || dx == nullptr || scratch == nullptr))
    return ESG_ERR_INVALID_ARG;
  if (tokens > 0 && scratch_bytes < need_scratch) return ESG_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  if (tokens == 0) {  // no tokens: the weight gradients are zero
    e = hip_status(launch_fill_i32((int32_t*)dw_up, 0, (size_t)d_ff * d_model / 2, st));
    if (e != ESG_OK) return e;
    return hip_status(launch_fill_i32((int32_t*)dw_down, 0, (size_t)d_ff * d_model / 2, st));
  }
  const size_t tf = align256((size_t)tokens * d_ff * 2);
  const void* post = saved;
  const void* act = (const char*)saved + tf;
  void* dpre = scratch;
  float* part = (float*)((char*)scratch + tf);
  return hip_status(launch_mlp_bwd(dy, x, w_up, w_down, tokens, d_model, d_ff, post, act, dx, dw_up, dw_down, dpre,
                                   part, st));
}

int esg_mhffn_supported(int tokens, int heads, int d_head, int subnets, int d_sub) {
  return mhffn_supported(tokens, heads, d_head, subnets, d_sub) ? 1 : 0;
}

int esg_mhffn_fwd(const void* q, const float* r, const void* k, const void* u, const void* v, int tokens, int heads,
                  int d_head, int subnets, int d_sub, void* out, void* stream) {
  if (tokens < 0 || heads <= 0 || subnets <= 0 || d_sub <= 0) return ESG_ERR_INVALID_ARG;
  if (!mhffn_supported(tokens, heads, d_head, subnets, d_sub)) return ESG_ERR_UNSUPPORTED;
  if (tokens == 0) return ESG_OK;
  for (const void* p : {q, (const void*)r, k, u, v, (const void*)out})
    if (p == nullptr || !aligned16(p)) return ESG_ERR_INVALID_ARG;
  return hip_status(launch_mhffn_fwd(q, r, k, u, v, tokens, heads, subnets, d_sub, out, (hipStream_t)stream));
}

int esg_mhffn_bwd(const void* dout, const void* q, const float* r, const void* k, const void* u, const void* v,
                  int tokens, int heads, int d_head, int subnets, int d_sub, void* dq, float* dr, void* dk, void* du,
                  void* dv, void* stream) {
  if (tokens < 0 || heads <= 0 || subnets <= 0 || d_sub <= 0) return ESG_ERR_INVALID_ARG;
  if (!mhffn_supported(tokens, heads, d_head, subnets, d_sub)) return ESG_ERR_UNSUPPORTED;
  for (const void* p : {k, u, v, (const void*)dk, (const void*)du, (const void*)dv})
    if (p == nullptr || !aligned16(p)) return ESG_ERR_INVALID_ARG;
  if (tokens > 0)
    for (const void* p : {dout, q, (const void*)r, (const void*)dq, (const void*)dr})
      if (p == nullptr || !aligned16(p)) return ESG_ERR_INVALID_ARG;
  return hip_status(launch_mhffn_bwd(dout, q, r, k, u, v, tokens, heads, subnets, d_sub, dq, dr, dk, du, dv,
                                     (hipStream_t)stream));
}

int esg_sigmoid_topk_supported(int num_experts, int topk) { return sigmoid_topk_supported(num_experts, topk) ? 1 : 0; }

int esg_sigmoid_topk_routing(const float* logits, const float* expert_bias, int bias_stride, int tokens,
                             int num_experts, int topk, float scaling_factor, int apply_scaling, float* probs,
                             int64_t* indices, void* stream) {
  if (tokens < 0 || bias_stride < 1) return ESG_ERR_INVALID_ARG;
  if (!sigmoid_topk_supported(num_experts, topk)) return ESG_ERR_UNSUPPORTED;
  if ((size_t)tokens * topk >= (1ull << 31) || (size_t)tokens * num_experts >= (1ull << 40))
    return ESG_ERR_UNSUPPORTED;
  if (tokens == 0) return ESG_OK;
  if (logits == nullptr || expert_bias == nullptr || probs == nullptr || indices == nullptr)
    return ESG_ERR_INVALID_ARG;
  return hip_status(launch_sigmoid_topk(logits, expert_bias, bias_stride, tokens, num_experts, topk, scaling_factor,
                                        apply_scaling, probs, indices, (hipStream_t)stream));
}

namespace {
// rows of cols elements quantised in blocks of 128: cols a multiple of 16, and
// the launch's threads (256 per 128 x 128 tile at most) within 2^32
int quant_shape(int dtype, int batch, int rows, int cols) {
  if (dtype != ESG_F32 && dtype != ESG_BF16) return ESG_ERR_UNSUPPORTED;
  if (batch < 0 || rows < 0 || cols <= 0) return ESG_ERR_INVALID_ARG;
  if (cols % 16 || rows > (1 << 30) || cols > (1 << 22)) return ESG_ERR_UNSUPPORTED;
  const double tiles = (double)batch * ((rows + 127) / 128) * ((cols + 127) / 128);
  return tiles < 16777216.0 ? ESG_OK : ESG_ERR_UNSUPPORTED;
}
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
}  // namespace

int esg_fp8_quant_rows(const void* x, int dtype, int rows, int cols, void* q, float* scale, void* qt, float* scale_t,
                       void* stream) {
  const int e = quant_shape(dtype, 1, rows, cols);
  if (e != ESG_OK) return e;
  if (rows == 0) return ESG_OK;
  if ((qt == nullptr) != (scale_t == nullptr)) return ESG_ERR_INVALID_ARG;
  for (const void* p : {x, (const void*)q, (const void*)(qt ? qt : q)})
    if (p == nullptr || !aligned16(p)) return ESG_ERR_INVALID_ARG;
  if (scale == nullptr || !aligned4(scale) || !aligned4(scale_t)) return ESG_ERR_INVALID_ARG;
  return hip_status(launch_quant_rows(dtype, x, rows, cols, q, scale, qt, scale_t, (hipStream_t)stream));
}

int esg_fp8_quant_tiles(const void* w, int dtype, int batch, int rows, int cols, void* q, float* scale, void* qt,
                        float* scale_t, void* stream) {
  const int e = quant_shape(dtype, batch, rows, cols);
  if (e != ESG_OK) return e;
  if (batch == 0 || rows == 0) return ESG_OK;
  if ((qt == nullptr) != (scale_t == nullptr)) return ESG_ERR_INVALID_ARG;
  for (const void* p : {w, (const void*)q, (const void*)(qt ? qt : q)})
    if (p == nullptr || !aligned16(p)) return ESG_ERR_INVALID_ARG;
  if (scale == nullptr || !aligned4(scale) || !aligned4(scale_t)) return ESG_ERR_INVALID_ARG;
  return hip_status(launch_quant_tiles(dtype, w, batch, rows, cols, q, scale, qt, scale_t, (hipStream_t)stream));
}

namespace {
int fp8_shape(int M, int N, int K) {
  if (M < 0 || N < 0 || K <= 0) return ESG_ERR_INVALID_ARG;
  if (K % 16 || K > (1 << 22) || M > (1 << 30) || N > (1 << 25)) return ESG_ERR_UNSUPPORTED;
  // a launch's threads within 2^32: 512 per output tile of 128 x 128 at most, 512 per 16 rows of b for few rows
  return (double)((M + 127) / 128) * ((N + 127) / 128) < 8388608.0 ? ESG_OK : ESG_ERR_UNSUPPORTED;
}
}  // namespace

int esg_fp8_matmul_workspace_size(int M, int N, int K, size_t* workspace_bytes) {
  if (workspace_bytes == nullptr) return ESG_ERR_INVALID_ARG;
  const int e = fp8_shape(M, N, K);
  if (e != ESG_OK) return e;
  *workspace_bytes = fp8_matmul_workspace_bytes(M, N, K);
  return ESG_OK;
}

int esg_fp8_matmul(const void* a, const float* a_scale, const void* b, const float* b_scale, int b_scale_rows,
                   int out_dtype, int M, int N, int K, void* y, void* workspace, size_t workspace_bytes,
                   void* stream) {
  const int e = fp8_shape(M, N, K);
  if (e != ESG_OK) return e;
  if (out_dtype != ESG_F32 && out_dtype != ESG_BF16) return ESG_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return ESG_OK;
  for (const void* p : {a, b, (const void*)y})
    if (p == nullptr || !aligned16(p)) return ESG_ERR_INVALID_ARG;
  if (a_scale == nullptr || b_scale == nullptr || !aligned4(a_scale) || !aligned4(b_scale))
    return ESG_ERR_INVALID_ARG;
  const size_t need = fp8_matmul_workspace_bytes(M, N, K);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return ESG_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return ESG_ERR_INVALID_ARG;
  return hip_status(launch_fp8_matmul(a, a_scale, b, b_scale, b_scale_rows != 0, out_dtype, M, N, K, y, workspace,
                                      (hipStream_t)stream));
}

namespace {
// Buffers of the linear layer: what the backward needs (the transposes), and scratch.
struct LinearLayout {
  size_t xqt = 0, xst = 0, wqt = 0, wst = 0, saved = 0;             // saved
  size_t xq = 0, xs = 0, wq = 0, ws = 0, fmm = 0, fwd = 0;          // forward scratch
  size_t dq = 0, ds = 0, dqt = 0, dst = 0, bmm = 0, bwd = 0;        // backward scratch
};
int linear_shape(int tokens, int d_in, int d_out) {
  if (tokens < 0 || d_in <= 0 || d_out <= 0) return ESG_ERR_INVALID_ARG;
  if (d_out % 16) return ESG_ERR_UNSUPPORTED;
  int e = quant_shape(ESG_BF16, 1, tokens, d_in);
  if (e == ESG_OK) e = quant_shape(ESG_BF16, 1, tokens, d_out);
  if (e == ESG_OK) e = fp8_shape(tokens, d_out, d_in);
  if (e == ESG_OK) e = fp8_shape(tokens, d_in, d_out);
  if (e == ESG_OK && tokens > 0) e = fp8_shape(d_out, d_in, (tokens + 15) / 16 * 16);
  return e;
}
LinearLayout linear_layout(int tokens, int d_in, int d_out, int need_dx, int need_dw) {
  LinearLayout L;
  const size_t T = tokens, T16 = (T + 15) / 16 * 16, K = d_in, N = d_out;
  const size_t tb = (T + 127) / 128, kb = (K + 127) / 128, nb = (N + 127) / 128;
  auto put = [](size_t& end, size_t bytes) {
    const size_t at = end;
    end += align256(bytes);
    return at;
  };
  if (need_dw) L.xqt = put(L.saved, K * T16), L.xst = put(L.saved, K * tb * 4);
  if (need_dx) L.wqt = put(L.saved, K * N), L.wst = put(L.saved, kb * nb * 4);
  L.xq = put(L.fwd, T * K);
  L.xs = put(L.fwd, T * kb * 4);
  L.wq = put(L.fwd, N * K);
  L.ws = put(L.fwd, nb * kb * 4);
  L.fmm = put(L.fwd, fp8_matmul_workspace_bytes(tokens, d_out, d_in));
  L.dq = put(L.bwd, T * N);
  L.ds = put(L.bwd, T * nb * 4);
  if (need_dw) L.dqt = put(L.bwd, N * T16), L.dst = put(L.bwd, N * tb * 4);
  const size_t a = need_dx ? fp8_matmul_workspace_bytes(tokens, d_in, d_out) : 0;
  const size_t b = need_dw ? fp8_matmul_workspace_bytes(d_out, d_in, (int)T16) : 0;
  L.bmm = put(L.bwd, a > b ? a : b);
  return L;
}
}  // namespace

int esg_fp8_linear_workspace_size(int tokens, int d_in, int d_out, int need_dx, int need_dw, size_t* saved_bytes,
                                  size_t* fwd_scratch_bytes, size_t* bwd_scratch_bytes) {
  if (saved_bytes == nullptr || fwd_scratch_bytes == nullptr || bwd_scratch_bytes == nullptr)
    return ESG_ERR_INVALID_ARG;
  const int e = linear_shape(tokens, d_in, d_out);
  if (e != ESG_OK) return e;
  const LinearLayout L = linear_layout(tokens, d_in, d_out, need_dx, need_dw);
  *saved_bytes = L.saved;
  *fwd_scratch_bytes = L.fwd;
  *bwd_scratch_bytes = L.bwd;
  return ESG_OK;
}

int esg_fp8_linear_fwd(const void* x, int x_dtype, const void* w, int w_dtype, int tokens, int d_in, int d_out,
                       int need_dx, int need_dw, void* y, void* saved, size_t saved_bytes, void* scratch,
                       size_t scratch_bytes, void* stream) {
  int e = linear_shape(tokens, d_in, d_out);
  if (e != ESG_OK) return e;
  const LinearLayout L = linear_layout(tokens, d_in, d_out, need_dx, need_dw);
  if ((x_dtype != ESG_F32 && x_dtype != ESG_BF16) || (w_dtype != ESG_F32 && w_dtype != ESG_BF16))
    return ESG_ERR_UNSUPPORTED;
  if (w == nullptr || !aligned16(w)) return ESG_ERR_INVALID_ARG;
  if (tokens > 0)
    for (const void* p : {x, (const void*)y})
      if (p == nullptr || !aligned16(p)) return ESG_ERR_INVALID_ARG;
  if ((L.saved > 0 && (saved == nullptr || saved_bytes < L.saved)) || scratch == nullptr || scratch_bytes < L.fwd)
    return ESG_ERR_WORKSPACE;
  if (!aligned16(scratch) || !aligned16(saved)) return ESG_ERR_INVALID_ARG;
  hipStream_t st = (hipStream_t)stream;
  void* const wqt = need_dx ? at<char>(saved, L.wqt) : nullptr;
  float* const wst = need_dx ? at<float>(saved, L.wst) : nullptr;
  hipError_t h;
  if (need_dw && tokens > 0) {
    h = launch_quant_pair(w_dtype, w, d_out, at<char>(scratch, L.wq), at<float>(scratch, L.ws), wqt, wst, x_dtype, x,
                          tokens, at<char>(scratch, L.xq), at<float>(scratch, L.xs), at<char>(saved, L.xqt),
                          at<float>(saved, L.xst), d_in, st);
  } else {
    h = launch_quant_tiles(w_dtype, w, 1, d_out, d_in, at<char>(scratch, L.wq), at<float>(scratch, L.ws), wqt, wst, st);
    if (h != hipSuccess || tokens == 0) return hip_status(h);
    h = launch_quant_rows(x_dtype, x, tokens, d_in, at<char>(scratch, L.xq), at<float>(scratch, L.xs), nullptr, nullptr,
                          st);
  }
  if (h == hipSuccess)
    h = launch_fp8_matmul(at<char>(scratch, L.xq), at<float>(scratch, L.xs), at<char>(scratch, L.wq),
                          at<float>(scratch, L.ws), 0, x_dtype, tokens, d_out, d_in, y, at<char>(scratch, L.fmm), st);
  return hip_status(h);
}

int esg_fp8_linear_bwd(const void* dy, int x_dtype, int w_dtype, int tokens, int d_in, int d_out, const void* saved,
                       size_t saved_bytes, void* dx, void* dw, void* scratch, size_t scratch_bytes, void* stream) {
  int e = linear_shape(tokens, d_in, d_out);
  if (e != ESG_OK) return e;
  if ((x_dtype != ESG_F32 && x_dtype != ESG_BF16) || (w_dtype != ESG_F32 && w_dtype != ESG_BF16))
    return ESG_ERR_UNSUPPORTED;
  const int need_dx = dx != nullptr, need_dw = dw != nullptr;
  if (!need_dx && !need_dw) return ESG_OK;
  hipStream_t st = (hipStream_t)stream;
  if (!aligned16(dx) || !aligned16(dw)) return ESG_ERR_INVALID_ARG;
  if (tokens == 0) {  // no tokens: the weight gradient is zero
    if (!need_dw) return ESG_OK;
    const size_t words = (size_t)d_out * d_in * (w_dtype == ESG_F32 ? 4 : 2) / 4;
    return hip_status(launch_fill_i32((int32_t*)dw, 0, words, st));
  }
  const LinearLayout L = linear_layout(tokens, d_in, d_out, need_dx, need_dw);
  if (dy == nullptr || !aligned16(dy)) return ESG_ERR_INVALID_ARG;
  if (saved == nullptr || saved_bytes < L.saved || scratch == nullptr || scratch_bytes < L.bwd)
    return ESG_ERR_WORKSPACE;
  if (!aligned16(scratch) || !aligned16(saved)) return ESG_ERR_INVALID_ARG;
  hipError_t h = launch_quant_rows(x_dtype, dy, tokens, d_out, at<char>(scratch, L.dq), at<float>(scratch, L.ds),
                                   need_dw ? at<char>(scratch, L.dqt) : nullptr,
                                   need_dw ? at<float>(scratch, L.dst) : nullptr, st);
  if (h == hipSuccess && need_dx)
    h = launch_fp8_matmul(at<char>(scratch, L.dq), at<float>(scratch, L.ds), at<char>(saved, L.wqt),
                          at<float>(saved, L.wst), 0, x_dtype, tokens, d_in, d_out, dx, at<char>(scratch, L.bmm), st);
  if (h == hipSuccess && need_dw)
    h = launch_fp8_matmul(at<char>(scratch, L.dqt), at<float>(scratch, L.dst), at<char>(saved, L.xqt),
                          at<float>(saved, L.xst), 1, w_dtype, d_out, d_in, (tokens + 15) / 16 * 16, dw,
                          at<char>(scratch, L.bmm), st);
  return hip_status(h);
}

int esg_moe_decode_supported(int tokens, int experts, int topk, int d_model, int d_ff, int w_dtype) {
  return tokens >= 0 && tokens <= kMoeMaxTokens && experts >= 1 && experts <= kMoeMaxExperts && topk >= 1 &&
         topk <= kRouteMaxK && topk <= experts && d_model >= 16 && d_model % 16 == 0 && d_model <= (1 << 17) &&
         d_ff >= 16 && d_ff % 16 == 0 && d_ff <= (1 << 17) && (w_dtype == ESG_BF16 || w_dtype == ESG_E4M3);
}

namespace {
thread_local int moe_patience = kMoePatience;
}

int esg_moe_decode_set_patience(int polls) {
  moe_patience = polls < 0 ? kMoePatience : polls;
  return ESG_OK;
}

int esg_moe_decode_workspace_size(int tokens, int experts, int topk, int d_model, int d_ff, size_t* workspace_bytes) {
  if (workspace_bytes == nullptr || tokens < 0) return ESG_ERR_INVALID_ARG;
  if (!esg_moe_decode_supported(tokens, experts, topk, d_model, d_ff, ESG_BF16)) return ESG_ERR_UNSUPPORTED;
  *workspace_bytes = moe_decode_workspace_bytes(tokens, experts, topk, d_model, d_ff);
  return ESG_OK;
}

int esg_moe_decode(const void* x, const void* w_router, const float* expert_bias, int bias_stride, const void* w_gate,
                   const void* w_up, const void* w_down, const float* s_gate, const float* s_up, const float* s_down,
                   int w_dtype, int tokens, int experts, int topk, int d_model, int d_ff, float scaling_factor,
                   int apply_scaling, void* y, float* probs, int64_t* indices, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (tokens < 0 || bias_stride < 1) return ESG_ERR_INVALID_ARG;
  if (!esg_moe_decode_supported(tokens, experts, topk, d_model, d_ff, w_dtype)) return ESG_ERR_UNSUPPORTED;
  if (tokens == 0) return ESG_OK;
  for (const void* p : {x, w_router, w_gate, w_up, w_down, (const void*)y})
    if (p == nullptr || !aligned16(p)) return ESG_ERR_INVALID_ARG;
  if (expert_bias == nullptr || probs == nullptr || indices == nullptr) return ESG_ERR_INVALID_ARG;
  if (w_dtype == ESG_E4M3 && (s_gate == nullptr || s_up == nullptr || s_down == nullptr)) return ESG_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < moe_decode_workspace_bytes(tokens, experts, topk, d_model, d_ff))
    return ESG_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ESG_ERR_INVALID_ARG;
  const MoeCall c{x,      w_router, expert_bias, bias_stride, w_gate, w_up,           w_down,        s_gate, s_up,  s_down,
                  w_dtype, tokens,  experts,     topk,        d_model, d_ff,          scaling_factor, apply_scaling, y,
                  probs,  indices, moe_patience};
  return hip_status(launch_moe_decode(c, workspace, (hipStream_t)stream));
}

int esg_mfma_rate_probe(int blocks, int iters, float* out, void* stream) {
  if (blocks <= 0 || iters <= 0 || out == nullptr) return ESG_ERR_INVALID_ARG;
  return hip_status(launch_mfma_probe(blocks, iters, out, (hipStream_t)stream));
}

int esg_timing_enable(int on) {
  timing_set(on != 0);
  return ESG_OK;
}

int esg_timing_reset(void) {
  timing_reset();
  return ESG_OK;
}

int esg_timing_read(const char* kernel, double* total_ms, int* launches) {
  if (kernel == nullptr || total_ms == nullptr || launches == nullptr) return ESG_ERR_INVALID_ARG;
  return timing_read(kernel, total_ms, launches) == 0 ? ESG_OK : ESG_ERR_HIP;
}

}  // extern "C"
