// C ABI of the operators that choose weights per token: routing and the chosen experts'
// product.  Argument checks, workspace layout and the launches of a call.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>

#include "gemvfuse.h"
#include "tile_host.cuh"

namespace gf {

static bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

static int issue_all(const LaunchRec* recs, int n, void* stream) {
  for (int i = 0; i < n; ++i) {
    const int e = issue(recs[i], static_cast<cudaStream_t>(stream));
    if (e != GF_OK) return e;
  }
  return GF_OK;
}

// ------------------------------------------------------------------ routing
static int plan_route(const float* logits, int64_t T, int64_t E, const gf_route_opts* o, int32_t* ids, float* weights,
                      LaunchRec* r, int* n) {
  *n = 0;
  if (!o || T < 0 || E < 1 || o->top_k < 1 || o->top_k > E) return GF_ERR_INVALID;
  if (o->score != GF_SCORE_SOFTMAX && o->score != GF_SCORE_SIGMOID) return GF_ERR_INVALID;
  if (!std::isfinite(o->scale)) return GF_ERR_INVALID;
  const int64_t ld = o->ld == 0 ? E : o->ld;
  if (ld < E) return GF_ERR_INVALID;
  const int64_t G = o->n_group == 0 ? 1 : o->n_group;
  if (G < 1 || E % G != 0) return GF_ERR_INVALID;
  if (G > 1 && (o->topk_group < 1 || o->topk_group > G || (o->group_top != 1 && o->group_top != 2)))
    return GF_ERR_INVALID;
  if (E > kRouteMaxExperts || o->top_k > kRouteMaxTopK || G > kRouteMaxGroups || T > (1 << 24) || ld > (1LL << 40))
    return GF_ERR_UNSUPPORTED;
  if (T == 0) return GF_OK;
  if (!logits || !ids || !weights) return GF_ERR_INVALID;
  if (!aligned_to(logits, 4) || !aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(o->bias, 4))
    return GF_ERR_ALIGN;
  const int64_t lb = ((T - 1) * ld + E) * 4, ob = T * o->top_k * 4;
  if (ranges_overlap(ids, ob, weights, ob) || ranges_overlap(ids, ob, logits, lb) ||
      ranges_overlap(weights, ob, logits, lb) || ranges_overlap(ids, ob, o->bias, E * 4) ||
      ranges_overlap(weights, ob, o->bias, E * 4))
    return GF_ERR_ALIAS;
  r->kind = REC_ROUTE;
  r->pdl = (o->flags & GF_FLAG_PDL) != 0;
  RouteArgs& a = r->route;
  a.logits = logits;
  a.bias = o->bias;
  a.ids = ids;
  a.weights = weights;
  a.T = T;
  a.ld = ld;
  a.E = static_cast<int>(E);
  a.k = static_cast<int>(o->top_k);
  a.sigmoid = o->score == GF_SCORE_SIGMOID;
  a.n_group = static_cast<int>(G);
  a.topk_group = static_cast<int>(G > 1 ? o->topk_group : 1);
  a.group_top = G > 1 ? o->group_top : 1;
  a.norm = o->norm != 0;
  a.scale = o->scale == 0.0f ? 1.0f : o->scale;
  *n = 1;
  return GF_OK;
}

// ------------------------------------------------------------------ experts
struct ExpertsLayout {
  int64_t slots, groups, n_groups, places, xrec, hrec, y, max_tiles, bytes;
};

static int experts_layout(int64_t E, int64_t T, int64_t k, int64_t M, int64_t K, ExpertsLayout& l) {
  if (E < 1 || T < 0 || k < 1 || M < 0 || K < 0) return GF_ERR_INVALID;
  if (E > kRouteMaxExperts || T > kExpMaxTokens || k > kRouteMaxTopK || M > (1 << 20) || K > (1 << 20))
    return GF_ERR_UNSUPPORTED;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const int64_t S = T * k, K32 = (K + 31) / 32, M32 = (M + 31) / 32;
  // every expert's slots in column tiles of cp: at most one part-filled tile an expert
  const int64_t cp = std::min<int64_t>(8, std::max<int64_t>(T, 1));
  l.max_tiles = std::min(S, std::min(E, S) + S / cp);
  l.n_groups = take(16);
  l.slots = take(std::max(S, l.max_tiles * 8) * 4);
  l.groups = take(S * 16);
  l.places = take(S * 8);
  l.xrec = take(l.max_tiles * K32 * record_bytes(static_cast<int>(cp)));
  l.hrec = take(std::max(l.max_tiles * M32 * record_bytes(static_cast<int>(cp)), S * M * 4));
  l.y = take(S * K * 4);
  l.bytes = at;
  return GF_OK;
}

static bool columns_ok(int wtype, int64_t n) {
  return wtype == GF_Q4_K ? n % 256 == 0 : (wtype == GF_Q8_0 || wtype == GF_Q4_0) ? n % 32 == 0 : true;
}

// Whether the tiled kernels take this call (both products or neither).
static bool experts_tiled(const gf_experts* x) {
  return x->K % 32 == 0 && x->M % 32 == 0 && x->M > 0 && !(x->flags & GF_FLAG_NO_TENSOR_CORES) &&
         aligned_to(x->W_gate, 16) && aligned_to(x->W_up, 16) && aligned_to(x->W_down, 16);
}

// Columns of a group.  Rows without codes are read once per group and decode for nothing:
// as many column tiles as the experts' mean fills (256 tokens on 8 F16 experts, 8 columns
// each: 374 us in groups of 8, 332 in groups of 16).  Block formats: groups of 16 on the wide
// kernel where that is estimated to be faster, else of 8.  One format of each kind: 8.
static int experts_cols(const gf_experts* x, int64_t T, int sms) {
  if (T < 8) return static_cast<int>(T);
  const double slots = static_cast<double>(T) * x->top_k;
  const double used = std::min<double>(static_cast<double>(x->E), slots), mean = slots / used;
  const int wg = x->wtype, wd = x->wtype_down;
  if (tile_plain(wg) && tile_plain(wd)) return mean <= 5.0 ? 8 : mean <= 10.0 ? 16 : 24;
  if (!wide_takes(wg, static_cast<int>(row_bytes_of(wg, x->K))) || !wide_takes(wd, static_cast<int>(row_bytes_of(wd, x->M))))
    return 8;
  // groups an expert's slots make, their number spread like a Poisson one: half a group is lost
  const double g8 = used * std::max(1.0, mean / 8.0 + 0.5), g16 = used * std::max(1.0, mean / 16.0 + 0.5);
  const double narrow = tile_cost(x->M, x->K, 32, g8, sms) + tile_cost(x->K, x->M, kTileRows, g8, sms);
  const double wide = wide_cost(wg, x->M, x->K, wide_rows(wg) / 2, g16, sms) + wide_cost(wd, x->K, x->M, wide_rows(wd), g16, sms);
  return mean > 5.0 && wide < narrow ? 16 : 8;
}

constexpr int kExpMaxRecs = 4;

// Every check of a call; its workspace layout.
static int check_experts(const gf_experts* ex, const float* x, int64_t T, const float* aux, const float* dst,
                         ExpertsLayout& l) {
  if (!ex) return GF_ERR_INVALID;
  const int wg = ex->wtype, wd = ex->wtype_down;
  if (wg < GF_F32 || wg > GF_Q4_K || wd < GF_F32 || wd > GF_Q4_K) return GF_ERR_INVALID;
  const int v = experts_layout(ex->E, T, ex->top_k, ex->M, ex->K, l);
  if (v != GF_OK) return v;
  if (!columns_ok(wg, ex->K) || !columns_ok(wd, ex->M)) return GF_ERR_UNSUPPORTED;
  if (T == 0 || ex->K == 0) return GF_OK;
  const bool some = ex->M > 0;
  if (!x || !dst || !ex->ids || !ex->weights || !ex->workspace || (some && (!ex->W_gate || !ex->W_up || !ex->W_down)))
    return GF_ERR_INVALID;
  if (ex->workspace_bytes < l.bytes) return GF_ERR_INVALID;
  const uintptr_t ag = wg == GF_F32 ? 4 : 2, adn = wd == GF_F32 ? 4 : 2;
  if (!aligned_to(ex->W_gate, ag) || !aligned_to(ex->W_up, ag) || !aligned_to(ex->W_down, adn) || !aligned_to(x, 4) ||
      !aligned_to(dst, 4) || !aligned_to(aux, 4) || !aligned_to(ex->ids, 4) || !aligned_to(ex->weights, 4) ||
      !aligned_to(ex->workspace, 256) || !aligned_to(ex->rms_norm_weight, 4))
    return GF_ERR_ALIGN;
  if (ex->rms_norm_weight && !(ex->rms_norm_eps >= 0.0f && ex->rms_norm_eps <= std::numeric_limits<float>::max()))
    return GF_ERR_INVALID;
  const int64_t xb = T * ex->K * 4, sb = T * ex->top_k * 4;
  const int64_t gb = ex->E * ex->M * row_bytes_of(wg, ex->K), db = ex->E * ex->K * row_bytes_of(wd, ex->M);
  const struct { const void* p; int64_t bytes; } in[7] = {{ex->W_gate, gb}, {ex->W_up, gb},  {ex->W_down, db},
                                                          {x, xb},          {ex->ids, sb},   {ex->weights, sb},
                                                          {ex->rms_norm_weight, ex->K * 4}};
  for (const auto& i : in)
    if (ranges_overlap(dst, xb, i.p, i.bytes) || ranges_overlap(ex->workspace, l.bytes, i.p, i.bytes)) return GF_ERR_ALIAS;
  if (ranges_overlap(ex->workspace, l.bytes, dst, xb) || ranges_overlap(ex->workspace, l.bytes, aux, xb) ||
      (aux != dst && ranges_overlap(dst, xb, aux, xb)))
    return GF_ERR_ALIAS;
  return GF_OK;
}

static int plan_experts(const gf_experts* ex, const float* x, int64_t T, const float* aux, float* dst, LaunchRec* recs,
                        int* n) {
  *n = 0;
  ExpertsLayout l;
  const int v = check_experts(ex, x, T, aux, dst, l);
  if (v != GF_OK || T == 0 || ex->K == 0) return v;
  const int wg = ex->wtype, wd = ex->wtype_down;
  const bool some = ex->M > 0;
  unsigned* err = device_error_word();
  if (!err) return cuda_fail(cudaGetLastError());
  const DeviceLimits lim = device_limits();
  uint8_t* ws = static_cast<uint8_t*>(ex->workspace);
  ExpertsArgs a = {};
  a.x = x;
  a.ids = ex->ids;
  a.weights = ex->weights;
  a.gamma = ex->rms_norm_weight;
  a.eps = ex->rms_norm_eps;
  a.aux = aux;
  a.dst = dst;
  a.err = err;
  a.E = static_cast<int>(ex->E);
  a.T = static_cast<int>(T);
  a.k = static_cast<int>(ex->top_k);
  a.M = static_cast<int>(ex->M);
  a.K = static_cast<int>(ex->K);
  a.n_groups = reinterpret_cast<int32_t*>(ws + l.n_groups);
  a.slots = reinterpret_cast<int32_t*>(ws + l.slots);
  a.groups = reinterpret_cast<int4*>(ws + l.groups);
  a.places = reinterpret_cast<int2*>(ws + l.places);
  a.xrec = ws + l.xrec;
  a.hrec = ws + l.hrec;
  a.cp = static_cast<int>(std::min<int64_t>(8, T));
  a.max_tiles = static_cast<int>(l.max_tiles);
  a.y = reinterpret_cast<float*>(ws + l.y);
  a.cols = experts_cols(ex, T, lim.sm_count);
  a.out_format = wd;
  a.sm_count = lim.sm_count;
  a.smem_optin = lim.smem_optin;
  bool pdl = (ex->flags & GF_FLAG_PDL) != 0;
  auto add = [&](int phase, int wtype, const void* W, const void* W2) {
    LaunchRec& r = recs[(*n)++];
    r.kind = REC_EXPERTS;
    r.pdl = pdl;
    r.experts = a;
    r.experts.phase = phase;
    r.experts.wtype = wtype;
    r.experts.W = static_cast<const uint8_t*>(W);
    r.experts.W2 = static_cast<const uint8_t*>(W2);
    pdl = true;  // each launch of a call may start early behind the one before it
  };
  if (some && experts_tiled(ex)) {
    add(EXP_PREP, wg, ex->W_gate, ex->W_up);
    add(EXP_GLU, wg, ex->W_gate, ex->W_up);
    add(EXP_DOWN, wd, ex->W_down, nullptr);
  } else {
    if (some) add(EXP_GLU_GENERIC, wg, ex->W_gate, ex->W_up);
    add(EXP_DOWN_GENERIC, wd, ex->W_down, nullptr);  // M == 0: empty sums, y = 0
  }
  add(EXP_COMBINE, wd, some && experts_tiled(ex) ? ex->W_down : nullptr, nullptr);
  return GF_OK;
}

}  // namespace gf

using namespace gf;

extern "C" {

int gf_route(const float* logits, int64_t T, int64_t E, const gf_route_opts* opts, int32_t* ids, float* weights,
             void* stream) {
  LaunchRec r;
  int n = 0;
  const int v = plan_route(logits, T, E, opts, ids, weights, &r, &n);
  return v != GF_OK ? v : issue_all(&r, n, stream);
}

int gf_prepare_route(const float* logits, int64_t T, int64_t E, const gf_route_opts* opts, int32_t* ids,
                     float* weights, gf_prepared** out) {
  if (!out) return GF_ERR_INVALID;
  *out = nullptr;
  LaunchRec r;
  int n = 0;
  const int v = plan_route(logits, T, E, opts, ids, weights, &r, &n);
  return v != GF_OK ? v : make_prepared(&r, n, out);
}

int64_t gf_experts_workspace(int64_t E, int64_t T, int64_t top_k, int64_t M, int64_t K) {
  ExpertsLayout l;
  const int v = experts_layout(E, T, top_k, M, K, l);
  return v != GF_OK ? v : l.bytes;
}

int gemv_experts(const gf_experts* ex, const float* x, int64_t T, const float* aux, float* dst, void* stream) {
  LaunchRec recs[kExpMaxRecs];
  int n = 0;
  const int v = plan_experts(ex, x, T, aux, dst, recs, &n);
  return v != GF_OK ? v : issue_all(recs, n, stream);
}

int gf_plan_experts(const gf_experts* ex, const float* x, int64_t T, const float* aux, const float* dst,
                    int64_t info[8]) {
  ExpertsLayout l;
  const int v = check_experts(ex, x, T, aux, dst, l);
  if (v != GF_OK || T == 0 || ex->K == 0) return v;
  const bool tiled = ex->M > 0 && experts_tiled(ex);
  if (info) {
    for (int i = 0; i < 8; ++i) info[i] = 0;
    if (tiled) {
      info[0] = experts_cols(ex, T, device_limits().sm_count);
      info[1] = info[0] > 8 && !tile_plain(ex->wtype);
      info[2] = info[0] > 8 && !tile_plain(ex->wtype_down);
    }
  }
  return tiled ? PATH_TILE : PATH_GENERIC;
}

int gf_prepare_experts(const gf_experts* ex, const float* x, int64_t T, const float* aux, float* dst,
                       gf_prepared** out) {
  if (!out) return GF_ERR_INVALID;
  *out = nullptr;
  LaunchRec recs[kExpMaxRecs];
  int n = 0;
  const int v = plan_experts(ex, x, T, aux, dst, recs, &n);
  return v != GF_OK ? v : make_prepared(recs, n, out);
}

}  // extern "C"
