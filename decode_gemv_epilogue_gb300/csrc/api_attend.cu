// C ABI of a decode step's attention: rotary positions, the 8-bit cache and attention over it.
// Argument checks and the launches of a call.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "gemvfuse.h"
#include "gf_internal.h"

namespace gf {

static bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int64_t kMaxTokens = 1 << 20;  // of a call on the cache
constexpr int64_t kMaxHeads = 1024;

static int elem_bytes(int type) { return type == GF_F32 ? 4 : 2; }

// Bytes of T rows of `width` elements, `ld` apart.
static int64_t rows_bytes(int64_t T, int64_t ld, int64_t width, int type) {
  return T > 0 ? ((T - 1) * ld + width) * elem_bytes(type) : 0;
}

// Rows of `heads` heads: their distance (0: dense), element type and alignment; `vec` is cleared where
// they cannot be read four elements at a time.
static int check_rows(const void* p, int64_t* ld, int64_t width, int type, int* vec) {
  if (*ld == 0) *ld = width;
  if (*ld < width) return GF_ERR_INVALID;
  if (*ld > (1LL << 40)) return GF_ERR_UNSUPPORTED;
  if (!p) return GF_ERR_INVALID;
  if (!aligned_to(p, static_cast<uintptr_t>(elem_bytes(type)))) return GF_ERR_ALIGN;
  if (!aligned_to(p, 4u * static_cast<unsigned>(elem_bytes(type))) || *ld % 4 != 0) *vec = 0;
  return GF_OK;
}

static bool type_ok(int type) { return type == GF_F32 || type == GF_F16; }

// Of a power of two, else -1 (for any v).
static int log2_of(int64_t v) {
  if (v < 1 || (v & (v - 1)) != 0) return -1;
  int l = 0;
  while (v >>= 1) ++l;
  return l;
}

// ------------------------------------------------------------------ rotary positions
int64_t rope_table_bytes(int64_t n_rot) { return 16 + n_rot / 2 * 8; }

static int plan_rope_table(void* table, int64_t n_rot, const gf_rope_freqs* f, RopeTableArgs& a) {
  if (!f || n_rot < 2 || n_rot % 2 != 0) return GF_ERR_INVALID;
  if (f->kind < GF_ROPE_PLAIN || f->kind > GF_ROPE_BANDS) return GF_ERR_INVALID;
  if (!(f->base > 1.0) || !std::isfinite(f->base) || !std::isfinite(f->magnitude) || f->magnitude < 0.0) return GF_ERR_INVALID;
  if (f->kind != GF_ROPE_PLAIN && (!(f->factor > 0.0) || !std::isfinite(f->factor))) return GF_ERR_INVALID;
  if (f->kind == GF_ROPE_RAMP || f->kind == GF_ROPE_BANDS) {
    if (f->span < 1 || !std::isfinite(f->fast) || !(f->slow > 0.0) || !(f->fast > f->slow)) return GF_ERR_INVALID;
  }
  if (n_rot > 1024) return GF_ERR_UNSUPPORTED;
  if (!table) return GF_ERR_INVALID;
  if (!aligned_to(table, 16) || !aligned_to(f->divisors, 4)) return GF_ERR_ALIGN;
  if (ranges_overlap(table, rope_table_bytes(n_rot), f->divisors, n_rot / 2 * 4)) return GF_ERR_ALIAS;
  a = {};
  a.table = table;
  a.divisors = f->divisors;
  a.base = f->base;
  a.factor = f->factor;
  a.span = static_cast<double>(f->span);
  a.fast = f->fast;
  a.slow = f->slow;
  const double stretched = f->kind == GF_ROPE_RAMP && f->factor > 1.0 ? 0.1 * std::log(f->factor) + 1.0 : 1.0;
  a.magnitude = static_cast<float>(f->magnitude > 0.0 ? f->magnitude : stretched);
  a.pairs = static_cast<int>(n_rot / 2);
  a.kind = f->kind;
  return GF_OK;
}

static int check_rotation(const gf_rope_opts* o, int64_t dim) {
  if (o->layout != GF_ROPE_HALVES && o->layout != GF_ROPE_PAIRS) return GF_ERR_INVALID;
  if (o->n_rot < 0 || o->n_rot % 2 != 0 || o->n_rot > dim) return GF_ERR_INVALID;
  if (o->n_rot == 0 && dim % 2 != 0) return GF_ERR_INVALID;
  if (!o->table) return GF_ERR_INVALID;
  return aligned_to(o->table, 16) ? GF_OK : GF_ERR_ALIGN;
}

static int plan_rope(const void* x, int64_t T, int64_t heads, int64_t dim, const int32_t* pos, const gf_rope_opts* o,
                     void* dst, LaunchRec* r, int* n) {
  *n = 0;
  if (!o || T < 0 || heads < 0 || dim < 2 || !type_ok(o->type)) return GF_ERR_INVALID;
  if (T > kMaxTokens || heads > kMaxHeads || dim > 1024) return GF_ERR_UNSUPPORTED;
  if (T == 0 || heads == 0) return GF_OK;
  int v = check_rotation(o, dim);
  if (v != GF_OK) return v;
  if (!pos) return GF_ERR_INVALID;
  if (!aligned_to(pos, 4)) return GF_ERR_ALIGN;
  const int64_t rot = o->n_rot == 0 ? dim : o->n_rot, width = heads * dim;
  int64_t ld = o->ld, ld_dst = o->ld_dst;
  int vec = dim % 8 == 0 && rot % 8 == 0;
  if ((v = check_rows(x, &ld, width, o->type, &vec)) != GF_OK) return v;
  if ((v = check_rows(dst, &ld_dst, width, o->type, &vec)) != GF_OK) return v;
  const int64_t xb = rows_bytes(T, ld, width, o->type), db = rows_bytes(T, ld_dst, width, o->type);
  if (ranges_overlap(dst, db, x, xb) && !(dst == x && ld == ld_dst)) return GF_ERR_ALIAS;
  if (ranges_overlap(dst, db, pos, T * 4) || ranges_overlap(dst, db, o->table, rope_table_bytes(rot))) return GF_ERR_ALIAS;
  unsigned* err = device_error_word();
  if (!err) return cuda_fail(cudaGetLastError());
  r->kind = REC_ROPE;
  r->pdl = (o->flags & GF_FLAG_PDL) != 0;
  RopeArgs& a = r->rope;
  a = {};
  a.x = x;
  a.dst = dst;
  a.pos = pos;
  a.table = o->table;
  a.err = err;
  a.T = T;
  a.ld = ld;
  a.ld_dst = ld_dst;
  a.heads = static_cast<int>(heads);
  a.dim = static_cast<int>(dim);
  a.n_rot = static_cast<int>(rot);
  a.halves = o->layout == GF_ROPE_HALVES;
  a.type = o->type;
  a.vec = vec;
  *n = 1;
  return GF_OK;
}

// ------------------------------------------------------------------ the cache
struct Range {
  const void* p;
  int64_t bytes;
};

static int64_t code_bytes(const gf_cache* c) { return c->n_pages * c->heads * c->page * c->dim; }
static int64_t scale_bytes(const gf_cache* c) { return c->n_pages * c->heads * (c->page / c->block) * 4; }

// Sizes and pointers of a cache; its arrays may not overlap one another.
static int check_cache(const gf_cache* c, CacheArgs& a) {
  if (!c || (c->format != GF_CACHE_I8 && c->format != GF_CACHE_E4M3)) return GF_ERR_INVALID;
  if (c->n_pages < 0 || c->heads < 1 || c->dim < 1 || c->n_seqs < 0 || c->table_ld < 0) return GF_ERR_INVALID;
  const int pl = log2_of(c->page), bl = log2_of(c->block);
  if (c->page < 1 || c->block < 1 || pl < 0 || bl < 0 || c->block > c->page) return GF_ERR_INVALID;
  if (c->page < 16 || c->page > (1 << 20) || c->block > kCacheMaxBlock || c->dim % 16 != 0 || c->dim > kCacheMaxDim ||
      c->heads > kMaxHeads || c->n_pages > INT32_MAX || c->n_seqs > INT32_MAX || c->table_ld > (1LL << 30) / c->page ||
      c->n_pages > (1LL << 46) / (c->heads * c->page * c->dim))
    return GF_ERR_UNSUPPORTED;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->table) return GF_ERR_INVALID;
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || !aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4) ||
      !aligned_to(c->table, 4))
    return GF_ERR_ALIGN;
  const Range all[5] = {{c->k, code_bytes(c)}, {c->v, code_bytes(c)}, {c->k_scale, scale_bytes(c)},
                        {c->v_scale, scale_bytes(c)}, {c->table, c->n_seqs * c->table_ld * 4}};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(all[i].p, all[i].bytes, all[j].p, all[j].bytes)) return GF_ERR_ALIAS;
  a = {};
  a.k = c->k;
  a.v = c->v;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.table = c->table;
  a.n_pages = c->n_pages;
  a.table_ld = c->table_ld;
  a.n_seqs = static_cast<int>(c->n_seqs);
  a.heads = static_cast<int>(c->heads);
  a.dim = static_cast<int>(c->dim);
  a.page_log2 = pl;
  a.block_log2 = bl;
  a.format = c->format;
  return GF_OK;
}

static bool overlaps_cache(const gf_cache* c, const void* p, int64_t bytes) {
  return ranges_overlap(p, bytes, c->k, code_bytes(c)) || ranges_overlap(p, bytes, c->v, code_bytes(c)) ||
         ranges_overlap(p, bytes, c->k_scale, scale_bytes(c)) || ranges_overlap(p, bytes, c->v_scale, scale_bytes(c));
}

// An output of a call: apart from the cache, its table and the tokens' lists.
static bool output_clear(const gf_cache* c, const void* p, int64_t bytes, int64_t T, const int32_t* seq, const int32_t* pos) {
  return !overlaps_cache(c, p, bytes) && !ranges_overlap(p, bytes, c->table, c->n_seqs * c->table_ld * 4) &&
         !ranges_overlap(p, bytes, seq, T * 4) && !ranges_overlap(p, bytes, pos, T * 4);
}

static int check_tokens(const int32_t* seq, const int32_t* pos) {
  if (!pos) return GF_ERR_INVALID;
  return aligned_to(seq, 4) && aligned_to(pos, 4) ? GF_OK : GF_ERR_ALIGN;
}

static int plan_store(const gf_cache* c, const void* k, const void* v, int64_t T, const int32_t* seq, const int32_t* pos,
                      const gf_store_opts* o, LaunchRec* r, int* n) {
  *n = 0;
  if (!o || T < 0 || !type_ok(o->type) || o->q_heads < 0) return GF_ERR_INVALID;
  CacheArgs ca;
  int e = check_cache(c, ca);
  if (e != GF_OK) return e;
  if (T > kMaxTokens || o->q_heads > kMaxHeads) return GF_ERR_UNSUPPORTED;
  if (o->rope && (e = check_rotation(o->rope, c->dim)) != GF_OK) return e;
  const int64_t rot = !o->rope ? 0 : o->rope->n_rot == 0 ? c->dim : o->rope->n_rot;
  if (rot % 8 != 0) return GF_ERR_UNSUPPORTED;
  if (!o->rope && (o->q || o->q_dst)) return GF_ERR_INVALID;  // queries are taken along for their rotation only
  if (T == 0) return GF_OK;
  if ((e = check_tokens(seq, pos)) != GF_OK) return e;
  int vec = 1;
  int64_t ldk = o->ldk, ldv = o->ldv, ldq = o->ldq, ldd = o->ld_q_dst;
  const int64_t width = c->heads * c->dim, qwidth = o->q_heads * c->dim;
  if ((e = check_rows(k, &ldk, width, o->type, &vec)) != GF_OK) return e;
  if ((e = check_rows(v, &ldv, width, o->type, &vec)) != GF_OK) return e;
  const int64_t kb = rows_bytes(T, ldk, width, o->type), vb = rows_bytes(T, ldv, width, o->type);
  if (overlaps_cache(c, k, kb) || overlaps_cache(c, v, vb) || overlaps_cache(c, seq, T * 4) ||
      overlaps_cache(c, pos, T * 4) ||
      (o->rope && overlaps_cache(c, o->rope->table, rope_table_bytes(rot))))
    return GF_ERR_ALIAS;
  const bool with_q = o->q != nullptr || o->q_dst != nullptr;
  if (with_q && o->q_heads > 0) {
    if ((e = check_rows(o->q, &ldq, qwidth, o->type, &vec)) != GF_OK) return e;
    if ((e = check_rows(o->q_dst, &ldd, qwidth, o->type, &vec)) != GF_OK) return e;
    const int64_t qb = rows_bytes(T, ldq, qwidth, o->type), db = rows_bytes(T, ldd, qwidth, o->type);
    if (overlaps_cache(c, o->q, qb) || !output_clear(c, o->q_dst, db, T, seq, pos) ||
        ranges_overlap(o->q_dst, db, o->rope->table, rope_table_bytes(rot)))
      return GF_ERR_ALIAS;
    if (ranges_overlap(o->q_dst, db, o->q, qb) && !(o->q_dst == o->q && ldq == ldd)) return GF_ERR_ALIAS;
    // rows of one fused q, k, v product lie between each other: only the elements themselves count
    const Range in[2] = {{k, kb}, {v, vb}};
    const int64_t ld_in[2] = {ldk, ldv};
    for (int i = 0; i < 2; ++i) {
      if (!ranges_overlap(o->q_dst, db, in[i].p, in[i].bytes)) continue;
      if (ldd != ld_in[i]) return GF_ERR_ALIAS;
      const int64_t eb = elem_bytes(o->type), step = ldd * eb;
      int64_t off = (reinterpret_cast<intptr_t>(in[i].p) - reinterpret_cast<intptr_t>(o->q_dst)) % step;
      if (off < 0) off += step;
      if (off < qwidth * eb || off + width * eb > step) return GF_ERR_ALIAS;
    }
  }
  unsigned* err = device_error_word();
  if (!err) return cuda_fail(cudaGetLastError());
  r->kind = REC_STORE;
  r->pdl = (o->flags & GF_FLAG_PDL) != 0;
  StoreArgs& a = r->store;
  a = {};
  a.c = ca;
  a.k = k;
  a.v = v;
  a.seq = seq;
  a.pos = pos;
  a.table = o->rope ? o->rope->table : nullptr;
  a.err = err;
  a.q = with_q && o->q_heads > 0 ? o->q : nullptr;
  a.q_dst = o->q_dst;
  a.T = T;
  a.ldk = ldk;
  a.ldv = ldv;
  a.ldq = ldq;
  a.ld_q_dst = ldd;
  a.n_rot = static_cast<int>(rot);
  a.halves = o->rope && o->rope->layout == GF_ROPE_HALVES;
  a.q_heads = static_cast<int>(o->q_heads);
  a.type = o->type;
  a.vec = vec;
  // Decode steps bring one token a block, a warp's work.  Prompts bring whole blocks: as many warps as hold
  // their values in registers between finding the scale and writing the codes.  Which of them a call is stands in its
  // lists on the device; without a list of sequences every token is one's own, else more than 256 tokens are taken for
  // prompts.  300 tokens of 8 heads of 128, f16, in the decode steps' plan and in the prompts', cold: one token a
  // sequence 13 and 18 us with blocks of 16, 13 and 38 with 64; one prompt 18 and 16, 42 and 17.  (64 tokens of one
  // prompt 16 and 12, 34 and 14: short prompts pay.)
  a.tpw = static_cast<int>(32 / (c->dim / 8));
  a.lane_inv = static_cast<int>(65536 / (c->dim / 8) + 1);
  const bool prompt = T > 256 && (seq || c->block <= a.tpw);
  while (prompt && (kStoreWarps >> a.wpu_log2) > 1 && (a.tpw * kStoreKept << a.wpu_log2) < c->block) ++a.wpu_log2;
  // (one token of each of 64 sequences with a scale each 9 us as units of a head and 13 as tasks, of 300 13 and 14, of
  // 512 16 and 14, of 1000 22 and 16)
  a.small = prompt && c->block <= a.tpw;
  if (a.small) {  // tasks of warps, two to a warp
    const int64_t tasks = 2 * ((c->heads + kStoreKept - 1) / kStoreKept);
    a.window = 8;
    a.unit_groups = static_cast<int>((a.window * tasks + 2 * kStoreWarps - 1) / (2 * kStoreWarps));
  } else {
    const int upg = kStoreWarps >> a.wpu_log2;
    a.unit_groups = static_cast<int>((2 * c->heads + upg - 1) / upg);
    // Each token may begin a block (decode steps); of a prompt's every block-th does, and CTAs that find none
    // only cost their start: as many tokens a CTA as leave sixteen CTAs to an SM.
    a.window = 1;
    const int64_t ctas = 16LL * device_limits().sm_count;
    while (a.window < 32 && a.window < c->block && T * a.unit_groups > ctas * a.window) a.window *= 2;
  }
  // (with 32 query heads to turn, blocks of 16: one token of each of 300 sequences 16 us by one row a lane and the decode
  // steps' plan, 22 by four and the prompts'; 300 tokens of a prompt 20 and 16)
  a.q_rows = prompt ? kStoreKept : 1;
  const int chunks = a.q ? (a.q_heads + a.q_rows * a.tpw - 1) / (a.q_rows * a.tpw) : 0;
  const int per_cta = kStoreWarps * (prompt ? 2 : 1);
  a.q_slices = (a.window * chunks + per_cta - 1) / per_cta;
  *n = 1;
  return GF_OK;
}

static int plan_load(const gf_cache* c, int64_t T, const int32_t* seq, const int32_t* pos, const gf_load_opts* o, void* k,
                     void* v, LaunchRec* r, int* n) {
  *n = 0;
  if (!o || T < 0 || !type_ok(o->type)) return GF_ERR_INVALID;
  CacheArgs ca;
  int e = check_cache(c, ca);
  if (e != GF_OK) return e;
  if (T > kMaxTokens) return GF_ERR_UNSUPPORTED;
  if (T == 0 || (!k && !v)) return GF_OK;
  if ((e = check_tokens(seq, pos)) != GF_OK) return e;
  int vec = 1;
  int64_t ldk = o->ldk, ldv = o->ldv;
  const int64_t width = c->heads * c->dim;
  if (k && (e = check_rows(k, &ldk, width, o->type, &vec)) != GF_OK) return e;
  if (v && (e = check_rows(v, &ldv, width, o->type, &vec)) != GF_OK) return e;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || (ldk | ldv) * elem_bytes(o->type) % 16 != 0) vec = 0;
  const int64_t kb = k ? rows_bytes(T, ldk, width, o->type) : 0, vb = v ? rows_bytes(T, ldv, width, o->type) : 0;
  if (!output_clear(c, k, kb, T, seq, pos) || !output_clear(c, v, vb, T, seq, pos) || ranges_overlap(k, kb, v, vb))
    return GF_ERR_ALIAS;
  r->kind = REC_LOAD;
  r->pdl = (o->flags & GF_FLAG_PDL) != 0;
  LoadArgs& a = r->load;
  a = {};
  a.c = ca;
  a.seq = seq;
  a.pos = pos;
  a.k = k;
  a.v = v;
  a.T = T;
  a.ldk = ldk;
  a.ldv = ldv;
  a.type = o->type;
  a.vec = vec;
  *n = 1;
  return GF_OK;
}

// ------------------------------------------------------------------ attention
// How the queries of a head of the cache fall into items of 8 or 16 rows.  Sixteen take two instructions'
// rows at once, on values decoded once; heads of more than 128 elements have no registers for that.
static void attend_shape(int64_t group, int64_t dim, int64_t run, AttendArgs& a) {
  a.tiles = dim <= 128 && group * run > 8 ? 2 : 1;
  const int most = 8 * a.tiles;
  a.subs = static_cast<int>((group + most - 1) / most);
  a.rows = static_cast<int>((group + a.subs - 1) / a.subs);
  const int64_t fit = std::max(1, most / a.rows), parts = (run + fit - 1) / fit;
  a.run = static_cast<int>(run);
  a.tokens = static_cast<int>((run + parts - 1) / parts);  // equal items of a run
}

static int64_t attend_bytes(int64_t T, int64_t q_heads, int64_t heads, int64_t dim, int64_t run) {
  if (T < 0 || heads < 1 || q_heads < 1 || q_heads % heads != 0 || dim < 1 || run < 0) return GF_ERR_INVALID;
  if (T > kAttMaxTokens || q_heads > kMaxHeads || dim % 16 != 0 || dim > kCacheMaxDim || run > kAttMaxTokens)
    return GF_ERR_UNSUPPORTED;
  AttendArgs a = {};
  attend_shape(q_heads / heads, dim, std::max<int64_t>(run, 1), a);
  return attend_workspace_bytes(static_cast<int>(dim), a.tiles, attend_ctas(device_limits().sm_count));
}

static int check_attend(const gf_cache* c, const void* q, int64_t T, int64_t q_heads, const int32_t* seq,
                        const int32_t* pos, const gf_attend_opts* o, const void* dst, AttendArgs& a) {
  if (!o || T < 0 || q_heads < 1 || !type_ok(o->type) || o->run < 0 || o->window < 0) return GF_ERR_INVALID;
  if (!std::isfinite(o->scale) || o->scale < 0.0f) return GF_ERR_INVALID;
  CacheArgs ca;
  int e = check_cache(c, ca);
  if (e != GF_OK) return e;
  if (q_heads % c->heads != 0) return GF_ERR_INVALID;
  if (T > kAttMaxTokens || q_heads > kMaxHeads || o->run > kAttMaxTokens || o->window > INT32_MAX)
    return GF_ERR_UNSUPPORTED;
  // (units of all items, counted in 64 bits times the warps that share them)
  if (static_cast<double>(T) * q_heads * (c->table_ld * c->page / 16 + 4) > 2251799813685248.0) return GF_ERR_UNSUPPORTED;
  if (T == 0) return GF_OK;
  if ((e = check_tokens(seq, pos)) != GF_OK) return e;
  int vec = 1;
  int64_t ldq = o->ldq, ldd = o->ld_dst;
  const int64_t width = q_heads * c->dim;
  int any = 1;
  if ((e = check_rows(q, &ldq, width, o->type, &vec)) != GF_OK) return e;
  if ((e = check_rows(dst, &ldd, width, o->type, &any)) != GF_OK) return e;
  if (!aligned_to(o->lse, 4)) return GF_ERR_ALIGN;
  const int64_t need = attend_bytes(T, q_heads, c->heads, c->dim, o->run);
  if (!o->workspace || o->workspace_bytes < need) return GF_ERR_INVALID;
  if (!aligned_to(o->workspace, 256)) return GF_ERR_ALIGN;
  const int64_t qb = rows_bytes(T, ldq, width, o->type), db = rows_bytes(T, ldd, width, o->type), lb = T * q_heads * 4;
  const Range out[3] = {{dst, db}, {o->lse, lb}, {o->workspace, need}};
  for (int i = 0; i < 3; ++i) {
    if (!output_clear(c, out[i].p, out[i].bytes, T, seq, pos) || ranges_overlap(out[i].p, out[i].bytes, q, qb))
      return GF_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return GF_ERR_ALIAS;
  }
  a = {};
  a.c = ca;
  a.q = q;
  a.dst = const_cast<void*>(dst);
  a.seq = seq;
  a.pos = pos;
  a.lse = o->lse;
  a.workspace = static_cast<float*>(o->workspace);
  a.ldq = ldq;
  a.ld_dst = ldd;
  a.scale = static_cast<float>((o->scale == 0.0f ? 1.0 / std::sqrt(static_cast<double>(c->dim)) : o->scale) *
                               1.4426950408889634);
  a.T = static_cast<int>(T);
  a.q_heads = static_cast<int>(q_heads);
  a.group = static_cast<int>(q_heads / c->heads);
  a.window = static_cast<int>(o->window);
  a.type = o->type;
  a.vec = vec;
  attend_shape(a.group, c->dim, std::max<int64_t>(o->run, 1), a);
  a.ctas = attend_ctas(device_limits().sm_count);
  return GF_OK;
}

constexpr int kAttMaxRecs = 2;

static int plan_attend(const gf_cache* c, const void* q, int64_t T, int64_t q_heads, const int32_t* seq, const int32_t* pos,
                       const gf_attend_opts* o, void* dst, LaunchRec* recs, int* n) {
  *n = 0;
  AttendArgs a;
  const int e = check_attend(c, q, T, q_heads, seq, pos, o, dst, a);
  if (e != GF_OK || T == 0) return e;
  bool pdl = (o->flags & GF_FLAG_PDL) != 0;
  for (const int phase : {ATT_PART, ATT_JOIN}) {
    LaunchRec& r = recs[(*n)++];
    r.kind = REC_ATTEND;
    r.pdl = pdl;
    r.attend = a;
    r.attend.phase = phase;
    pdl = true;
  }
  return GF_OK;
}

static int run_recs(const LaunchRec* recs, int n, void* stream) {
  for (int i = 0; i < n; ++i) {
    const int e = issue(recs[i], static_cast<cudaStream_t>(stream));
    if (e != GF_OK) return e;
  }
  return GF_OK;
}

}  // namespace gf

using namespace gf;

extern "C" {

int64_t gf_rope_table_bytes(int64_t n_rot) {
  if (n_rot < 2 || n_rot % 2 != 0) return GF_ERR_INVALID;
  return n_rot > 1024 ? GF_ERR_UNSUPPORTED : rope_table_bytes(n_rot);
}

int gf_rope_table(void* table, int64_t n_rot, const gf_rope_freqs* freqs, void* stream) {
  RopeTableArgs a;
  const int v = plan_rope_table(table, n_rot, freqs, a);
  if (v != GF_OK) return v;
  const int e = launch_rope_table(a, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_fail(static_cast<cudaError_t>(e)) : GF_OK;
}

int gf_rope(const void* x, int64_t T, int64_t heads, int64_t dim, const int32_t* pos, const gf_rope_opts* opts, void* dst,
            void* stream) {
  LaunchRec r;
  int n = 0;
  const int v = plan_rope(x, T, heads, dim, pos, opts, dst, &r, &n);
  return v != GF_OK ? v : run_recs(&r, n, stream);
}

int gf_prepare_rope(const void* x, int64_t T, int64_t heads, int64_t dim, const int32_t* pos, const gf_rope_opts* opts,
                    void* dst, gf_prepared** out) {
  if (!out) return GF_ERR_INVALID;
  *out = nullptr;
  LaunchRec r;
  int n = 0;
  const int v = plan_rope(x, T, heads, dim, pos, opts, dst, &r, &n);
  return v != GF_OK ? v : make_prepared(&r, n, out);
}

int gf_cache_store(const gf_cache* cache, const void* k, const void* v, int64_t T, const int32_t* seq, const int32_t* pos,
                   const gf_store_opts* opts, void* stream) {
  LaunchRec r;
  int n = 0;
  const int e = plan_store(cache, k, v, T, seq, pos, opts, &r, &n);
  return e != GF_OK ? e : run_recs(&r, n, stream);
}

int gf_prepare_cache_store(const gf_cache* cache, const void* k, const void* v, int64_t T, const int32_t* seq,
                           const int32_t* pos, const gf_store_opts* opts, gf_prepared** out) {
  if (!out) return GF_ERR_INVALID;
  *out = nullptr;
  LaunchRec r;
  int n = 0;
  const int e = plan_store(cache, k, v, T, seq, pos, opts, &r, &n);
  return e != GF_OK ? e : make_prepared(&r, n, out);
}

int gf_cache_load(const gf_cache* cache, int64_t T, const int32_t* seq, const int32_t* pos, const gf_load_opts* opts, void* k,
                  void* v, void* stream) {
  LaunchRec r;
  int n = 0;
  const int e = plan_load(cache, T, seq, pos, opts, k, v, &r, &n);
  return e != GF_OK ? e : run_recs(&r, n, stream);
}

int gf_prepare_cache_load(const gf_cache* cache, int64_t T, const int32_t* seq, const int32_t* pos, const gf_load_opts* opts,
                          void* k, void* v, gf_prepared** out) {
  if (!out) return GF_ERR_INVALID;
  *out = nullptr;
  LaunchRec r;
  int n = 0;
  const int e = plan_load(cache, T, seq, pos, opts, k, v, &r, &n);
  return e != GF_OK ? e : make_prepared(&r, n, out);
}

int64_t gf_attend_workspace(int64_t T, int64_t q_heads, int64_t heads, int64_t dim, int64_t run) {
  return attend_bytes(T, q_heads, heads, dim, run);
}

int gf_attend(const gf_cache* cache, const void* q, int64_t T, int64_t q_heads, const int32_t* seq, const int32_t* pos,
              const gf_attend_opts* opts, void* dst, void* stream) {
  LaunchRec recs[kAttMaxRecs];
  int n = 0;
  const int e = plan_attend(cache, q, T, q_heads, seq, pos, opts, dst, recs, &n);
  return e != GF_OK ? e : run_recs(recs, n, stream);
}

int gf_prepare_attend(const gf_cache* cache, const void* q, int64_t T, int64_t q_heads, const int32_t* seq,
                      const int32_t* pos, const gf_attend_opts* opts, void* dst, gf_prepared** out) {
  if (!out) return GF_ERR_INVALID;
  *out = nullptr;
  LaunchRec recs[kAttMaxRecs];
  int n = 0;
  const int e = plan_attend(cache, q, T, q_heads, seq, pos, opts, dst, recs, &n);
  return e != GF_OK ? e : make_prepared(recs, n, out);
}

}  // extern "C"
