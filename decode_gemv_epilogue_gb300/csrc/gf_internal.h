// Host/device shared declarations for the gemvfuse library (not part of the C ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "smem_limit.h"

struct CUtensorMap_st;  // the driver's tensor-map descriptor (cuda.h)
struct gf_prepared;

namespace gf {

// Kernel-side limits of the TMA-streamed GEMV.
constexpr int kMaxCols = 8;      // columns per GEMV launch
constexpr int kMaxBatch = 256;   // columns per call (wider batches run in blocks of kMaxCols)
constexpr int kMaxStages = 8;
constexpr int kBarBytes = 256;              // mbarrier area at the start of shared memory
constexpr int kXsMaxBytes = 64 * 1024;      // x chunk (all columns) kept in shared memory
constexpr int kXStageMaxBytes = 32 * 1024;  // x staged without a prologue (whole rows only)
constexpr int kSegMaxBytes = 32 * 1024;     // bytes of one row's K chunk
constexpr int kStageMaxBytes = 72 * 1024;
constexpr int kRedMaxBytes = 16 * 1024;
constexpr int kRingSlackBytes = 16;         // aligned-word decoders may read 3 bytes past a row
constexpr int kMaxFusedFwhtBlock = 8192;
constexpr int kUnitElems = 16;              // weights per decode unit (half a quant block)
constexpr int kMaxSplit = 8;                // CTAs of a split-K cluster (portable cluster size)
constexpr int kMaxSeg = 4;                  // matrices sharing x in one multi-matrix launch

// Tiling of the consumer warps, per (format, columns):
//  U   units (16 weights) per thread per K chunk, RT rows per thread per tile;
//  NCT columns per thread, CS = ceil(NC / NCT) column groups.
// A tile of R = G * RT rows is split over G row groups of consumer warps; a row group is
// CS column groups of wpc warps; within a column group every thread owns U units of the
// K chunk and keeps their x values (NCT columns) in registers for the whole chunk.
// F32/F16 decode is cheap, so batches are split two columns per thread (more warps);
// Q8_0/Q4_0 keep up to four columns per thread so each weight is decoded once per four
// columns.  Q4_K threads always own one unit pair (two units sharing a code load) and
// one column: with 17 warps a thread has at most 96 registers (a quarter of the SM's
// register file serves up to five warps), and a second column of x spills.  Single-
// column Q4_0 and Q8_0 (integer dot products, below) keep one unit and eight rows per
// thread per tile: the x conversion per unit is the costly part of a chunk's start, the
// rows share it, and the per-tile reduction is spread over more rows (Q8_0 with four
// rows per thread: 5-8% slower at 4096..14336 rows).
__host__ __device__ constexpr bool stream_quant(int wt) { return wt == 2 || wt == 3 || wt == 4; }
__host__ __device__ constexpr int stream_nct(int wt, int nc) {
  return wt == 4 ? 1 : stream_quant(wt) ? (nc <= 4 ? nc : 4) : (nc <= 2 ? nc : 2);
}
__host__ __device__ constexpr int stream_cs(int wt, int nc) {
  return (nc + stream_nct(wt, nc) - 1) / stream_nct(wt, nc);
}
__host__ __device__ constexpr int stream_u(int wt, int nc) {
  return wt == 4 ? 2 : ((wt == 3 || wt == 2) && nc == 1) ? 1 : (nc == 1 && stream_quant(wt)) ? 2 : 1;
}
__host__ __device__ constexpr int stream_rt(int wt, int nc) {
  return (nc == 1 && (wt == 3 || wt == 2)) ? 8 : 4;
}
__host__ __device__ constexpr int stream_max_cw(int wt, int nc) { return stream_nct(wt, nc) <= 2 ? 16 : 8; }
__host__ __device__ constexpr int stream_threads(int wt, int nc) { return 32 * (1 + stream_max_cw(wt, nc)); }
// Q4_0, Q8_0 and Q4_K with up to kIntMaxCols columns take integer dot products (x as
// shared-exponent 24-bit integers, dp4a on the codes): a third to a half of the
// instructions per weight of the float decode.  With more columns per thread the float
// decode, done once for all of them, is cheaper.
constexpr int kIntMaxCols = 1;
__host__ __device__ constexpr bool stream_int(int wt, int nc) { return (wt >= 2 && wt <= 4) && nc <= kIntMaxCols; }

struct StreamArgs {
  const uint8_t* W;
  const float* x;
  const float* aux;
  float* dst;
  const float* signs;
  unsigned* err;
  int64_t M;
  int K;
  int epi;
  int row_bytes;     // bytes of a full row
  int kc_len;        // elements per K chunk
  int n_kc;          // K chunks
  int R;             // rows per tile (= G * RT)
  int G;             // row groups of consumer warps
  int wpg;           // warps per row group (= CS * wpc)
  int wpc;           // warps per column group
  int NS;            // ring stages
  int stage_bytes;   // bytes reserved per stage
  int RC;            // rows per finalize chunk
  int ncw;           // consumer warps (= G * wpg)
  int rows_base;     // granules of rows per CTA (the first rows_extra CTAs take one more)
  int rows_extra;
  int gran;          // rows per granule: 1, or a full tile's real rows
  int fwht_B;        // 0 = no prologue
  int nsigns;
  float fwht_scale;
  const uint8_t* W2; // up-projection rows of the gated dual GEMV (nullptr: one matrix)
  const float* gamma;  // RMS-normalisation weight [K] (nullptr: no normalisation)
  float norm_eps;
  // Several matrices sharing x in one pass (nseg > 0): virtual row r belongs to segment
  // i = the first with r < seg_end[i]; its rows are seg_W[i], its tail seg_epi[i] with
  // seg_aux[i], its output seg_dst[i] ([ncols][rows of the segment]).  W, epi, aux and dst
  // above are then unused.
  int nseg;
  const uint8_t* seg_W[kMaxSeg];
  int64_t seg_end[kMaxSeg];
  int seg_epi[kMaxSeg];
  const float* seg_aux[kMaxSeg];
  float* seg_dst[kMaxSeg];
  int S;             // CTAs per cluster sharing a row range, each a slice of the K chunks
  int stage_x;       // 1: the producer bulk-copies x (one K chunk, every column) into xs
  int off_xs, off_aux, off_red, off_norm, off_xchg, off_ring;
};

struct GenericArgs {
  const uint8_t* W;
  const float* x;
  const float* aux;
  float* dst;
  const float* signs;
  unsigned* err;
  int64_t M;
  int K;
  int epi;
  int64_t row_bytes;
  int fwht_B;
  int nsigns;
  float fwht_scale;
  const uint8_t* W2;
  const float* gamma;
  float norm_eps;
};

struct DeviceLimits;

// Tensor-core GEMV (F16 weights, batches): see gemv_tc.cu.
struct TcArgs {
  const float* x;
  const float* aux;
  float* dst;
  unsigned* err;
  int64_t M;
  int K;
  int epi;
  int ncols;          // columns of this launch (<= kTcMaxCols)
  int Np;             // columns rounded up to 8: B holds Np rows of hi, then Np of lo
  int S;              // CTAs per cluster splitting K (1: none)
  int subs;           // 64-element sub-tiles per stage
  int nst;            // stages of a row (K / (64 subs))
  int NS;             // pipeline stages
  int tmem_cols;      // tensor-memory columns allocated (power of two >= 2 Np, >= 32)
  int off_a, off_b;   // stage offsets from the 1024-aligned shared-memory base
  int b_stage_bytes;  // 2 Np rows of 128 bytes
  int off_x;          // x stages: ncols rows of 64 * subs floats per stage
  int x_stage_bytes;
};

struct TcPlan {
  int grid, smem;
  TcArgs a;
};

constexpr int kTcMaxCols = 16;  // columns per tensor-core launch (one B chunk per converter thread)

// Shapes only (pointers are filled by the caller); false if the kernel cannot take them.
bool plan_tc(int64_t M, int64_t K, int ncols, int epi, const DeviceLimits& lim, TcPlan& p);
// Encodes the tensor map of W ([M][K] f16, row stride 2K) and launches.
int launch_tc(const TcPlan& p, const void* W, cudaStream_t st, bool pdl);

// A 2-D tensor map of element type dtype (kMapU8, kMapF16, kMapF32) over rows of `inner`
// elements, `stride_bytes` apart, with boxes of box_inner x box_rows (128-byte swizzle or
// none).  `map` points to a 64-byte aligned CUtensorMap.  Returns a cudaError_t.
enum { kMapU8 = 0, kMapF16 = 1, kMapF32 = 2 };
// The same over a dense [rows][inner] operand, from the cache of recent maps.
int cached_map_2d(const void* base, int dtype, uint64_t inner, uint64_t rows, uint32_t box_inner, uint32_t box_rows,
                  bool swizzle128, ::CUtensorMap_st* out);
int encode_map_2d(::CUtensorMap_st* map, int dtype, const void* base, uint64_t inner, uint64_t rows,
                  uint64_t stride_bytes, uint32_t box_inner, uint32_t box_rows, bool swizzle128);


// Generic kernel: 256 threads; shared memory x [ncols][K], 1/rms [ncols], warp
// partials [8][ncols].
constexpr int kGenericWarps = 8;
__host__ __device__ constexpr int64_t generic_smem_floats(int64_t ncols, int64_t K) {
  return ncols * K + ncols + kGenericWarps * ncols;
}

enum { PATH_STREAM = 1, PATH_GENERIC = 2, PATH_TC = 3, PATH_TILE = 4 };

struct Plan {
  int path;
  int grid, threads, smem;
  StreamArgs s;   // valid when path == PATH_STREAM (pointers filled by the caller)
};

struct DeviceLimits {
  int sm_count;
  int smem_optin;
};

// Kernel feature sets of the streamed GEMV (separate instantiations).
enum { FEAT_PLAIN = 0, FEAT_EXT = 1, FEAT_SPLIT = 2 };

// Launchers (return cudaError_t).  `pdl` requests programmatic stream serialization.
// FEAT_SPLIT launches group the grid into clusters of p.s.S CTAs.  One function per
// (format family, feature set), each in its own translation unit.
int launch_stream_float_plain(int wtype, int ncols, const Plan& p, cudaStream_t st, bool pdl);  // F32, F16
int launch_stream_float_ext(int wtype, int ncols, const Plan& p, cudaStream_t st, bool pdl);
int launch_stream_float_split(int wtype, int ncols, const Plan& p, cudaStream_t st, bool pdl);
int launch_stream_block_plain(int wtype, int ncols, const Plan& p, cudaStream_t st, bool pdl);  // Q8_0, Q4_0
int launch_stream_block_ext(int wtype, int ncols, const Plan& p, cudaStream_t st, bool pdl);
int launch_stream_block_split(int wtype, int ncols, const Plan& p, cudaStream_t st, bool pdl);
int launch_stream_q4k_plain(int ncols, const Plan& p, cudaStream_t st, bool pdl);              // Q4_K
int launch_stream_q4k_ext(int ncols, const Plan& p, cudaStream_t st, bool pdl);
int launch_stream_q4k_split(int ncols, const Plan& p, cudaStream_t st, bool pdl);
// Resident clusters of the split-K kernel for this plan (0 if unknown, e.g. no device).
int stream_split_max_clusters_float(int wtype, int ncols, const Plan& p);
int stream_split_max_clusters_block(int wtype, int ncols, const Plan& p);
int stream_split_max_clusters_q4k(int ncols, const Plan& p);
int launch_generic(int wtype, int ncols, const GenericArgs& a, int grid, int smem,
                   cudaStream_t st, bool pdl);
int launch_fwht(const float* x, const float* signs, float* dst, int64_t n, int B, int nsigns,
                cudaStream_t st);
// Kernel copy of `bytes` (a multiple of 16) between device-addressable ranges.
int launch_copy(void* dst, const void* src, int64_t bytes, cudaStream_t st, bool pdl);
int launch_elementwise(int op, const float* a, const float* b, int64_t nb, float* dst, int64_t n,
                       cudaStream_t st);
int launch_dequantize(int wtype, const uint8_t* W, int64_t M, int64_t K, int64_t row_bytes,
                      float* out, cudaStream_t st);

// ------------------------------------------------------------------ weights chosen per column
// Routing to experts (route.cu).
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteMaxGroups = 32;
struct RouteArgs {
  const float* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t T, ld;
  int E, k, sigmoid, n_group, topk_group, group_top, norm;
  float scale;
};
int launch_route(const RouteArgs& a, cudaStream_t st, bool pdl);

// The chosen experts' gated product (experts.cu): one launch of one phase.
constexpr int kExpMaxTokens = 256;
enum { EXP_PREP = 0, EXP_GLU = 1, EXP_DOWN = 2, EXP_COMBINE = 3, EXP_GLU_GENERIC = 4, EXP_DOWN_GENERIC = 5 };
struct ExpertsArgs {
  int phase;
  int wtype;            // of this phase's matrices
  int out_format;       // of the weights that take the gated product's records
  const uint8_t* W;     // gate (EXP_PREP, EXP_GLU*) or down (EXP_DOWN*; EXP_COMBINE behind the tiles)
  const uint8_t* W2;    // up
  const float* x;
  const int32_t* ids;
  const float* weights;
  const float* gamma;   // RMS normalisation of x (nullptr: none)
  float eps;
  const float* aux;
  float* dst;
  unsigned* err;
  int E, T, k;
  int M, K;             // ffn width, model width
  int cols;             // columns per group (8, 16 or 24, or the tokens if fewer than 8)
  int cp;               // columns stored per column tile: min(8, T)
  int max_tiles;        // upper bound on the column tiles of all experts
  // workspace
  int32_t* slots;       // the slots of each group, one after another
  int4* groups;         // {expert, first entry, columns, first column tile} of each column group
  int32_t* n_groups;    // their number; the items of the two products taken so far
  int2* places;         // [T k] {column tile, column | columns stored << 8} of each slot, or {-1, 0}
  uint8_t* xrec;        // [column tile][K / 32] records of packed x (see tile_mma.cuh)
  uint8_t* hrec;        // the same of the gated values, or [T k][M] float32 (generic)
  float* y;             // [T k][K]
  int sm_count, smem_optin;
};
int launch_experts(const ExpertsArgs& a, cudaStream_t st, bool pdl);

// Low-rank adapters (lora.cu): one launch of one phase.
constexpr int kLoraMaxRank = 256;
enum { LORA_SHRINK = 0, LORA_EXPAND = 1 };
struct LoraArgs {
  int phase;
  int atype;            // GF_F16 or GF_F32
  const uint8_t* A;     // [n][r][K]
  const uint8_t* B;     // [n][M][r]
  const int32_t* ids;
  const float* scales;
  const float* x;       // [ncols][K]
  const float* gamma;
  float eps;
  const float* aux;     // added by the expansion (nullptr: none)
  float* v;             // [ncols][r]
  float* out;           // [ncols][M]
  int n, r, M, K, ncols;
  int beside_pack;      // behind the launch that packs x, of the same call
};
int launch_lora(const LoraArgs& a, cudaStream_t st, bool pdl);

// The shared projection of a batch on the tensor cores (tile_lin.cu).
enum { LIN_PACK = 0, LIN_PRODUCT = 1, LIN_TAIL = 2 };
struct LinArgs {
  int phase;
  int wtype;            // any format
  const uint8_t* W;
  const float* x;       // [ncols][K]
  const float* gamma;
  float eps;
  const float* aux;
  float* dst;           // [ncols][M]
  uint8_t* records;     // packed x
  unsigned* err;
  int M, K, row_bytes, epi, ncols;
  int cols, cp;         // columns per group, stored per column tile
  int sm_count, smem_optin;
};
int launch_lin(const LinArgs& a, cudaStream_t st, bool pdl);
// Columns of a group.
int lin_cols(int wtype, int64_t M, int64_t K, int row_bytes, int ncols, int sms);

// ------------------------------------------------------------------ attention over an 8-bit cache
// Rotary positions (rope.cu).
struct RopeTableArgs {
  void* table;
  const float* divisors;
  double base, factor, span, fast, slow;
  float magnitude;
  int pairs, kind;
};
int launch_rope_table(const RopeTableArgs& a, cudaStream_t st);
struct RopeArgs {
  const void* x;
  void* dst;
  const int32_t* pos;
  const void* table;
  unsigned* err;        // device error word
  int64_t T, ld, ld_dst;
  int heads, dim, n_rot, halves;
  int type;             // GF_F32 or GF_F16
  int vec;              // units of eight elements, 16-byte (F16: 8-byte) aligned
};
int launch_rope(const RopeArgs& a, cudaStream_t st, bool pdl);

// The cache (cache.cu).
constexpr int kStoreWarps = 8;
constexpr int kStoreKept = 4;  // iterations whose values stay in registers between the store's two passes
constexpr int kCacheMaxBlock = 64;
constexpr int kCacheMaxDim = 256;
struct CacheArgs {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  int64_t n_pages, table_ld;
  int n_seqs, heads, dim, page_log2, block_log2, format;
};
struct StoreArgs {
  CacheArgs c;
  const void* k;
  const void* v;
  const int32_t* seq;   // nullptr: token t is of sequence t
  const int32_t* pos;
  const void* table;    // rotation (nullptr: none)
  unsigned* err;        // device error word
  const void* q;
  void* q_dst;
  int64_t T, ldk, ldv, ldq, ld_q_dst;
  int n_rot, halves, q_heads, type, vec;
  int wpu_log2;         // warps that share a block of a head
  int tpw, lane_inv;    // tokens a warp holds at a time; 65536 over a token's lanes, rounded up
  int small;            // blocks no longer than tpw, of a prompt
  int unit_groups;      // CTAs that have work for a block (small: for a window)
  int q_rows, q_slices; // heads a lane turns at a time; CTAs that share a window's queries
  int window;           // tokens that a CTA looks through, up to 32
};
int launch_store(const StoreArgs& a, int sms, cudaStream_t st, bool pdl);
struct LoadArgs {
  CacheArgs c;
  const int32_t* seq;
  const int32_t* pos;
  void* k;              // nullptr: not read back
  void* v;
  int64_t T, ldk, ldv;
  int type, vec;
};
int launch_load(const LoadArgs& a, cudaStream_t st, bool pdl);

// Attention (attend.cu): one launch of one phase.
enum { ATT_PART = 0, ATT_JOIN = 1 };
constexpr int kAttMaxTokens = 1 << 16;  // tokens of a call
struct AttendArgs {
  CacheArgs c;
  const void* q;
  void* dst;
  const int32_t* seq;
  const int32_t* pos;
  float* lse;           // [T][q_heads] or nullptr
  float* workspace;
  int64_t ldq, ld_dst;
  float scale;          // of q . k, times log2(e)
  int phase;
  int T, q_heads, group;
  int window;           // keys back from a token's own (0: all)
  int type, vec;        // vec: queries are read four elements at a time
  int tiles;            // of 8 rows an item has (1 or 2)
  int subs, rows;       // parts that the heads of a group fall into, heads of a part
  int run, tokens;      // tokens of a sequence expected next to each other; most tokens of an item
  int ctas;
};
int64_t attend_workspace_bytes(int dim, int tiles, int ctas);
int attend_ctas(int sms);  // two an SM
int launch_attend(const AttendArgs& a, cudaStream_t st, bool pdl);

// One kernel launch with every argument resolved: what a call plans, and what a
// prepared call keeps (gf_prepare) so that launching it does no planning at all.
enum {
  REC_FWHT = 0, REC_TC = 1, REC_STREAM = 2, REC_GENERIC = 3, REC_COPY = 4, REC_ROUTE = 5, REC_EXPERTS = 6,
  REC_LORA = 7, REC_EW = 8, REC_LIN = 9, REC_ROPE = 10, REC_STORE = 11, REC_LOAD = 12, REC_ATTEND = 13
};
struct LaunchRec {
  int kind;
  bool pdl;
  int wtype, ncols;  // REC_STREAM, REC_GENERIC
  union {            // by kind
    struct {         // REC_COPY: host staging copy (device-addressable pointers)
      const void* csrc;
      void* cdst;
      int64_t cbytes;
    };
    struct {  // REC_FWHT: stand-alone FWHT; REC_EW: element-wise op over fx and fsigns (fn elements)
      const float* fx;
      const float* fsigns;
      float* fdst;
      int64_t fn;
      int fB, fnsigns, ewop;
    };
    struct {  // REC_TC
      TcPlan tp;
      const void* W;  // the matrix of the tensor map
    };
    Plan p;   // REC_STREAM
    struct {  // REC_GENERIC
      GenericArgs g;
      int ggrid, gsmem;
    };
    RouteArgs route;
    ExpertsArgs experts;
    LoraArgs lora;
    LinArgs lin;
    RopeArgs rope;
    StoreArgs store;
    LoadArgs load;
    AttendArgs attend;
  };
};
// (a direct call plans into kMaxRecs of them on its stack)
static_assert(sizeof(LaunchRec) <= sizeof(Plan) + 16, "the streamed kernel's plan is the largest");
constexpr int kMaxRecs = 1 + kMaxSeg * (kMaxBatch / kMaxCols);  // transform + column blocks (per matrix)

// Shared by the entry points (api.cu, api_select.cu, api_attend.cu).
int64_t row_bytes_of(int wtype, int64_t K);
bool ranges_overlap(const void* a, int64_t abytes, const void* b, int64_t bbytes);
int cuda_fail(cudaError_t e);
DeviceLimits device_limits();
int issue(const LaunchRec& r, cudaStream_t st);
// A handle over n planned launches; a gf_status.
int make_prepared(const LaunchRec* recs, int n, gf_prepared** out);

unsigned* device_error_word();  // this device's error word (nullptr on failure)
int launch_selftest_wait(unsigned* err, uint64_t limit_ns, int* out, cudaStream_t st);

}  // namespace gf
