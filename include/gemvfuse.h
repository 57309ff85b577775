/*
 * gemvfuse -- decode-path GEMV with a fused element-wise epilogue and a signed
 * Walsh-Hadamard prologue, for GB300 (sm_103a).  C ABI.
 *
 * Operations defined by the pages this library restates (cited by title, section):
 *  [EPI]  "feat(cuda): fuse activations and residual add into mmv f/q epilogues",
 *         Summary / What changed: y = W x for one output column (ncols_dst == 1), with
 *         the tail sigmoid | silu | silu(y)*m | y + r folded into the GEMV; a reshape
 *         between the product and the tail is an index identity; the destination may
 *         alias the mul/add operand (same element index) but never the product inputs.
 *  [FWHT] "vulkan: fuse the sign multiply into the Hadamard FWHT", Overview: the sign
 *         vector is multiplied in while the row is loaded, before the transform, and is
 *         broadcast over its own length.
 *  [CPU]  "ggml-cpu: fuse element-wise epilogues (ADD, MUL, SILU) into
 *         ggml_compute_forward_mul_mat", Guards / Correctness: epilogue operands are F32,
 *         same shape, contiguous; F32/F16/Q8_0/Q4_0 weights; fused == unfused values.
 *         What: the SwiGLU gate (MUL_MAT + SILU) and the gate x up product (MUL_MAT +
 *         MUL) of one FFN -- taken together as the gated dual GEMV gemv_glu() -- and
 *         the RMS_NORM + MUL pair ahead of a matmul (the RMS-normalisation prologue).
 *
 * Conventions for every entry point:
 *  - All array pointers are DEVICE pointers owned by the caller (gf_copy's may also be
 *    pinned host memory).  The library never allocates, frees or keeps a pointer after
 *    the call returns, except for handles: a prepared call keeps its pointers (host
 *    memory only), and a step graph owns its CUDA graph.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  Work is enqueued
 *    asynchronously; the call returns once it is launched.
 *  - Arguments are validated on the host before anything is launched.  A non-zero
 *    return means nothing was launched, except GF_ERR_CUDA (launch failure; see
 *    gf_last_cuda_error()).
 *  - Vectors are contiguous float32.  A batch of ncols columns is column-major:
 *    x is [ncols][K], aux and dst are [ncols][M].
 *  - The library holds no state between calls other than per-device launch limits,
 *    a device error word (see gf_device_status()), a repair counter
 *    (gf_repair_count()) and a host-side cache of encoded tensor maps (address, shape
 *    and box of recent tensor-core operands; an entry never goes stale, as it holds
 *    no data).
 */
#ifndef GEMVFUSE_H
#define GEMVFUSE_H

#include <stdint.h>

#if defined(__GNUC__)
#define GF_API __attribute__((visibility("default")))
#else
#define GF_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Weight storage formats; each row of W holds K elements, rows are contiguous.
 *  GF_F32  : float32 [M][K].
 *  GF_F16  : IEEE binary16 [M][K].
 *  GF_Q8_0 : per 32 elements a 34-byte block {binary16 d; int8 q[32]}; w = d*q.
 *  GF_Q4_0 : per 32 elements an 18-byte block {binary16 d; uint8 qs[16]}; byte j holds
 *            element j (low nibble) and element j+16 (high nibble); w = d*(nibble-8).
 *  GF_Q4_K : per 256 elements a 144-byte super-block {binary16 d; binary16 dmin;
 *            uint8 scales[12]; uint8 qs[128]}: eight 32-element sub-blocks j with 6-bit
 *            scale sc[j] and min m[j] (scales[j] low 6 bits = sc[j], scales[j+4] low 6
 *            bits = m[j] for j < 4; for j >= 4 the low 4 bits are the low/high nibble of
 *            scales[j+4] and the top 2 bits those of scales[j-4] / scales[j]); qs holds
 *            four 32-byte groups, group g sub-block 2g in the low nibbles and 2g+1 in the
 *            high nibbles; w = d*sc[j]*q - dmin*m[j].  K % 256 == 0.
 * (Format names from [CPU] Correctness; the layouts are the ggml block convention.) */
typedef enum { GF_F32 = 0, GF_F16 = 1, GF_Q8_0 = 2, GF_Q4_0 = 3, GF_Q4_K = 4 } gf_wtype;

/* Fused tails ([EPI] What changed; [CPU] What):
 *  NONE      dst = y
 *  SIGMOID   dst = 1/(1+exp(-y))
 *  SILU      dst = y*sigmoid(y)
 *  SILU_MUL  dst = silu(y)*aux          (aux = the per-row activation_mul operand)
 *  ADD       dst = y + aux              (residual add; dst == aux allowed, in place) */
typedef enum {
  GF_EPI_NONE = 0, GF_EPI_SIGMOID = 1, GF_EPI_SILU = 2, GF_EPI_SILU_MUL = 3, GF_EPI_ADD = 4
} gf_epilogue;

/* Stand-alone element-wise ops (the unfused control path): dst[i] = op(a[i], b[i % nb]). */
typedef enum { GF_EW_SIGMOID = 1, GF_EW_SILU = 2, GF_EW_MUL = 3, GF_EW_ADD = 4 } gf_ewop;

typedef enum {
  GF_OK = 0,
  GF_ERR_INVALID = -1,      /* bad enum, size, null pointer or view shape            */
  GF_ERR_ALIAS = -2,        /* dst overlaps an input it may not alias                */
  GF_ERR_UNSUPPORTED = -3,  /* valid but outside what is implemented (e.g. K%32 != 0 */
                            /* for a block format, ncols > 256, FWHT block > 8192)   */
  GF_ERR_ALIGN = -4,        /* pointer not aligned to its element type               */
  GF_ERR_CUDA = -5,         /* a CUDA runtime call or launch failed                  */
  GF_ERR_TIMEOUT = -6       /* a kernel gave up on a bounded wait (device status)    */
} gf_status;

/* gf_opts.flags */
#define GF_FLAG_PDL 1u   /* launch with programmatic dependent launch: the kernel may
                            start while the previous kernel in `stream` still runs and
                            streams W before waiting for it.  Only valid when no kernel
                            still running in `stream` writes W. */
#define GF_FLAG_NO_TENSOR_CORES 4u  /* use the CUDA-core kernels only.  By default F16 weights
                            with 3 or more columns (16 per launch), K % 64 == 0 and
                            16-byte aligned W and x run on the tensor cores: tcgen05 MMAs
                            of the f16 weights with x split into scaled f16 hi + lo parts,
                            fp32 accumulation. */
#define GF_FLAG_NO_SPLIT_K 2u  /* never split K over a cluster of CTAs (by default a GEMV
                            with M <= SMs/2 rows gives each row range to a cluster of
                            2..8 CTAs that each stream a slice of K and add their
                            partial sums in a fixed order through distributed shared
                            memory; the result is deterministic either way, but the
                            summation order, hence the rounding, differs). */

typedef struct {
  int64_t ncols;             /* columns in the batch, 1..256 (0 is read as 1); up to 8 */
                             /* share one pass over W, wider batches run as blocks of 8 */
  const float* fwht_signs;   /* non-NULL: signed-FWHT prologue on every column of x     */
  int64_t fwht_block;        /* FWHT block B: power of two, 1..8192, K % B == 0         */
  int64_t nsigns;            /* length of fwht_signs; K % nsigns == 0; element k of a   */
                             /* column uses fwht_signs[k % nsigns]                      */
  int64_t view_ne[4];        /* optional view of each dst column (all 0 = none); the    */
                             /* product of the non-zero entries must equal M. A view of */
                             /* contiguous memory is an index identity ([EPI] What      */
                             /* changed: result written with the matmul geometry).      */
  uint32_t flags;            /* GF_FLAG_*                                              */
  float* fwht_workspace;     /* optional device buffer of ncols*K floats (16-byte       */
                             /* aligned, overlapping no other argument).  Given, the    */
                             /* prologue runs once as a stand-alone transform into it   */
                             /* and the GEMV reads it, chained with programmatic        */
                             /* dependent launch; NULL: every CTA transforms x on chip. */
  const float* rms_norm_weight;  /* non-NULL: RMS-normalisation prologue on every column */
                             /* of x: x'_c = x_c / sqrt(mean_k(x_c[k]^2) + eps) * gamma, */
                             /* gamma = rms_norm_weight [K] (device float32, overlapping */
                             /* no output).  Not combinable with the FWHT prologue       */
                             /* (GF_ERR_UNSUPPORTED).                                    */
  float rms_norm_eps;        /* eps of the normalisation: finite, >= 0                 */
} gf_opts;

/* y = W x with the fused tail, one column.  [EPI] Summary, What changed.
 *  W    : device, M rows in format `wtype` (see gf_wtype).  Alignment: 4 B for F32,
 *         2 B otherwise; 16 B (and K % 256 == 0 for block formats) selects the
 *         TMA-streamed fast kernel, anything else the generic kernel.
 *  x    : device float32 [K].           aux : device float32 [M], required iff the
 *  dst  : device float32 [M].                 epilogue is SILU_MUL or ADD.
 *  Aliasing: dst may equal aux exactly; any other overlap of dst with W, x or aux
 *  returns GF_ERR_ALIAS.  M == 0 launches nothing.  K == 0 gives y = 0. */
GF_API int gemv_fused(const void* W, int wtype, const float* x, int64_t M, int64_t K,
               int epilogue, const float* aux, float* dst, void* stream);

/* gemv_fused plus the options in `opts` (may be NULL): a batch of ncols independent
 * columns sharing one pass over W; the signed-FWHT prologue
 *     x'_c[b*B + j] = (1/sqrt(B)) sum_t H_B[j][t] s[(b*B + t) % nsigns] x_c[b*B + t]
 * (Sylvester H, [FWHT] Overview) applied to each column before the product -- on chip
 * in every CTA, or once into opts->fwht_workspace; the dst view check; and
 * GF_FLAG_PDL.  fwht_signs must not overlap dst.  With a workspace two kernels are
 * launched (the transform, then the GEMV). */
GF_API int gemv_fused_ex(const void* W, int wtype, const float* x, int64_t M, int64_t K,
                  int epilogue, const float* aux, float* dst, const gf_opts* opts,
                  void* stream);

/* Gated dual GEMV, the gate and up projections of one FFN in a single pass:
 *     dst_c[i] = silu(G_i . x'_c) * (U_i . x'_c),   silu(g) = g / (1 + exp(-g))
 * ([CPU] What: MUL_MAT + SILU on the gate, then MUL by the up projection; [EPI] Summary
 * names this gated branch, which it leaves to its own GLU path).  W_gate and W_up are
 * two M x K matrices of the same format `wtype` (same rules as W of gemv_fused); x'
 * is x after the prologue chosen in `opts` (none, signed FWHT, RMS normalisation).
 * Every tile the kernel streams holds rows of both matrices, so each weight byte is
 * read once and the gate result never leaves the chip.  opts may be NULL; its ncols,
 * prologues, view and flags apply as in gemv_fused_ex.  dst may not overlap W_gate,
 * W_up, x or the prologue operands. */
GF_API int gemv_glu(const void* W_gate, const void* W_up, int wtype, const float* x, int64_t M,
                    int64_t K, float* dst, const gf_opts* opts, void* stream);

/* Several matrices that share x, in one pass (no counterpart on the pages; it carries
 * their fusion one step further): for each item i,
 *     dst_i = epilogue_i(W_i x')          (x' = x after the prologue in `opts`)
 * e.g. a layer's q, k and v projections (and a small gate such as a sigmoid head) on the
 * same activations, without concatenating their weights.  One launch streams every
 * matrix once, as one matrix of sum_i M_i rows: the fixed cost of a launch is paid once.
 *  items : n items (1 <= n <= GF_MULTI_MAX, else GF_ERR_INVALID / GF_ERR_UNSUPPORTED),
 *          each a matrix W (M rows of format `wtype`, K columns; the rules of W in
 *          gemv_fused) with its own epilogue, aux ([ncols][M], required iff SILU_MUL or
 *          ADD) and dst ([ncols][M]).
 *  x, K, wtype, opts : shared; opts as in gemv_fused_ex (ncols, either prologue,
 *          flags) except `view_ne`, which must be all zero.
 *  Aliasing: each dst as in gemv_fused against its own operands, and it may not overlap
 *  any other item's W, aux or dst (GF_ERR_ALIAS).  The results equal those of the n
 *  separate calls bit for bit (the same per-row arithmetic).  Shapes the streamed kernel
 *  cannot take in one pass run as one launch per matrix. */
#define GF_MULTI_MAX 4
typedef struct {
  const void* W;
  int64_t M;
  int epilogue;
  const float* aux;
  float* dst;
} gf_multi_item;
GF_API int gemv_multi(const gf_multi_item* items, int n, int wtype, const float* x, int64_t K,
                      const gf_opts* opts, void* stream);

/* Prepared calls: plan once, launch many times.  A decode loop issues the same GEMVs
 * with the same buffers every step; gf_prepare / gf_prepare_glu validate and plan a
 * call exactly as gemv_fused_ex / gemv_glu would (same arguments, same rules, same
 * status codes) and keep every launch argument, so gf_launch_prepared only issues the
 * kernels: no validation, planning or allocation per step.  The results are the ones
 * the direct call gives (the same kernels with the same arguments).
 *  out      : receives a handle owned by the caller, released with gf_free_prepared;
 *             NULL on failure.  A call with M == 0 gives a handle that launches nothing.
 *  (gf_prepare_multi plans gemv_multi the same way.)
 *  Buffers  : the handle holds the device pointers given here (W, x, aux, dst, opts'
 *             signs, workspace and RMS weight); their contents may change between
 *             launches, the allocations must stay valid while the handle is used.
 *  Device   : the handle belongs to the device current at gf_prepare; launching it
 *             with another device current returns GF_ERR_INVALID. */
typedef struct gf_prepared gf_prepared;
GF_API int gf_prepare(const void* W, int wtype, const float* x, int64_t M, int64_t K, int epilogue,
                      const float* aux, float* dst, const gf_opts* opts, gf_prepared** out);
GF_API int gf_prepare_glu(const void* W_gate, const void* W_up, int wtype, const float* x, int64_t M,
                          int64_t K, float* dst, const gf_opts* opts, gf_prepared** out);
GF_API int gf_prepare_multi(const gf_multi_item* items, int n, int wtype, const float* x, int64_t K,
                            const gf_opts* opts, gf_prepared** out);
/* Issues the launches of calls[0], ..., calls[n-1] in order on `stream` (n >= 0; the
 * calls' GF_FLAG_PDL settings apply as given to gf_prepare).  Stops at the first
 * failing launch and returns its status; GF_ERR_INVALID (nothing launched) for a NULL
 * handle or one prepared on another device. */
GF_API int gf_launch_prepared(const gf_prepared* const* calls, int n, void* stream);
/* Releases a handle (NULL is ignored).  Launches already issued are not affected. */
GF_API void gf_free_prepared(gf_prepared* p);

/* Host staging of a decode step by a kernel instead of the copy engine, so that a step's
 * input upload, its GEMVs and its result download can be one stream sequence or one CUDA
 * graph (gf_graph_create takes the handle of gf_prepare_copy like any prepared call).
 * Copies `bytes` bytes from src to dst; each range may be device memory of the current
 * device, managed memory, or pinned host memory (cudaHostAlloc / cudaMallocHost, or
 * registered with cudaHostRegister).
 *  - src and dst 16-byte aligned (GF_ERR_ALIGN), bytes >= 0 and a multiple of 16
 *    (GF_ERR_INVALID), the ranges disjoint (GF_ERR_ALIAS); pageable host memory, or
 *    device memory of another device: GF_ERR_INVALID (nothing launched).  bytes == 0
 *    launches nothing.
 *  - flags: GF_FLAG_PDL launches it with programmatic dependent launch; the kernel
 *    waits for the preceding grid before reading src, so it may read what that grid
 *    wrote, and the next launch may start early (every kernel of this library waits
 *    before reading what a preceding grid writes).
 *  - Host memory written here is complete when the stream (or graph launch) is; the
 *    copy uses no copy engine and is not ordered with copies in other streams. */
GF_API int gf_copy(void* dst, const void* src, int64_t bytes, uint32_t flags, void* stream);
GF_API int gf_prepare_copy(void* dst, const void* src, int64_t bytes, uint32_t flags, gf_prepared** out);

/* A decode step as one launch: gf_graph_create records the launches of calls[0..n)
 * (n >= 1, in order, as gf_launch_prepared would issue them, programmatic dependent
 * launches included) into a CUDA graph and instantiates it; gf_graph_launch replays it
 * on `stream` -- one host call for the whole sequence, and the launch overhead of a
 * graph instead of one per kernel.  The graph keeps the prepared calls' arguments
 * (the handles may be freed afterwards; their buffers must stay allocated).  It belongs
 * to the device current at creation (another one: GF_ERR_INVALID).  Errors: NULL or
 * foreign handles GF_ERR_INVALID; a failing capture or instantiation GF_ERR_CUDA. */
typedef struct gf_graph gf_graph;
GF_API int gf_graph_create(const gf_prepared* const* calls, int n, gf_graph** out);
GF_API int gf_graph_launch(const gf_graph* g, void* stream);
GF_API void gf_graph_free(gf_graph* g);

/* Allocation-free variant of gemv_fused_ex with the signed-FWHT prologue.  The pages
 * have no counterpart: this entry point exists for callers that cannot allocate a
 * device workspace -- a C host that links only this library and has no device
 * allocator of its own, or a serving process whose device memory is fixed at start-up
 * and may not grow while requests run.  It computes exactly what gemv_fused_ex computes
 * with opts = {ncols, fwht_signs, fwht_block, nsigns, flags} and a workspace, but the
 * workspace (the transformed x', ncols*K floats) is a static device array inside the
 * library; nothing is allocated or freed.
 *  - Limit: ncols*K <= GF_NOALLOC_MAX_WORKSPACE_FLOATS, else GF_ERR_UNSUPPORTED with
 *    nothing launched.  fwht_signs must be non-NULL (GF_ERR_INVALID otherwise).
 *  - The array (1 MiB) is held on every GPU that loads the library until the process
 *    exits.  The first call on a device looks up its address (cudaGetSymbolAddress,
 *    with that device current); make that first call before any stream capture.
 *  - Every call on a device shares the one array and overwrites it before reading it;
 *    calls whose work overlaps on the GPU (e.g. on different streams without ordering)
 *    race on it and give undefined results: order them, e.g. on one stream.
 *  - The address is kept for the life of the process.  Destroying the device's primary
 *    context (cudaDeviceReset) invalidates it, as it does the library's device error
 *    word: after a reset, reload the library before calling it again. */
#define GF_NOALLOC_MAX_WORKSPACE_FLOATS 262144
GF_API int gemv_fused_fwht_noalloc(const void* W, int wtype, const float* x, int64_t M, int64_t K,
                                   int epilogue, const float* aux, float* dst, int64_t ncols,
                                   const float* fwht_signs, int64_t fwht_block, int64_t nsigns,
                                   uint32_t flags, void* stream);

/* ---- Products whose weights are chosen per column (no counterpart on the pages; the
 * operators a decode step with a mixture of experts or with per-request adapters needs
 * next to the products above).  The conventions of this header hold: device pointers,
 * checks before any launch, nothing allocated; each call has a prepared form. */

/* Routing: for each token t (a row of E logits, `ld` elements apart)
 *     s = softmax(l_t)  or  1 / (1 + exp(-l_t));      key_e = s_e + bias_e
 *     with n_group > 1: the experts form n_group groups of E / n_group neighbours; a group's
 *         score is its largest key (group_top 1) or the sum of its two largest (group_top 2;
 *         one where only one is choosable); the topk_group best groups stay
 *     ids_t     = the top_k experts of the largest keys, descending
 *     weights_t = scale * s of those, first divided by their sum if `norm`
 * Ties (of keys and of group scores) go to the lowest index; which of two near keys is the
 * larger is decided in 64 bits.  Without a bias the order is that of the logits.  Logits of
 * -inf or NaN (and keys made so by the bias) are never chosen and count for nothing; +inf
 * counts as the largest float.  Places that find no expert get id -1 and weight 0, so a
 * wholly masked row gives only those.
 *  ids : int32 [T][top_k], weights : float32 [T][top_k]; neither may overlap an input or the
 *  other.  T == 0 launches nothing.
 *  Limits (GF_ERR_UNSUPPORTED beyond): E <= 1024, top_k <= 32, n_group <= 32, T <= 2^24.
 *  GF_ERR_INVALID: E < 1, top_k < 1 or > E, n_group not dividing E, topk_group outside
 *  1..n_group, group_top not 1 or 2, 0 < ld < E, a scale that is not finite.  */
typedef enum { GF_SCORE_SOFTMAX = 0, GF_SCORE_SIGMOID = 1 } gf_score;
typedef struct {
  int64_t top_k;
  int score;           /* gf_score                                                  */
  int norm;            /* non-zero: divide the chosen weights by their sum          */
  float scale;         /* factor of every weight (0 is read as 1)                   */
  const float* bias;   /* [E], added for the choice only; NULL: none                */
  int64_t n_group;     /* 0 or 1: no groups                                         */
  int64_t topk_group;  /* groups that stay (read only with n_group > 1)             */
  int group_top;       /* keys a group's score is made of: 1 or 2 (n_group > 1)     */
  int64_t ld;          /* elements between rows of logits; 0: E                     */
  uint32_t flags;      /* GF_FLAG_PDL                                               */
} gf_route_opts;
GF_API int gf_route(const float* logits, int64_t T, int64_t E, const gf_route_opts* opts, int32_t* ids,
                    float* weights, void* stream);
GF_API int gf_prepare_route(const float* logits, int64_t T, int64_t E, const gf_route_opts* opts, int32_t* ids,
                            float* weights, gf_prepared** out);

/* The gated feed-forward product of the chosen experts:
 *     dst_t = aux_t + sum_j weights_tj * Wd_e (silu(Wg_e x'_t) * (Wu_e x'_t)),   e = ids_tj
 * for T tokens, each chosen expert's matrices read once for all the tokens that take it
 * (up to 24 at a time).  The sums of a token run over j in order: deterministic.
 *  W_gate, W_up : E matrices of M rows and K columns one after another, format `wtype`;
 *  W_down       : E matrices of K rows and M columns, format `wtype_down`.
 *  ids          : int32 [T][top_k]; a value outside 0..E-1 takes no expert and adds nothing.
 *  weights      : float32 [T][top_k].          x : [T][K].
 *  x'           : x, or with rms_norm_weight its RMS normalisation (as in gf_opts).
 *  aux          : [T][K] or NULL (0); dst == aux is allowed (in place).
 *  workspace    : device memory of at least gf_experts_workspace() bytes, 256-byte aligned,
 *                 contents undefined before and after; not shared by calls that may overlap.
 *  Shapes: K and M multiples of 32 (256 for a Q4_K matrix's columns) with 16-byte aligned
 *  matrices take the tiled kernels on the tensor cores (x and the gated values as f16 hi + lo
 *  parts), anything else, and GF_FLAG_NO_TENSOR_CORES, the generic ones in 32 bits.
 *  dst may not overlap W_*, x, ids, weights, rms_norm_weight or the workspace; the workspace
 *  no argument.
 *  Limits (GF_ERR_UNSUPPORTED beyond): T <= 256, top_k <= 32, E <= 1024, M and K <= 2^20,
 *  columns no whole number of the format's blocks.  T == 0 or K == 0 launches nothing. */
typedef struct {
  const void* W_gate;
  const void* W_up;
  const void* W_down;
  int wtype, wtype_down;
  int64_t E, M, K;
  const int32_t* ids;
  const float* weights;
  int64_t top_k;
  void* workspace;
  int64_t workspace_bytes;
  const float* rms_norm_weight;  /* [K] or NULL: no normalisation of x              */
  float rms_norm_eps;
  uint32_t flags;      /* GF_FLAG_PDL, GF_FLAG_NO_TENSOR_CORES (the generic kernels) */
} gf_experts;
GF_API int gemv_experts(const gf_experts* ex, const float* x, int64_t T, const float* aux, float* dst,
                        void* stream);
GF_API int gf_prepare_experts(const gf_experts* ex, const float* x, int64_t T, const float* aux, float* dst,
                              gf_prepared** out);
/* Which kernels gemv_experts would launch for these arguments (host only, launches nothing):
 * 0 = none, 2 = generic, 4 = tiled, <0 = the gf_status the call would return.  `info` (may be
 * NULL) receives of the tiled kernels {columns a group may have, wide kernel for gate and up
 * (0, 1), wide kernel for down (0, 1)}. */
GF_API int gf_plan_experts(const gf_experts* ex, const float* x, int64_t T, const float* aux, const float* dst,
                           int64_t info[8]);
/* Bytes of workspace for these sizes (any format); negative: a gf_status. */
GF_API int64_t gf_experts_workspace(int64_t E, int64_t T, int64_t top_k, int64_t M, int64_t K);

/* A shared projection with a low-rank adapter per column:
 *     dst_c = tail(W x'_c + scales_a * B_a (A_a x'_c), aux_c),   a = ids_c
 * i.e. gemv_fused_ex (W .. dst, opts as there) with the adapters' products added before the
 * tail.  x' is x after the prologue in `opts`; the FWHT prologue needs opts->fwht_workspace
 * (GF_ERR_UNSUPPORTED without).
 *  A      : n matrices of rank rows and K columns, B : n matrices of M rows and rank columns,
 *           one after another, format atype (GF_F16 or GF_F32).
 *  ids    : int32 [ncols]; a value outside 0..n-1 takes no adapter (dst_c = tail(W x'_c)).
 *  scales : float32 [n] or NULL (1).
 *  workspace : device memory of at least gf_lora_workspace() bytes, 256-byte aligned,
 *           contents undefined before and after.
 *  Limits: rank 1..256 (GF_ERR_INVALID below, GF_ERR_UNSUPPORTED above).  dst may not
 *  overlap A, B, ids, scales or the workspace; the workspace no argument. */
typedef struct {
  const void* A;
  const void* B;
  int atype;
  int64_t n, rank;
  const int32_t* ids;
  const float* scales;
  void* workspace;
  int64_t workspace_bytes;
} gf_lora;
GF_API int gemv_lora(const void* W, int wtype, const float* x, int64_t M, int64_t K, int epilogue, const float* aux,
                     float* dst, const gf_lora* lora, const gf_opts* opts, void* stream);
GF_API int gf_prepare_lora(const void* W, int wtype, const float* x, int64_t M, int64_t K, int epilogue,
                           const float* aux, float* dst, const gf_lora* lora, const gf_opts* opts, gf_prepared** out);
/* Which kernel gemv_lora would run the shared product on (host only, launches nothing): as
 * gf_plan, or 4 = tiled.  `info` (may be NULL) is gf_plan's, or of the tiled kernels {columns
 * a group may have, wide kernel (0, 1)}. */
GF_API int gf_plan_lora(const void* W, int wtype, const float* x, int64_t M, int64_t K, int epilogue, const float* aux,
                        const float* dst, const gf_lora* lora, const gf_opts* opts, int64_t info[8]);
/* Bytes of workspace for these sizes (any format); negative: a gf_status. */
GF_API int64_t gf_lora_workspace(int64_t ncols, int64_t M, int64_t K, int64_t rank, int64_t n);

/* ---- Attention of a decode step over a cache held in 8 bits (no counterpart on the pages): what
 * stands between a layer's q, k, v products and its output projection.  The conventions of this header
 * hold; each call has a prepared form.  Vectors here are rows of heads, [T][heads][dim], float32 or
 * binary16 (`type`: GF_F32, GF_F16), rows `ld` elements apart (0: dense).
 *
 * Tokens are named by two lists on the device, which may change between launches of a prepared call:
 * token t of a call is position pos[t] of sequence seq[t] (seq == NULL: of sequence t). */

/* Rotary positions.  A pair (a, b) of a head at position p becomes
 *     m (a cos(p f) - b sin(p f)),  m (a sin(p f) + b cos(p f)),      pair i: f_i = base^(-2i / n_rot)
 * HALVES: the pair is elements (i, i + n_rot/2) of the head; PAIRS: (2i, 2i + 1).  Elements from n_rot
 * on stay.  Frequencies and m are held in a table that a program makes once (gf_rope_table):
 *  PLAIN  : f_i.       LINEAR : f_i / factor.
 *  RAMP   : (1 - r) f_i + r f_i / factor, r rising linearly in i from 0 at the pair that makes `fast`
 *           turns over `span` positions, i = floor(x(fast)), to 1 at i = ceil(x(slow)), with x(turns) =
 *           n_rot/2 * ln(span / (2 pi turns)) / ln(base); floor and ceil are held within 0..n_rot - 1.
 *  BANDS  : (1 - r) f_i + r f_i / factor, r falling linearly in the turns span f_i / 2 pi, from 1 at
 *           `slow` and fewer to 0 at `fast` and more.
 *  divisors[i] (device float32 [n_rot/2] or NULL) divides f_i last.
 *  m = magnitude, or where that is 0: 0.1 ln(factor) + 1 for RAMP with factor > 1, else 1.
 * Frequencies are computed in 64 bits and held as 64-bit fractions of a turn; the product with a 32-bit
 * position is exact, and so is the quarter turn that is taken off it before the rest is rounded to 32 bits.  An
 * angle is off by 2^-28 turns (2^-24 of its distance from that quarter turn), and by the frequency's own error, some
 * 2^-49 of the whole angle: 2^-18 radians at position 2^31.  A negative position turns back. */
typedef enum { GF_ROPE_HALVES = 0, GF_ROPE_PAIRS = 1 } gf_rope_layout;
typedef enum { GF_ROPE_PLAIN = 0, GF_ROPE_LINEAR = 1, GF_ROPE_RAMP = 2, GF_ROPE_BANDS = 3 } gf_rope_kind;
typedef struct {
  double base;             /* > 1                                                    */
  int kind;                /* gf_rope_kind                                           */
  double factor;           /* > 0; read unless PLAIN                                 */
  int64_t span;            /* positions of the unscaled context (RAMP, BANDS)        */
  double fast, slow;       /* turns over the span, fast > slow > 0 (RAMP, BANDS)     */
  double magnitude;        /* of cosine and sine; 0: see above                       */
  const float* divisors;
} gf_rope_freqs;
/* Bytes of a table, and its making (16-byte aligned, on the device): n_rot even, 2..1024. */
GF_API int64_t gf_rope_table_bytes(int64_t n_rot);
GF_API int gf_rope_table(void* table, int64_t n_rot, const gf_rope_freqs* freqs, void* stream);
typedef struct {
  const void* table;   /* made for n_rot, else nothing is written (gf_device_status) */
  int64_t n_rot;       /* elements of a head that turn; 0: all                       */
  int layout;          /* gf_rope_layout                                             */
  int type;            /* of x and dst (gf_rope only)                                */
  int64_t ld, ld_dst;  /* gf_rope only                                               */
  uint32_t flags;      /* GF_FLAG_PDL (gf_rope only)                                 */
} gf_rope_opts;
/* dst = x rotated by pos (int32 [T]).  dst == x with equal ld is allowed, no other overlap.  dim 2..1024,
 * T <= 2^20, heads <= 1024. */
GF_API int gf_rope(const void* x, int64_t T, int64_t heads, int64_t dim, const int32_t* pos, const gf_rope_opts* opts,
                   void* dst, void* stream);
GF_API int gf_prepare_rope(const void* x, int64_t T, int64_t heads, int64_t dim, const int32_t* pos,
                           const gf_rope_opts* opts, void* dst, gf_prepared** out);

/* A cache of keys and values in pages of `page` tokens, one byte an element and a float32 scale for every
 * `block` tokens of a page and head:
 *   k, v             : [n_pages][heads][page][dim] codes, 16-byte aligned
 *   k_scale, v_scale : [n_pages][heads][page / block]
 *   table            : int32 [n_seqs][table_ld]; position p of sequence s lies in page table[s][p / page]
 * A value is code * scale.  I8: codes -127..127, scales of 12 significant bits; E4M3: 4-bit exponents and
 * 3-bit mantissas up to 448, scales that are powers of two.  Codes that are no values (E4M3's NaN, which the library
 * does not write) may reach rows that share the reading of their keys.
 *  Limits (GF_ERR_UNSUPPORTED beyond): page 16..2^20 and block 1..64, powers of two, block <= page; dim a
 *  multiple of 16 up to 256; heads <= 1024; page * table_ld <= 2^30.
 * A token has no place where its seq is outside 0..n_seqs - 1, its pos below 0 or not under page *
 * table_ld, or the page outside 0..n_pages - 1: such rows (of a padded batch) are not stored, load as
 * zeros, and see no keys. */
typedef enum { GF_CACHE_I8 = 0, GF_CACHE_E4M3 = 1 } gf_cache_format;
typedef struct {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int format;
  int64_t n_pages, heads, page, dim, block;
  const int32_t* table;
  int64_t n_seqs, table_ld;
} gf_cache;

/* Writes T tokens' keys and values [T][heads][dim].  With opts->rope the keys are rotated by their
 * position first, and the queries q [T][q_heads][dim], if given, into q_dst (q_dst == q allowed).
 * For every block of tokens of a head that is written to, with a the largest magnitude of its new values:
 *     need  = the least scale of the format with 127 (E4M3: 448) * need >= a, within 2^-112..2^121 (2^119)
 *     scale = need, or where the block holds earlier tokens the larger of need and its scale before
 *     code  = value / scale rounded to the nearest code, ties to even
 * and where the scale grew, the earlier tokens' codes become code * old scale / scale, rounded the same
 * way.  A block holds earlier tokens if its first position of this call is not its first one; later
 * positions of it count as new.  A value that is not finite makes its block's scale NaN: the block reads
 * back as NaN until its first position is written again.
 * Tokens of one sequence stand next to each other in the call, each at the position behind the one before it
 * (else the blocks concerned hold some of the values, and nothing else is touched).
 * More than 256 tokens with a list of sequences are taken for prompts, without one for a token of each: only speed
 * depends on it.
 * n_rot must be a multiple of 8 here (GF_ERR_UNSUPPORTED); T <= 2^20, q_heads <= 1024.  No argument may
 * overlap the cache's arrays, and q_dst no input but q (rows of one fused q, k, v buffer may lie between
 * each other). */
typedef struct {
  int type;                   /* of k, v, q, q_dst                                    */
  int64_t ldk, ldv;
  const gf_rope_opts* rope;   /* table, n_rot and layout are read; NULL: no rotation  */
  const void* q;              /* NULL: none (must be NULL without rope)               */
  void* q_dst;
  int64_t q_heads, ldq, ld_q_dst;
  uint32_t flags;             /* GF_FLAG_PDL                                          */
} gf_store_opts;
GF_API int gf_cache_store(const gf_cache* cache, const void* k, const void* v, int64_t T, const int32_t* seq,
                          const int32_t* pos, const gf_store_opts* opts, void* stream);
GF_API int gf_prepare_cache_store(const gf_cache* cache, const void* k, const void* v, int64_t T, const int32_t* seq,
                                  const int32_t* pos, const gf_store_opts* opts, gf_prepared** out);

/* Reads T tokens' keys and values back as [T][heads][dim] (k or v may be NULL: not wanted).  The outputs
 * overlap nothing else.  T <= 2^20. */
typedef struct {
  int type;
  int64_t ldk, ldv;
  uint32_t flags;  /* GF_FLAG_PDL */
} gf_load_opts;
GF_API int gf_cache_load(const gf_cache* cache, int64_t T, const int32_t* seq, const int32_t* pos,
                         const gf_load_opts* opts, void* k, void* v, void* stream);
GF_API int gf_prepare_cache_load(const gf_cache* cache, int64_t T, const int32_t* seq, const int32_t* pos,
                                 const gf_load_opts* opts, void* k, void* v, gf_prepared** out);

/* Attention of T tokens over the cache: query head h of token t sees the keys of head h / (q_heads / heads)
 * at positions max(0, pos - window + 1) .. pos of its sequence,
 *     s_j = scale * q . K_j,   dst = sum_j softmax(s)_j V_j,   lse = ln sum_j exp(s_j)
 * in 32-bit arithmetic.  q is taken as pairs of binary16, to 2^-22 of an element or 2^-39 of its row's largest; so
 * are the softmax's weights (1 for the largest) times their values' scales: to 2^-22 of each, or 2^-30 of the scale,
 * or, where the scales of neighbouring keys lie more than 2^8 apart, 2^-31 of the largest weight times scale that
 * the row has met.  Weights below 2^-126 are zero, and a key whose score times log2(e) leaves the
 * finite numbers downwards has none.  The tokens' own keys have been stored before.
 * Positions in pages that the table does not have are not seen; a row that sees nothing (of a token without a
 * place, for instance) is 0, its lse -inf.  A token whose pos reaches beyond the table sees what lies in it.
 *  q, dst    : [T][q_heads][dim]; q_heads a multiple of heads, <= 1024.  T <= 2^16, and T * q_heads times
 *              (page * table_ld / 16 + 4) <= 2^51.
 *  run       : how many tokens of one sequence stand next to each other (drafted tokens, a prompt's part;
 *              0 or 1: a decode step).  They then share one reading of the keys.  Only speed depends on it.
 *  workspace : device memory of at least gf_attend_workspace() bytes, 256-byte aligned, contents undefined
 *              before and after; not shared by calls that may overlap.
 *  dst, lse and the workspace overlap nothing else. */
typedef struct {
  int type;
  int64_t ldq, ld_dst;
  float scale;          /* > 0; 0: 1 / sqrt(dim)                                      */
  int64_t window;       /* keys that a token sees, itself among them; 0: all          */
  int64_t run;
  float* lse;           /* [T][q_heads] or NULL                                       */
  void* workspace;
  int64_t workspace_bytes;
  uint32_t flags;       /* GF_FLAG_PDL                                                */
} gf_attend_opts;
GF_API int gf_attend(const gf_cache* cache, const void* q, int64_t T, int64_t q_heads, const int32_t* seq,
                     const int32_t* pos, const gf_attend_opts* opts, void* dst, void* stream);
GF_API int gf_prepare_attend(const gf_cache* cache, const void* q, int64_t T, int64_t q_heads, const int32_t* seq,
                             const int32_t* pos, const gf_attend_opts* opts, void* dst, gf_prepared** out);
/* Bytes of workspace for these sizes on the current device; negative: a gf_status. */
GF_API int64_t gf_attend_workspace(int64_t T, int64_t q_heads, int64_t heads, int64_t dim, int64_t run);

/* Signed FWHT, stand-alone ([FWHT] Overview): for every block of `block` consecutive
 * elements of x[0..n), dst_b = H_block (x_b * s) / sqrt(block), with element i using
 * signs[i % nsigns]; signs == NULL means all +1 (the plain normalised transform).
 *  block : power of two, 1..16384, n % block == 0;  n % nsigns == 0 when signs != NULL.
 *  dst == x is allowed (in place); other overlaps with x or signs: GF_ERR_ALIAS. */
GF_API int fwht_signed(const float* x, const float* signs, float* dst, int64_t n,
                int64_t block, int64_t nsigns, void* stream);

/* Unfused control ([CPU] Correctness compares fused against unfused outputs):
 * dst[i] = op(a[i], b[i % nb]) for i < n; SIGMOID and SILU ignore b.  Uses the same
 * device functions as the fused tails.  dst may equal a or b exactly. */
GF_API int gf_elementwise(int op, const float* a, const float* b, int64_t nb, float* dst,
                   int64_t n, void* stream);

/* Test hook: out[i*K + k] = decoded W[i][k] as float32, through the same unit decoders
 * the fast GEMV kernel uses.  Every decoded value is exact in float32. */
GF_API int gf_dequantize(const void* W, int wtype, int64_t M, int64_t K, float* out, void* stream);

/* Which kernel gemv_fused_ex would launch for these arguments (host only, launches
 * nothing): 0 = none (M == 0), 1 = TMA-streamed kernel, 2 = generic kernel, 3 = tensor-core
 * kernel (F16 batches), <0 = the gf_status the call would return.  `info` (may be NULL) receives
 *   {grid, block_threads, stage_rows, stages, k_chunk, smem_bytes, row_chunk,
 *    ctas_per_cluster (split K; 1 = no split)}. */
GF_API int gf_plan(const void* W, int wtype, const float* x, int64_t M, int64_t K, int epilogue,
            const float* aux, const float* dst, const gf_opts* opts, int64_t info[8]);

/* gf_plan for gemv_glu. */
GF_API int gf_plan_glu(const void* W_gate, const void* W_up, int wtype, const float* x, int64_t M,
                       int64_t K, const float* dst, const gf_opts* opts, int64_t info[8]);

/* Failure-path self-test (no GEMV): one GPU thread waits, through the same bounded wait
 * every kernel uses, on a barrier that nothing completes.  After limit_us microseconds
 * (1..1000000) the wait gives up, sets the device error word (gf_device_status then
 * reports GF_ERR_TIMEOUT) and the kernel returns; the context stays usable.  out: device
 * int[4] = {first wait succeeded (0), second wait succeeded (0: it returns at once on the
 * abort flag), microseconds spent in the first wait, microseconds in the second}. */
GF_API int gf_selftest_wait_timeout(int64_t limit_us, int* out, void* stream);

/* Device error word of the current device: GF_OK, GF_ERR_TIMEOUT if a kernel gave up
 * on a bounded wait since the last reset, or GF_ERR_INVALID if gf_rope or gf_cache_store
 * met a rotation table of another n_rot than its own (it then wrote nothing).
 * Synchronises with the device.  reset != 0 clears it. */
GF_API int gf_device_status(int reset);

/* Row chunks (a CTA's rows of one launch, or of one row chunk of it) whose sums the
 * single-column Q4_0 / Q8_0 / Q4_K kernels recomputed in fp32 because some 16-element
 * unit of x could not be carried by their integer dot products (an outlier far above
 * the values around it, or a NaN / Inf): a count since the last reset, on the current
 * device.  Such a launch reads its weights twice; the count says how often that
 * happens for a workload.  The tiled kernels of gemv_experts and gemv_lora count here too: a
 * column of packed x that they do not carry (a NaN / Inf, or an outlier far above an eighth of
 * the other values), once for the gated products of an
 * expert and once for every 32 rows of a shared projection, and every output of a down product
 * computed again; such a call takes many times as long.  Synchronises with the device; reset != 0 clears it.
 * Negative: a gf_status (GF_ERR_CUDA). */
GF_API int64_t gf_repair_count(int reset);

/* Human-readable name of a gf_status value. */
GF_API const char* gf_status_string(int status);

/* cudaError_t of the last failing CUDA call made by this library in this thread. */
GF_API int gf_last_cuda_error(void);

/* Library ABI version. */
GF_API int gf_version(void);

#ifdef __cplusplus
}
#endif
#endif /* GEMVFUSE_H */
