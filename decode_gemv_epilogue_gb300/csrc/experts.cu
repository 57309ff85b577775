// The chosen experts' gated product:
//   dst_t = aux_t + sum_j w_tj Wd_e (silu(Wg_e x_t) * (Wu_e x_t)),   e = ids_tj.
// A "slot" is one (token, choice) pair, s = t k + j.
//
// Tiled path, four launches chained with programmatic dependent launch:
//   prep     lists the slots of every expert (stable, so that nothing depends on the order
//            in which threads run), cuts them into column groups, and packs x;
//   gate/up  every chosen expert's gate and up rows are read once per column group; the
//            gated values go out packed for the next product;
//   down     the same for the down matrices, each slot's column times its weight;
//   combine  adds a token's slots in the order of its choices.
// Generic path, for shapes and alignments (and F32) that the tiles do not take: a warp per
// row of a slot's expert, weights decoded element by element, then the same combination.
#include <algorithm>

#include "tile_mma.cuh"

namespace gf {

constexpr int kExpGenericWarps = 8;

template <int WT>
__host__ __device__ constexpr int64_t expert_row_bytes(int64_t K) {
  return WT == WT_F32    ? 4 * K
         : WT == WT_F16  ? 2 * K
         : WT == WT_Q8_0 ? (K / 32) * 34
         : WT == WT_Q4_0 ? (K / 32) * 18
                         : (K / 256) * 144;
}

// GLU: h[s][m] = silu(Wg_e x_t) * (Wu_e x_t); otherwise y[s][m] = w_s Wd_e h_s.
template <int WT, bool GLU>
__global__ void __launch_bounds__(32 * kExpGenericWarps) experts_generic_kernel(const __grid_constant__ ExpertsArgs a) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.y;
  const int e = a.ids[s];
  if (e < 0 || e >= a.E) return;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kExpGenericWarps + (threadIdx.x >> 5);
  const int rows = GLU ? a.M : a.K, K = GLU ? a.K : a.M;
  if (row >= rows) return;
  const int64_t rb = expert_row_bytes<WT>(K), off = (static_cast<int64_t>(e) * rows + row) * rb;
  const float* x = GLU ? a.x + static_cast<int64_t>(s / a.k) * K
                       : reinterpret_cast<const float*>(a.hpack) + static_cast<int64_t>(s) * K;
  float g = 0.0f, u = 0.0f;
  for (int k = lane; k < K; k += 32) {
    const float xv = x[k];
    g = fmaf(decode_elem<WT>(a.W + off, k), xv, g);
    if constexpr (GLU) u = fmaf(decode_elem<WT>(a.W2 + off, k), xv, u);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    g += __shfl_xor_sync(0xffffffffu, g, o);
    if constexpr (GLU) u += __shfl_xor_sync(0xffffffffu, u, o);
  }
  if (lane == 0) {
    if constexpr (GLU)
      reinterpret_cast<float*>(a.hpack)[static_cast<int64_t>(s) * a.M + row] = tail_silu(g) * u;
    else
      a.y[static_cast<int64_t>(s) * a.K + row] = a.weights[s] * g;
  }
}

__global__ void __launch_bounds__(256) experts_combine_kernel(const __grid_constant__ ExpertsArgs a) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.y;
  const int m = blockIdx.x * 256 + threadIdx.x;
  if (m >= a.K) return;
  const int64_t o = static_cast<int64_t>(t) * a.K + m;
  float s = a.aux ? a.aux[o] : 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int e = a.ids[t * a.k + j];
    if (e >= 0 && e < a.E) s += a.y[static_cast<int64_t>(t * a.k + j) * a.K + m];
  }
  a.dst[o] = s;
}

static cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t st, bool pdl, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = st;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cfg;
}

// ------------------------------------------------------------------ lists and packed x
constexpr int kPrepThreads = 1024;
constexpr int kPrepMaxIter = kExpMaxTokens * kRouteMaxTopK / kPrepThreads;  // 32-slot steps of a warp

static int prep_smem(int E) { return 32 * E * 2 + E * 4 + 32 * 4; }

// The slots of each expert in slot order: a counting sort whose counts are kept per warp
// (each warp owns a run of consecutive slots) and ranked within a 32-slot step by matching.
__device__ void list_slots(const ExpertsArgs& a, uint16_t* cnt, uint32_t* offs, uint32_t* wsum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int S = a.T * a.k, run = ((S + 31) / 32 + 31) / 32 * 32;  // slots of a warp
  for (int i = threadIdx.x; i < 32 * a.E; i += kPrepThreads) cnt[i] = 0;
  __syncthreads();
  int ex[kPrepMaxIter], rank[kPrepMaxIter];
  uint16_t* mine = cnt + w * a.E;
#pragma unroll
  for (int j = 0; j < kPrepMaxIter; ++j) {
    ex[j] = -1;
    rank[j] = 0;
    if (32 * j < run) {
      const int s = w * run + 32 * j + lane;
      const int e = s < S ? a.ids[s] : -1;
      const bool valid = e >= 0 && e < a.E;
      const uint32_t same = __match_any_sync(0xffffffffu, valid ? e : -1);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int base = valid ? mine[e] : 0;
      __syncwarp();
      if (valid && before == 0) mine[e] = static_cast<uint16_t>(base + __popc(same));
      __syncwarp();
      if (valid) {
        ex[j] = e;
        rank[j] = base + before;
      }
    }
  }
  __syncthreads();
  // per expert: offsets of the warps' runs, then of the experts and of their column groups
  // (slots in the low half of a word, groups in the high one: both at most 8192 in all)
  const int e = threadIdx.x;
  uint32_t total = 0;
  if (e < a.E)
    for (int q = 0; q < 32; ++q) {
      const uint32_t c = cnt[q * a.E + e];
      cnt[q * a.E + e] = static_cast<uint16_t>(total);
      total += c;
    }
  const uint32_t ng = (total + a.cols - 1) / a.cols;
  const uint32_t v = total | (ng << 16);
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) wsum[w] = incl;
  __syncthreads();
  uint32_t before = 0;
  for (int q = 0; q < w; ++q) before += wsum[q];
  const uint32_t excl = before + incl - v;
  const uint32_t off = excl & 0xffffu, gbase = excl >> 16;
  if (e < a.E) {
    offs[e] = off;
    for (uint32_t i = 0; i < ng; ++i)
      a.groups[gbase + i] = make_int4(e, static_cast<int>(off + i * a.cols),
                                      static_cast<int>(min(static_cast<uint32_t>(a.cols), total - i * a.cols)), 0);
  }
  if (e == kPrepThreads - 1) *a.n_groups = static_cast<int>((before + incl) >> 16);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPrepMaxIter; ++j)
    if (ex[j] >= 0) a.slots[offs[ex[j]] + mine[ex[j]] + rank[j]] = w * run + 32 * j + lane;
}

// Column c of x packed with one scale for the whole column.
__device__ void pack_column(const float* x, int K, uint8_t* xp, float2* meta, bool swapped, float* wmax) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, n4 = K / 4;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
  auto load = [&](int i) -> float4 {
    if (vec) return reinterpret_cast<const float4*>(x)[i];
    return make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  };
  constexpr int kKeep = 2;  // groups of four a thread keeps between the two passes
  float4 keep[kKeep];
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int i = threadIdx.x + j * kPrepThreads;
    keep[j] = i < n4 ? load(i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    m = fmaxf(fmaxf(m, fmaxf(finite_abs(keep[j].x), finite_abs(keep[j].y))),
              fmaxf(finite_abs(keep[j].z), finite_abs(keep[j].w)));
  }
  for (int i = threadIdx.x + kKeep * kPrepThreads; i < n4; i += kPrepThreads) {
    const float4 v = load(i);
    m = fmaxf(fmaxf(m, fmaxf(finite_abs(v.x), finite_abs(v.y))), fmaxf(finite_abs(v.z), finite_abs(v.w)));
  }
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  if (lane == 0) wmax[w] = m;
  __syncthreads();
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(wmax[lane])));
  const float sc = pack_scale(m), inv = pow2_inverse(sc);
  auto put = [&](int i, float4 v) {
    v.x *= sc; v.y *= sc; v.z *= sc; v.w *= sc;
    float sum = (v.x + v.y) + (v.z + v.w);
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (i < n4) {
      reinterpret_cast<uint4*>(xp)[i] = pack_group(v, swapped);
      if ((i & 7) == 0) meta[i >> 3] = make_float2(inv, sum);
    }
  };
#pragma unroll
  for (int j = 0; j < kKeep; ++j) put(threadIdx.x + j * kPrepThreads, keep[j]);
  for (int i0 = kKeep * kPrepThreads; i0 < n4; i0 += kPrepThreads) {
    const int i = i0 + threadIdx.x;
    put(i, i < n4 ? load(i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f));
  }
}

__global__ void __launch_bounds__(kPrepThreads) experts_prep_kernel(const __grid_constant__ ExpertsArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) {
    uint32_t* offs = reinterpret_cast<uint32_t*>(smem);
    uint32_t* wsum = offs + a.E;
    list_slots(a, reinterpret_cast<uint16_t*>(wsum + 32), offs, wsum);
  } else {
    const int64_t c = blockIdx.x - 1;
    pack_column(a.x + c * a.K, a.K, a.xpack + c * a.K * 4, a.xmeta + c * expert_meta_stride(a.K), pack_swapped(a.wtype),
                reinterpret_cast<float*>(smem));
  }
}

// ------------------------------------------------------------------ tiled products
template <int WT, int MODE, int NT, int WR>
static cudaError_t launch_tile_t(const TileArgs& t, int grid, int smem, cudaStream_t st, bool pdl) {
  auto kern = tile_kernel<WT, MODE, NT, WR>;
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && configured[dev] < smem) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[dev] = smem;
  }
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>(grid)), 32 * (1 + kTileWarpsK * WR), st, pdl, &attr);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  return cudaLaunchKernelEx(&cfg, kern, t);
}

template <int WT, int MODE, int NT, int WR>
static cudaError_t launch_tile_shape(TileArgs t, const ExpertsArgs& a, cudaStream_t st, bool pdl) {
  constexpr int kCtas = (WR == 1 && NT <= 2) ? 2 : 1;  // CTAs per SM the registers allow
  const int stage = tile_stage_bytes<WT, NT>(WR, a.cols), fixed = kTileBarBytes + tile_red_bytes(WR);
  // as many CTAs per SM as leave each three stages
  int ctas = kCtas, ns = 0;
  for (; ctas >= 1; --ctas) {
    const int budget = ctas == 1 ? a.smem_optin : (a.smem_optin + 1024) / ctas - 1024;  // 1 KB a CTA is the system's
    ns = std::min(kTileMaxStages, (budget - fixed) / stage);
    if (ns >= 3 || ctas == 1) break;
  }
  if (ns < 2) return cudaErrorInvalidConfiguration;
  t.NS = ns;
  return launch_tile_t<WT, MODE, NT, WR>(t, ctas * a.sm_count, fixed + ns * stage, st, pdl);
}

template <int WT, int MODE>
static cudaError_t launch_tile_cols(const TileArgs& t, const ExpertsArgs& a, cudaStream_t st, bool pdl) {
  if (a.cols <= 8) return launch_tile_shape<WT, MODE, 1, 1>(t, a, st, pdl);
  if (a.cols <= 16) return launch_tile_shape<WT, MODE, 2, 1>(t, a, st, pdl);
  return launch_tile_shape<WT, MODE, 4, 1>(t, a, st, pdl);
}

template <int MODE>
static cudaError_t launch_tiles(const ExpertsArgs& a, cudaStream_t st, bool pdl) {
  TileArgs t = {};
  t.W = a.W;
  t.W2 = a.W2;
  t.rows = MODE == TILE_GLU ? a.M : a.K;
  t.K = MODE == TILE_GLU ? a.K : a.M;
  t.groups = a.groups;
  t.n_groups = a.n_groups;
  t.slots = a.slots;
  t.slot_div = MODE == TILE_GLU ? a.k : 1;
  t.xpack = MODE == TILE_GLU ? a.xpack : a.hpack;
  t.xmeta = MODE == TILE_GLU ? a.xmeta : a.hmeta;
  t.cols = a.cols;
  t.err = a.err;
  t.hpack = a.hpack;
  t.hmeta = a.hmeta;
  t.h_swapped = a.order;
  t.weights = a.weights;
  t.y = a.y;
  t.row_bytes = static_cast<int>(row_bytes_of(a.wtype, t.K));
  t.total_bytes = static_cast<int64_t>(a.E) * t.rows * t.row_bytes;
  switch (a.wtype) {
    case WT_F16: return launch_tile_cols<WT_F16, MODE>(t, a, st, pdl);
    case WT_Q8_0: return launch_tile_cols<WT_Q8_0, MODE>(t, a, st, pdl);
    case WT_Q4_0: return launch_tile_cols<WT_Q4_0, MODE>(t, a, st, pdl);
    case WT_Q4_K: return launch_tile_cols<WT_Q4_K, MODE>(t, a, st, pdl);
    default: return cudaErrorInvalidValue;
  }
}

template <bool GLU>
static cudaError_t launch_generic_phase(const ExpertsArgs& a, cudaStream_t st, bool pdl) {
  const int rows = GLU ? a.M : a.K;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>((rows + kExpGenericWarps - 1) / kExpGenericWarps),
                                             static_cast<unsigned>(a.T * a.k)),
                                        32 * kExpGenericWarps, st, pdl, &attr);
  switch (a.wtype) {
    case WT_F32: return cudaLaunchKernelEx(&cfg, experts_generic_kernel<WT_F32, GLU>, a);
    case WT_F16: return cudaLaunchKernelEx(&cfg, experts_generic_kernel<WT_F16, GLU>, a);
    case WT_Q8_0: return cudaLaunchKernelEx(&cfg, experts_generic_kernel<WT_Q8_0, GLU>, a);
    case WT_Q4_0: return cudaLaunchKernelEx(&cfg, experts_generic_kernel<WT_Q4_0, GLU>, a);
    case WT_Q4_K: return cudaLaunchKernelEx(&cfg, experts_generic_kernel<WT_Q4_K, GLU>, a);
    default: return cudaErrorInvalidValue;
  }
}

int launch_experts(const ExpertsArgs& a, cudaStream_t st, bool pdl) {
  cudaLaunchAttribute attr;
  switch (a.phase) {
    case EXP_PREP: {
      static int configured[64] = {0};
      int dev = 0;
      cudaGetDevice(&dev);
      const int smem = prep_smem(a.E);
      if (smem > 48 * 1024 && dev < 64 && configured[dev] < smem) {
        const cudaError_t e = cudaFuncSetAttribute(experts_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured[dev] = smem;
      }
      cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>(1 + a.T)), kPrepThreads, st, pdl, &attr);
      cfg.dynamicSmemBytes = static_cast<size_t>(smem);
      return cudaLaunchKernelEx(&cfg, experts_prep_kernel, a);
    }
    case EXP_GLU: return launch_tiles<TILE_GLU>(a, st, pdl);
    case EXP_DOWN: return launch_tiles<TILE_DOWN>(a, st, pdl);
    case EXP_GLU_GENERIC: return launch_generic_phase<true>(a, st, pdl);
    case EXP_DOWN_GENERIC: return launch_generic_phase<false>(a, st, pdl);
    case EXP_COMBINE: {
      const cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>((a.K + 255) / 256), static_cast<unsigned>(a.T)),
                                            256, st, pdl, &attr);
      return cudaLaunchKernelEx(&cfg, experts_combine_kernel, a);
    }
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gf
