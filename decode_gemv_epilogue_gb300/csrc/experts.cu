// The chosen experts' gated product:
//   dst_t = aux_t + sum_j w_tj Wd_e (silu(Wg_e x_t) * (Wu_e x_t)),   e = ids_tj.
// A "slot" is one (token, choice) pair, s = t k + j.
//
// Tiled path, four launches chained with programmatic dependent launch:
//   prep     lists the slots of every expert (stable, so that nothing depends on the order
//            in which threads run), cuts them into column groups, and packs x (two launches
//            where the list is long);
//   gate/up  every chosen expert's gate and up rows are read once per column group; the
//            gated values go out packed for the next product;
//   down     the same for the down matrices, each slot's column times its weight;
//   combine  adds a token's slots in the order of its choices.
// Generic path, for shapes and alignments that the tiles do not take: a warp per
// row of a slot's expert, weights decoded element by element, then the same combination.
#include <algorithm>

#include "tile_host.cuh"

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
                       : reinterpret_cast<const float*>(a.hrec) + static_cast<int64_t>(s) * K;
  float g = 0.0f, u = 0.0f, ss = 0.0f;
  for (int k = lane; k < K; k += 32) {
    float xv = x[k];
    if constexpr (GLU)
      if (a.gamma) {
        ss = fmaf(xv, xv, ss);
        xv *= a.gamma[k];
      }
    g = fmaf(decode_elem<WT>(a.W + off, k), xv, g);
    if constexpr (GLU) u = fmaf(decode_elem<WT>(a.W2 + off, k), xv, u);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    g += __shfl_xor_sync(0xffffffffu, g, o);
    if constexpr (GLU) {
      u += __shfl_xor_sync(0xffffffffu, u, o);
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
  }
  if constexpr (GLU)
    if (a.gamma) {
      const float inv = 1.0f / sqrtf(ss / static_cast<float>(K) + a.eps);
      g *= inv;
      u *= inv;
    }
  if (lane == 0) {
    if constexpr (GLU)
      reinterpret_cast<float*>(a.hrec)[static_cast<int64_t>(s) * a.M + row] = tail_silu(g) * u;
    else
      a.y[static_cast<int64_t>(s) * a.K + row] = a.weights[s] * g;
  }
}

// The gated values of slot s, a raw column (column c of `tile`), by the CTA that packed it.
template <int WT>
__device__ __forceinline__ void exact_gated(const ExpertsArgs& a, int s, int tile, uint32_t c, uint32_t cp) {
  const int64_t rb = expert_row_bytes<WT>(a.K);
  const uint8_t* rec = a.xrec + static_cast<int64_t>(tile) * (a.K / 32) * record_bytes(a.cp);
  if (threadIdx.x == 0) atomicAdd(a.err + 1, 1u);  // counted for gf_repair_count
#pragma unroll 1
  for (int b = threadIdx.x >> 5; b < a.M / 32; b += blockDim.x >> 5) {
    const int64_t at = (static_cast<int64_t>(a.ids[s]) * a.M + 32 * b) * rb;
    float g = 0.0f, u = 0.0f;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      g = u;
      u = exact_block<WT, 4>((i ? a.W2 : a.W) + at, rb, rec, c, cp, a.K);
    }
    write_gated(tail_silu(g) * u,
                a.hrec + static_cast<int64_t>(tile) * (a.M / 32) * record_bytes(a.cp) +
                    static_cast<int64_t>(b) * record_bytes(static_cast<int>(cp)),
                c, cp, a.out_format);
  }
}

// W: the down matrices, where their products are the tiles' (nullptr: the generic kernel's).  A
// product that a raw block among its gated values made NaN is taken again, element by element.
// (Six CTAs an SM, five of the packing: the code of raw columns must not cost the others their warps.)
template <int WT>
__global__ void __launch_bounds__(256, 6) experts_combine_kernel(const __grid_constant__ ExpertsArgs a) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.y;
  const int m = blockIdx.x * 256 + threadIdx.x;
  const bool in = m < a.K;
  const int64_t o = static_cast<int64_t>(t) * a.K + m;
  const float first = in && a.aux ? a.aux[o] : 0.0f;
  float s = first;
  if (in)
    for (int j = 0; j < a.k; ++j) {
      const int e = a.ids[t * a.k + j];
      if (e >= 0 && e < a.E) s += a.y[static_cast<int64_t>(t * a.k + j) * a.K + m];
    }
  // (the slots one by one only here: a look at each of them above took 9 -> 25 us of 256 tokens)
  const uint32_t odd = __ballot_sync(0xffffffffu, in && !is_finite(s));
  if (odd && a.W) {
    if (odd >> (threadIdx.x & 31) & 1u) s = first;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
      const int e = a.ids[t * a.k + j];
      if (e < 0 || e >= a.E) continue;
      float y = in ? a.y[static_cast<int64_t>(t * a.k + j) * a.K + m] : 0.0f;
      const int2 p = a.places[t * a.k + j];
      const uint32_t c = static_cast<uint32_t>(p.y) & 255u, cp = static_cast<uint32_t>(p.y) >> 8;
      const uint8_t* rec = a.hrec + static_cast<int64_t>(p.x) * (a.M / 32) * record_bytes(a.cp);
      bool raw = false;
      for (int b = threadIdx.x & 31; b < a.M / 32 && !is_finite(y); b += 32)
        raw |= *reinterpret_cast<const uint32_t*>(rec + b * record_bytes(static_cast<int>(cp)) + cp * 128u + c * 8u) == kRawBlock;
      if (__any_sync(0xffffffffu, raw)) {
        if ((threadIdx.x & 31) == 0) atomicAdd(a.err + 1, 1u);  // counted for gf_repair_count
        const int64_t rb = expert_row_bytes<WT>(a.M);
        const int m0 = m - static_cast<int>(threadIdx.x & 31);
        const float v = exact_block<WT, 2>(a.W + (static_cast<int64_t>(e) * a.K + m0) * rb, rb, rec, c, cp, a.M);
        if (!is_finite(y)) y = a.weights[t * a.k + j] * v;
      }
      if (odd >> (threadIdx.x & 31) & 1u) s += y;
    }
  }
  if (!in) return;
  a.dst[o] = s;
}

// ------------------------------------------------------------------ lists and packed x
constexpr int kPrepThreads = kPackThreads;
constexpr int kPrepMaxIter = kExpMaxTokens * kRouteMaxTopK / kPrepThreads;  // 32-slot steps of a warp

constexpr int kPackSlotThreads = 256;

static int prep_smem(int E) { return 32 * E * 2 + 3 * E * 4; }

// A short list (at most a slot a thread, groups of one column tile): every CTA packs one
// slot's column, and finds its place by counting over all slots; the first one writes the
// groups too.  Groups are numbered in the order of their first slots.
template <int WT>
__global__ void __launch_bounds__(kPackSlotThreads, 4) experts_prep_short_kernel(const __grid_constant__ ExpertsArgs a) {
  __shared__ int ids[kPackSlotThreads];
  __shared__ uint32_t leaders[kPackSlotThreads / 32];
  __shared__ int place[3];  // of this CTA's slot: group (-1: none), column, columns of the group
  __shared__ float wmax[kPackWords];
  pdl_wait();
  pdl_trigger();
  const int S = a.T * a.k, s = threadIdx.x, mine = blockIdx.x, lane = s & 31;
  int e = s < S ? a.ids[s] : -1;
  if (e >= a.E) e = -1;
  if (e < 0) e = -1;
  ids[s] = e;
  __syncthreads();
  // (a group has no more columns than its records have room for: a token may name an expert twice)
  const int width = a.cp;
  // slots of the same expert before this one, in all; the group's first; the next slot's column
  int before = 0, all = 0, first = 0, next = 0;
  if (e >= 0) {
    for (int q = 0; q < S; ++q) {
      const bool same = ids[q] == e;
      if (same && q <= s && next == 0) first = q;
      if (same && q < s) ++before;
      if (same) {
        ++all;
        next = next + 1 == width ? 0 : next + 1;
      }
    }
  }
  const uint32_t lead = __ballot_sync(0xffffffffu, e >= 0 && first == s);
  if (lane == 0) leaders[s >> 5] = lead;
  __syncthreads();
  if (e >= 0) {
    int g = __popc(leaders[first >> 5] & ((1u << (first & 31)) - 1u));
    for (int q = 0; q < (first >> 5); ++q) g += __popc(leaders[q]);
    const int col = before % width, count = min(width, all - (before - col));
    if (mine == 0) {
      a.slots[8 * g + col] = s;
      if (first == s) a.groups[g] = make_int4(e, 8 * g, count, g);
    }
    if (s == mine) {
      place[0] = g;
      place[1] = col;
      place[2] = count;
    }
  } else if (s == mine) {
    place[0] = -1;
  }
  if (mine == 0 && s == 0) {
    int n = 0;
    for (int q = 0; q < kPackSlotThreads / 32; ++q) n += __popc(leaders[q]);
    *a.n_groups = n;
  }
  __syncthreads();
  if (s == 0) a.places[mine] = place[0] < 0 ? make_int2(-1, 0) : make_int2(place[0], place[1] | (place[2] << 8));
  if (place[0] < 0) return;
  const bool raw = pack_column<kPackSlotThreads>(a.x + static_cast<int64_t>(mine / a.k) * a.K, place[1], a.gamma, a.eps,
                                                 a.K, WT, place[2],
                                                 a.xrec + static_cast<int64_t>(place[0]) * (a.K / 32) * record_bytes(a.cp),
                                                 wmax);
  if (raw) exact_gated<WT>(a, mine, place[0], static_cast<uint32_t>(place[1]), static_cast<uint32_t>(place[2]));
}

// The slots of each expert in slot order: a counting sort whose counts are kept per warp
// (each warp owns a run of consecutive slots) and ranked within a 32-slot step by matching.
// One CTA; a launch of a CTA per slot then packs.
__global__ void __launch_bounds__(kPrepThreads) experts_list_kernel(const __grid_constant__ ExpertsArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t wsum[32];
  uint32_t* offs = reinterpret_cast<uint32_t*>(smem);
  uint32_t *first_tile = offs + a.E, *totals = first_tile + a.E;
  uint16_t* cnt = reinterpret_cast<uint16_t*>(totals + a.E);
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int S = a.T * a.k;
  const int run = ((S + 31) / 32 + 31) / 32 * 32;  // slots of a warp
  const int nw = (S + run - 1) / run;              // warps that have some
  int ex[kPrepMaxIter], rank[kPrepMaxIter];
#pragma unroll
  for (int j = 0; j < kPrepMaxIter; ++j) {
    const int s = w * run + 32 * j + lane;
    ex[j] = 32 * j < run && s < S ? a.ids[s] : -1;
    if (ex[j] >= a.E) ex[j] = -1;
  }
  for (int i = threadIdx.x; i < nw * a.E; i += kPrepThreads) cnt[i] = 0;
  __syncthreads();
  uint16_t* mine = cnt + w * a.E;
#pragma unroll
  for (int j = 0; j < kPrepMaxIter; ++j) {
    rank[j] = 0;
    if (32 * j < run && w < nw) {
      const bool valid = ex[j] >= 0;
      const uint32_t same = __match_any_sync(0xffffffffu, valid ? ex[j] : -1);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int base = valid ? mine[ex[j]] : 0;
      __syncwarp();
      if (valid && before == 0) mine[ex[j]] = static_cast<uint16_t>(base + __popc(same));
      __syncwarp();
      rank[j] = base + before;
    }
  }
  __syncthreads();
  // per expert: offsets of the warps' runs, then of the experts and of their column tiles
  // (slots in the low half of a word, tiles in the high one: both at most 8192 in all)
  const int e = threadIdx.x;
  uint32_t total = 0;
  if (e < a.E)
    for (int q0 = 0; q0 < nw; q0 += 8) {
      uint32_t c[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) c[q] = q0 + q < nw ? cnt[(q0 + q) * a.E + e] : 0u;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (q0 + q < nw) cnt[(q0 + q) * a.E + e] = static_cast<uint16_t>(total);
        total += c[q];
      }
    }
  const uint32_t nt = (total + 7) / 8, gt = (a.cols + 7) / 8;  // column tiles of the expert, of a full group
  const uint32_t ng = (nt + gt - 1) / gt;
  auto scan = [&](uint32_t v, uint32_t& all) -> uint32_t {  // exclusive over the CTA
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) wsum[w] = incl;
    __syncthreads();
    const uint32_t ws = wsum[lane];
    uint32_t before = ws;  // every warp scans the warps' sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += up;
    }
    all = __shfl_sync(0xffffffffu, before, 31);
    const uint32_t mine_before = __shfl_sync(0xffffffffu, before - ws, w);
    __syncthreads();
    return mine_before + incl - v;
  };
  uint32_t all;
  const uint32_t ex0 = scan(total | (nt << 16), all);
  const uint32_t off = ex0 & 0xffffu, t0 = ex0 >> 16;
  if (e < a.E) {
    offs[e] = off;
    first_tile[e] = t0;
    totals[e] = total;
  }
  // every expert's first group, the largest, before the others'
  uint32_t experts, groups;
  const uint32_t g0 = scan(ng > 0 ? 1u : 0u, experts), g1 = experts + scan(ng > 0 ? ng - 1u : 0u, groups);
  for (uint32_t i = 0; i < ng; ++i) {
    const uint32_t f = i * gt * 8u;
    a.groups[i == 0 ? g0 : g1 + i - 1u] = make_int4(e, static_cast<int>(off + f), static_cast<int>(min(gt * 8u, total - f)),
                                                    static_cast<int>(t0 + i * gt));
  }
  if (threadIdx.x == 0) {
    a.n_groups[0] = static_cast<int>(experts + groups);
    a.n_groups[1] = a.n_groups[2] = 0;  // items of the two products taken
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPrepMaxIter; ++j) {
    const int s = w * run + 32 * j + lane;
    if (ex[j] >= 0) {
      const uint32_t f = mine[ex[j]] + rank[j], group = f / (gt * 8u) * (gt * 8u);  // among the expert's slots
      a.slots[offs[ex[j]] + f] = s;
      a.places[s] = make_int2(static_cast<int>(first_tile[ex[j]] + f / 8u),
                              static_cast<int>((f % 8u) | (min(8u, totals[ex[j]] - group) << 8)));
    } else if (32 * j < run && s < S) {
      a.places[s] = make_int2(-1, 0);
    }
  }
}

template <int WT>
__global__ void __launch_bounds__(kPackSlotThreads, 5) experts_pack_kernel(const __grid_constant__ ExpertsArgs a) {
  __shared__ float wmax[kPackWords];
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x;
  const int2 p = a.places[s];  // {column tile, column | columns stored << 8}
  if (p.x < 0) return;
  const bool raw = pack_column<kPackSlotThreads>(a.x + static_cast<int64_t>(s / a.k) * a.K, p.y & 255, a.gamma,
                                                 a.eps, a.K, WT, p.y >> 8,
                                                 a.xrec + static_cast<int64_t>(p.x) * (a.K / 32) * record_bytes(a.cp), wmax);
  if (raw) exact_gated<WT>(a, s, p.x, static_cast<uint32_t>(p.y) & 255u, static_cast<uint32_t>(p.y) >> 8);
}

// ------------------------------------------------------------------ tiled products
template <int WT, int MODE, bool PER1>
static int launch_tile_cols(const TileArgs& t, const ExpertsArgs& a, cudaStream_t st, bool pdl) {
  const TileOperands o = {a.W, a.W2, static_cast<int64_t>(a.E) * t.rows, a.max_tiles, a.sm_count, a.smem_optin};
  if constexpr (tile_plain(WT)) {
    if (a.cols > 16) return launch_tile<WT, MODE, 3, PER1>(t, o, st, pdl);
    if (a.cols > 8) return launch_tile<WT, MODE, 2, PER1>(t, o, st, pdl);
  } else if constexpr (PER1) {
    if (a.cols > 8) return launch_wide<WT, MODE>(t, o, st, pdl);
  }
  return launch_tile<WT, MODE, 1, PER1>(t, o, st, pdl);
}

template <int MODE>
static int launch_tiles(const ExpertsArgs& a, cudaStream_t st, bool pdl) {
  TileArgs t = {};
  t.rows = MODE == TILE_GLU ? a.M : a.K;
  t.K = MODE == TILE_GLU ? a.K : a.M;
  t.row_bytes = static_cast<int>(row_bytes_of(a.wtype, t.K));
  t.period = tile_period(t.row_bytes);
  t.groups = a.groups;
  t.n_groups = a.n_groups;
  t.max_groups = a.T * a.k;
  t.next = reinterpret_cast<uint32_t*>(a.n_groups) + (MODE == TILE_GLU ? 1 : 2);
  t.slots = a.slots;
  t.records = MODE == TILE_GLU ? a.xrec : a.hrec;
  t.cp = a.cp;
  t.err = a.err;
  t.out_records = a.hrec;
  t.out_format = a.out_format;
  t.factors = a.weights;
  t.out = a.y;
  t.out_ld = t.rows;
  switch (a.wtype) {
    case WT_F32: return launch_tile_cols<WT_F32, MODE, true>(t, a, st, pdl);
    case WT_F16: return launch_tile_cols<WT_F16, MODE, true>(t, a, st, pdl);
    case WT_Q8_0:
      return t.period == 1 ? launch_tile_cols<WT_Q8_0, MODE, true>(t, a, st, pdl)
                           : launch_tile_cols<WT_Q8_0, MODE, false>(t, a, st, pdl);
    case WT_Q4_0:
      return t.period == 1 ? launch_tile_cols<WT_Q4_0, MODE, true>(t, a, st, pdl)
                           : launch_tile_cols<WT_Q4_0, MODE, false>(t, a, st, pdl);
    case WT_Q4_K: return launch_tile_cols<WT_Q4_K, MODE, true>(t, a, st, pdl);
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

// The kernels that hold the raw columns' code, one for each format.
struct ExpertsShort {
  template <int WT>
  static constexpr auto kernel() { return experts_prep_short_kernel<WT>; }
};
struct ExpertsPack {
  template <int WT>
  static constexpr auto kernel() { return experts_pack_kernel<WT>; }
};
struct ExpertsCombine {
  template <int WT>
  static constexpr auto kernel() { return experts_combine_kernel<WT>; }
};
template <class KERNEL>
static cudaError_t launch_wt(const ExpertsArgs& a, const cudaLaunchConfig_t& cfg) {
  switch (a.wtype) {
    case WT_F32: return cudaLaunchKernelEx(&cfg, KERNEL::template kernel<WT_F32>(), a);
    case WT_F16: return cudaLaunchKernelEx(&cfg, KERNEL::template kernel<WT_F16>(), a);
    case WT_Q8_0: return cudaLaunchKernelEx(&cfg, KERNEL::template kernel<WT_Q8_0>(), a);
    case WT_Q4_0: return cudaLaunchKernelEx(&cfg, KERNEL::template kernel<WT_Q4_0>(), a);
    case WT_Q4_K: return cudaLaunchKernelEx(&cfg, KERNEL::template kernel<WT_Q4_K>(), a);
    default: return cudaErrorInvalidValue;
  }
}

int launch_experts(const ExpertsArgs& a, cudaStream_t st, bool pdl) {
  cudaLaunchAttribute attr;
  switch (a.phase) {
    case EXP_PREP: {
      const cudaLaunchConfig_t pack =
          config(dim3(static_cast<unsigned>(a.T * a.k)), kPackSlotThreads, st, pdl, &attr);
      // (fewer than eight tokens always come this way: their groups are narrower than a column
      // tile; measured, 8 and 42 slots: 6.5 us through the list, 3.7 and 4.6 so)
      if (a.T * a.k <= kPackSlotThreads && a.cols <= 8) return launch_wt<ExpertsShort>(a, pack);
      static SmemLimit limit;
      cudaError_t e = limit.raise(reinterpret_cast<const void*>(experts_list_kernel));
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t list = config(dim3(1), kPrepThreads, st, pdl, &attr);
      list.dynamicSmemBytes = static_cast<size_t>(prep_smem(a.E));
      e = cudaLaunchKernelEx(&list, experts_list_kernel, a);
      if (e != cudaSuccess) return e;
      cudaLaunchAttribute behind;
      const cudaLaunchConfig_t cfg = config(pack.gridDim, kPackSlotThreads, st, true, &behind);
      return launch_wt<ExpertsPack>(a, cfg);
    }
    case EXP_GLU: return launch_tiles<TILE_GLU>(a, st, pdl);
    case EXP_DOWN: return launch_tiles<TILE_DOWN>(a, st, pdl);
    case EXP_GLU_GENERIC: return launch_generic_phase<true>(a, st, pdl);
    case EXP_DOWN_GENERIC: return launch_generic_phase<false>(a, st, pdl);
    case EXP_COMBINE: {
      const cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>((a.K + 255) / 256), static_cast<unsigned>(a.T)),
                                            256, st, pdl, &attr);
      return launch_wt<ExpertsCombine>(a, cfg);
    }
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gf
