// Host side of the tiled products (tile_mma.cuh): tensor maps, stages, launch.
#pragma once

#include <algorithm>
#include <cmath>

#include "tile_wide.cuh"

namespace gf {

inline cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t st, bool pdl, cudaLaunchAttribute* attr) {
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

// Tensor map over the rows of all matrices of one kind.
template <int WT>
int tile_map(const void* W, int64_t all_rows, int row_bytes, CUtensorMap* out) {
  if (WT == WT_F16)
    return cached_map_2d(W, kMapF16, static_cast<uint64_t>(row_bytes / 2), static_cast<uint64_t>(all_rows), 64, 32, true, out);
  if (WT == WT_F32)
    return cached_map_2d(W, kMapF32, static_cast<uint64_t>(row_bytes / 4), static_cast<uint64_t>(all_rows), 32, 32, true, out);
  const int p = tile_period(row_bytes);
  return cached_map_2d(W, kMapF16, static_cast<uint64_t>(row_bytes) * p / 2, static_cast<uint64_t>(all_rows / p),
                       static_cast<uint32_t>(tile_pitch<WT>(p) / 2), static_cast<uint32_t>(32 / p), false, out);
}

struct TileOperands {
  const void* W;
  const void* W2;
  int64_t all_rows;       // of all matrices of W
  int max_groups;         // upper bound on the column groups
  int sm_count, smem_optin;
};

template <int WT, int MODE, int NT, bool PER1>
int launch_tile(TileArgs t, const TileOperands& o, cudaStream_t st, bool pdl) {
  auto kern = tile_kernel<WT, MODE, NT, PER1>;
  CUtensorMap m0, m1;
  int e = tile_map<WT>(o.W, o.all_rows, t.row_bytes, &m0);
  if (e != cudaSuccess) return e;
  m1 = m0;
  t.W = static_cast<const uint8_t*>(o.W);
  if (MODE == TILE_GLU) e = tile_map<WT>(o.W2, o.all_rows, t.row_bytes, &m1);
  if (e != cudaSuccess) return e;
  // The columns' records of whole groups where they leave three chunks of weights or more, in
  // two buffers where those leave a stage more, with as many CTAs per SM as the registers allow;
  // else the records go with the weights.  1 KB a CTA is the system's.
  const int fixed = kTileHeadBytes + kTileRedBytes + 1024;
  const int64_t xb = tile_x_bytes(t.K, NT, t.cp);
  int ctas = tile_ctas(WT, NT), ns = 0, stage = 0;
  int64_t x_all = 0;
  auto plan = [&](int n, int buffers, int want) {
    const int budget = n == 1 ? o.smem_optin : (o.smem_optin + 1024) / n - 1024;
    if (fixed + buffers * xb >= budget) return false;
    stage = tile_chunks(WT, NT) * tile_stage_bytes<WT>(t.period, NT, t.cp, buffers > 0);
    ns = static_cast<int>(std::min<int64_t>(kTileMaxStages, (budget - fixed - buffers * xb) / stage));
    ctas = n;
    t.xbuffers = buffers;
    x_all = buffers * xb;
    return ns >= want;
  };
  const int most = tile_ctas(WT, NT);
  constexpr int kFew = tile_chunks(WT, NT) == 2 ? 2 : 3;  // stages
  if (!plan(most, 2, kFew + 1) && !plan(most, 1, kFew) && !plan(most, 0, kFew) && !plan(1, 1, kFew)) plan(1, 0, 2);
  if (ns < 2 || o.max_groups / (ctas * o.sm_count) + 2 > kTileMaxGroups) return cudaErrorInvalidConfiguration;
  t.NS = ns;
  const int smem = fixed + static_cast<int>(x_all) + ns * stage;
  static SmemLimit limit;
  e = limit.raise(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>(ctas * o.sm_count)), kTileThreads, st, pdl, &attr);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  return cudaLaunchKernelEx(&cfg, kern, m0, m1, t);
}

// The wide kernel takes block formats whose rows are whole 16-byte words.
inline bool wide_takes(int wt, int row_bytes) { return !tile_plain(wt) && row_bytes % 16 == 0; }

// Time of a product of `rows` outputs and K columns over `groups` column groups, in units of
// one K-sharing item: items run in waves of as many as fit the device (the K-sharing kernel's
// many small ones level out, the wide kernel's few large ones do not).  A wide item takes as
// long as 3.7 K-sharing ones of 64 rows and 8 columns, 2.6 for Q8_0 with half the rows
// (measured at 14336 x 4096: 67, 46 and 18 us).
inline double tile_cost(int64_t rows, int64_t K, int tile_rows, double groups, int sms) {
  const double items = groups * static_cast<double>((rows + tile_rows - 1) / tile_rows);
  return static_cast<double>(K) * std::max(1.0, items / (2.0 * sms));
}
inline double wide_cost(int wt, int64_t rows, int64_t K, int tile_rows, double groups, int sms) {
  const double items = groups * static_cast<double>((rows + tile_rows - 1) / tile_rows);
  return static_cast<double>(K) * (wt == WT_Q8_0 ? 2.6 : 3.7) * std::ceil(items / sms);
}
inline int wide_rows(int wt) { return wt == WT_Q8_0 ? 32 * wide_warps<WT_Q8_0>() : 32 * wide_warps<WT_Q4_0>(); }

// A batch's items are alike and handed out in equal shares, so what counts is how many a CTA gets:
// fewer rows an item where that saves a wave or fills one.  An item's time goes by the warps that
// share a scheduler (Q4_0, K 4096: 64 us with 16 warps, 62 with 14, 50 with 12 or 10, 40 with 8):
// the rows of 16, 12 or 8 warps (Q8_0: 8).  64 columns of 14336 x 4096 with rank-16 adapters:
// 90 us, 76, 107.
inline double wide_lin_cost(int wt, int64_t rows, int64_t K, double groups, int sms, int* item_rows) {
  const int most = wide_rows(wt) / 32;
  double best = 0.0;
  for (int n = most; n >= 8; n -= 4) {
    const double items = groups * static_cast<double>((rows + 32 * n - 1) / (32 * n));
    const double us = std::ceil(items / sms) * (wt == WT_Q8_0 ? 46.0 : 16.0 + 3.0 * n) * static_cast<double>(K) / 4096.0;
    if (n == most || us < best) {
      best = us;
      *item_rows = 32 * n;
    }
  }
  return best;
}
// The K-sharing kernel's for the same, in groups of 8: 5 us and, by format, 11 to 15 a wave.  Whole
// calls with rank-16 adapters, this kernel and the wide one: Q4_0, 32 columns of 14336 x 4096 55
// us and 60, 48 of 11008 x 4096 68 and 62, 48 of 14336 x 4096 86 and 73; Q4_K, the same 64 and
// 64, 80 and 66, 92 and 78; Q8_0, 256 of 4096 x 4096 144 and 131.
inline double tile_lin_cost(int wt, int64_t rows, int64_t K, double groups, int sms) {
  const double items = groups * static_cast<double>((rows + kTileRows - 1) / kTileRows);
  const double wave = wt == WT_Q4_0 ? 11.0 : wt == WT_Q4_K ? 12.0 : 15.0;
  return (5.0 + wave * std::max(1.0, items / (2.0 * sms))) * static_cast<double>(K) / 4096.0;
}

template <int WT, int MODE>
int launch_wide(TileArgs t, const TileOperands& o, cudaStream_t st, bool pdl) {
  auto kern = wide_kernel<WT, MODE>;
  CUtensorMap m0, m1;
  int e = tile_map<WT>(o.W, o.all_rows, t.row_bytes, &m0);
  if (e != cudaSuccess) return e;
  m1 = m0;
  t.W = static_cast<const uint8_t*>(o.W);
  if (MODE == TILE_GLU) e = tile_map<WT>(o.W2, o.all_rows, t.row_bytes, &m1);
  if (e != cudaSuccess) return e;
  const int stage = wide_stage_bytes<WT>(), fixed = kTileHeadBytes + wide_xchg<WT>() + 1024;
  t.NS = std::min(kTileMaxStages, (o.smem_optin - fixed) / stage);
  if (t.NS < 2) return cudaErrorInvalidConfiguration;
  const int smem = fixed + t.NS * stage;
  static SmemLimit limit;
  e = limit.raise(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>(o.sm_count)), 32 * (1 + wide_warps<WT>()), st, pdl, &attr);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  return cudaLaunchKernelEx(&cfg, kern, m0, m1, t);
}

}  // namespace gf
