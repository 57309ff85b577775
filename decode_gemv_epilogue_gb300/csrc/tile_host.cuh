// Host side of the tiled products (tile_mma.cuh): tensor maps, stages, launch.
#pragma once

#include <algorithm>

#include "tile_mma.cuh"

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
  if (MODE == TILE_GLU) e = tile_map<WT>(o.W2, o.all_rows, t.row_bytes, &m1);
  if (e != cudaSuccess) return e;
  const int stage = tile_stage_bytes<WT>(t.period, NT, t.cp), fixed = kTileHeadBytes + kTileRedBytes + 1024;
  // as many CTAs per SM as leave each three stages; 1 KB a CTA is the system's
  int ctas = tile_ctas(NT), ns = 0;
  for (; ctas >= 1; --ctas) {
    const int budget = ctas == 1 ? o.smem_optin : (o.smem_optin + 1024) / ctas - 1024;
    ns = std::min(kTileMaxStages, (budget - fixed) / stage);
    if (ns >= 3 || ctas == 1) break;
  }
  if (ns < 2 || o.max_groups / (ctas * o.sm_count) + 2 > kTileMaxGroups) return cudaErrorInvalidConfiguration;
  t.NS = ns;
  const int smem = fixed + ns * stage;
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && configured[dev] < smem) {
    const cudaError_t c = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (c != cudaSuccess) return c;
    configured[dev] = smem;
  }
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>(ctas * o.sm_count)), kTileThreads, st, pdl, &attr);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  return cudaLaunchKernelEx(&cfg, kern, m0, m1, t);
}

}  // namespace gf
