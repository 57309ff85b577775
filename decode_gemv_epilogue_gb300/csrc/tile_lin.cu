// The shared projection of a batch with adapters on the tensor cores: y = W x for all columns
// of the batch with the adapters' sums as the tail's addend (see tile_mma.cuh).
// Two launches: x packed (with the RMS normalisation, if any), the product; a third for the
// few rows at the end that a tensor map over several rows at once cannot reach.
#include "tile_host.cuh"

namespace gf {

__global__ void __launch_bounds__(kPackThreads) tile_pack_kernel(const __grid_constant__ LinArgs a) {
  __shared__ float wmax[kPackWords];
  pdl_wait();
  pdl_trigger();
  // a CTA a column
  const int col = static_cast<int>(blockIdx.x), tile = col / 8;
  const int first = tile * 8 / a.cols * a.cols;  // of the column group
  const int cp = min(8, min(a.cols, a.ncols - first));
  pack_column<kPackThreads>(a.x + static_cast<int64_t>(col) * a.K, col % 8, a.gamma, a.eps, a.K, a.wtype, cp,
              a.records + static_cast<int64_t>(tile) * (a.K / 32) * record_bytes(a.cp), wmax);
}

// The last rows of a matrix whose rows are no whole 16-byte words and whose number is no
// multiple of its period: a warp per (row, column).
template <int WT>
__global__ void __launch_bounds__(32) lin_tail_kernel(const __grid_constant__ LinArgs a, int row0) {
  pdl_wait();
  pdl_trigger();
  const int r = row0 + blockIdx.x, c = blockIdx.y, lane = threadIdx.x;
  const uint8_t* w = a.W + static_cast<int64_t>(r) * a.row_bytes;
  const float* x = a.x + static_cast<int64_t>(c) * a.K;
  float s = 0.0f, ss = 0.0f;
  for (int k = lane; k < a.K; k += 32) {
    float v = x[k];
    ss = fmaf(v, v, ss);
    if (a.gamma) v *= a.gamma[k];
    s = fmaf(decode_elem<WT>(w, k), v, s);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  if (lane == 0) {
    if (a.gamma) s *= 1.0f / sqrtf(ss / static_cast<float>(a.K) + a.eps);
    const int64_t o = static_cast<int64_t>(c) * a.M + r;
    a.dst[o] = apply_tail(a.epi, s, epi_takes_aux(a.epi) ? a.aux[o] : 0.0f);
  }
}

int lin_cols(int wtype, int64_t M, int64_t K, int row_bytes, int ncols, int sms) {
  if (ncols <= 8) return ncols;
  if (tile_plain(wtype)) return 16;
  int item_rows;
  return wide_takes(wtype, row_bytes) && wide_lin_cost(wtype, M, K, (ncols + 15) / 16, sms, &item_rows) <
                                             tile_lin_cost(wtype, M, K, (ncols + 7) / 8, sms)
             ? 16
             : 8;
}

template <int WT, bool PER1>
static int launch_lin_cols(const TileArgs& t, const LinArgs& a, cudaStream_t st, bool pdl) {
  const TileOperands o = {a.W, nullptr, t.rows, (a.ncols + a.cols - 1) / a.cols, a.sm_count, a.smem_optin};
  if constexpr (tile_plain(WT)) {
    if (a.cols > 8) return launch_tile<WT, TILE_LIN, 2, PER1>(t, o, st, pdl);
  } else if constexpr (PER1) {
    if (a.cols > 8) return launch_wide<WT, TILE_LIN>(t, o, st, pdl);
  }
  return launch_tile<WT, TILE_LIN, 1, PER1>(t, o, st, pdl);
}

int launch_lin(const LinArgs& a, cudaStream_t st, bool pdl) {
  cudaLaunchAttribute attr;
  if (a.phase == LIN_PACK) {
    const cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>(a.ncols)), kPackThreads, st, pdl, &attr);
    return cudaLaunchKernelEx(&cfg, tile_pack_kernel, a);
  }
  const int period = tile_period(a.row_bytes), main_rows = a.M / period * period;
  if (a.phase == LIN_TAIL) {
    const cudaLaunchConfig_t cfg =
        config(dim3(static_cast<unsigned>(a.M - main_rows), static_cast<unsigned>(a.ncols)), 32, st, pdl, &attr);
    return a.wtype == WT_Q8_0 ? cudaLaunchKernelEx(&cfg, lin_tail_kernel<WT_Q8_0>, a, main_rows)
                              : cudaLaunchKernelEx(&cfg, lin_tail_kernel<WT_Q4_0>, a, main_rows);
  }
  TileArgs t = {};
  t.rows = main_rows;
  t.K = a.K;
  t.row_bytes = a.row_bytes;
  t.period = period;
  t.records = a.records;
  t.cp = a.cp;
  t.err = a.err;
  t.out = a.dst;
  t.out_ld = a.M;
  t.aux = a.aux;
  t.epi = a.epi;
  t.ncols = a.ncols;
  t.group_cols = a.cols;
  if (!tile_plain(a.wtype)) wide_lin_cost(a.wtype, t.rows, a.K, (a.ncols + 15) / 16, a.sm_count, &t.item_rows);
  switch (a.wtype) {
    case WT_F32: return launch_lin_cols<WT_F32, true>(t, a, st, pdl);
    case WT_F16: return launch_lin_cols<WT_F16, true>(t, a, st, pdl);
    case WT_Q8_0: return period == 1 ? launch_lin_cols<WT_Q8_0, true>(t, a, st, pdl) : launch_lin_cols<WT_Q8_0, false>(t, a, st, pdl);
    case WT_Q4_0: return period == 1 ? launch_lin_cols<WT_Q4_0, true>(t, a, st, pdl) : launch_lin_cols<WT_Q4_0, false>(t, a, st, pdl);
    case WT_Q4_K: return launch_lin_cols<WT_Q4_K, true>(t, a, st, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gf
