// The shared projection of a batch with adapters on the tensor cores: y = W x for all columns
// of the batch with the adapters' sums as the tail's addend (block formats; see
// tile_mma.cuh).  Two launches: x packed (with the RMS normalisation, if any), the product.
#include "tile_host.cuh"

namespace gf {

__global__ void __launch_bounds__(kPackThreads) tile_pack_kernel(const __grid_constant__ LinArgs a) {
  __shared__ float wmax[2 * kPackThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tile = static_cast<int>(blockIdx.x), col = tile * 8 + threadIdx.x / kPackColumn;
  const int first = tile * 8 / a.cols * a.cols;  // of the column group
  const int cp = min(8, min(a.cols, a.ncols - first));
  pack_tile(col < a.ncols ? a.x + static_cast<int64_t>(col) * a.K : nullptr, a.gamma, a.eps, a.K, a.wtype, cp,
            a.records + static_cast<int64_t>(blockIdx.x) * (a.K / 32) * record_bytes(a.cp), wmax);
}

template <int WT>
static int launch_lin_cols(const TileArgs& t, const LinArgs& a, cudaStream_t st, bool pdl) {
  const TileOperands o = {a.W, nullptr, a.M, (a.ncols + a.cols - 1) / a.cols, a.sm_count, a.smem_optin};
  if (a.cols <= 8) return launch_tile<WT, TILE_LIN, 1, true>(t, o, st, pdl);

  return launch_wide<WT, TILE_LIN>(t, o, st, pdl);
}

int launch_lin(const LinArgs& a, cudaStream_t st, bool pdl) {
  if (a.phase == LIN_PACK) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(dim3(static_cast<unsigned>((a.ncols + 7) / 8)), kPackThreads, st, pdl, &attr);
    return cudaLaunchKernelEx(&cfg, tile_pack_kernel, a);
  }
  TileArgs t = {};
  t.rows = a.M;
  t.K = a.K;
  t.row_bytes = static_cast<int>(row_bytes_of(a.wtype, a.K));
  t.period = 1;
  t.records = a.records;
  t.cp = a.cp;
  t.err = a.err;
  t.out = a.dst;
  t.aux = a.aux;
  t.epi = a.epi;
  t.ncols = a.ncols;
  t.group_cols = a.cols;
  switch (a.wtype) {
    case WT_Q8_0: return launch_lin_cols<WT_Q8_0>(t, a, st, pdl);
    case WT_Q4_0: return launch_lin_cols<WT_Q4_0>(t, a, st, pdl);
    case WT_Q4_K: return launch_lin_cols<WT_Q4_K>(t, a, st, pdl);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gf
