// The chosen experts' gated product:
//   dst_t = aux_t + sum_j w_tj Wd_e (silu(Wg_e x_t) * (Wu_e x_t)),   e = ids_tj.
// A "slot" is one (token, choice) pair, s = t k + j.  Kernels for any shape and alignment:
// a warp per row of a slot's expert, weights decoded element by element from global memory,
// 32-bit sums; then the combination, which adds a token's slots in the order of its choices
// (deterministic).
#include "gf_device.cuh"
#include "gf_internal.h"

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
