// Low-rank adapters beside a shared projection: y_c = tail(W x'_c + s_a B_a (A_a x'_c)),
// a = ids[c] (outside 0 .. n-1: no adapter).  Two launches run ahead of the shared product,
//
//   shrink:  v_c = s_a (A_a x'_c)          [r values per column]
//   expand:  out_c = B_a v_c (+ aux_c)     [M values per column]
//
// and the shared product then adds out in its epilogue, before the activation.  In this
// order the shared product, launched with programmatic dependent launch, already streams its
// weights while the two small kernels run, and the output is read and written once more only.
//
// Shrink: a CTA takes eight rows of one column's A; its 256 threads share the K axis, every
// thread holding eight row sums, so that one round of independent 16-byte loads covers
// 2048 elements of the eight rows and a decode-sized K is a latency of one or two rounds.
// Sums: 32 bits, per thread in K order, then a shuffle tree, then the warps in order.
// Expand: a thread per output row walks its r contiguous values of B.
#include "gf_device.cuh"
#include "gf_internal.h"

namespace gf {

constexpr int kLoraThreads = 256;
constexpr int kShrinkRows = 8;

// Eight consecutive adapter weights.
template <int AT>
__device__ __forceinline__ void load8(const uint8_t* p, float (&w)[8]) {
  if constexpr (AT == WT_F16) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const float2 a = h2pair(u.x), b = h2pair(u.y), c = h2pair(u.z), d = h2pair(u.w);
    w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
    w[4] = c.x; w[5] = c.y; w[6] = d.x; w[7] = d.y;
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}

template <int AT>
__device__ __forceinline__ float load1(const uint8_t* base, int64_t i) {
  if constexpr (AT == WT_F16)
    return __half2float(reinterpret_cast<const __half*>(base)[i]);
  else
    return reinterpret_cast<const float*>(base)[i];
}

// VEC: rows of A, x and gamma are read 16 bytes at a time (K a multiple of 8, all 16-byte
// aligned); otherwise element by element.
template <int AT, bool VEC>
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_kernel(const __grid_constant__ LoraArgs a) {
  constexpr int kEl = AT == WT_F16 ? 2 : 4;
  __shared__ float part[kLoraThreads / 32][kShrinkRows + 1];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.y, j0 = blockIdx.x * kShrinkRows;
  const int rows = min(kShrinkRows, a.r - j0);
  const int ad = a.ids[c];
  if (ad < 0 || ad >= a.n) return;  // the expansion does not read v for this column
  const float* x = a.x + static_cast<int64_t>(c) * a.K;
  const uint8_t* A = a.A + (static_cast<int64_t>(ad) * a.r + j0) * a.K * kEl;
  float acc[kShrinkRows], ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kShrinkRows; ++i) acc[i] = 0.0f;
  if constexpr (VEC) {
    for (int k = threadIdx.x * 8; k < a.K; k += kLoraThreads * 8) {
      float xv[8];
      load8<WT_F32>(reinterpret_cast<const uint8_t*>(x + k), xv);
      if (a.gamma) {
        float g[8];
        load8<WT_F32>(reinterpret_cast<const uint8_t*>(a.gamma + k), g);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          ss = fmaf(xv[q], xv[q], ss);
          xv[q] *= g[q];
        }
      }
#pragma unroll
      for (int i = 0; i < kShrinkRows; ++i)
        if (i < rows) {
          float w[8];
          load8<AT>(A + (static_cast<int64_t>(i) * a.K + k) * kEl, w);
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[i] = fmaf(w[q], xv[q], acc[i]);
        }
    }
  } else {
    for (int k = threadIdx.x; k < a.K; k += kLoraThreads) {
      float xv = x[k];
      if (a.gamma) {
        ss = fmaf(xv, xv, ss);
        xv *= a.gamma[k];
      }
#pragma unroll
      for (int i = 0; i < kShrinkRows; ++i)
        if (i < rows) acc[i] = fmaf(load1<AT>(A, static_cast<int64_t>(i) * a.K + k), xv, acc[i]);
    }
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const float t = WarpVecReduce<kShrinkRows>::run(acc, lane);
  if (lane % (32 / kShrinkRows) == 0) part[w][lane / (32 / kShrinkRows)] = t;
  if (a.gamma) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) part[w][kShrinkRows] = ss;
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < rows) {
    float s = 0.0f;
    for (int q = 0; q < kLoraThreads / 32; ++q) s += part[q][threadIdx.x];
    if (a.gamma) {
      float q2 = 0.0f;
      for (int q = 0; q < kLoraThreads / 32; ++q) q2 += part[q][kShrinkRows];
      s *= 1.0f / sqrtf(q2 / static_cast<float>(a.K) + a.eps);
    }
    a.v[static_cast<int64_t>(c) * a.r + j0 + threadIdx.x] = a.scales ? s * a.scales[ad] : s;
  }
}

// VEC: rows of B read 16 bytes at a time (r a multiple of 8, B 16-byte aligned).
template <int AT, bool VEC>
__global__ void __launch_bounds__(kLoraThreads) lora_expand_kernel(const __grid_constant__ LoraArgs a) {
  constexpr int kEl = AT == WT_F16 ? 2 : 4;
  __shared__ __align__(16) float vs[kLoraMaxRank];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.y;
  const int ad = a.ids[c];
  const bool live = ad >= 0 && ad < a.n;
  if (live) {
    for (int j = threadIdx.x; j < a.r; j += kLoraThreads) vs[j] = a.v[static_cast<int64_t>(c) * a.r + j];
  }
  __syncthreads();
  const int m = blockIdx.x * kLoraThreads + threadIdx.x;
  if (m >= a.M) return;
  const int64_t o = static_cast<int64_t>(c) * a.M + m;
  float s = 0.0f;
  if (live) {
    const uint8_t* B = a.B + (static_cast<int64_t>(ad) * a.M + m) * a.r * kEl;
    if constexpr (VEC) {
      for (int j = 0; j < a.r; j += 8) {
        float w[8];
        load8<AT>(B + j * kEl, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) s = fmaf(w[q], vs[j + q], s);
      }
    } else {
      for (int j = 0; j < a.r; ++j) s = fmaf(load1<AT>(B, j), vs[j], s);
    }
  }
  a.out[o] = a.aux ? a.aux[o] + s : s;
}

static bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int AT>
static cudaError_t launch_lora_t(const LoraArgs& a, cudaStream_t st, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kLoraThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (a.phase == LORA_SHRINK) {
    cfg.gridDim = dim3(static_cast<unsigned>((a.r + kShrinkRows - 1) / kShrinkRows), static_cast<unsigned>(a.ncols));
    const bool vec = a.K % 8 == 0 && al16(a.A) && al16(a.x) && al16(a.gamma);
    return vec ? cudaLaunchKernelEx(&cfg, lora_shrink_kernel<AT, true>, a)
               : cudaLaunchKernelEx(&cfg, lora_shrink_kernel<AT, false>, a);
  }
  cfg.gridDim = dim3(static_cast<unsigned>((a.M + kLoraThreads - 1) / kLoraThreads), static_cast<unsigned>(a.ncols));
  const bool vec = a.r % 8 == 0 && al16(a.B);
  return vec ? cudaLaunchKernelEx(&cfg, lora_expand_kernel<AT, true>, a)
             : cudaLaunchKernelEx(&cfg, lora_expand_kernel<AT, false>, a);
}

int launch_lora(const LoraArgs& a, cudaStream_t st, bool pdl) {
  return a.atype == WT_F16 ? launch_lora_t<WT_F16>(a, st, pdl) : launch_lora_t<WT_F32>(a, st, pdl);
}

}  // namespace gf
