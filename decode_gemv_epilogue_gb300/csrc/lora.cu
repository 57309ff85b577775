// Low-rank adapters beside a shared projection: y_c = tail(W x'_c + s_a B_a (A_a x'_c)),
// a = ids[c] (outside 0 .. n-1: no adapter).  Two launches run ahead of the shared product,
//
//   shrink:  v_c = s_a (A_a x'_c)          [r values per column]
//   expand:  out_c = B_a v_c (+ aux_c)     [M values per column]
//
// and the shared product then adds out in its epilogue, before the activation.  In this
// order the output is read and written once more only, and the kernels of plain batches, launched
// with programmatic dependent launch, already stream their weights while the two small kernels
// run (the tiled ones wait for both before their first copy).
//
// Columns that share an adapter are served together, so that an adapter's rows are fetched
// once per four columns (shrink) or once (expand): with fewer adapters than columns a CTA is
// an adapter's (and one row of CTAs more the columns' without), else a column's, and the CTA
// of the first column of an adapter takes all of them.
//
// Shrink: a CTA takes a few rows of an adapter's A; its 256 threads share the K axis, every
// thread holding the sums of its rows and up to four columns, so that one round of
// independent 16-byte loads covers 2048 elements and a decode-sized K is a latency of one or
// two rounds.  Two rows a CTA while that leaves SMs idle (16 rows of 4096 for one column: 6.1
// -> 3.4 us against eight), four once the columns fill them.  Sums: 32 bits, per thread in K
// order, then a shuffle tree, then the warps in order.
// Expand: a CTA takes 128 rows of B, 64 (f32: 32) values of each at a time through shared
// memory, a thread per row walks them for four columns at a time.
#include "gf_device.cuh"
#include "gf_internal.h"

namespace gf {

constexpr int kLoraThreads = 256;
constexpr int kLoraCols = 4;      // columns of an adapter served at once
constexpr int kExpandRows = 128;  // rows, and threads, of an expansion CTA

__host__ __device__ __forceinline__ bool lora_by_adapter(const LoraArgs& a) { return a.n < a.ncols; }

// The columns that the CTAs of index y serve, in order, into cols; their number (0: another
// index serves them), and their adapter (-1: none).  Called by every thread of a CTA.
__device__ __forceinline__ int lora_columns(const LoraArgs& a, int y, int threads, int* cols, int* seen, int& ad) {
  const bool by = lora_by_adapter(a);
  ad = by ? y : a.ids[y];
  if (ad < 0 || ad >= a.n) ad = -1;
  if (!by) {
    if (ad < 0 || a.ncols == 1) {  // a column without an adapter is served alone
      if (threadIdx.x == 0) cols[0] = y;
      __syncthreads();
      return 1;
    }
    if (threadIdx.x == 0) seen[0] = 0;
    __syncthreads();
    for (int q = threadIdx.x; q < y; q += threads)
      if (a.ids[q] == ad) seen[0] = 1;
    __syncthreads();
    if (seen[0]) return 0;
  }
  if (threadIdx.x < 32) {  // one warp lists them
    int n = 0;
    for (int q0 = 0; q0 < a.ncols; q0 += 32) {
      const int q = q0 + static_cast<int>(threadIdx.x);
      const int id = q < a.ncols ? a.ids[q] : -2;
      const bool is = q < a.ncols && (ad >= 0 ? id == ad : id < 0 || id >= a.n);
      const uint32_t m = __ballot_sync(0xffffffffu, is);
      if (is) cols[n + __popc(m & ((1u << threadIdx.x) - 1u))] = q;
      n += __popc(m);
    }
    if (threadIdx.x == 0) seen[1] = n;
  }
  __syncthreads();
  return seen[1];
}

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
// aligned); otherwise element by element.  RB rows, up to CT columns at once.
template <int AT, bool VEC, int RB, int CT>
__device__ __forceinline__ void lora_shrink(const LoraArgs& a) {
  constexpr int kEl = AT == WT_F16 ? 2 : 4, V = RB * CT;
  __shared__ float part[kLoraThreads / 32][V + CT];
  __shared__ int cols[256], seen[2];
  const int j0 = blockIdx.x * RB;
  const int rows = min(RB, a.r - j0);
  int ad;
  const int n = lora_columns(a, blockIdx.y, kLoraThreads, cols, seen, ad);
  if (n == 0 || ad < 0) return;  // the expansion does not read v of a column without an adapter
  const uint8_t* A = a.A + (static_cast<int64_t>(ad) * a.r + j0) * a.K * kEl;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int q0 = 0; q0 < n; q0 += CT) {
    const int nc = min(CT, n - q0);
    const float* x[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) x[t] = a.x + static_cast<int64_t>(cols[q0 + min(t, nc - 1)]) * a.K;
    float acc[V], ss[CT];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int t = 0; t < CT; ++t) ss[t] = 0.0f;
    if constexpr (VEC) {
#pragma unroll 2
      for (int k = threadIdx.x * 8; k < a.K; k += kLoraThreads * 8) {
        float xv[CT][8], g[8];
#pragma unroll
        for (int t = 0; t < CT; ++t)
          if (t < nc) load8<WT_F32>(reinterpret_cast<const uint8_t*>(x[t] + k), xv[t]);
        if (a.gamma) {
          load8<WT_F32>(reinterpret_cast<const uint8_t*>(a.gamma + k), g);
#pragma unroll
          for (int t = 0; t < CT; ++t)
            if (t < nc)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                ss[t] = fmaf(xv[t][e], xv[t][e], ss[t]);
                xv[t][e] *= g[e];
              }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
          if (i < rows) {
            float wv[8];
            load8<AT>(A + (static_cast<int64_t>(i) * a.K + k) * kEl, wv);
#pragma unroll
            for (int t = 0; t < CT; ++t)
              if (t < nc)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[i * CT + t] = fmaf(wv[e], xv[t][e], acc[i * CT + t]);
          }
      }
    } else {
      for (int k = threadIdx.x; k < a.K; k += kLoraThreads) {
        float xv[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) {
          xv[t] = x[t][k];
          if (a.gamma) {
            ss[t] = fmaf(xv[t], xv[t], ss[t]);
            xv[t] *= a.gamma[k];
          }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
          if (i < rows) {
            const float wv = load1<AT>(A, static_cast<int64_t>(i) * a.K + k);
#pragma unroll
            for (int t = 0; t < CT; ++t) acc[i * CT + t] = fmaf(wv, xv[t], acc[i * CT + t]);
          }
      }
    }
    const float t = WarpVecReduce<V>::run(acc, lane);
    if (lane % (32 / V) == 0) part[w][lane / (32 / V)] = t;
    if (a.gamma) {
#pragma unroll
      for (int q = 0; q < CT; ++q) {
        float v = ss[q];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) part[w][V + q] = v;
      }
    }
    __syncthreads();
    const int i = threadIdx.x / CT, q = threadIdx.x % CT;
    if (i < rows && q < nc) {
      float s = 0.0f;
      for (int p = 0; p < kLoraThreads / 32; ++p) s += part[p][i * CT + q];
      if (a.gamma) {
        float z = 0.0f;
        for (int p = 0; p < kLoraThreads / 32; ++p) z += part[p][V + q];
        s *= 1.0f / sqrtf(z / static_cast<float>(a.K) + a.eps);
      }
      a.v[static_cast<int64_t>(cols[q0 + q]) * a.r + j0 + i] = a.scales ? s * a.scales[ad] : s;
    }
    __syncthreads();  // part is written again
  }
}

// Behind the launch that packs x for the shared product it runs beside that: every CTA there
// has waited for what precedes the call before this grid starts, and nothing here is packed.
// It waits at the end instead, so that the product, which waits for the expansion only, finds
// x packed.
template <int AT, bool VEC, int RB, int CT>
__global__ void __launch_bounds__(kLoraThreads) lora_shrink_kernel(const __grid_constant__ LoraArgs a) {
  if (!a.beside_pack) pdl_wait();
  pdl_trigger();
  lora_shrink<AT, VEC, RB, CT>(a);
  if (a.beside_pack) pdl_wait();
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A chunk of B, `len` values of `rows` rows, into bs.  VEC: asynchronous copies, all in flight at
// once, that copies_wait() waits for.
template <int AT, bool VEC, int PITCH>
__device__ __forceinline__ void stage_b(const LoraArgs& a, const uint8_t* B, int rows, int k0, int len, uint8_t* bs) {
  constexpr int kEl = AT == WT_F16 ? 2 : 4;
  if constexpr (VEC) {
    const int words = len * kEl / 16;
    const uint32_t to = smem_u32(bs);
    for (int i = threadIdx.x; i < rows * words; i += kExpandRows) {
      const int r = i / words, q = i - r * words;
      copy16_async(to + r * PITCH + q * 16, B + (static_cast<int64_t>(r) * a.r + k0) * kEl + q * 16);
    }
  } else {
    for (int i = threadIdx.x; i < rows * len; i += kExpandRows) {
      const int r = i / len, q = i - r * len;
      const int64_t at = static_cast<int64_t>(r) * a.r + k0 + q;
      if constexpr (AT == WT_F16)
        reinterpret_cast<uint16_t*>(bs + r * PITCH)[q] = reinterpret_cast<const uint16_t*>(B)[at];
      else
        reinterpret_cast<uint32_t*>(bs + r * PITCH)[q] = reinterpret_cast<const uint32_t*>(B)[at];
    }
  }
}

// The first chunk of B and the ids are read before the wait for the shrinking grid: whatever
// precedes that one is complete once its CTAs have triggered.  The product may start as soon as
// every CTA here has started (and, but for the tiled one, reads W before its own wait).  With the asynchronous copies, the
// whole call: one column of 4096 x 4096 Q4_0 13.7 -> 13.0 us, eight of F16 24.0 -> 22.8, 64 of
// 14336 x 4096 Q4_0 106 -> 103.
// VEC: rows of B are whole 16-byte words.
template <int AT, bool VEC>
__global__ void __launch_bounds__(kExpandRows) lora_expand_kernel(const __grid_constant__ LoraArgs a) {
  constexpr int kEl = AT == WT_F16 ? 2 : 4;
  constexpr int kChunk = 128 / kEl;    // values of a row at a time
  constexpr int kPitch = 128 + 16;     // bytes: rows a bank row and a word apart
  __shared__ __align__(16) uint8_t bs[kExpandRows * kPitch];
  __shared__ __align__(16) float vs[kLoraCols][kChunk];
  __shared__ int cols[256], seen[2];
  pdl_trigger();
  const int m0 = blockIdx.x * kExpandRows, m = m0 + threadIdx.x;
  int ad;
  const int n = lora_columns(a, blockIdx.y, kExpandRows, cols, seen, ad);
  if (ad < 0) {  // no adapter: the addend alone
    pdl_wait();
    for (int q = 0; q < n && m < a.M; ++q) {
      const int64_t o = static_cast<int64_t>(cols[q]) * a.M + m;
      a.out[o] = a.aux ? a.aux[o] : 0.0f;
    }
    return;
  }
  if (n == 0) {
    pdl_wait();
    return;
  }
  const int rows = min(kExpandRows, a.M - m0);
  const uint8_t* B = a.B + (static_cast<int64_t>(ad) * a.M + m0) * a.r * kEl;
  stage_b<AT, VEC, kPitch>(a, B, rows, 0, min(kChunk, a.r), bs);
  pdl_wait();
  for (int k0 = 0; k0 < a.r; k0 += kChunk) {
    const int len = min(kChunk, a.r - k0);
    if (k0 > 0) {
      __syncthreads();  // the previous chunk has been read
      stage_b<AT, VEC, kPitch>(a, B, rows, k0, len, bs);
    }
    if constexpr (VEC) copies_wait();
    for (int q0 = 0; q0 < n; q0 += kLoraCols) {
      const int nc = min(kLoraCols, n - q0);
      __syncthreads();  // the rows are staged; the previous columns' v has been read
      for (int i = threadIdx.x; i < kLoraCols * kChunk; i += kExpandRows) {
        const int t = i / kChunk, j = i - t * kChunk;
        vs[t][j] = t < nc && j < len ? a.v[static_cast<int64_t>(cols[q0 + t]) * a.r + k0 + j] : 0.0f;
      }
      __syncthreads();
      if (m < a.M) {
        float s[kLoraCols] = {0.0f, 0.0f, 0.0f, 0.0f};
        const uint8_t* b = bs + threadIdx.x * kPitch;
        int j = 0;
        for (; j + 8 <= len; j += 8) {
          float wv[8];
          load8<AT>(b + j * kEl, wv);
#pragma unroll
          for (int t = 0; t < kLoraCols; ++t)
            if (t < nc) {
              const float4 v0 = *reinterpret_cast<const float4*>(&vs[t][j]), v1 = *reinterpret_cast<const float4*>(&vs[t][j + 4]);
              s[t] = fmaf(wv[0], v0.x, s[t]); s[t] = fmaf(wv[1], v0.y, s[t]);
              s[t] = fmaf(wv[2], v0.z, s[t]); s[t] = fmaf(wv[3], v0.w, s[t]);
              s[t] = fmaf(wv[4], v1.x, s[t]); s[t] = fmaf(wv[5], v1.y, s[t]);
              s[t] = fmaf(wv[6], v1.z, s[t]); s[t] = fmaf(wv[7], v1.w, s[t]);
            }
        }
        for (; j < len; ++j) {
          const float wv = load1<AT>(b, j);
#pragma unroll
          for (int t = 0; t < kLoraCols; ++t) s[t] = fmaf(wv, vs[t][j], s[t]);
        }
#pragma unroll
        for (int t = 0; t < kLoraCols; ++t)
          if (t < nc) {
            const int64_t o = static_cast<int64_t>(cols[q0 + t]) * a.M + m;
            const float base = k0 > 0 ? a.out[o] : a.aux ? a.aux[o] : 0.0f;  // later chunks add to the first one's
            a.out[o] = base + s[t];
          }
      }
    }
  }
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
    const bool vec = a.K % 8 == 0 && al16(a.A) && al16(a.x) && al16(a.gamma);
    const int served = lora_by_adapter(a) ? a.n : a.ncols;
    const bool few = a.ncols * ((a.r + 7) / 8) <= 32;  // two rows a CTA, a column at a time
    const int rb = few ? 2 : 4;
    cfg.gridDim = dim3(static_cast<unsigned>((a.r + rb - 1) / rb), static_cast<unsigned>(served));
    if (few)
      return vec ? cudaLaunchKernelEx(&cfg, lora_shrink_kernel<AT, true, 2, 1>, a)
                 : cudaLaunchKernelEx(&cfg, lora_shrink_kernel<AT, false, 2, 1>, a);
    return vec ? cudaLaunchKernelEx(&cfg, lora_shrink_kernel<AT, true, 4, kLoraCols>, a)
               : cudaLaunchKernelEx(&cfg, lora_shrink_kernel<AT, false, 4, kLoraCols>, a);
  }
  cfg.blockDim = dim3(kExpandRows);
  cfg.gridDim = dim3(static_cast<unsigned>((a.M + kExpandRows - 1) / kExpandRows),
                     static_cast<unsigned>(lora_by_adapter(a) ? a.n + 1 : a.ncols));
  const bool vec = a.r * (AT == WT_F16 ? 2 : 4) % 16 == 0 && al16(a.B);
  return vec ? cudaLaunchKernelEx(&cfg, lora_expand_kernel<AT, true>, a)
             : cudaLaunchKernelEx(&cfg, lora_expand_kernel<AT, false>, a);
}

int launch_lora(const LoraArgs& a, cudaStream_t st, bool pdl) {
  return a.atype == WT_F16 ? launch_lora_t<WT_F16>(a, st, pdl) : launch_lora_t<WT_F32>(a, st, pdl);
}

}  // namespace gf
