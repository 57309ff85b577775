// The 8-bit cache of keys and values: new tokens quantised as they are written (gf_cache_store, with the
// rotation of queries and keys if wanted) and read back (gf_cache_load).
//
// A block of tokens of one head shares a scale, the least one that its values need.  New tokens that
// need a larger one than the block's earlier tokens have make the earlier codes be rounded again under
// it; a block whose first token is written starts anew.
#include "cache_device.cuh"
#include "gf_device.cuh"
#include "rope_device.cuh"

namespace gf {

constexpr int kStoreWarps = 8;
constexpr int kStoreKept = 4;  // iterations whose values stay in registers between the two passes

__device__ __forceinline__ int seq_of(const int32_t* seq, int64_t t) { return seq ? seq[t] : static_cast<int>(t); }

template <typename E, bool VEC>
__device__ __forceinline__ void load8(const E* row, int o0, int o1, float (&v)[8]) {
  if constexpr (VEC) {
    const float4 l = load4(row + o0), r = load4(row + o1);
    v[0] = l.x, v[1] = l.y, v[2] = l.z, v[3] = l.w, v[4] = r.x, v[5] = r.y, v[6] = r.z, v[7] = r.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = load1(row + o0 + i);
      v[4 + i] = load1(row + o1 + i);
    }
  }
}

template <typename E, bool VEC>
__device__ __forceinline__ void store8(E* row, int o0, int o1, const float (&v)[8]) {
  if constexpr (VEC) {
    store4(row + o0, v[0], v[1], v[2], v[3]);
    store4(row + o1, v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      store1(row + o0 + i, v[i]);
      store1(row + o1 + i, v[4 + i]);
    }
  }
}

// Rotates a unit by its four pairs' cosines and sines.
__device__ __forceinline__ void turn8(float (&v)[8], const float2* cs, bool halves) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = cs[i];
    if (halves)
      rope_turn(v[i], v[4 + i], t);
    else
      rope_turn(v[2 * i], v[2 * i + 1], t);
  }
}

// A CTA takes the new tokens of one block (those behind the first find that they are not the first and
// leave), and of its work, units of (block, head, keys or values) and rows of queries, every gridDim.y-th
// group of kStoreWarps warps.  A unit is wpu warps'; a warp holds 32 / (dim / 8) tokens at a time, eight
// elements a lane.
template <int FMT, typename E, bool VEC>
__global__ void __launch_bounds__(32 * kStoreWarps) store_kernel(const __grid_constant__ StoreArgs a) {
  extern __shared__ float2 cs[];  // [token][pair]
  __shared__ uint32_t tops[kStoreWarps];
  __shared__ int first_other;
  pdl_wait();
  pdl_trigger();
  const CacheArgs& c = a.c;
  const int64_t t = blockIdx.x;
  const int seq = seq_of(a.seq, t), pos = a.pos[t];
  const int64_t page = cache_page(c, seq, pos);
  if (page < 0) return;
  const int block = 1 << c.block_log2, i0 = pos & (block - 1);
  if (t > 0 && i0 > 0 && seq_of(a.seq, t - 1) == seq && a.pos[t - 1] == pos - 1) return;
  int n = 1;
  if (block > 1) {
    if (threadIdx.x == 0) first_other = block - i0;
    __syncthreads();
    const int i = threadIdx.x;
    if (i > 0 && i < block - i0 &&
        !(t + i < a.T && seq_of(a.seq, t + i) == seq && a.pos[t + i] == pos + i))
      atomicMin(&first_other, i);
    __syncthreads();
    n = first_other;
  }
  const int pairs = a.n_rot / 2;
  if (a.table) {
    const float mag = static_cast<const RopeHeader*>(a.table)->magnitude;
    for (int i = threadIdx.x; i < n * pairs; i += blockDim.x)
      cs[i] = rope_cs(rope_turns(a.table)[i % pairs], pos + i / pairs, mag);
    __syncthreads();
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = c.dim >> 3, tpw = 32 / L, lg = lane / L, u = lane - lg * L;
  const bool on = lg < tpw, halves = a.halves != 0, turns = a.table && 8 * u < a.n_rot;
  int o0, o1;
  unit_offsets(u, a.table ? a.n_rot : 0, halves, o0, o1);
  const int slot0 = pos & ((1 << c.page_log2) - 1);
  const int upg = kStoreWarps / a.wpu, unit_groups = (2 * c.heads + upg - 1) / upg;
  const int q_groups = a.q ? (a.q_heads + kStoreWarps * tpw - 1) / (kStoreWarps * tpw) : 0;
  for (int item = blockIdx.y; item < unit_groups + q_groups; item += gridDim.y) {
    if (item >= unit_groups) {
      const int h = ((item - unit_groups) * kStoreWarps + warp) * tpw + lg;
      if (!on || h >= a.q_heads) continue;
      for (int i = 0; i < n; ++i) {
        float v[8];
        load8<E, VEC>(static_cast<const E*>(a.q) + (t + i) * a.ldq + static_cast<int64_t>(h) * c.dim, o0, o1, v);
        if (turns) turn8(v, cs + i * pairs + 4 * u, halves);
        store8<E, VEC>(static_cast<E*>(a.q_dst) + (t + i) * a.ld_q_dst + static_cast<int64_t>(h) * c.dim, o0, o1, v);
      }
      continue;
    }
    const int unit = item * upg + warp / a.wpu, w = warp % a.wpu;
    const bool live = unit < 2 * c.heads, is_v = unit >= c.heads;
    const int head = is_v ? unit - c.heads : unit;
    const int step = a.wpu * tpw, iters = (n + step - 1) / step;
    // values are at their plain places in V and, where nothing turns, in K
    const int p0 = is_v ? 8 * u : o0, p1 = is_v ? 8 * u + 4 : o1;
    const E* src = static_cast<const E*>(is_v ? a.v : a.k) + static_cast<int64_t>(head) * c.dim;
    const int64_t ld = is_v ? a.ldv : a.ldk;
    auto fetch = [&](int i, float (&v)[8]) {
      load8<E, VEC>(src + (t + i) * ld, p0, p1, v);
      if (turns && !is_v) turn8(v, cs + i * pairs + 4 * u, halves);
    };
    float kept[kStoreKept][8];
    uint32_t top = 0;
    auto widen = [&](const float (&v)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);  // NaN is the largest
    };
#pragma unroll
    for (int k = 0; k < kStoreKept; ++k) {
      const int i = k * step + w * tpw + lg;
      if (live && on && i < n) {
        fetch(i, kept[k]);
        widen(kept[k]);
      }
    }
    for (int k = kStoreKept; k < iters; ++k) {
      const int i = k * step + w * tpw + lg;
      if (live && on && i < n) {
        float v[8];
        fetch(i, v);
        widen(v);
      }
    }
    float* scale = live ? (is_v ? c.v_scale : c.k_scale) + cache_scale(c, page, head, slot0) : nullptr;
    const float old = live && i0 > 0 ? *scale : 0.0f;
    top = __reduce_max_sync(0xffffffffu, top);
    if (a.wpu > 1) {
      __syncthreads();  // the group before has read its tops
      if (lane == 0) tops[warp] = top;
      __syncthreads();
      for (int i = 0; i < a.wpu; ++i) top = max(top, tops[warp - w + i]);
    }
    if (!live) continue;
    float d;
    if (top >= 0x7f800000u || !(old == old))
      d = __uint_as_float(0x7fffffffu);  // not finite: the block reads back as NaN
    else
      d = fmaxf(scale_for<FMT>(__uint_as_float(top)), old);
    const bool number = d == d;
    const float inv = number ? 1.0f / d : 0.0f;
    if (lane == 0 && w == 0) *scale = d;
    uint8_t* codes = (is_v ? c.v : c.k) + cache_row(c, page, head, slot0);
    auto write = [&](int i, const float (&v)[8]) {
      uint8_t* row = codes + static_cast<int64_t>(i) * c.dim;
      const uint32_t x = number ? codes4<FMT>(v[0], v[1], v[2], v[3], d, inv) : 0u;
      const uint32_t y = number ? codes4<FMT>(v[4], v[5], v[6], v[7], d, inv) : 0u;
      *reinterpret_cast<uint32_t*>(row + p0) = x;
      *reinterpret_cast<uint32_t*>(row + p1) = y;
    };
#pragma unroll
    for (int k = 0; k < kStoreKept; ++k) {
      const int i = k * step + w * tpw + lg;
      if (on && i < n) write(i, kept[k]);
    }
    for (int k = kStoreKept; k < iters; ++k) {
      const int i = k * step + w * tpw + lg;
      if (on && i < n) {
        float v[8];
        fetch(i, v);
        write(i, v);
      }
    }
    if (number && i0 > 0 && d > old && on) {  // the block's earlier tokens, under the larger scale
      for (int i = w * tpw + lg; i < i0; i += step) {
        uint2* row = reinterpret_cast<uint2*>(codes - static_cast<int64_t>(i0 - i) * c.dim + 8 * u);
        const uint2 raw = *row;
        float x[4], y[4];
        values4<FMT>(raw.x, x);
        values4<FMT>(raw.y, y);
        // i8: code * old is exact; e4m3: the scales' quotient is
        const float f = FMT == 0 ? old : 1.0f, r = FMT == 0 ? inv : old * inv;
        *row = make_uint2(codes4<FMT>(x[0] * f, x[1] * f, x[2] * f, x[3] * f, d, r),
                          codes4<FMT>(y[0] * f, y[1] * f, y[2] * f, y[3] * f, d, r));
      }
    }
  }
}

template <int FMT, typename E, bool VEC>
static int launch_store_t(const StoreArgs& a, int sms, cudaStream_t st, bool pdl) {
  const int64_t tpw = 32 / (a.c.dim / 8), upg = kStoreWarps / a.wpu;
  int64_t groups = (2 * a.c.heads + upg - 1) / upg;
  if (a.q) groups += (a.q_heads + kStoreWarps * tpw - 1) / (kStoreWarps * tpw);
  // Groups spread over as many CTAs as keep eight on every SM, counting whole blocks of new tokens
  // (a prompt's); every CTA of a block computes its tokens' cosines again.
  const int64_t blocks = (a.T + (1 << a.c.block_log2) - 1) >> a.c.block_log2;
  int64_t y = (8 * sms + blocks - 1) / blocks;
  if (y > groups) y = groups;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.T), static_cast<unsigned>(y));
  cfg.blockDim = dim3(32 * kStoreWarps);
  cfg.dynamicSmemBytes = a.table ? static_cast<size_t>(a.n_rot / 2) << (3 + a.c.block_log2) : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (cfg.dynamicSmemBytes > 40 * 1024) {
    static SmemLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(store_kernel<FMT, E, VEC>));
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, store_kernel<FMT, E, VEC>, a);
}

int launch_store(const StoreArgs& a, int sms, cudaStream_t st, bool pdl) {
  if (a.type == 0) {
    if (a.c.format == 0)
      return a.vec ? launch_store_t<0, float, true>(a, sms, st, pdl) : launch_store_t<0, float, false>(a, sms, st, pdl);
    return a.vec ? launch_store_t<1, float, true>(a, sms, st, pdl) : launch_store_t<1, float, false>(a, sms, st, pdl);
  }
  if (a.c.format == 0)
    return a.vec ? launch_store_t<0, __half, true>(a, sms, st, pdl) : launch_store_t<0, __half, false>(a, sms, st, pdl);
  return a.vec ? launch_store_t<1, __half, true>(a, sms, st, pdl) : launch_store_t<1, __half, false>(a, sms, st, pdl);
}

// A lane takes eight elements of a (token, head) row.
template <int FMT, typename E, bool VEC>
__global__ void __launch_bounds__(256) load_kernel(const __grid_constant__ LoadArgs a) {
  pdl_wait();
  pdl_trigger();
  const CacheArgs& c = a.c;
  const int L = c.dim >> 3;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, row = i / L;
  const int u = static_cast<int>(i - row * L);
  const int64_t t = row / c.heads;
  const int h = static_cast<int>(row - t * c.heads);
  if (t >= a.T) return;
  const int pos = a.pos[t], slot = pos & ((1 << c.page_log2) - 1);
  const int64_t page = cache_page(c, seq_of(a.seq, t), pos);
  const int64_t at = cache_row(c, page, h, slot) + 8 * u, sc = cache_scale(c, page, h, slot);
#pragma unroll
  for (int is_v = 0; is_v < 2; ++is_v) {
    E* out = static_cast<E*>(is_v ? a.v : a.k);
    if (!out) continue;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (page >= 0) {
      const uint2 raw = *reinterpret_cast<const uint2*>((is_v ? c.v : c.k) + at);
      const float d = (is_v ? c.v_scale : c.k_scale)[sc];
      float x[4], y[4];
      values4<FMT>(raw.x, x);
      values4<FMT>(raw.y, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = x[e] * d;
        v[4 + e] = y[e] * d;
      }
    }
    store8<E, VEC>(out + t * (is_v ? a.ldv : a.ldk) + static_cast<int64_t>(h) * c.dim, 8 * u, 8 * u + 4, v);
  }
}

template <int FMT, typename E>
static int launch_load_t(const LoadArgs& a, cudaStream_t st, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.T * a.c.heads * (a.c.dim / 8) + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return a.vec ? cudaLaunchKernelEx(&cfg, load_kernel<FMT, E, true>, a)
               : cudaLaunchKernelEx(&cfg, load_kernel<FMT, E, false>, a);
}

int launch_load(const LoadArgs& a, cudaStream_t st, bool pdl) {
  if (a.type == 0) return a.c.format == 0 ? launch_load_t<0, float>(a, st, pdl) : launch_load_t<1, float>(a, st, pdl);
  return a.c.format == 0 ? launch_load_t<0, __half>(a, st, pdl) : launch_load_t<1, __half>(a, st, pdl);
}

}  // namespace gf
