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

// Queries of a window's tokens: a warp takes q_rows times tpw heads of a token at a time, every (q_slices *
// kStoreWarps)th such task; a lane turns its four pairs of all of them by the same angles.  (As rows of a block's
// work, behind its scan and between its CTAs' cosines, they made 86 us of 66 for 8191 tokens of 32 query and 8 key
// heads.)
template <typename E, bool VEC>
__device__ __forceinline__ void store_queries(const StoreArgs& a, int task, int lg, int u, bool on, int o0, int o1) {
  const CacheArgs& c = a.c;
  const int heads = a.q_rows * a.tpw, chunks = (a.q_heads + heads - 1) / heads;
  const bool halves = a.halves != 0, turns = 8 * u < a.n_rot;
  for (; task < a.window * chunks; task += a.q_slices * kStoreWarps) {
    const int i = task / chunks, h0 = (task - i * chunks) * heads + lg;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * a.window + i;
    if (t >= a.T) return;
    const E* from = static_cast<const E*>(a.q) + t * a.ldq;
    E* to = static_cast<E*>(a.q_dst) + t * a.ld_q_dst;
    const int pos = a.pos[t], seq = seq_of(a.seq, t);
    float v[kStoreKept][8];
#pragma unroll
    for (int k = 0; k < kStoreKept; ++k) {
      const int h = h0 + k * a.tpw;
      if (on && k < a.q_rows && h < a.q_heads) load8<E, VEC>(from + static_cast<int64_t>(h) * c.dim, o0, o1, v[k]);
    }
    float2 cs[4];
    if (turns) {
      const float mag = static_cast<const RopeHeader*>(a.table)->magnitude;
      const uint64_t* f = rope_turns(a.table) + 4 * u;
#pragma unroll
      for (int e = 0; e < 4; ++e) cs[e] = rope_cs(f[e], pos, mag);
    }
    if (cache_page(c, seq, pos) < 0) continue;
#pragma unroll
    for (int k = 0; k < kStoreKept; ++k) {
      const int h = h0 + k * a.tpw;
      if (on && k < a.q_rows && h < a.q_heads) {
        if (turns) turn8(v[k], cs, halves);
        store8<E, VEC>(to + static_cast<int64_t>(h) * c.dim, o0, o1, v[k]);
      }
    }
  }
}

// A block's scale: what its new values of magnitude up to `top` (as bits) and its earlier ones need; NaN where
// a value is not finite, and the block then reads back as NaN.
template <int FMT>
__device__ __forceinline__ float block_scale(uint32_t top, float old) {
  if (top >= 0x7f800000u || !(old == old)) return __uint_as_float(0x7fffffffu);
  return fmaxf(scale_for<FMT>(__uint_as_float(top)), old);
}

// Eight codes of an earlier token, under the larger scale d.  i8: code * old is exact; e4m3: the scales' quotient is.
template <int FMT>
__device__ __forceinline__ void rescale8(uint2* row, float old, float d, float inv) {
  const uint2 raw = *row;
  float x[4], y[4];
  values4<FMT>(raw.x, x);
  values4<FMT>(raw.y, y);
  const float f = FMT == 0 ? old : 1.0f, r = FMT == 0 ? inv : old * inv;
  const float v[8] = {x[0] * f, x[1] * f, x[2] * f, x[3] * f, y[0] * f, y[1] * f, y[2] * f, y[3] * f};
  *row = codes8<FMT>(v, d, r);
}

// Codes of a unit of eight, which lie at p0 and p1 of a row.
__device__ __forceinline__ void put_codes(uint8_t* row, int p0, int p1, uint2 w) {
  if (p1 == p0 + 4) {
    *reinterpret_cast<uint2*>(row + p0) = w;
  } else {
    *reinterpret_cast<uint32_t*>(row + p0) = w.x;
    *reinterpret_cast<uint32_t*>(row + p1) = w.y;
  }
}

// Blocks no longer than a warp's tokens, of a prompt: a task is a window's token and kStoreKept heads, all values
// of the token's block on their way together if it begins one.  (As units of a head, 8191 tokens with a scale each
// took 90 us where 44.)
template <int FMT, typename E, bool VEC>
__device__ __forceinline__ void store_small(const StoreArgs& a, int task, int step, int lg, int u, bool on, int o0, int o1) {
  const CacheArgs& c = a.c;
  const int block = 1 << c.block_log2, chunks = (c.heads + kStoreKept - 1) / kStoreKept, lane = threadIdx.x & 31;
  const bool halves = a.halves != 0;
  for (; task < a.window * 2 * chunks; task += step) {
    const int j = task / (2 * chunks), part = task - j * 2 * chunks;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * a.window + j;
    if (t >= a.T) return;
    const int seq = seq_of(a.seq, t), pos = a.pos[t], i0 = pos & (block - 1);
    if (t > 0 && i0 > 0 && seq_of(a.seq, t - 1) == seq && a.pos[t - 1] == pos - 1) continue;
    const uint32_t same = __ballot_sync(0xffffffffu, lane < block - i0 && t + lane < a.T && seq_of(a.seq, t + lane) == seq &&
                                                         a.pos[t + lane] == pos + lane);
    const int n = __ffs(~same) - 1;  // (blocks are shorter than a warp)
    const bool is_v = part >= chunks, turns = a.table && !is_v && 8 * u < a.n_rot;
    const int head0 = (is_v ? part - chunks : part) * kStoreKept, slot0 = pos & ((1 << c.page_log2) - 1);
    const int p0 = is_v ? 8 * u : o0, p1 = is_v ? 8 * u + 4 : o1, i = min(lg, n - 1);
    const E* src = static_cast<const E*>(is_v ? a.v : a.k) + (t + i) * (is_v ? a.ldv : a.ldk);
    float v[kStoreKept][8];
#pragma unroll
    for (int k = 0; k < kStoreKept; ++k)
      load8<E, VEC>(src + static_cast<int64_t>(min(head0 + k, c.heads - 1)) * c.dim, p0, p1, v[k]);
    float2 cs[4];
    if (turns) {
      const float mag = static_cast<const RopeHeader*>(a.table)->magnitude;
#pragma unroll
      for (int e = 0; e < 4; ++e) cs[e] = rope_cs(rope_turns(a.table)[4 * u + e], pos + i, mag);
    }
    const int64_t page = cache_page(c, seq, pos);
    if (page < 0) continue;
    float* scales = is_v ? c.v_scale : c.k_scale;
    uint8_t* codes = is_v ? c.v : c.k;
#pragma unroll
    for (int k = 0; k < kStoreKept; ++k) {
      if (head0 + k >= c.heads) break;
      float* scale = scales + cache_scale(c, page, head0 + k, slot0);
      const float old = i0 > 0 ? *scale : 0.0f;
      if (turns) turn8(v[k], cs, halves);
      float widest = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) widest = top_of(widest, v[k][e]);
      const float d = block_scale<FMT>(__reduce_max_sync(0xffffffffu, __float_as_uint(widest)), old);
      const bool number = d == d;
      const float inv = number ? 1.0f / d : 0.0f;
      __syncwarp();  // the scale before has been read
      if (lane == 0) *scale = d;
      uint8_t* rows = codes + cache_row(c, page, head0 + k, slot0);
      if (on && lg < n) put_codes(rows + lg * c.dim, p0, p1, number ? codes8<FMT>(v[k], d, inv) : make_uint2(0u, 0u));
      if (number && on && lg < i0 && d > old)
        rescale8<FMT>(reinterpret_cast<uint2*>(rows + (lg - i0) * c.dim + 8 * u), old, d, inv);
    }
  }
}

// A CTA looks for first tokens of blocks among `window` tokens of the call, and takes the new tokens of each one's
// block in turn: of their units of (block, head, keys or values), every (gridDim.y - q_slices)th group of
// kStoreWarps warps.  A unit is 1 << wpu_log2 warps'; a warp holds 32 / (dim / 8) tokens at a time, eight elements
// a lane.  The last q_slices CTAs of a window turn its queries.
// Every value is read once, every code written once; 8191 tokens of 8 heads of 128 in blocks of 32, f16, take 32 us
// (50 MB, 7.5 us of the memory's): the chain from positions to values, scale and codes is what a CTA waits for.
// With a CTA to every token, those of a prompt that begin no block cost more than the others: 120 us.
template <int FMT, typename E, bool VEC, bool SMALL>
__global__ void __launch_bounds__(32 * kStoreWarps, 3) store_kernel(const __grid_constant__ StoreArgs a) {
  extern __shared__ float2 cs[];  // [token][pair]
  __shared__ uint32_t tops[kStoreWarps];
  pdl_wait();
  pdl_trigger();
  const CacheArgs& c = a.c;
  const int block = 1 << c.block_log2, pairs = a.n_rot / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = c.dim >> 3, tpw = a.tpw, lg = lane * a.lane_inv >> 16, u = lane - lg * L;  // lane / L; lanes over: unit 0 ..
  const bool on = lg < tpw, halves = a.halves != 0, turns = a.table && 8 * u < a.n_rot;
  int o0, o1;
  unit_offsets(u, a.table ? a.n_rot : 0, halves, o0, o1);
  const int slices = gridDim.y - a.q_slices;
  if (static_cast<int>(blockIdx.y) >= slices) {
    if (!rope_fits(a.table, a.n_rot, a.err)) return;
    store_queries<E, VEC>(a, (blockIdx.y - slices) * kStoreWarps + warp, lg, u, on, o0, o1);
    return;
  }
  if constexpr (SMALL) {
    if (a.table && !rope_fits(a.table, a.n_rot, a.err)) return;
    store_small<FMT, E, VEC>(a, blockIdx.y * kStoreWarps + warp, slices * kStoreWarps, lg, u, on, o0, o1);
    return;
  }
  const int wpu = 1 << a.wpu_log2, upg = kStoreWarps >> a.wpu_log2, unit_groups = a.unit_groups;
  uint32_t firsts;  // of the window's tokens, those that begin a block's new ones
  {
    const uint32_t table_pairs = a.table ? static_cast<const RopeHeader*>(a.table)->pairs : 0;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * a.window + lane;
    bool first = false;
    if (lane < a.window && t < a.T) {
      const int pos = a.pos[t], seq = seq_of(a.seq, t);
      first = !(t > 0 && (pos & (block - 1)) > 0 && seq_of(a.seq, t - 1) == seq && a.pos[t - 1] == pos - 1);
    }
    firsts = __ballot_sync(0xffffffffu, first);
    if (a.table && !rope_fits(table_pairs, a.n_rot, a.err)) return;  // (positions do not wait for it)
  }
  for (; firsts; firsts &= firsts - 1) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * a.window + __ffs(firsts) - 1;
    const int seq = seq_of(a.seq, t), pos = a.pos[t], i0 = pos & (block - 1);
    int n = 0;  // tokens of the run within the block
    for (int k = 0; k < block - i0; k += 32) {
      const int i = k + lane;
      const uint32_t same = __ballot_sync(0xffffffffu, i < block - i0 && t + i < a.T && seq_of(a.seq, t + i) == seq &&
                                                           a.pos[t + i] == pos + i);
      n += __ffs(~same) ? __ffs(~same) - 1 : 32;
      if (~same) break;
    }
    const int slot0 = pos & ((1 << c.page_log2) - 1);
    bool turned = false;  // the run's cosines are there
    for (int item = blockIdx.y; item < unit_groups; item += slices) {
      if (a.table && item * upg < c.heads && !turned) {
        turned = true;
        __syncthreads();  // the block before is done with
        const float mag = static_cast<const RopeHeader*>(a.table)->magnitude;
        for (int i = threadIdx.x; i < n * pairs; i += blockDim.x)
          cs[i] = rope_cs(rope_turns(a.table)[i % pairs], pos + i / pairs, mag);
        __syncthreads();
      }
      const int unit = item * upg + (warp >> a.wpu_log2), w = warp & (wpu - 1);
      bool live = unit < 2 * c.heads;
      const bool is_v = unit >= c.heads;
      const int head = is_v ? unit - c.heads : unit;
      const int step = tpw << a.wpu_log2;
      // values are at their plain places in V and, where nothing turns, in K
      const int p0 = is_v ? 8 * u : o0, p1 = is_v ? 8 * u + 4 : o1;
      const E* src = static_cast<const E*>(is_v ? a.v : a.k) + static_cast<int64_t>(head) * c.dim;
      const int64_t ld = is_v ? a.ldv : a.ldk;
      auto turn = [&](int i, float (&v)[8]) {
        if (turns && !is_v) turn8(v, cs + i * pairs + 4 * u, halves);
      };
      float widest = 0.0f;
      auto widen = [&](const float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) widest = top_of(widest, v[e]);
      };
      // All of the kept values are on their way before the first is waited for: lanes and iterations that have no token
      // take the run's last one.
      float kept[kStoreKept][8];
      if (live) {
#pragma unroll
        for (int k = 0; k < kStoreKept; ++k)
          if (k == 0 || k * step < n) load8<E, VEC>(src + (t + min(k * step + w * tpw + lg, n - 1)) * ld, p0, p1, kept[k]);
      }
      // (looked up behind the loads, so that they do not wait for it)
      const int64_t page = cache_page(c, seq, pos);
      live = live && page >= 0;
      float* scale = live ? (is_v ? c.v_scale : c.k_scale) + cache_scale(c, page, head, slot0) : nullptr;
      const float old = live && i0 > 0 ? *scale : 0.0f;
      if (live) {
#pragma unroll
        for (int k = 0; k < kStoreKept; ++k) {
          if (k > 0 && k * step >= n) break;
          turn(min(k * step + w * tpw + lg, n - 1), kept[k]);
          widen(kept[k]);
        }
#pragma unroll 2
        for (int k = kStoreKept; k * step < n; ++k) {
          const int i = min(k * step + w * tpw + lg, n - 1);
          float v[8];
          load8<E, VEC>(src + (t + i) * ld, p0, p1, v);
          turn(i, v);
          widen(v);
        }
      }
      uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(widest));  // NaN is the largest
      if (wpu > 1) {
        __syncthreads();  // the group before has read its tops
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        for (int i = 0; i < wpu; ++i) top = max(top, tops[warp - w + i]);
      }
      if (!live) continue;
      const float d = block_scale<FMT>(top, old);
      const bool number = d == d;
      const float inv = number ? 1.0f / d : 0.0f;
      if (lane == 0 && w == 0) *scale = d;
      uint8_t* codes = (is_v ? c.v : c.k) + cache_row(c, page, head, slot0);
      auto write = [&](int i, const float (&v)[8]) {
        uint8_t* row = codes + static_cast<int64_t>(i) * c.dim;
        put_codes(row, p0, p1, number ? codes8<FMT>(v, d, inv) : make_uint2(0u, 0u));
      };
#pragma unroll
      for (int k = 0; k < kStoreKept; ++k) {
        const int i = k * step + w * tpw + lg;
        if (on && i < n) write(i, kept[k]);
      }
      for (int k = kStoreKept; k * step < n; ++k) {
        const int i = k * step + w * tpw + lg;
        if (on && i < n) {
          float v[8];
          load8<E, VEC>(src + (t + i) * ld, p0, p1, v);
          turn(i, v);
          write(i, v);
        }
      }
      if (number && i0 > 0 && d > old && on) {  // the block's earlier tokens, under the larger scale
        for (int i = w * tpw + lg; i < i0; i += step)
          rescale8<FMT>(reinterpret_cast<uint2*>(codes - static_cast<int64_t>(i0 - i) * c.dim + 8 * u), old, d, inv);
      }
    }
  }
}

template <int FMT, typename E, bool VEC>
static int launch_store_t(const StoreArgs& a, int sms, cudaStream_t st, bool pdl) {
  // A block's units are spread over as many CTAs as make 32 for every SM, counting those that find a block (a
  // prompt's): a CTA waits for its values once, and others fill the time; every CTA of a block computes its
  // tokens' cosines again.
  const int64_t windows = (a.T + a.window - 1) / a.window, blocks = (a.T + (1 << a.c.block_log2) - 1) >> a.c.block_log2;
  const int64_t busy = windows < blocks ? windows : blocks, wanted = (32 * sms + busy - 1) / busy;
  const int64_t y = wanted < a.unit_groups ? wanted : a.unit_groups;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(windows), static_cast<unsigned>(y + a.q_slices));
  cfg.blockDim = dim3(32 * kStoreWarps);
  cfg.dynamicSmemBytes = a.table && !a.small ? static_cast<size_t>(a.n_rot / 2) << (3 + a.c.block_log2) : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const auto kernel = a.small ? store_kernel<FMT, E, VEC, true> : store_kernel<FMT, E, VEC, false>;
  if (cfg.dynamicSmemBytes > 40 * 1024) {
    static SmemLimit limit;  // (blocks that a warp holds take less)
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a);
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

// A thread takes 16 bytes of output, at the same place of TOKENS tokens' rows: all their positions, then
// all their pages, then all their codes are on the way together.  8191 tokens of 8 heads of 128 into f16: 13 us (50 MB).
template <int FMT, typename E, bool VEC, int TOKENS>
__global__ void __launch_bounds__(256) load_kernel(const __grid_constant__ LoadArgs a) {
  constexpr int N = 16 / sizeof(E), WORDS = N / 4;
  pdl_wait();
  pdl_trigger();
  const CacheArgs& c = a.c;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TOKENS;
  int pos[TOKENS], seq[TOKENS];
  int64_t page[TOKENS];
#pragma unroll
  for (int i = 0; i < TOKENS; ++i) {
    pos[i] = t0 + i < a.T ? a.pos[t0 + i] : -1;
    seq[i] = t0 + i < a.T ? seq_of(a.seq, t0 + i) : -1;
  }
#pragma unroll
  for (int i = 0; i < TOKENS; ++i) page[i] = cache_page(c, seq[i], pos[i]);
  for (int at = (threadIdx.x + blockIdx.y * blockDim.x) * N; at < c.heads * c.dim; at += blockDim.x * gridDim.y * N) {
    const int h = at / c.dim, d = at - h * c.dim;
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
      E* out = static_cast<E*>(is_v ? a.v : a.k);
      if (!out) continue;
      uint32_t raw[TOKENS][WORDS];
      float scale[TOKENS];
#pragma unroll
      for (int i = 0; i < TOKENS; ++i) {
        const int slot = pos[i] & ((1 << c.page_log2) - 1);
        scale[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) raw[i][w] = 0;
        if (page[i] >= 0) {
          const uint8_t* p = (is_v ? c.v : c.k) + cache_row(c, page[i], h, slot) + d;
          if constexpr (WORDS == 2) {
            const uint2 r = *reinterpret_cast<const uint2*>(p);
            raw[i][0] = r.x, raw[i][1] = r.y;
          } else {
            raw[i][0] = *reinterpret_cast<const uint32_t*>(p);
          }
          scale[i] = (is_v ? c.v_scale : c.k_scale)[cache_scale(c, page[i], h, slot)];
        }
      }
#pragma unroll
      for (int i = 0; i < TOKENS; ++i) {
        if (t0 + i >= a.T) break;
        E* to = out + (t0 + i) * (is_v ? a.ldv : a.ldk) + at;
        float v[N];
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
          float x[4];
          values4<FMT>(raw[i][w], x);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * w + e] = page[i] >= 0 ? x[e] * scale[i] : 0.0f;
        }
        if constexpr (!VEC) {
#pragma unroll
          for (int e = 0; e < N; ++e) store1(to + e, v[e]);
        } else if constexpr (WORDS == 2) {
          const __half2 q[4] = {__floats2half2_rn(v[0], v[1]), __floats2half2_rn(v[2], v[3]), __floats2half2_rn(v[4], v[5]),
                                __floats2half2_rn(v[6], v[7])};
          *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(q);
        } else {
          store4(to, v[0], v[1], v[2], v[3]);
        }
      }
    }
  }
}

template <int FMT, typename E>
static int launch_load_t(const LoadArgs& a, cudaStream_t st, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  // Few tokens: one a CTA, its heads spread over CTAs.  64 tokens of 32 heads of 128, f16, 9.3 us so and 11.4 with four
  // tokens a CTA; of 8 heads 9.3 either way up to 1000; 2000 of them, f32, 13.4 and 11.4, 4000 20 and 16.
  const bool few = a.T < 1024;
  const int64_t units = static_cast<int64_t>(a.c.heads) * a.c.dim * sizeof(E) / 16;
  cfg.blockDim = dim3(static_cast<unsigned>(units < 256 ? (units + 31) / 32 * 32 : 256));
  cfg.gridDim = few ? dim3(static_cast<unsigned>(a.T), static_cast<unsigned>((units + 255) / 256))
                    : dim3(static_cast<unsigned>((a.T + 3) / 4));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (few)
    return a.vec ? cudaLaunchKernelEx(&cfg, load_kernel<FMT, E, true, 1>, a)
                 : cudaLaunchKernelEx(&cfg, load_kernel<FMT, E, false, 1>, a);
  return a.vec ? cudaLaunchKernelEx(&cfg, load_kernel<FMT, E, true, 4>, a)
               : cudaLaunchKernelEx(&cfg, load_kernel<FMT, E, false, 4>, a);
}

int launch_load(const LoadArgs& a, cudaStream_t st, bool pdl) {
  if (a.type == 0) return a.c.format == 0 ? launch_load_t<0, float>(a, st, pdl) : launch_load_t<1, float>(a, st, pdl);
  return a.c.format == 0 ? launch_load_t<0, __half>(a, st, pdl) : launch_load_t<1, __half>(a, st, pdl);
}

}  // namespace gf
