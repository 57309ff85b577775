// Tiled products of block-format weights with several columns on the tensor cores: the
// device code of the chosen experts' kernels and of wide batches beside adapters.
//
// x is "packed" first: its elements become pairs of f16,
//     x * 2^s = hi + lo,   hi = f16(x 2^s),   lo = f16(x 2^s - hi)
// with a power of two 2^s, one for a column of x and one for every 32 gated values, that puts the
// largest magnitude under it into [2^14, 2^15): hi + lo carries x to 2^-22 of itself or 2^-39 of
// the largest, whichever is more (columns for which that is too much go another way, below): 22
// bits where 24 would need a third product.  The weights' codes are exact in f16, the products of f16 are exact in
// the 32-bit accumulators, and the blocks' scales multiply the accumulated sum of a block in
// 32 bits: the only roundings are those of 32-bit sums (truncated ones in the matrix unit,
// which is why its sums end with the block, and take the low parts first).
//
// Codes become f16 by masks and, where the format has an offset (8 and 128), one packed
// operation for two of them: the f16 with the bits 0x6400 | c is 1024 + c, and taking 1024 and
// the offset off is exact.  (Leaving the offset to the block's sum, as -offset times the sum of
// x, saves that operation but not a sum's rounding: an x of 1e5 among units on a weight of zero
// moved the other weights' products by more than the parity bound.)  Q4_K's codes have none,
// its mins being a term of the format's own definition: masked in place, the f16 with the bits
// of 64 c is the subnormal c 2^-18, which the matrix unit takes exactly.  It lines its products
// up by the operands' exponents, though, a subnormal's being that of 2^-14: a code is placed
// high enough that what it drops stays at the level of a 32-bit sum's rounding (in the lowest
// bits: an error of 5e-6 of the result; 16 times the code: 5e-7).  Its sums are in units of
// 2^-18, taken back in the tail.
//
// Why mma.sync: a block format's scale belongs to 32 weights of one row, and here a block's sum is
// scaled where it arises, in registers; with accumulators in tensor memory that would be one
// read-back per two instructions.  (The asynchronous unit could take weights that are scaled
// already: two f16 parts hold a scale times a code exactly, 11 bits times 4, 8 or 10, under a
// power of two per row, at three products instead of two and a way through shared memory for
// every decoded weight.  That is not built.  F16 batches of up to 16 columns a pass, which
// have no scales, go that way in gemv_tc.cu.)
//
// F32 weights take tf32 instructions: w = hi + lo in two tf32 (to 2^-22 of it), and the sums
// hi(w) hi(x) + lo(w) hi(x) + hi(w) lo(x); hi(x) and lo(x), f16, are exact in tf32.
#pragma once

#include "gf_internal.h"
#include "tc_device.cuh"

namespace gf {

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = A B.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// tf32 operands (f32 registers whose low 13 bits do not count), k = 8.
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t to_tf32(float v) {  // to nearest
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
  return r;
}
template <int N>
struct TileConst {
  static constexpr int value = N;
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

constexpr int kTileK = 256;  // K of a chunk
constexpr int kTileBlocks = kTileK / 32;
template <int WT>
__host__ __device__ constexpr int tile_seg() {  // bytes of a row and chunk
  return WT == WT_F32 ? 4 * kTileK : WT == WT_F16 ? 2 * kTileK : WT == WT_Q8_0 ? kTileBlocks * 34 : 144;
}

// ------------------------------------------------------------------ packing x
// Packed columns lie in the order in which the matrix instruction takes them.  Eight columns
// form a column tile, and for every 32 elements a column tile has one record:
//   [step s of 2][column of cp][thread t of 4] 16 bytes {hi, hi, hi, hi, lo, lo, lo, lo},
//   then per column {2^-s, for Q4_K the block's sum of x 2^s in the units of its sums};
// or, in a block that the two parts cannot carry (below), four 32-bit elements in place of the 16
// bytes and {kRawBlock, their factor} behind them (all blocks of a packed column, single blocks
// of the gated values);
// cp = min(8, columns of the group) columns are stored, so that a single column does not move
// eight (column tiles are allocated for the most any group of the call can have).  A warp's
// 16-byte reads of a step are then consecutive, and the records of a K chunk are one piece of
// memory for one bulk copy.  Which four elements (s, t) holds is the
// weights' choice: 16 s + 4 t + .. in the order 0, 2, 1, 3 for the nibble formats (two masks
// take a code word apart in that order), 16 s + 4 t + 0..3 for Q8_0 and F32, and 8 t + 4 s + 0..3
// for F16 (a thread then reads 16 bytes of a row at once).
enum { ORDER_NIBBLE = 0, ORDER_BYTE = 1, ORDER_F16 = 2 };
__host__ __device__ constexpr int pack_order(int wt) {
  return wt == WT_F16 ? ORDER_F16 : wt == WT_Q8_0 || wt == WT_F32 ? ORDER_BYTE : ORDER_NIBBLE;
}
// Q4_K's mins multiply the sum of x over a block.
__host__ __device__ constexpr bool pack_sums(int wt) { return wt == WT_Q4_K; }
// Unit of the accumulators.
__host__ __device__ constexpr float tile_unit(int wt) { return wt == WT_Q4_K ? 0x1p18f : 1.0f; }
__host__ __device__ constexpr int record_bytes(int cp) { return cp * 128 + (cp * 8 + 15) / 16 * 16; }
// Byte offset in a record of the four elements 4q .. 4q + 3 of column c.
__device__ __forceinline__ uint32_t record_offset(uint32_t q, uint32_t c, uint32_t cp, int order) {
  const uint32_t s = order == ORDER_F16 ? (q & 1u) : (q >> 2), t = order == ORDER_F16 ? (q >> 1) : (q & 3u);
  return (s * cp + c) * 64u + t * 16u;
}

// 2^s for the largest magnitude m (finite), s in [-113, 126]; 1 for m = 0.
__device__ __forceinline__ float pack_scale(float m) {
  const int e = static_cast<int>((__float_as_uint(m) >> 23) & 0xFFu);  // m in [2^(e-127), 2^(e-126))
  const int s = m == 0.0f ? 0 : max(-126, min(126, 14 + 127 - e));
  return __uint_as_float(static_cast<uint32_t>(s + 127) << 23);
}
// The inverse of a power of two in [2^-126, 2^126].
__device__ __forceinline__ float pow2_inverse(float p) {
  return __uint_as_float((254u << 23) - __float_as_uint(p));
}

// What the two parts carry.  Under one scale for a packed column (a block of gated values) whose
// largest magnitude is m, hi + lo moves a value by at most 2^-22 of itself or 2^-39 m, whichever
// is more.  That is little next to the products of a row unless many values lie far below m and
// the weights of those near m are zero; and a NaN or an infinity in hi makes NaN of what should be
// an infinity (the other part, or Q4_K's mins, take it off again).  A value is tiny where it is
// not zero and below 2^-18 m (the others move by at most 2^-21 of themselves).  Carried is what
// holds a NaN, since nothing but NaN comes of it, and are finite values
//  - of a packed column, if m times the sum over every four neighbours of 1 / q, q the sum of the
//    two smaller of them, is at most 2^16 K (the four then move by at most 2^-19 q on the mean) or
//    if at most an eighth of them are tiny (normal values: m up to 40000 standard deviations; the
//    first rule needs no second look at the column);
//  - of a block of 32 gated values, if none is tiny or four or more are at least 2^-14 m (all
//    together then move by at most 2^-21 of the two smaller of these).
// (A row whose weights are zero but where x is smallest can still exceed the parity bound.)
constexpr float kCarryTiny = 0x1p-18f, kCarryFours = 0x1p-16f, kCarryBlock = 0x1p-14f;

// In place of a block's 2^-s where its elements are stored as they are: a NaN that no arithmetic
// makes, so that every sum with that block is NaN too.
constexpr uint32_t kRawBlock = 0x7FC0AC7Fu;
__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) <= 3.402823466e38f; }

struct HiLo {
  __half hi, lo;
};
// x must be scaled already.
__device__ __forceinline__ HiLo split_hi_lo(float v) {
  HiLo r;
  r.hi = __float2half_rn(v);
  const float rest = v - __half2float(r.hi);
  r.lo = __float2half_rn(rest);
  return r;
}

__device__ __forceinline__ uint32_t half_pair(__half a, __half b) {
  return static_cast<uint32_t>(__half_as_ushort(a)) | (static_cast<uint32_t>(__half_as_ushort(b)) << 16);
}

__device__ __forceinline__ float value_of(const HiLo& p) { return __half2float(p.hi) + __half2float(p.lo); }

// Four consecutive scaled elements as the 16 bytes of a packed group, and the sum of what these
// hold: the mins multiply the sum of the same values that the codes multiply.
__device__ __forceinline__ uint4 pack_group(float4 v, bool swapped, float& sum) {
  const HiLo a = split_hi_lo(v.x), b = split_hi_lo(v.y), c = split_hi_lo(v.z), d = split_hi_lo(v.w);
  sum = (value_of(a) + value_of(b)) + (value_of(c) + value_of(d));
  return swapped ? make_uint4(half_pair(a.hi, c.hi), half_pair(b.hi, d.hi), half_pair(a.lo, c.lo), half_pair(b.lo, d.lo))
                 : make_uint4(half_pair(a.hi, b.hi), half_pair(c.hi, d.hi), half_pair(a.lo, b.lo), half_pair(c.lo, d.lo));
}

// Column c of a column tile's records, by a CTA of THREADS (at most kPackThreads); one scale
// for the whole column.  With gamma the column is first normalised, x / sqrt(mean(x^2) + eps)
// gamma: gamma multiplies before packing, the root enters through the stored scale.  wmax:
// kPackWords floats of shared memory.  Returns whether the column went raw.
constexpr int kPackThreads = 1024;
constexpr int kPackWords = 4 * kPackThreads / 32;
template <int THREADS>
__device__ __forceinline__ bool pack_column(const float* x, int c, const float* gamma, float eps, int K, int fmt, int cp, uint8_t* base,
                                   float* wmax) {
  const int i0 = threadIdx.x;
  const int lane = threadIdx.x & 31;
  const int n4 = K / 4, order = pack_order(fmt);
  const bool sums = pack_sums(fmt);
  const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(gamma)) & 15u) == 0;
  auto four = [&](const float* p, int i) -> float4 {
    if (vec) return reinterpret_cast<const float4*>(p)[i];
    return make_float4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
  };
  float ss = 0.0f;
  auto load = [&](int i, bool sq) -> float4 {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < n4) {
      v = four(x, i);
      if (gamma != nullptr) {
        if (sq) ss = fmaf(v.x, v.x, fmaf(v.y, v.y, fmaf(v.z, v.z, fmaf(v.w, v.w, ss))));
        const float4 g = four(gamma, i);
        v.x *= g.x; v.y *= g.y; v.z *= g.z; v.w *= g.w;
      }
    }
    return v;
  };
  bool nan = false, inf = false;  // of any element
  float small = 0.0f;             // sum over every four elements of 1 / (the two smaller magnitudes)
  auto top = [&](float4 v) {
    const float a = fabsf(v.x), b = fabsf(v.y), c4 = fabsf(v.z), d = fabsf(v.w), all = (a + b) + (c4 + d);
    nan |= all != all;
    inf |= all > 3.402823466e38f;
    const float h0 = fmaxf(a, b), h1 = fmaxf(c4, d), l0 = fminf(a, b), l1 = fminf(c4, d);
    small += __frcp_rn(fminf(l0, l1) + fminf(fmaxf(l0, l1), fminf(h0, h1)));
    return is_finite(fmaxf(h0, h1)) ? fmaxf(h0, h1) : 0.0f;  // (the others do not set the scale)
  };
  auto tiny = [&](float4 v, float edge) {
    auto is = [&](float e) { return e != 0.0f && fabsf(e) < edge ? 1u : 0u; };
    return is(v.x) + is(v.y) + is(v.z) + is(v.w);
  };
  constexpr int kKeep = 2;  // groups of four a thread keeps between the two passes
  float4 keep[kKeep];
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < kKeep; ++j) keep[j] = load(i0 + THREADS * j, true);
#pragma unroll
  for (int j = 0; j < kKeep; ++j)
    if (i0 + THREADS * j < n4) m = fmaxf(m, top(keep[j]));
  for (int i = i0 + THREADS * kKeep; i < n4; i += THREADS) m = fmaxf(m, top(load(i, true)));
  m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    small += __shfl_xor_sync(0xffffffffu, small, o);
  }
  nan = __any_sync(0xffffffffu, nan);
  inf = __any_sync(0xffffffffu, inf);
  if (lane == 0) {
    wmax[threadIdx.x >> 5] = m;
    wmax[kPackThreads / 32 + (threadIdx.x >> 5)] = ss;
    wmax[2 * kPackThreads / 32 + (threadIdx.x >> 5)] = nan ? 2.0f : inf ? 1.0f : 0.0f;
    wmax[3 * kPackThreads / 32 + (threadIdx.x >> 5)] = small;
  }
  __syncthreads();
  ss = small = 0.0f;
  for (int q = 0; q < THREADS / 32; ++q) {
    m = fmaxf(m, wmax[q]);
    ss += wmax[kPackThreads / 32 + q];
    nan |= wmax[2 * kPackThreads / 32 + q] == 2.0f;
    inf |= wmax[2 * kPackThreads / 32 + q] == 1.0f;
    small += wmax[3 * kPackThreads / 32 + q];
  }
  // (normalised by an infinite mean square, what is finite is zero and the rest NaN: as packed)
  bool raw = inf && !nan && (gamma == nullptr || is_finite(ss));
  if (!inf && !nan && !(m * kCarryFours * small <= static_cast<float>(K))) {  // (the same for the whole column)
    unsigned n = 0;
#pragma unroll 1
    for (int i = i0; i < n4; i += THREADS) n += tiny(load(i, false), m * kCarryTiny);
    n = __reduce_add_sync(0xffffffffu, n);
    __syncthreads();
    if (lane == 0) wmax[threadIdx.x >> 5] = static_cast<float>(n);
    __syncthreads();
    float all = 0.0f;
    for (int q = 0; q < THREADS / 32; ++q) all += wmax[q];
    raw = 8.0f * all > static_cast<float>(K);
  }
  const float sc = pack_scale(m);
  const float root = gamma != nullptr ? 1.0f / sqrtf(ss / static_cast<float>(K) + eps) : 1.0f;
  const float inv = pow2_inverse(sc) * root;
  const int rec = record_bytes(cp);
  auto put = [&](int i, float4 v) {
    if (raw) {
      if (i < n4) {
        uint8_t* r = base + static_cast<int64_t>(i >> 3) * rec;
        *reinterpret_cast<float4*>(r + record_offset(i & 7, c, cp, order)) = v;
        if ((i & 7) == 0) *reinterpret_cast<float2*>(r + cp * 128 + c * 8) = make_float2(__uint_as_float(kRawBlock), root);
      }
      return;
    }
    v.x *= sc; v.y *= sc; v.z *= sc; v.w *= sc;
    float sum;
    const uint4 packed = pack_group(v, order == ORDER_NIBBLE, sum);
    if (sums)
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (i < n4) {
      uint8_t* r = base + static_cast<int64_t>(i >> 3) * rec;
      *reinterpret_cast<uint4*>(r + record_offset(i & 7, c, cp, order)) = packed;
      if ((i & 7) == 0) *reinterpret_cast<float2*>(r + cp * 128 + c * 8) = make_float2(inv, sums ? sum / tile_unit(WT_Q4_K) : 0.0f);
    }
  };
#pragma unroll
  for (int j = 0; j < kKeep; ++j) put(i0 + THREADS * j, keep[j]);
  for (int b = THREADS * kKeep; b < n4; b += THREADS) put(b + i0, load(b + i0, false));
  __syncthreads();  // the column is written; wmax may be used again
  return raw;
}

// ------------------------------------------------------------------ A fragments
// d * sc[j] and dmin * m[j] of a Q4_K super-block from its first 16 bytes (both exact).  The
// 6-bit integers become floats in the low bits of 2^23: a conversion instruction has a
// quarter of an addition's rate.
__device__ __forceinline__ void q4k_scale_of(const uint4 hd, uint32_t j, float& dsc, float& dmn) {
  const uint32_t sh = 8u * (j & 3u);
  const uint32_t x = hd.y >> sh, y = hd.z >> sh, z = hd.w >> sh;
  const uint32_t sc = j < 4u ? (x & 63u) : ((z & 15u) | ((x >> 2) & 48u));
  const uint32_t mn = j < 4u ? (y & 63u) : (((z >> 4) & 15u) | ((y >> 2) & 48u));
  dsc = h2f(hd.x & 0xFFFFu) * (__uint_as_float(0x4B000000u | sc) - kMagic);
  dmn = h2f(hd.x >> 16) * (__uint_as_float(0x4B000000u | mn) - kMagic);
}

constexpr uint32_t kNibbles = 0x03C003C0u;  // two 4-bit codes as c 2^-18

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_half2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
// 1024 + c of two codes (f16) -> c - OFF.
template <int OFF>
__device__ __forceinline__ uint32_t code_pair(uint32_t u) {
  return half2_bits(__hsub2(bits_half2(u), __half2half2(__int2half_rn(1024 + OFF))));
}
// 1024 + 16 c -> c - 8.
__device__ __forceinline__ uint32_t code_pair_16(uint32_t u) {
  return half2_bits(__hfma2(bits_half2(u), __float2half2_rn(0.0625f), __float2half2_rn(-72.0f)));
}

// One lane's place in a row of a stage: what it reads of its warp's block.
struct RowPlace {
  uint32_t code;   // first aligned word of its codes
  uint32_t scale;  // the block's scale (Q4_0, Q8_0)
  uint32_t shift;  // bits the codes start above that word's first (0 or 16)
  uint32_t left, right;  // Q4_K: shifts that bring its nibbles into place
};
template <int WT>
__device__ __forceinline__ RowPlace row_place(uint32_t row, uint32_t blk, uint32_t t) {
  RowPlace p = {};
  if constexpr (WT == WT_Q8_0 || WT == WT_Q4_0) {
    p.scale = row + blk * (WT == WT_Q8_0 ? 34u : 18u);
    const uint32_t c = p.scale + 2u + 4u * t;
    p.code = c & ~3u;
    p.shift = (c & 3u) * 8u;
  } else if constexpr (WT == WT_Q4_K) {
    p.code = row + 16u + ((blk >> 1) & 3u) * 32u + 4u * t;
    p.left = 6u - 4u * (blk & 1u);
    p.right = 2u + 4u * (blk & 1u);
  } else {
    p.code = row;  // F16: swizzled by the caller
  }
  return p;
}

// One 32-element block of a row, at `off` bytes from the place, as A operands of two
// m16n8k16 steps: a[step] = {k-slots 2t, 2t+1; 2t+8, 2t+9}.  Which element sits in which
// k-slot is free as long as the packed x has the same one (see pack_order).
// WHOLE: the codes start on a word (shift 0).  d: the block's scale.
template <int WT, bool WHOLE>
__device__ __forceinline__ void load_block_row(const RowPlace& p, uint32_t off, uint32_t (&a0)[2], uint32_t (&a1)[2],
                                               float& d) {
  if constexpr (WT == WT_F16) {
    const uint4 u = lds128(p.code + off);
    a0[0] = u.x; a0[1] = u.y;
    a1[0] = u.z; a1[1] = u.w;
    d = 1.0f;
  } else if constexpr (WT == WT_Q8_0) {
    d = h2f(lds16(p.scale + off));
    uint32_t u = lds32(p.code + off), v = lds32(p.code + off + 16u);
    if constexpr (!WHOLE) {
      u = __funnelshift_r(u, lds32(p.code + off + 4u), p.shift);
      v = __funnelshift_r(v, lds32(p.code + off + 20u), p.shift);
    }
    u ^= 0x80808080u;  // q + 128
    v ^= 0x80808080u;
    a0[0] = code_pair<128>(__byte_perm(u, 0x64646464u, 0x4140));
    a0[1] = code_pair<128>(__byte_perm(u, 0x64646464u, 0x4342));
    a1[0] = code_pair<128>(__byte_perm(v, 0x64646464u, 0x4140));
    a1[1] = code_pair<128>(__byte_perm(v, 0x64646464u, 0x4342));
  } else if constexpr (WT == WT_Q4_K) {  // scale and min come apart elsewhere
    const uint32_t w = lds32(p.code + off), v = lds32(p.code + off + 16u);
    a0[0] = (w << p.left) & kNibbles;
    a0[1] = (w >> p.right) & kNibbles;
    a1[0] = (v << p.left) & kNibbles;
    a1[1] = (v >> p.right) & kNibbles;
    d = 1.0f;
  } else {  // Q4_0
    d = h2f(lds16(p.scale + off));
    uint32_t w = lds32(p.code + off);
    if constexpr (!WHOLE) w = __funnelshift_r(w, lds32(p.code + off + 4u), p.shift);
    const uint32_t v = w >> 8;
    a0[0] = code_pair<8>((w & 0x000F000Fu) | 0x64006400u);   // elements 4t, 4t + 2
    a0[1] = code_pair<8>((v & 0x000F000Fu) | 0x64006400u);   // 4t + 1, 4t + 3
    a1[0] = code_pair_16((w & 0x00F000F0u) | 0x64006400u);   // the same + 16
    a1[1] = code_pair_16((v & 0x00F000F0u) | 0x64006400u);
  }
}

// ------------------------------------------------------------------ the tiled kernel
// A work item is (column group, row tile): up to 8 NT columns that share one matrix, and
// 64 rows of it (gated: 32 gate rows and the same up rows).  Warp 0 streams the rows' weights
// in K chunks of 256, by tensor-map copies of 32 rows, through a ring of shared-memory
// stages.  The columns' records are brought in once for all the row tiles of a group that a
// CTA has (items are handed out in that order) where the whole K of them fits beside three
// stages, else chunk by chunk with the weights.  The eight
// consumer warps share the K axis: a warp takes one 32-element block of the chunk for all 64
// rows (four 16-row matrix tiles), so that a packed x fragment, once loaded, serves four
// matrix tiles.  At the end of an item the warps' accumulators are added through shared
// memory in warp order (deterministic) and the tail is applied.  Up to two column tiles two
// CTAs share an SM, so that one's reduction overlaps the other's stream; three take the
// registers of one.
//
// (A first version copied every row of a chunk by its own bulk copy: each took about 90
// cycles of an SM's copy engine whatever its size, three to ten times the time of the bytes.
// One without a copying warp, whose warps took turns refilling a stage, fell into step with
// itself and was 10 to 30% slower.)
//
// Rows in a stage.  Q4_0, Q4_K: 144 bytes a row and chunk, Q8_0: 272, odd multiples of 16, so
// that the eight rows a warp reads together fall on distinct banks.  Where K is no multiple
// of 256, rows of these formats are no whole number of 16-byte words, which a tensor map
// cannot express; but `period` = 2, 4 or 8 rows together are, and the map is laid over
// those: the rows of each residue are copied apart, from the 16-byte boundary before them
// and 32 bytes wider.  F16: four boxes of 64 elements, 128-byte swizzled; lanes 2q and
// 2q + 1 take rows q and q + 4 of eight, so that a quarter warp's reads cover all banks.
//
// Every wait is bounded; a timeout sets the device error word, and the kernel returns after
// draining its own copies.
constexpr int kTileRows = 64;
constexpr int kTileWarps = 8;           // consumer warps, sharing K
constexpr int kTileThreads = 32 * (1 + kTileWarps);
constexpr int kTileMaxStages = 8;
constexpr int kTileMaxGroups = 64;      // column groups a CTA's items may touch
constexpr int kTileHeadBytes = 256 + 16 * kTileMaxGroups;  // barriers, abort flag, groups
constexpr int kTileMaxXBuffers = 2;
constexpr int kRedPitch = kTileRows + 4;
constexpr int kTileRedBytes = kTileWarps * 8 * kRedPitch * 4;  // the warps' sums of eight columns
// The gated product; one that scales each column by a factor of its own; the plain product
// of all columns of a batch with a fused tail.
enum { TILE_GLU = 0, TILE_DOWN = 1, TILE_LIN = 2 };
// Rows without codes: swizzled 128-byte boxes.
__host__ __device__ constexpr bool tile_plain(int wt) { return wt == WT_F16 || wt == WT_F32; }
// (F32's stages are too large for two CTAs.)
__host__ __device__ constexpr int tile_ctas(int wt, int nt) { return nt <= 2 && wt != WT_F32 ? 2 : 1; }

// Rows that make a whole number of 16-byte words.
__host__ __device__ constexpr int tile_period(int row_bytes) {
  return row_bytes % 16 == 0 ? 1 : row_bytes % 8 == 0 ? 2 : row_bytes % 4 == 0 ? 4 : 8;
}
template <int WT>
__host__ __device__ constexpr int tile_pitch(int period) { return tile_seg<WT>() + (period > 1 ? 32 : 0); }
// Bytes of the rows of one residue in a 32-row half (boxes start on 128-byte boundaries).
template <int WT>
__host__ __device__ constexpr int tile_part(int period) {
  return (32 / period * tile_pitch<WT>(period) + 127) / 128 * 128;
}
template <int WT>
__host__ __device__ constexpr int tile_weight_bytes(int period) {
  return tile_plain(WT) ? kTileRows * tile_seg<WT>() : 2 * period * tile_part<WT>(period);
}
// Chunks of a stage: two where a stage of one holds little (a wait serves two blocks of each
// warp then, whose instructions interleave).
__host__ __device__ constexpr int tile_chunks(int wt, int nt) { return (wt == WT_Q4_0 || wt == WT_Q4_K) && nt == 1 ? 2 : 1; }
// One chunk of a stage: weights, and in the chunk by chunk case its records.
template <int WT>
__host__ __device__ constexpr int tile_stage_bytes(int period, int nt, int cp, bool resident) {
  return (tile_weight_bytes<WT>(period) + 16 + (resident ? 0 : nt * kTileBlocks * record_bytes(cp)) + 1023) / 1024 * 1024;
}
// Records of a group's whole K.
__host__ __device__ constexpr int64_t tile_x_bytes(int K, int nt, int cp) {
  return (static_cast<int64_t>(nt) * (K / 32) * record_bytes(cp) + 127) / 128 * 128;
}

struct TileArgs {
  int rows, K, row_bytes;   // rows of one matrix (outputs), columns
  int period;
  const int4* groups;       // {matrix, first entry, columns, first column tile}
  const int32_t* n_groups;
  int max_groups;           // entries `groups` has room for
  uint32_t* next;           // wide kernel, but for TILE_LIN: the next item to be taken (zero at the start)
  const int32_t* slots;     // slot of each entry
  const uint8_t* W;         // TILE_LIN: the matrix, for raw columns (the stages are filled by tensor maps)
  const uint8_t* records;   // [column tile][K / 32] records of x
  int cp;                   // most columns stored per column tile
  int NS;
  int xbuffers;             // 1 or 2 buffers of a group's records; 0: they come chunk by chunk
  unsigned* err;
  // tails
  uint8_t* out_records;     // TILE_GLU: records of the next product's x
  int out_format;           // of the next product's weights
  const float* factors;     // TILE_DOWN: factor of a slot
  float* out;               // TILE_DOWN: [slot][out_ld]; TILE_LIN: [column][out_ld]
  int64_t out_ld;
  const float* aux;         // TILE_LIN: may be `out`
  int epi;
  int ncols, group_cols;    // TILE_LIN: columns of the batch, of a group (no list of groups)
  int item_rows;            // wide kernel, TILE_LIN: rows of an item
};

// ------------------------------------------------------------------ raw columns
// A raw column's sums in the tiles go nowhere.  Its products are taken element by
// element: the gated ones by the launch that packs it, which the tiles follow (in the tiles'
// kernel this code took 3 to 7% of every call's time without running), a batch's behind the
// tiles' own; and a down product that a raw block made NaN by the combination.
//
// R rows, `stride` bytes apart, times one packed column in 32 bits, by a warp; every lane gets the
// sums.  Lean: the kernels that hold it pay for its registers and, where it needs a stack, at
// every launch.  rec: the column tile's first record, cp columns stored, this one c.
template <int WT, int R>
__device__ __forceinline__ void exact_products(const uint8_t* row, int64_t stride, const uint8_t* rec, uint32_t c, uint32_t cp,
                                               int K, float (&s)[R]) {
  constexpr int kOrder = pack_order(WT);
  const uint32_t lane = threadIdx.x & 31u, i = lane & 3u;
  const uint32_t at = record_offset(lane >> 2, c, cp, kOrder), half = kOrder == ORDER_NIBBLE ? ((i & 1u) << 1) | (i >> 1) : i;
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = 0.0f;
#pragma unroll 1
  for (int b = 0; b < K / 32; ++b) {  // a lane's element of each block
    const float2 meta = *reinterpret_cast<const float2*>(rec + cp * 128u + c * 8u);
    float x;
    if (__float_as_uint(meta.x) == kRawBlock) {
      x = meta.y * reinterpret_cast<const float*>(rec + at)[i];
    } else {
      const __half* h = reinterpret_cast<const __half*>(rec + at) + half;
      x = meta.x * (__half2float(h[0]) + __half2float(h[4]));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = fmaf(decode_elem<WT>(row + r * stride, 32 * (b & 7) + static_cast<int>(lane)), x, s[r]);
    rec += record_bytes(static_cast<int>(cp));
    if ((b & 7) == 7) row += tile_seg<WT>();
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
}
// 32 rows from `row` on, R at a time: lane r gets the r-th.
template <int WT, int R>
__device__ __forceinline__ float exact_block(const uint8_t* row, int64_t stride, const uint8_t* rec, uint32_t c, uint32_t cp,
                                             int K) {
  float y = 0.0f, s[R];
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += R) {
    exact_products<WT, R>(row + r0 * stride, stride, rec, c, cp, K, s);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (static_cast<int>(threadIdx.x & 31u) == r0 + r) y = s[r];
  }
  return y;
}

// A block of 32 gated values of one column, a lane's each, into its record r (cp columns stored,
// this one c) for a product in format fmt.
__device__ __forceinline__ void write_gated(float h, uint8_t* r, uint32_t c, uint32_t cp, int fmt) {
  const uint32_t lane = threadIdx.x & 31u, i = lane & 3u;
  const int order = pack_order(fmt);
  const uint32_t at = record_offset(lane >> 2, c, cp, order);
  float2 meta;
  const bool nan = __any_sync(0xffffffffu, h != h);
  const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, h == h ? __float_as_uint(fabsf(h)) : 0u));
  const uint32_t big = __ballot_sync(0xffffffffu, fabsf(h) >= m * kCarryBlock);
  const uint32_t not_tiny = __ballot_sync(0xffffffffu, h == 0.0f || fabsf(h) >= m * kCarryTiny);
  if (!nan && (!is_finite(m) || (__popc(big) < 4 && not_tiny != 0xffffffffu))) {
    *reinterpret_cast<float*>(r + at + 4u * i) = h;
    meta = make_float2(__uint_as_float(kRawBlock), 1.0f);
  } else {
    const float sc = pack_scale(is_finite(m) ? m : 0.0f);
    const HiLo p = split_hi_lo(h * sc);
    float sum = value_of(p);
    if (pack_sums(fmt))
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const uint32_t place = at + 2u * (order == ORDER_NIBBLE ? ((i & 1u) << 1) | (i >> 1) : i);
    *reinterpret_cast<__half*>(r + place) = p.hi;
    *reinterpret_cast<__half*>(r + place + 8u) = p.lo;
    meta = make_float2(pow2_inverse(sc), pack_sums(fmt) ? sum / tile_unit(WT_Q4_K) : 0.0f);
  }
  if (lane == 0) *reinterpret_cast<float2*>(r + cp * 128u + c * 8u) = meta;
}

__device__ __forceinline__ const uint8_t* column_records(const TileArgs& a, const int4& g, int col) {
  return a.records + (g.w + col / 8) * (static_cast<int64_t>(a.K / 32) * record_bytes(a.cp));
}
// Whether column col of group g is raw.
__device__ __forceinline__ bool raw_column(const TileArgs& a, const int4& g, int col) {
  const uint32_t cp = static_cast<uint32_t>(min(8, g.z));
  return *reinterpret_cast<const uint32_t*>(column_records(a, g, col) + cp * 128u + (col & 7) * 8u) == kRawBlock;
}
// TILE_LIN: the 32 output rows from row0 of a raw column of group g, by a warp.
template <int WT>
__device__ __forceinline__ void exact_rows(const TileArgs& a, const int4& g, int col, int row0) {
  const int lane = threadIdx.x & 31, r = row0 + lane;
  if (lane == 0) atomicAdd(a.err + 1, 1u);  // counted for gf_repair_count
  const uint8_t *W = a.W + static_cast<int64_t>(row0) * a.row_bytes, *rec = column_records(a, g, col);
  const uint32_t c = static_cast<uint32_t>(col) & 7u, cp = static_cast<uint32_t>(min(8, g.z));
  float y = 0.0f;
  if (row0 + 32 <= a.rows) {
    y = exact_block<WT, 4>(W, a.row_bytes, rec, c, cp, a.K);
  } else {
#pragma unroll 1
    for (int i = 0; i < a.rows - row0; ++i) {
      float s[1];
      exact_products<WT, 1>(W + i * static_cast<int64_t>(a.row_bytes), 0, rec, c, cp, a.K, s);
      if (i == lane) y = s[0];
    }
  }
  if (r < a.rows) {
    const int64_t o = (static_cast<int64_t>(g.w) * 8 + col) * a.out_ld + r;
    a.out[o] = apply_tail(a.epi, y, epi_takes_aux(a.epi) ? a.aux[o] : 0.0f);  // aux may be out
  }
}

// One lane's constants of the walk over a stage.
struct TileLane {
  uint32_t rowbase, step8, step16, half;  // rows row8, + 8, + 16, + 32
  uint32_t row8, t4;
  uint32_t xlane, m0, m1, cp, rec;        // of the group's records
  uint32_t xtile;                         // distance of column tiles in shared memory
};

// This warp's block `blk` of a stage (weights at st, its records at xs): acc += W x for 64
// rows and NTA column tiles.  PER1: rows lie at the constant pitch of period 1.  FEW: up to four
// columns, whose hi parts are the columns 0..3 and whose lo parts are the columns 4..7 of one
// matrix tile: half the matrix instructions, and half as many in a row (whole calls with cold
// weights: one token through 8 of 128 Q4_0 experts of 768 x 2048 24.0 -> 23.2 us, Q8_0 26.8 ->
// 26.0; 4 columns of 14336 x 4096 Q4_0 with adapters 28.0 -> 27.1, Q4_K 31.7 -> 30.6).
template <int WT, int MODE, int NTA, int NT, bool PER1, bool WHOLE, bool FEW>
__device__ __forceinline__ void tile_block(const TileLane& l, uint32_t st, uint32_t xs, uint32_t blk,
                                           float (&acc)[4][NT][4]) {
  constexpr bool kMeta = MODE == TILE_DOWN || pack_sums(WT);  // per-block scales or sums are read here
  constexpr uint32_t kP = tile_pitch<WT>(1);
  const uint32_t step8 = WT == WT_F16 ? 1024u : PER1 ? 8u * kP : l.step8;
  const uint32_t step16 = WT == WT_F16 ? 2048u : PER1 ? 16u * kP : l.step16;
  const uint32_t half = WT == WT_F16 ? 4096u : PER1 ? static_cast<uint32_t>(tile_part<WT>(1)) : l.half;
  uint4 b[NTA][2];
  float2 meta[NTA][2];  // of columns 2t and 2t + 1 of each column tile
#pragma unroll
  for (int n = 0; n < NTA; ++n) {
    const uint32_t xa = xs + static_cast<uint32_t>(n) * l.xtile;
    if constexpr (FEW) {
      const uint2 u = lds64(xa + l.xlane), v = lds64(xa + l.xlane + l.cp * 64u);
      b[n][0] = make_uint4(u.x, u.y, 0u, 0u);
      b[n][1] = make_uint4(v.x, v.y, 0u, 0u);
    } else {
      b[n][0] = lds128(xa + l.xlane);
      b[n][1] = lds128(xa + l.xlane + l.cp * 64u);
    }
    if constexpr (kMeta) {
      const uint2 u = lds64(xa + l.m0), v = lds64(xa + l.m1);
      meta[n][0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      meta[n][1] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
      if constexpr (FEW && pack_sums(WT)) {  // a column's sum counts once, beside its hi part
        meta[n][0].y = l.t4 < 2u ? meta[n][0].y : 0.0f;
        meta[n][1].y = l.t4 < 2u ? meta[n][1].y : 0.0f;
      }
    }
  }
  const uint32_t row = st + l.rowbase;
  RowPlace place = row_place<WT>(row, blk, l.t4);
  if constexpr (WT == WT_F16)  // box blk / 2, 16-byte word 4 (blk % 2) + t of the 128, swizzled by the row
    place.code += (blk >> 1) * 8192u + ((((blk & 1u) * 4u + l.t4) ^ l.row8) << 4);
  // Q4_K: taking a row's 6-bit scale and min apart costs as much as its codes; the four
  // lanes of a row would all do it, so lane t does it for matrix tile t only
  float qd[2], qm[2];
  if constexpr (WT == WT_Q4_K) {
    const uint32_t mine = row + (l.t4 & 1u) * step16 + (l.t4 >> 1) * half;
    q4k_scale_of(lds128(mine), blk, qd[0], qm[0]);
    q4k_scale_of(lds128(mine + step8), blk, qd[1], qm[1]);
  }
  // A matrix instruction takes long to give its sum back and the four of a block follow one
  // another in it: MG matrix tiles are taken side by side
  constexpr int MG = 2;
#pragma unroll
  for (int mg = 0; mg < 4; mg += MG) {
    uint32_t a0[MG][2][2], a1[MG][2][2];
    float d[MG][2], dm[MG][2];
#pragma unroll
    for (int j = 0; j < MG; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = mg + j;
        load_block_row<WT, WHOLE>(place, (m & 1) * step16 + (m >> 1) * half + h * step8, a0[j][h], a1[j][h], d[j][h]);
        dm[j][h] = 0.0f;
        if constexpr (WT == WT_Q4_K) {
          d[j][h] = __shfl_sync(0xffffffffu, qd[h], m, 4);
          dm[j][h] = __shfl_sync(0xffffffffu, qm[h], m, 4);
        }
      }
    // lo of both k-steps, then hi: the matrix unit cuts its sums off, toward zero, at the size
    // they have reached.  For the same reason they end with the block (a sum over all of K in its
    // accumulators was off by 2e-6 of itself, all to one side)
    float s[MG][NTA][4];
    auto step = [&](int i) {
#pragma unroll
      for (int j = 0; j < MG; ++j)
#pragma unroll
        for (int n = 0; n < NTA; ++n) {
          const uint32_t (&x)[2][2] = (i & 1) ? a1[j] : a0[j];
          const uint4 v = b[n][i & 1];
          const uint32_t p = i < 2 && !FEW ? v.z : v.x, q = i < 2 && !FEW ? v.w : v.y;
          if (i == 0)
            mma_f16_first(s[j][n], x[0][0], x[1][0], x[0][1], x[1][1], p, q);
          else
            mma_f16(s[j][n], x[0][0], x[1][0], x[0][1], x[1][1], p, q);
        }
    };
    step(0);
    step(1);
    if constexpr (!FEW) {
      step(2);
      step(3);
    }
#pragma unroll
    for (int j = 0; j < MG; ++j)
#pragma unroll
      for (int n = 0; n < NTA; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // row row8 (0, 1) or row8 + 8 (2, 3), column 2t + (i & 1)
          const int h = i >> 1, c = i & 1;
          float& o = acc[mg + j][n][i];
          if constexpr (MODE == TILE_DOWN) {
            float v = WT == WT_F16 ? s[j][n][i] : d[j][h] * s[j][n][i];
            if constexpr (WT == WT_Q4_K) v = fmaf(-dm[j][h], meta[n][c].y, v);
            o = fmaf(meta[n][c].x, v, o);
          } else if constexpr (WT == WT_F16) {  // one scale per column
            o += s[j][n][i];
          } else {
            o = fmaf(d[j][h], s[j][n][i], o);
            if constexpr (WT == WT_Q4_K) o = fmaf(-dm[j][h], meta[n][c].y, o);
          }
        }
  }
}

// The same for F32 rows: boxes of one block each, 16-byte words 4 s + t of the 128 swizzled by
// the row.
template <int MODE, int NTA, int NT>
__device__ __forceinline__ void tile_block_f32(const TileLane& l, uint32_t st, uint32_t xs, uint32_t blk,
                                               float (&acc)[4][NT][4]) {
  const uint32_t row = st + l.rowbase + blk * 8192u;
  float sum[4][NTA][4];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < NTA; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[m][n][i] = 0.0f;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float xh[NTA][4], xl[NTA][4];  // elements 16 s + 4 t + 0..3 of column g
#pragma unroll
    for (int n = 0; n < NTA; ++n) {
      const uint4 b = lds128(xs + static_cast<uint32_t>(n) * l.xtile + l.xlane + s * l.cp * 64u);
      const float2 h0 = h2pair(b.x), h1 = h2pair(b.y), l0 = h2pair(b.z), l1 = h2pair(b.w);
      xh[n][0] = h0.x; xh[n][1] = h0.y; xh[n][2] = h1.x; xh[n][3] = h1.y;
      xl[n][0] = l0.x; xl[n][1] = l0.y; xl[n][2] = l1.x; xl[n][3] = l1.y;
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t wh[2][4], wl[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 u = lds128(row + (m & 1) * 2048u + (m >> 1) * 4096u + h * 1024u + (((4u * s + l.t4) ^ l.row8) << 4));
        const float w[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          wh[h][k] = to_tf32(w[k]);
          const float rest = w[k] - __uint_as_float(wh[h][k]);
          wl[h][k] = to_tf32(fabsf(w[k]) <= 3.402823466e38f ? rest : 0.0f);  // no NaN beside an infinite weight
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)  // k-slots t and t + 4 hold elements 2j and 2j + 1
#pragma unroll
        for (int n = 0; n < NTA; ++n) {
          const uint32_t h0 = __float_as_uint(xh[n][2 * j]), h1 = __float_as_uint(xh[n][2 * j + 1]);
          const uint32_t l0 = __float_as_uint(xl[n][2 * j]), l1 = __float_as_uint(xl[n][2 * j + 1]);
          mma_tf32(sum[m][n], wh[0][2 * j], wh[1][2 * j], wh[0][2 * j + 1], wh[1][2 * j + 1], h0, h1);
          mma_tf32(sum[m][n], wl[0][2 * j], wl[1][2 * j], wl[0][2 * j + 1], wl[1][2 * j + 1], h0, h1);
          mma_tf32(sum[m][n], wh[0][2 * j], wh[1][2 * j], wh[0][2 * j + 1], wh[1][2 * j + 1], l0, l1);
        }
    }
  }
#pragma unroll
  for (int n = 0; n < NTA; ++n) {
    const float sx[2] = {__uint_as_float(lds32(xs + static_cast<uint32_t>(n) * l.xtile + l.m0)),
                         __uint_as_float(lds32(xs + static_cast<uint32_t>(n) * l.xtile + l.m1))};
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[m][n][i] = MODE == TILE_DOWN ? fmaf(sx[i & 1], sum[m][n][i], acc[m][n][i]) : acc[m][n][i] + sum[m][n][i];
  }
}

template <int WT, int MODE, int NT, bool PER1>
__global__ void __launch_bounds__(kTileThreads, tile_ctas(WT, NT))
    tile_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                const __grid_constant__ TileArgs a) {
  constexpr int kOutRows = MODE == TILE_GLU ? 32 : kTileRows;
  constexpr int CH = tile_chunks(WT, NT);
  constexpr bool kFew = NT == 1 && !tile_plain(WT);
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem), full0 = sbase, empty0 = sbase + 8u * kTileMaxStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 248);
  int4* groups = reinterpret_cast<int4*>(smem + 256);
  float* red = reinterpret_cast<float*>(smem + kTileHeadBytes);
  const uint32_t xfull0 = sbase + 128u, xempty0 = xfull0 + 8u * kTileMaxXBuffers;
  const bool resident = a.xbuffers > 0;
  const uint32_t xbytes = resident ? static_cast<uint32_t>(tile_x_bytes(a.K, NT, a.cp)) : 0u;
  const uint32_t xres = sbase + kTileHeadBytes + kTileRedBytes;
  const uint32_t ring = (xres + a.xbuffers * xbytes + 1023u) & ~1023u;
  const uint32_t stage_bytes = tile_stage_bytes<WT>(a.period, NT, a.cp, resident);
  const uint32_t xoff = tile_weight_bytes<WT>(a.period) + 16;  // slack: words are read up to 3 bytes past a row
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < a.NS; ++i) {
      mbar_init(full0 + 8u * i, 1);
      mbar_init(empty0 + 8u * i, kTileWarps);
    }
    for (int i = 0; i < kTileMaxXBuffers; ++i) {
      mbar_init(xfull0 + 8u * i, 1);
      mbar_init(xempty0 + 8u * i, kTileWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&map0);
    if (MODE == TILE_GLU) prefetch_tmap(&map1);
  }
  pdl_trigger();
  pdl_wait();
  const int tiles = (a.rows + kOutRows - 1) / kOutRows;
  // (a call of few groups: the list is fetched beside its length, not after it)
  if (MODE != TILE_LIN)
    for (int i = threadIdx.x; i < min(kTileMaxGroups, a.max_groups); i += kTileThreads) groups[i] = a.groups[i];
  const int n_groups = MODE == TILE_LIN ? (a.ncols + a.group_cols - 1) / a.group_cols : *a.n_groups;
  const int64_t items = static_cast<int64_t>(n_groups) * tiles;
  const int64_t lo = items * blockIdx.x / gridDim.x, hi = items * (blockIdx.x + 1) / gridDim.x;
  const bool all = MODE != TILE_LIN && n_groups <= kTileMaxGroups;
  const int g_lo = static_cast<int>(lo / tiles), g_at = all ? g_lo : 0;  // the first group's place in `groups`
  if (lo < hi && !all)
    for (int i = threadIdx.x; i <= static_cast<int>((hi - 1) / tiles) - g_lo; i += kTileThreads)
      groups[i] = MODE == TILE_LIN ? make_int4(0, 0, min(a.group_cols, a.ncols - (g_lo + i) * a.group_cols),
                                               (g_lo + i) * ((a.group_cols + 7) / 8))
                                   : a.groups[g_lo + i];
  __syncthreads();
  const int n_kc = (a.K + kTileK - 1) / kTileK, nblk = a.K / 32;
  const int n_items = static_cast<int>(hi - lo);
  const int tile_lo = static_cast<int>(lo - static_cast<int64_t>(g_lo) * tiles);
  const int64_t tile_stride = static_cast<int64_t>(nblk) * record_bytes(a.cp);  // of column tiles in memory

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int slot = 0, issued = 0, gi = 0, tile = tile_lo, xgroups = 0;  // gi: groups since the first
      uint32_t phase = 1u;
      bool ok = true;
      const uint32_t wlen = 32u * static_cast<uint32_t>(tile_plain(WT) ? tile_seg<WT>() : tile_pitch<WT>(a.period));
      for (int it = 0; it < n_items && ok; ++it) {
        const int4 g = groups[g_at + gi];
        const int row0 = tile * kOutRows;
        const int halves = MODE == TILE_GLU || row0 + 32 < a.rows ? 2 : 1;
        const int nt = (g.z + 7) / 8;
        const int first = g.x * a.rows + row0;
        const uint8_t* xsrc = a.records + g.w * tile_stride;
        const uint32_t rec = static_cast<uint32_t>(record_bytes(min(8, g.z)));
        if (resident && (it == 0 || tile == 0)) {  // a new group: its records, once the buffer is free
          const int b = gi % a.xbuffers;
          if (gi >= a.xbuffers &&
              !mbar_wait_or_abort(xempty0 + 8u * b, static_cast<uint32_t>((gi / a.xbuffers - 1) & 1), abort_flag, a.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(xfull0 + 8u * b, static_cast<uint32_t>(nt * nblk) * rec);
          for (int n = 0; n < nt; ++n)
            bulk_g2s(xres + b * xbytes + static_cast<uint32_t>(n * nblk) * rec, xsrc + n * tile_stride,
                     static_cast<uint32_t>(nblk) * rec, xfull0 + 8u * b);
          xgroups = gi + 1;
        }
        for (int kc0 = 0; kc0 < n_kc; kc0 += CH) {
          if (issued >= a.NS && !mbar_wait_or_abort(empty0 + 8u * slot, phase, abort_flag, a.err)) {
            ok = false;
            break;
          }
          const uint32_t full = full0 + 8u * slot;
          const int chunks = min(CH, n_kc - kc0);
          const uint32_t blocks = static_cast<uint32_t>(min(CH * kTileBlocks, nblk - kc0 * kTileBlocks));
          mbar_arrive_expect_tx(full, chunks * halves * wlen + (resident ? 0u : nt * blocks * rec));
          for (int ch = 0; ch < chunks; ++ch) {
            const int kc = kc0 + ch;
            const uint32_t st = ring + static_cast<uint32_t>(slot * CH + ch) * stage_bytes;
            for (int h = 0; h < halves; ++h) {
              const CUtensorMap* map = MODE == TILE_GLU && h ? &map1 : &map0;
              const int row = first + (MODE == TILE_GLU ? 0 : 32 * h);
              if constexpr (tile_plain(WT)) {
                constexpr int kBox = WT == WT_F16 ? 64 : 32;  // elements of 128 bytes
#pragma unroll
                for (int q = 0; q < kTileK / kBox; ++q)
                  tma_load_2d(st + static_cast<uint32_t>((2 * q + h) * 4096), map, kc * kTileK + kBox * q, row, full);
              } else if constexpr (PER1) {
                tma_load_2d(st + static_cast<uint32_t>(h * tile_part<WT>(1)), map, kc * (tile_seg<WT>() / 2), row, full);
              } else {
                for (int i = 0; i < a.period; ++i)
                  tma_load_2d(st + static_cast<uint32_t>((h * a.period + i) * tile_part<WT>(a.period)), map,
                              ((i * a.row_bytes + kc * tile_seg<WT>()) & ~15) / 2, row / a.period, full);
              }
            }
            const uint32_t xlen = static_cast<uint32_t>(min(kTileBlocks, nblk - kc * kTileBlocks)) * rec;
            for (int n = 0; n < nt && !resident; ++n)
              bulk_g2s(st + xoff + static_cast<uint32_t>(n) * kTileBlocks * rec,
                       xsrc + n * tile_stride + static_cast<uint32_t>(kc * kTileBlocks) * rec, xlen, full);
          }
          ++issued;
          if (++slot == a.NS) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (++tile == tiles) {
          tile = 0;
          ++gi;
        }
      }
      // Drain after an abort: every copy this thread issued lands before the CTA leaves.
      if (!ok) {
        for (int i = max(0, issued - a.NS); i < issued; ++i)
          (void)mbar_wait(full0 + 8u * (i % a.NS), static_cast<uint32_t>((i / a.NS) & 1));
        for (int i = max(0, xgroups - a.xbuffers); i < xgroups; ++i)
          (void)mbar_wait(xfull0 + 8u * (i % a.xbuffers), static_cast<uint32_t>((i / a.xbuffers) & 1));
      }
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int wk = warp - 1;
    TileLane l;
    {
      const uint32_t g4 = static_cast<uint32_t>(lane) >> 2, per = static_cast<uint32_t>(a.period);
      l.t4 = static_cast<uint32_t>(lane) & 3u;
      l.row8 = tile_plain(WT) ? ((g4 >> 1) | ((g4 & 1u) << 2)) : g4;  // the row of eight that this lane takes
      l.step8 = l.step16 = l.half = 0;
      if constexpr (tile_plain(WT)) {
        l.rowbase = l.row8 * 128u;
      } else if constexpr (PER1) {
        l.rowbase = l.row8 * tile_pitch<WT>(1);
      } else {
        const uint32_t P = tile_pitch<WT>(a.period), res = l.row8 % per;
        l.rowbase = res * tile_part<WT>(a.period) + l.row8 / per * P + ((res * static_cast<uint32_t>(a.row_bytes)) & 15u);
        l.step8 = 8u / per * P;
        l.step16 = 16u / per * P;
        l.half = per * tile_part<WT>(a.period);
      }
    }
    auto group_bar = [&]() { named_bar_sync(1u, 32u * kTileWarps); };
    int slot = 0, gi = 0, tile = tile_lo;
    uint32_t phase = 0;
    bool ok = true, raw = false;  // raw: one of this warp's columns was
    for (int it = 0; it < n_items; ++it) {
      const int4 g = groups[g_at + gi];
      const int row0 = tile * kOutRows;
      const int ncol = g.z;
      const bool few = kFew && ncol <= 4;
      {
        const uint32_t g4 = static_cast<uint32_t>(lane) >> 2;
        l.cp = static_cast<uint32_t>(min(8, ncol));
        l.rec = static_cast<uint32_t>(record_bytes(static_cast<int>(l.cp)));
        l.xtile = (resident ? static_cast<uint32_t>(nblk) : static_cast<uint32_t>(kTileBlocks)) * l.rec;
        l.xlane = min(g4, l.cp - 1u) * 64u + l.t4 * 16u;  // lanes past the columns read the last one
        l.m0 = l.cp * 128u + min(2u * l.t4, l.cp - 1u) * 8u;
        l.m1 = l.cp * 128u + min(2u * l.t4 + 1u, l.cp - 1u) * 8u;
        if (few) {
          l.xlane = min(g4 & 3u, l.cp - 1u) * 64u + l.t4 * 16u + (g4 >> 2) * 8u;
          l.m0 = l.cp * 128u + min(2u * (l.t4 & 1u), l.cp - 1u) * 8u;
          l.m1 = l.cp * 128u + min(2u * (l.t4 & 1u) + 1u, l.cp - 1u) * 8u;
        }
      }
      const uint32_t xbuf = resident ? static_cast<uint32_t>(gi % a.xbuffers) : 0u;
      if (resident && (it == 0 || tile == 0))
        ok = ok && mbar_wait_or_abort(xfull0 + 8u * xbuf, static_cast<uint32_t>((gi / a.xbuffers) & 1), abort_flag, a.err);
      // what the tail needs of this warp's columns 8n + wk, on its way during the K loop
      float factor[NT];
      int sl[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        factor[n] = 0.0f;
        sl[n] = 0;
        if (8 * n + wk < ncol) {
          if constexpr (MODE != TILE_DOWN) {
            factor[n] = *reinterpret_cast<const float*>(a.records + (g.w + n) * tile_stride + l.cp * 128u +
                                                        static_cast<uint32_t>(wk) * 8u);
          } else {
            sl[n] = a.slots[g.y + 8 * n + wk];
            factor[n] = a.factors[sl[n]];
          }
        }
      }
      float acc[4][NT][4];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
      // the K chunks, for NTA column tiles
      auto walk = [&](auto nta, auto few_columns) {
        constexpr int NTA = decltype(nta)::value;
        constexpr bool FEW = decltype(few_columns)::value != 0;
#pragma unroll 1
        for (int kc0 = 0; kc0 < n_kc; kc0 += CH) {
          ok = __all_sync(0xffffffffu, ok && mbar_wait_or_abort(full0 + 8u * slot, phase, abort_flag, a.err));
#pragma unroll
          for (int ch = 0; ch < CH; ++ch) {
            const int kc = kc0 + ch;
            const uint32_t st = ring + static_cast<uint32_t>(slot * CH + ch) * stage_bytes;
            if (ok && kc * kTileBlocks + wk < nblk) {
              const uint32_t blk = static_cast<uint32_t>(wk);
              const uint32_t xs = resident ? xres + xbuf * xbytes + (static_cast<uint32_t>(kc * kTileBlocks) + blk) * l.rec
                                           : st + xoff + blk * l.rec;
              // codes behind a two-byte scale start on a word in every other block (in rows that
              // themselves do)
              if constexpr (WT == WT_F32)
                tile_block_f32<MODE, NTA, NT>(l, st, xs, blk, acc);
              else if (PER1 && (WT == WT_Q4_0 || WT == WT_Q8_0) && (wk & 1))
                tile_block<WT, MODE, NTA, NT, PER1, true, FEW>(l, st, xs, blk, acc);
              else
                tile_block<WT, MODE, NTA, NT, PER1, false, FEW>(l, st, xs, blk, acc);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty0 + 8u * slot);
          if (++slot == a.NS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      };
      if (NT >= 3 && ncol > 16) walk(TileConst<NT >= 3 ? 3 : 1>(), TileConst<0>());
      else if (NT >= 2 && ncol > 8) walk(TileConst<NT >= 2 ? 2 : 1>(), TileConst<0>());
      else if (few) walk(TileConst<1>(), TileConst<kFew ? 1 : 0>());
      else walk(TileConst<1>(), TileConst<0>());
      if (resident && (tile + 1 == tiles || it + 1 == n_items)) {  // done with the group's records
        __syncwarp();
        if (lane == 0) mbar_arrive(xempty0 + 8u * xbuf);
      }
      // the warps' sums through shared memory, eight columns at a time: red[warp][column][row];
      // then warp wk takes column 8n + wk
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= ncol) break;
        group_bar();  // everyone has read the previous sums
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            red[(wk * 8 + 2 * l.t4 + (i & 1)) * kRedPitch + 16 * m + l.row8 + 8 * (i >> 1)] = acc[m][n][i];
        group_bar();
        const int c = 8 * n + wk;
        if (MODE != TILE_DOWN && c < ncol && __float_as_uint(factor[n]) == kRawBlock) {
          raw = true;  // not this kernel's (TILE_GLU), or later
        } else if (c < ncol && ok && !*abort_flag) {
          float v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float s = 0.0f;
            if (few)  // the lo parts
#pragma unroll
              for (int w = 0; w < kTileWarps; ++w) s += red[(w * 8 + wk + 4) * kRedPitch + 32 * h + lane];
#pragma unroll
            for (int w = 0; w < kTileWarps; ++w) s += red[(w * 8 + wk) * kRedPitch + 32 * h + lane];
            v[h] = s;
          }
          if constexpr (MODE == TILE_GLU) {
            // 32 output rows of the gated product (rows are a multiple of 32): one record's column
            const float gv = v[0] * tile_unit(WT) * factor[n], uv = v[1] * tile_unit(WT) * factor[n];
            write_gated(tail_silu(gv) * uv,
                        a.out_records + static_cast<int64_t>(g.w + n) * (a.rows / 32) * record_bytes(a.cp) +
                            static_cast<int64_t>(row0 / 32) * l.rec,
                        static_cast<uint32_t>(wk), l.cp, a.out_format);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = row0 + 32 * h + lane;
              if (r < a.rows) {
                const int64_t col = MODE == TILE_LIN ? (g.w + n) * 8 + wk : sl[n];
                const int64_t o = col * a.out_ld + r;
                const float y = factor[n] * (v[h] * tile_unit(WT));
                if constexpr (MODE == TILE_LIN)
                  a.out[o] = apply_tail(a.epi, y, epi_takes_aux(a.epi) ? a.aux[o] : 0.0f);  // aux may be out
                else
                  a.out[o] = y;
              }
            }
          }
        }
      }
      if (++tile == tiles) {
        tile = 0;
        ++gi;
      }
    }
    // a batch's raw columns
    if (MODE == TILE_LIN && raw && ok && !*abort_flag)
      for (int64_t it = lo; it < hi; ++it) {
        const int4 g = groups[g_at + static_cast<int>(it / tiles) - g_lo];
        const int row0 = static_cast<int>(it % tiles) * kOutRows;
        for (int c = wk; c < g.z; c += 8)
          if (raw_column(a, g, c))
            for (int r = row0; r < min(row0 + kOutRows, a.rows); r += 32) exact_rows<WT>(a, g, c, r);
      }
  }
  __syncthreads();
}

}  // namespace gf
