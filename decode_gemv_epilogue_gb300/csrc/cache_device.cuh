// The 8-bit cache of keys and values: where a token's codes and scale lie, and the two code formats.
//   i8   : value = scale * int8 code in -127..127; scales have 12 significant bits, so that
//          code * scale, and x - code * scale for the x it stands for, are exact in 32 bits.
//   e4m3 : value = scale * e4m3 code; scales are powers of two (the code carries an exponent).
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "gf_internal.h"

namespace gf {

constexpr float kScaleMin = 0x1p-112f;  // 1 / scale and code * scale stay normal

// Where token `pos` of sequence `seq` lies: its page, or -1 where it has none.
__device__ __forceinline__ int64_t cache_page(const CacheArgs& c, int seq, int pos) {
  if (pos < 0 || seq < 0 || seq >= c.n_seqs) return -1;
  const int64_t i = pos >> c.page_log2;
  if (i >= c.table_ld) return -1;
  const int p = c.table[seq * c.table_ld + i];
  return p >= 0 && p < c.n_pages ? p : -1;
}

__device__ __forceinline__ int64_t cache_row(const CacheArgs& c, int64_t page, int head, int slot) {
  return (((page * c.heads + head) << c.page_log2) + slot) * c.dim;
}

__device__ __forceinline__ int64_t cache_scale(const CacheArgs& c, int64_t page, int head, int slot) {
  return ((page * c.heads + head) << (c.page_log2 - c.block_log2)) + (slot >> c.block_log2);
}

// The least scale for values of magnitude up to `top` (finite).
template <int FMT>
__device__ __forceinline__ float scale_for(float top) {
  if constexpr (FMT == 0) {
    // 12 significant bits: the mantissa's upper 11.  One step either way is settled by the exact
    // product 127 d.
    const float lim = 0x1p121f;  // 127 of them are finite
    uint32_t b = __float_as_uint(top / 127.0f) & 0xfffff000u;
    float d = __uint_as_float(b);
    while (127.0f * d < top && d < lim) {  // at most twice
      b += 0x1000u;
      d = __uint_as_float(b);
    }
    return fminf(fmaxf(d, kScaleMin), lim);
  } else {
    const float lim = 0x1p119f;
    float d = __uint_as_float(__float_as_uint(top * (1.0f / 512.0f)) & 0x7f800000u);  // 512 d <= top < 1024 d
    while (448.0f * d < top && d < lim) d = d == 0.0f ? kScaleMin : d + d;
    return fminf(fmaxf(d, kScaleMin), lim);
  }
}

// x / d rounded to the nearest integer, ties to even, exactly: the estimate is off by one step at
// most, and what it leaves of x is exact in 32 bits.
__device__ __forceinline__ int code_i8(float x, float d, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, d, x), h = 0.5f * d;
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (r > h || (r == h && odd)) q += 1.0f;
  if (r < -h || (r == -h && odd)) q -= 1.0f;
  return static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
}

__device__ __forceinline__ uint2 codes8_slow(float4 a, float4 b, float d, float inv) {
  uint2 w;
  w.x = (code_i8(a.x, d, inv) & 255) | (code_i8(a.y, d, inv) & 255) << 8 | (code_i8(a.z, d, inv) & 255) << 16 |
        static_cast<uint32_t>(code_i8(a.w, d, inv)) << 24;
  w.y = (code_i8(b.x, d, inv) & 255) | (code_i8(b.y, d, inv) & 255) << 8 | (code_i8(b.z, d, inv) & 255) << 16 |
        static_cast<uint32_t>(code_i8(b.w, d, inv)) << 24;
  return w;
}

// Eight values as code bytes.  inv = 1 / d (exact for e4m3, whose quotient is then exact too).
// i8: adding 1.5 * 2^23 rounds x * inv to an integer and leaves it in the low bits; it is the right one if what it
// leaves of x is less than half a step.  Ties, the few estimates next to them and the largest scale, whose
// codes may have to be cut, are looked at one by one (all of them in that way: 42 us for a prompt of 8191
// tokens of 8 heads of 128, where 32).
template <int FMT>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float d, float inv) {
  uint2 w;
  if constexpr (FMT == 0) {
    constexpr float kRound = 12582912.0f;
    uint32_t t[8];
    float left = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = fmaf(v[i], inv, kRound);
      t[i] = __float_as_uint(y);
      left = fmaxf(left, fabsf(fmaf(kRound - y, d, v[i])));
    }
    w.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    w.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
    if (!(left < 0.5f * d) || d >= 0x1p121f)
      w = codes8_slow(make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7]), d, inv);
  } else {
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(v[2 * i + 1] * inv), "f"(v[2 * i] * inv));
    w = make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
  }
  return w;
}

// The larger magnitude; NaN if either is.
__device__ __forceinline__ float top_of(float top, float x) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(top), "f"(fabsf(x)));
  return y;
}

// The values of four code bytes (without their scale).
template <int FMT>
__device__ __forceinline__ void values4(uint32_t w, float (&v)[4]) {
  if constexpr (FMT == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * i))));
      const __half2 p = *reinterpret_cast<const __half2*>(&h);
      v[2 * i] = __low2float(p);
      v[2 * i + 1] = __high2float(p);
    }
  }
}

}  // namespace gf
