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

// Four values as code bytes.  inv = 1 / d (exact for e4m3, whose quotient is then exact too).
template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float e, float d, float inv) {
  if constexpr (FMT == 0) {
    return (code_i8(a, d, inv) & 255) | ((code_i8(b, d, inv) & 255) << 8) | ((code_i8(c, d, inv) & 255) << 16) |
           (static_cast<uint32_t>(code_i8(e, d, inv)) << 24);
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(e * inv), "f"(c * inv));
    return lo | (static_cast<uint32_t>(hi) << 16);
  }
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
