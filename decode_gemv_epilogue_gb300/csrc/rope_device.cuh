// Rotary positions: the angle of a pair and the rotation of a head's row, shared by gf_rope and the
// cache store.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "gf_device.cuh"
#include "gf_internal.h"

namespace gf {

// The table of gf_rope_table: a header, then one word a pair.
struct RopeHeader {
  float magnitude;  // of cosine and sine
  uint32_t pairs;
  uint32_t unused[2];
};

// Cosine and sine of pi x, |x| <= 1/4, by their Taylor series (the terms left out are below 2^-29): within one unit
// of the last place.
__device__ __forceinline__ void cos_sin_pi(float x, float& c, float& s) {
  const float y = x * x;
  float p = fmaf(0.0821458846f, y, -0.599264503f);  // pi^9 / 9!, -pi^7 / 7!, ..
  p = fmaf(p, y, 2.55016398f);
  p = fmaf(p, y, -5.16771269f);
  p = fmaf(p, y, -8.74227766e-08f);  // what 32 bits leave of pi
  s = fmaf(x, 3.14159274f, x * p);
  float q = fmaf(-0.0258068908f, y, 0.235330626f);  // -pi^10 / 10!, pi^8 / 8!, ..
  q = fmaf(q, y, -1.33526278f);
  q = fmaf(q, y, 4.05871201f);
  q = fmaf(q, y, -4.93480206f);
  c = fmaf(q, y, 1.0f);
}

// Cosine and sine of position `pos` for a pair that makes turns * 2^-64 turns a position.  The product modulo one
// turn is exact in 64-bit integers, and so is the nearest quarter turn that is taken off it; what is left, an eighth of
// a turn at most, is rounded to 32 bits: by 2^-28 turns, or some 2^-24 of itself.  (The whole angle rounded to 32 bits was
// off by 2^-26 turns.)
__device__ __forceinline__ float2 rope_cs(uint64_t turns, int pos, float magnitude) {
  const uint64_t a = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint32_t b = static_cast<uint32_t>(a >> 32) + (1u << 29), quarter = b >> 30;
  const int left = static_cast<int>(b & 0x3fffffffu) - (1 << 29);  // and the low word: in 2^-64 turns
  // Its upper 24 bits and the 32 behind them.  (One conversion of 64 bits and sincospif: a prompt's 8191 tokens stored
  // with 32 query heads 70 us, where 66.)
  const uint32_t low = static_cast<uint32_t>(left) << 26 | static_cast<uint32_t>(a) >> 6;
  const float rest = fmaf(static_cast<float>(left >> 6), 0x1p32f, static_cast<float>(low));
  float s, c;
  cos_sin_pi(rest * 0x1p-57f, c, s);  // half turns
  const float x = quarter & 1u ? s : c, y = quarter & 1u ? c : s;
  return make_float2(__uint_as_float(__float_as_uint(x) ^ ((quarter + 1u) & 2u) << 30) * magnitude,
                     __uint_as_float(__float_as_uint(y) ^ (quarter & 2u) << 30) * magnitude);
}

// Whether the table is one for n_rot elements.  Where it is not, what lies behind its header is not read and the
// device error word says so.
__device__ __forceinline__ bool rope_fits(uint32_t pairs, int n_rot, unsigned* err) {
  if (pairs == static_cast<uint32_t>(n_rot) / 2) return true;
  if (threadIdx.x == 0) set_error(err, ERRBIT_TABLE);
  return false;
}
__device__ __forceinline__ bool rope_fits(const void* table, int n_rot, unsigned* err) {
  return rope_fits(static_cast<const RopeHeader*>(table)->pairs, n_rot, err);
}

__device__ __forceinline__ const uint64_t* rope_turns(const void* table) {
  return reinterpret_cast<const uint64_t*>(static_cast<const uint8_t*>(table) + sizeof(RopeHeader));
}

__device__ __forceinline__ void rope_turn(float& a, float& b, float2 cs) {
  const float u = fmaf(a, cs.x, -(b * cs.y)), v = fmaf(a, cs.y, b * cs.x);
  a = u;
  b = v;
}

// Eight elements of a row: unit u (four adjacent pairs) of a head whose first n_rot elements turn.
// They lie at o0 .. o0 + 3 and o1 .. o1 + 3; pair i is (v[i], v[4 + i]) in halves, else (v[2i],
// v[2i + 1]).
__device__ __forceinline__ void unit_offsets(int u, int n_rot, bool halves, int& o0, int& o1) {
  if (halves && 8 * u < n_rot) {
    o0 = 4 * u;
    o1 = n_rot / 2 + 4 * u;
  } else {
    o0 = 8 * u;
    o1 = 8 * u + 4;
  }
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __half* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__half* p, float a, float b, float c, float d) {
  const __half2 x = __floats2half2_rn(a, b), y = __floats2half2_rn(c, d);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__half* p, float v) { *p = __float2half_rn(v); }

}  // namespace gf
