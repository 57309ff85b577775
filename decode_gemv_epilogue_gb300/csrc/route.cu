// Routing to experts: scores, the choice of top_k experts per token, their weights.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e));   key_e = s_e + bias_e (the choice only);
//   with groups, the topk_group groups with the largest (best, or sum of two best) keys stay;
//   the top_k largest keys, descending, ties to the lowest index;  w = s of the chosen,
//   optionally divided by their sum, times scale.
//
// One warp per token: lane L holds experts L, L + 32, ... in registers (VPL of them), so a
// row of logits is read once, coalesced, and nothing else is shared.  A round of the choice
// is a per-lane maximum, one warp-wide integer maximum of the keys as ordered integers
// (redux) and one minimum of the indices that hold it: no sort, and ties fall to the lowest
// index by construction.
//
// Which expert is taken has to be right where two keys are closer than 32 bits can tell.
// Without a bias and without groups the key is the logit itself (both scores grow with it),
// exact.  Otherwise the keys are computed in 32 bits, and a warp that finds two neighbours
// of its choice within the error bound of that arithmetic (and not made of the same logit
// and bias) computes the keys that can matter again in 64 bits.  Roughly one row in a hundred
// to a thousand does; an exponential and a division in 64 bits take a warp some 1000 cycles
// at this machine's two double operations per clock and SM, so a row is not computed so
// throughout (a batch with one such row, 256 experts in groups: 28 us for all its keys, 13 for
// those that matter).
#include <cfloat>
#include <cmath>

#include "gf_device.cuh"
#include "gf_internal.h"

namespace gf {

constexpr int kRouteWarps = 8;
// Bounds on the error of a 32-bit key: the exponential and the division (a few units in the
// last place of a value <= 1), the row sum of up to 1024 terms (32 adds per lane and five
// shuffles) and the rounding of the sum with the bias.
constexpr float kKeyTolAbs = 0x1p-18f, kKeyTolRel = 0x1p-22f;

// Keys as integers in the same order (-inf lowest of all values used here; 0 is below it).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 64-bit keys as integers in the same order: comparing doubles costs a trip through the few
// double units each.
__device__ __forceinline__ long long ordered64(double v) {
  const long long u = __double_as_longlong(v + 0.0);
  return u ^ ((u >> 63) & 0x7fffffffffffffffLL);
}
__device__ __forceinline__ double from_ordered64(long long k) {
  return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffLL));
}
constexpr long long kLowest64 = -0x7ff0000000000001LL;  // of -inf

__device__ __forceinline__ float lowest(float) { return -INFINITY; }
__device__ __forceinline__ long long lowest(long long) { return kLowest64; }
__device__ __forceinline__ float add_keys(float a, float b) { return a + b; }
__device__ __forceinline__ long long add_keys(long long a, long long b) {
  return ordered64(from_ordered64(a) + from_ordered64(b));
}

// The best key of a warp in 64 bits: largest, ties to the lowest index.
__device__ __forceinline__ void warp_best(long long& key, int& e) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const long long k2 = __shfl_xor_sync(0xffffffffu, key, o);
    const int e2 = __shfl_xor_sync(0xffffffffu, e, o);
    if (k2 > key || (k2 == key && e2 < e)) {
      key = k2;
      e = e2;
    }
  }
}

// The two largest values of a warp's lanes, each lane giving its own two (a >= b).
template <class T>
__device__ __forceinline__ void warp_top2(T& a, T& b) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const T a2 = __shfl_xor_sync(0xffffffffu, a, o), b2 = __shfl_xor_sync(0xffffffffu, b, o);
    const T lo = a < a2 ? a : a2, hb = b > b2 ? b : b2;
    a = a < a2 ? a2 : a;
    b = lo > hb ? lo : hb;
  }
}

// Groups that stay, as a bit mask, from the keys kv (float or ordered64; the lowest: not
// choosable).  unsure (may be NULL; floats): the last kept and the first dropped score are
// within tol.
template <int VPL, class T>
__device__ __forceinline__ uint32_t choose_groups(const RouteArgs& a, const T (&kv)[VPL], int lane, float tol, bool* unsure) {
  const T low = lowest(T());
  const int gs = a.E / a.n_group;
  T mine = low;
  for (int g = 0; g < a.n_group; ++g) {
    T t1 = low, t2 = low;
    const int lo = g * gs, hi = lo + gs;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e >= lo && e < hi) {
        const T v = kv[i];
        t2 = v > t1 ? t1 : (v > t2 ? v : t2);
        t1 = v > t1 ? v : t1;
      }
    }
    warp_top2(t1, t2);
    const T s = (a.group_top == 2 && t2 > low) ? add_keys(t1, t2) : t1;
    if (lane == g) mine = s;
  }
  int rank = 0;
  for (int g = 0; g < a.n_group; ++g) {
    const T o = __shfl_sync(0xffffffffu, mine, g);
    rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
  }
  const bool in = lane < a.n_group;
  const uint32_t kept = __ballot_sync(0xffffffffu, in && rank < a.topk_group);
  if (unsure) {
    const uint32_t last = __ballot_sync(0xffffffffu, in && rank == a.topk_group - 1);
    const uint32_t next = __ballot_sync(0xffffffffu, in && rank == a.topk_group);
    if (next) {
      const T v = __shfl_sync(0xffffffffu, mine, __ffs(last) - 1), w = __shfl_sync(0xffffffffu, mine, __ffs(next) - 1);
      // nothing in doubt where the next group is empty
      *unsure = w > low && static_cast<float>(v - w) <= tol;
    }
  }
  return kept;
}

// Keys in 64 bits, as ordered64, of the experts in `need` (bit i: expert lane + 32 i); the
// others get the lowest.  Each lane takes its next needed expert in each round: a few rounds,
// where computing all of them would take VPL.
template <int VPL>
__device__ __forceinline__ void exact_keys(const RouteArgs& a, const float (&l)[VPL], int lane, uint32_t need, float m,
                                           double z, long long (&key)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = kLowest64;
  while (__any_sync(0xffffffffu, need != 0u)) {
    const int at = __ffs(need) - 1;
    need &= need - 1u;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i == at) v = l[i];
    double k = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(v)))
                         : exp(static_cast<double>(v) - static_cast<double>(m)) / z;
    if (a.bias && at >= 0) k += static_cast<double>(a.bias[lane + 32 * at]);
    const long long o = ordered64(k);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i == at) key[i] = o;
  }
}

// The row's groups once more in 64 bits.  s: the 32-bit keys, the lowest where not choosable.
template <int VPL>
__device__ __noinline__ uint32_t exact_groups(const RouteArgs& a, const float (&l)[VPL], const float (&s)[VPL], int lane,
                                              float tol, float m, double z) {
  // all that can be among a group's two best
  const int gs = a.E / a.n_group;
  uint32_t need = 0;
  for (int g = 0; g < a.n_group; ++g) {
    float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e >= g * gs && e < (g + 1) * gs) {
        t2 = s[i] > t1 ? t1 : fmaxf(s[i], t2);
        t1 = fmaxf(s[i], t1);
      }
    }
    warp_top2(t1, t2);
    const float edge = (a.group_top == 2 ? t2 : t1) - tol;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e >= g * gs && e < (g + 1) * gs && s[i] > -INFINITY && !(s[i] < edge)) need |= 1u << i;
    }
  }
  long long key[VPL];
  exact_keys<VPL>(a, l, lane, need, m, z, key);
  return choose_groups<VPL, long long>(a, key, lane, 0.0f, nullptr);
}

// The row's choice once more in 64 bits, among the experts whose 32-bit keys s reach `edge`.
// Returns the expert that lane j takes in round j.
template <int VPL>
__device__ __noinline__ int exact_choice(const RouteArgs& a, const float (&l)[VPL], const float (&s)[VPL], int lane,
                                         float edge, float m, double z) {
  uint32_t need = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (s[i] > -INFINITY && !(s[i] < edge)) need |= 1u << i;
  long long key[VPL];
  exact_keys<VPL>(a, l, lane, need, m, z, key);
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    long long bk = kLowest64;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > bk) {
        bk = key[i];
        be = lane + 32 * i;
      }
    warp_best(bk, be);
    if (bk <= kLowest64) break;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 32 * i == be) key[i] = kLowest64;
    if (lane == j) mine = be;
  }
  return mine;
}

// Sum of the row's exponentials in 64 bits (softmax).
template <int VPL>
__device__ __noinline__ double exact_sum(const float (&l)[VPL], float m) {
  double z = 0.0;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (l[i] > -INFINITY) z += exp(static_cast<double>(l[i]) - static_cast<double>(m));
  return warp_sum(z);
}

// PLAIN: no bias and no groups, the key is the logit (64 -> 25 registers a thread with
// four experts a lane, and as many warps as an SM holds).
template <int VPL, bool PLAIN>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const __grid_constant__ RouteArgs a) {
  pdl_wait();  // the logits may be the preceding grid's
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= a.T) return;
  const float* lp = a.logits + row * a.ld;
  // An expert is choosable where its logit is a number above -inf; +inf counts as the largest
  // float (so that a softmax row with it stays defined).
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    const float v = e < a.E ? lp[e] : -INFINITY;
    l[i] = v == v ? fminf(v, FLT_MAX) : -INFINITY;
  }
  float key[VPL], b[VPL];
  const bool biased = !PLAIN && a.bias != nullptr;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    b[i] = (biased && e < a.E) ? a.bias[e] : 0.0f;
    key[i] = l[i] + 0.0f;  // -0 and +0 tie
  }
  float top = 0.0f, tol = 0.0f;  // largest logit; bound on the error of a 32-bit key
  if constexpr (!PLAIN) {
    float s[VPL];
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = tail_sigmoid(l[i]);
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
      top = warp_max(m);
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        s[i] = l[i] > -INFINITY ? expf(l[i] - top) : 0.0f;
        z += s[i];
      }
      const float inv = 1.0f / warp_sum(z);
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] *= inv;
    }
    // s + bias; without a bias the groups are chosen by s and the experts by the logit
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = l[i] > -INFINITY ? s[i] + b[i] : -INFINITY;
      if (!(s[i] == s[i])) s[i] = -INFINITY;  // a NaN bias: not choosable
      s[i] += 0.0f;
      if (s[i] > -INFINITY && s[i] < INFINITY) big = fmaxf(big, fabsf(s[i]));
    }
    tol = kKeyTolAbs + kKeyTolRel * warp_max(big);
    uint32_t kept = 0xffffffffu;
    if (a.n_group > 1) {
      bool unsure = false;
      kept = choose_groups<VPL, float>(a, s, lane, 4.0f * tol, &unsure);
      if (unsure) kept = exact_groups<VPL>(a, l, s, lane, 2.0f * tol, top, a.sigmoid ? 1.0 : exact_sum<VPL>(l, top));
    }
    const int gs = a.E / a.n_group;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (biased) key[i] = s[i];
      if (a.n_group > 1 && e < a.E && !((kept >> (e / gs)) & 1u)) key[i] = -INFINITY;
    }
  }
  // top_k rounds (one more where the keys are rounded, to see the first one left out)
  int mine = -1;
  float pk = 0.0f, pl = 0.0f, pb = 0.0f;  // the previous round's key, logit and bias
  float last = -INFINITY;                 // the k-th key
  uint32_t left[VPL];                     // ordered keys of this lane's experts not taken yet, 0: none
#pragma unroll
  for (int i = 0; i < VPL; ++i) left[i] = key[i] > -INFINITY ? ordered(key[i]) : 0u;
  bool unsure = false;
  const int rounds = biased ? a.k + 1 : a.k;
  for (int j = 0; j < rounds; ++j) {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) u = max(u, left[i]);
    const uint32_t best = __reduce_max_sync(0xffffffffu, u);
    if (best == 0u) break;
    uint32_t cand = 0xffffffffu;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i)
      if (left[i] == best) cand = static_cast<uint32_t>(lane + 32 * i);
    const uint32_t e = __reduce_min_sync(0xffffffffu, cand);
    if (biased) {
      float bk = 0.0f, bl = 0.0f, bb = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (static_cast<uint32_t>(i) == e >> 5) {
          bk = key[i];
          bl = l[i];
          bb = b[i];
        }
      const int owner = static_cast<int>(e & 31u);
      const float kk = __shfl_sync(0xffffffffu, bk, owner), kl = __shfl_sync(0xffffffffu, bl, owner),
                  kb = __shfl_sync(0xffffffffu, bb, owner);
      if (j > 0 && !(kl == pl && kb == pb) && pk - kk <= 2.0f * tol) unsure = true;
      pk = kk;
      pl = kl;
      pb = kb;
      if (j == a.k - 1) last = kk;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (static_cast<uint32_t>(lane + 32 * i) == e) left[i] = 0u;
    if (lane == j && j < a.k) mine = static_cast<int>(e);
  }
  if (!PLAIN && unsure) mine = exact_choice<VPL>(a, l, key, lane, last - 2.0f * tol, top, a.sigmoid ? 1.0 : exact_sum<VPL>(l, top));

  // weights of the chosen, one lane each.  Normalised ones are taken relative to the largest
  // of them, so that scores that would vanish in 32 bits still share the whole.
  float lm = -INFINITY;
  if (mine >= 0) lm = fminf(lp[mine], FLT_MAX);
  float w = 0.0f;
  if (a.norm) {
    const float top = warp_max(lm);
    if (mine >= 0) {
      if (!a.sigmoid) {
        w = expf(lm - top);
      } else {
        const float ref = fminf(top, 0.0f);  // the scores times exp(-ref)
        w = lm >= 0.0f ? tail_sigmoid(lm) : expf(lm - ref) / (1.0f + expf(lm));
      }
    }
    const float z = warp_sum(w);
    w = z > 0.0f ? w / z : 0.0f;
  } else if (a.sigmoid) {
    if (mine >= 0) w = tail_sigmoid(lm);
  } else {
    float m = -INFINITY, z = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < VPL; ++i) z += l[i] > -INFINITY ? expf(l[i] - m) : 0.0f;
    z = warp_sum(z);
    if (mine >= 0) w = expf(lm - m) / z;
  }
  if (lane < a.k) {
    a.ids[row * a.k + lane] = mine;
    a.weights[row * a.k + lane] = w * a.scale;
  }
}

template <int VPL>
static cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t st, bool pdl) {
  // one warp per token; small batches take one warp per CTA, so that their rows spread over
  // the SMs and none waits for another's slots
  const int warps = a.T <= 256 ? 1 : kRouteWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.T + warps - 1) / warps));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return !a.bias && a.n_group <= 1 ? cudaLaunchKernelEx(&cfg, route_kernel<VPL, true>, a)
                                   : cudaLaunchKernelEx(&cfg, route_kernel<VPL, false>, a);
}

int launch_route(const RouteArgs& a, cudaStream_t st, bool pdl) {
  if (a.E <= 32) return launch_route_t<1>(a, st, pdl);
  if (a.E <= 64) return launch_route_t<2>(a, st, pdl);
  if (a.E <= 128) return launch_route_t<4>(a, st, pdl);
  if (a.E <= 256) return launch_route_t<8>(a, st, pdl);
  if (a.E <= 512) return launch_route_t<16>(a, st, pdl);
  return launch_route_t<32>(a, st, pdl);
}

}  // namespace gf
