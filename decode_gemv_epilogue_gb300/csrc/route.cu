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
// and bias) computes its row again in 64 bits.  Roughly one row in a hundred to a thousand
// does; computing every row in 64 bits would cost an exp of ~30 double operations per
// expert at a rate of two per clock and SM.
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

// The best key of a warp in 64 bits: largest, ties to the lowest index.
__device__ __forceinline__ void warp_best(double& key, int& e) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const double k2 = __shfl_xor_sync(0xffffffffu, key, o);
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

// Groups that stay, as a bit mask, from the keys kv (value type T, -inf: not choosable).
// ambiguous: the last kept and the first dropped score are within tol.
template <int VPL, class T>
__device__ __forceinline__ uint32_t choose_groups(const RouteArgs& a, const T (&kv)[VPL], int lane, T tol,
                                                  bool& ambiguous) {
  const T ninf = -static_cast<T>(INFINITY);
  const int gs = a.E / a.n_group;
  T mine = ninf;
  for (int g = 0; g < a.n_group; ++g) {
    T t1 = ninf, t2 = ninf;
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
    const T s = (a.group_top == 2 && t2 > ninf) ? t1 + t2 : t1;
    if (lane == g) mine = s;
  }
  int rank = 0;
  for (int g = 0; g < a.n_group; ++g) {
    const T o = __shfl_sync(0xffffffffu, mine, g);
    rank += (o > mine || (o == mine && g < lane)) ? 1 : 0;
  }
  const bool in = lane < a.n_group;
  const uint32_t kept = __ballot_sync(0xffffffffu, in && rank < a.topk_group);
  const uint32_t last = __ballot_sync(0xffffffffu, in && rank == a.topk_group - 1);
  const uint32_t next = __ballot_sync(0xffffffffu, in && rank == a.topk_group);
  if (next) {
    const T v = __shfl_sync(0xffffffffu, mine, __ffs(last) - 1), w = __shfl_sync(0xffffffffu, mine, __ffs(next) - 1);
    ambiguous = w > ninf && v - w <= tol;  // nothing in doubt where the next group is empty
  }
  return kept;
}

// The row once more in 64 bits.  Returns the expert that lane j takes in round j.
template <int VPL>
__device__ __noinline__ int route_row_f64(const RouteArgs& a, const float (&l)[VPL], int lane) {
  const double ninf = -static_cast<double>(INFINITY);
  double key[VPL];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = 1.0 / (1.0 + exp(-static_cast<double>(l[i])));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      key[i] = l[i] > -INFINITY ? exp(static_cast<double>(l[i]) - static_cast<double>(m)) : 0.0;
      z += key[i];
    }
    z = warp_sum(z);
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] /= z;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    if (!(l[i] > -INFINITY)) key[i] = ninf;
    else if (a.bias) key[i] += static_cast<double>(a.bias[e]);
    if (!(key[i] == key[i])) key[i] = ninf;
  }
  if (a.n_group > 1) {
    bool unused = false;
    const uint32_t kept = choose_groups<VPL, double>(a, key, lane, 0.0, unused);
    const int gs = a.E / a.n_group;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (!a.bias && key[i] > ninf) key[i] = static_cast<double>(l[i]);  // the order of the logits
      if (e < a.E && !((kept >> (e / gs)) & 1u)) key[i] = ninf;
    }
  }
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    double bk = ninf;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > bk) {
        bk = key[i];
        be = lane + 32 * i;
      }
    warp_best(bk, be);
    if (!(bk > ninf)) break;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 32 * i == be) key[i] = ninf;
    if (lane == j) mine = be;
  }
  return mine;
}

template <int VPL>
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
  const bool plain_key = !a.bias && a.n_group <= 1;
  bool redo = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    b[i] = (a.bias && e < a.E) ? a.bias[e] : 0.0f;
    key[i] = l[i] + 0.0f;  // -0 and +0 tie
  }
  if (!plain_key) {
    float s[VPL];
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = tail_sigmoid(l[i]);
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) m = fmaxf(m, l[i]);
      m = warp_max(m);
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        s[i] = l[i] > -INFINITY ? expf(l[i] - m) : 0.0f;
        z += s[i];
      }
      const float inv = 1.0f / warp_sum(z);
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] *= inv;
    }
    // s + bias; without a bias the groups are chosen by s and the experts by the logit
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = l[i] > -INFINITY ? s[i] + b[i] : -INFINITY;
      if (!(s[i] == s[i])) s[i] = -INFINITY;  // a NaN bias: not choosable
      s[i] += 0.0f;
    }
    uint32_t kept = 0xffffffffu;
    if (a.n_group > 1) {
      float big = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (s[i] > -INFINITY) big = fmaxf(big, fabsf(s[i]));
      kept = choose_groups<VPL, float>(a, s, lane, 4.0f * (kKeyTolAbs + kKeyTolRel * warp_max(big)), redo);
    }
    const int gs = a.E / a.n_group;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (a.bias) key[i] = s[i];
      if (a.n_group > 1 && e < a.E && !((kept >> (e / gs)) & 1u)) key[i] = -INFINITY;
    }
  }
  // top_k rounds (one more where the keys are rounded, to see the first one left out)
  int mine = -1;
  float pk = 0.0f, pl = 0.0f, pb = 0.0f;  // the previous round's key, logit and bias
  const int rounds = a.bias ? a.k + 1 : a.k;
  for (int j = 0; j < rounds && !redo; ++j) {
    float bk = key[0], bl = l[0], bb = b[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bl = l[i];
        bb = b[i];
        bi = i;
      }
    const uint32_t u = ordered(bk), best = __reduce_max_sync(0xffffffffu, u);
    if (best <= ordered(-INFINITY)) break;
    const uint32_t cand = u == best ? static_cast<uint32_t>(lane + 32 * bi) : 0xffffffffu;
    const uint32_t e = __reduce_min_sync(0xffffffffu, cand);
    const int owner = static_cast<int>(e & 31u);
    if (a.bias) {
      const float kk = __shfl_sync(0xffffffffu, bk, owner), kl = __shfl_sync(0xffffffffu, bl, owner),
                  kb = __shfl_sync(0xffffffffu, bb, owner);
      if (j > 0 && !(kl == pl && kb == pb) &&
          pk - kk <= 2.0f * (kKeyTolAbs + kKeyTolRel * fmaxf(fabsf(pk), fabsf(kk))))
        redo = true;
      pk = kk;
      pl = kl;
      pb = kb;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 32 * i == static_cast<int>(e)) key[i] = -INFINITY;
    if (lane == j && j < a.k) mine = static_cast<int>(e);
  }
  if (redo) mine = route_row_f64<VPL>(a, l, lane);

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
  return cudaLaunchKernelEx(&cfg, route_kernel<VPL>, a);
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
