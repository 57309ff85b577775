// Rotary positions: the table of frequencies (gf_rope_table) and the rotation (gf_rope).
//
// A pair (a, b) of a head's row at position p becomes m (a cos t - b sin t, a sin t + b cos t),
// t = p f.  Every element is read and written once; cosine and sine of a token's pair are computed
// once for all the heads that a thread takes.  8191 tokens of 40 heads of 128 take 54 us in f32, 6.2 TB/s: memory
// bounds it; a few tokens are a launch's latency.
#include <cmath>

#include "rope_device.cuh"
#include "gf_device.cuh"

namespace gf {

// One thread a pair, in 64 bits; a program makes the table once.
__global__ void rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  const double n = a.pairs, pi = 3.14159265358979323846;
  if (i == 0) {
    RopeHeader h = {};
    h.magnitude = a.magnitude;
    h.pairs = static_cast<uint32_t>(a.pairs);
    *static_cast<RopeHeader*>(a.table) = h;
  }
  if (i >= a.pairs) return;
  double f = exp(-static_cast<double>(i) / n * log(a.base));
  if (a.kind == 1) {
    f /= a.factor;
  } else if (a.kind == 2) {
    // the pair that makes `turns` turns over the span
    const double lo0 = floor(n * log(a.span / (2.0 * pi * a.fast)) / log(a.base));
    const double hi0 = ceil(n * log(a.span / (2.0 * pi * a.slow)) / log(a.base));
    const double lo = fmax(lo0, 0.0), hi = fmin(hi0, 2.0 * n - 1.0);
    const double r = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
    f = f * (1.0 - r) + f / a.factor * r;
  } else if (a.kind == 3) {
    const double r = fmin(fmax((a.span * f / (2.0 * pi) - a.slow) / (a.fast - a.slow), 0.0), 1.0);
    f = f * r + f / a.factor * (1.0 - r);
  }
  if (a.divisors) f /= static_cast<double>(a.divisors[i]);
  // the fraction of a turn, 2^64 a turn; whole turns drop out of an integer position's angle
  double t = f / (2.0 * pi);
  t -= floor(t);
  const double hi = floor(t * 4294967296.0), lo = (t * 4294967296.0 - hi) * 4294967296.0;
  uint64_t* turns = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(a.table) + sizeof(RopeHeader));
  turns[i] = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(fmin(rint(lo), 4294967295.0));
}

int launch_rope_table(const RopeTableArgs& a, cudaStream_t st) {
  rope_table_kernel<<<(a.pairs + 127) / 128, 128, 0, st>>>(a);
  return cudaGetLastError();
}

// VEC: a thread holds unit u (four pairs) of a token and goes through heads, blockDim / units at a time.  ONCE: it has
// one at most, whose row is on its way before the table's header is looked at.
template <typename E, bool HALVES, bool ONCE>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int units = a.dim >> 3, u = threadIdx.x % units, hp = blockDim.x / units;
  const int64_t t = blockIdx.x;
  const E* x = static_cast<const E*>(a.x) + t * a.ld;
  E* y = static_cast<E*>(a.dst) + t * a.ld_dst;
  const uint32_t table_pairs = static_cast<const RopeHeader*>(a.table)->pairs;
  const int pos = a.pos[t], first = threadIdx.x / units + hp * blockIdx.y;
  int o0, o1;
  unit_offsets(u, a.n_rot, HALVES, o0, o1);
  float4 l = {}, r = {};
  if (ONCE && first < a.heads) {
    const E* p = x + static_cast<int64_t>(first) * a.dim;
    l = load4(p + o0), r = load4(p + o1);
  }
  if (!rope_fits(table_pairs, a.n_rot, a.err)) return;
  float2 cs[4];
  const bool turns = 8 * u < a.n_rot;
  if (turns) {
    const float mag = static_cast<const RopeHeader*>(a.table)->magnitude;
    const uint64_t* f = rope_turns(a.table) + 4 * u;
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = rope_cs(f[i], pos, mag);
  }
  for (int h = first; h < a.heads; h += hp * gridDim.y) {
    if (!ONCE) {
      const E* p = x + static_cast<int64_t>(h) * a.dim;
      l = load4(p + o0), r = load4(p + o1);
    }
    float v[8] = {l.x, l.y, l.z, l.w, r.x, r.y, r.z, r.w};
    if (turns) {
#pragma unroll
      for (int i = 0; i < 4; ++i) HALVES ? rope_turn(v[i], v[4 + i], cs[i]) : rope_turn(v[2 * i], v[2 * i + 1], cs[i]);
    }
    E* q = y + static_cast<int64_t>(h) * a.dim;
    store4(q + o0, v[0], v[1], v[2], v[3]);
    store4(q + o1, v[4], v[5], v[6], v[7]);
    if (ONCE) break;
  }
}

// Any size and alignment: a thread takes one pair, or one element behind the rotated part.
template <typename E>
__global__ void __launch_bounds__(256) rope_generic_kernel(const __grid_constant__ RopeArgs a) {
  pdl_wait();
  pdl_trigger();
  if (!rope_fits(a.table, a.n_rot, a.err)) return;
  const int pairs = a.n_rot / 2, units = pairs + a.dim - a.n_rot;
  const int64_t t = blockIdx.x;
  const E* x = static_cast<const E*>(a.x) + t * a.ld;
  E* y = static_cast<E*>(a.dst) + t * a.ld_dst;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    float2 cs = make_float2(1.0f, 0.0f);
    if (u < pairs) cs = rope_cs(rope_turns(a.table)[u], a.pos[t], static_cast<const RopeHeader*>(a.table)->magnitude);
    for (int h = blockIdx.y; h < a.heads; h += gridDim.y) {
      const int64_t at = static_cast<int64_t>(h) * a.dim;
      if (u >= pairs) {
        y[at + pairs + u] = x[at + pairs + u];
      } else {
        const int64_t i = at + (a.halves ? u : 2 * u), j = at + (a.halves ? pairs + u : 2 * u + 1);
        float p = load1(x + i), q = load1(x + j);
        rope_turn(p, q, cs);
        store1(y + i, p);
        store1(y + j, q);
      }
    }
  }
}

template <typename E, bool ONCE>
static int launch_rope_t(const cudaLaunchConfig_t& cfg, const RopeArgs& a) {
  return a.halves ? cudaLaunchKernelEx(&cfg, rope_kernel<E, true, ONCE>, a) : cudaLaunchKernelEx(&cfg, rope_kernel<E, false, ONCE>, a);
}

int launch_rope(const RopeArgs& a, cudaStream_t st, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const bool f32 = a.type == 0;
  if (a.vec) {
    const int units = a.dim / 8, most = 256 / units;
    // Whole passes over the heads, equally full; few tokens spread their heads over CTAs: 40 heads of 128, f32, for 32
    // tokens 7.3 us where a CTA a token takes 9.3, for 200 9.3 and 10.3, for 256 10.4 either way, for 1000 17.5 and 14.4.
    const int passes = (a.heads + most - 1) / most, hp = (a.heads + passes - 1) / passes;
    cfg.blockDim = dim3(static_cast<unsigned>(units * hp));
    cfg.gridDim = dim3(static_cast<unsigned>(a.T), static_cast<unsigned>(a.T <= 256 ? passes : 1));
    const bool once = static_cast<int>(cfg.gridDim.y) == passes;
    if (f32) return once ? launch_rope_t<float, true>(cfg, a) : launch_rope_t<float, false>(cfg, a);
    return once ? launch_rope_t<__half, true>(cfg, a) : launch_rope_t<__half, false>(cfg, a);
  }
  cfg.blockDim = dim3(128);
  cfg.gridDim = dim3(static_cast<unsigned>(a.T), static_cast<unsigned>(a.heads < 64 ? a.heads : 64));
  return f32 ? cudaLaunchKernelEx(&cfg, rope_generic_kernel<float>, a)
             : cudaLaunchKernelEx(&cfg, rope_generic_kernel<__half>, a);
}

}  // namespace gf
