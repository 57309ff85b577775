// Attention of a decode step over the 8-bit cache (gf_attend).
//
// One pass over a row's keys and values with the running maximum and sum of the softmax.  What bounds it
// is reading the codes: each warp copies (cp.async) chunks of CT tokens, whole lines of consecutive addresses, into
// stages of its own, a chunk ahead.  (Copies of just the bytes that a lane decodes itself, in fours of rows, left
// the memory at 5.0 TB/s where consecutive ones reach 6.4.)  With the arithmetic, 938 instructions a chunk at three
// warps a scheduler, 256 sequences of 4000 to 8000 keys and 32 query heads over 8 of 128 take 556 us, 5.5 TB/s.
//
// A warp takes a chunk of CT tokens.  m16n8k16 with the queries as the 16 rows: eight rows' f16 high parts and
// the same rows' low parts (q = hi + lo to 22 bits under a power of two a row), so that one instruction
// gives both and a lane holds the two halves of its own sums.  Codes are exact in f16.  The contraction
// over dims and the order of the tokens are free, so that
//   keys  : lane (g, c) takes 16-byte units c, c + 4, .. of token g; the four bytes of a word are the
//           two k pairs of one instruction;
//   values: lane (g, c) takes a unit of the four tokens that its k indices mean; the bytes of four
//           tokens' words are paired by dim, and dim j of column g's unit is column g of instruction j.
// The weights p * scale_v are split into hi + lo like the queries, under a power of two a row.  A chunk's products are
// added to the running ones in 32 bits, outside the matrix unit (which truncates).
//
// Items, (tokens of a sequence next to each other, head of the cache, part of its queries), are laid end
// to end by their number of chunks and some more for their start and end; every CTA takes an equal stretch
// and every warp an equal stretch of that, whatever the sequences' lengths.  Warps know nothing of each other
// until they are done: the parts of an item that reaches over several go through the workspace, where the CTA
// joins its own and a second launch joins the CTAs', both in order.  (A CTA to an item, its warps joined in shared
// memory at each one's end, took twice as long for 61 sequences of 100 to 8000 keys: short ones cost it a
// barrier's round each.)
#include <cfloat>

#include "cache_device.cuh"
#include "gf_device.cuh"
#include "rope_device.cuh"

namespace gf {

// Warps of a CTA, two of which share an SM: as many as the registers allow (NM: tiles of eight rows).  Six for two
// tiles of 64 dims take 77 us where four take 86 (33 sequences, two tokens of 64 query heads each).
__host__ __device__ constexpr int att_warps(int dc, int nm) { return dc == 64 || (dc == 128 && nm == 1) ? 6 : 4; }

template <int DC, int NM>
struct AttShape {
  static constexpr int kTokens = DC == 256 ? 16 : 32;               // of a chunk
  static constexpr bool kQRegs = DC <= 128 && NM == 1;              // queries in registers, else in shared memory
  static constexpr int kWarps = att_warps(DC, NM);
  static constexpr int kRows = 8 * NM;
  static constexpr int kSteps = DC / 16;                            // instructions along the dims
  static constexpr int kStage = kTokens * DC;                       // a chunk's keys or values; two of each
  static constexpr int kScalesAt = kWarps * 4 * kStage;             // of all warps: keys' and values' scales
  static constexpr int kQueriesAt = kScalesAt + kWarps * 8 * kTokens;
  static constexpr int kSmem = kQueriesAt + (kQRegs ? 0 : kWarps * NM * kSteps * 512);
  static constexpr int kSlices = kRows * DC / 128;                  // float4 a lane of a row part
  static constexpr int64_t kPart = kRows * (DC + 2);                // floats: sums, maxima, sums of weights
};
template <int DC>
constexpr int kUnitBytes = DC == 64 ? 8 : 16;  // of a value row, in a lane's hands

// An item's start and end in units of a chunk's time.  At one unit 61 sequences of 100 to 8000 keys take 66 us where
// 63, 244 of them 226 where 212; at six 64 and 220.  They come first, and a share that ends within them leaves the
// item to the next: only a share's chunks make a part.
constexpr int kItemUnits = 3;
// Running maximum of a row without keys: no finite score lies below it, and a masked one, -inf, has no weight under it.
constexpr float kNoMax = -FLT_MAX;
// Weights times their values' scales, as f16 parts, reach 2^15 in units of a power of two a row.  A unit serves
// chunks whose scales lie within 2^-9 of it: the parts' last step, 2^-24, is then 2^-30 of the smallest of them.
constexpr int kWeightBits = 15;
constexpr int kScaleSpread = 8;  // exponents below the unit's
// A unit may fall to 2^-56 of what earlier keys have left in the sums, as far as that is known (2^kScaleSpread more at
// worst): those reach 2^(24 + 56 + 8) then, times the keys.
constexpr float kUnitFall = 56.0f;
// Parts hold their sums times this: a mean of the largest values is finite, and so is what a million of them add up to.
constexpr float kPartScale = 0x1p-20f;

// A stage is lines of 128 bytes (two tokens of 64, half a token of 256) whose 16-byte units are exchanged by
// the line's number.  Unit u of token r of a chunk:
template <int DC>
__device__ __forceinline__ uint32_t smem_place(int r, int u) {
  const int line = r * (DC / 64) / 2 + (DC == 256 ? u >> 3 : 0), at = DC == 64 ? (r & 1) * 4 + u : u & 7;
  return line * 128 + ((at ^ (line & 7)) * 16);
}
// The same eight tokens n times further on (from an offset within the first eight).
template <int DC>
__device__ __forceinline__ uint32_t further(uint32_t place, int n) {
  return (DC == 64 && n % 2 ? place ^ 64u : place) + n * 8 * DC;
}

// The token of eight that is column n of the instructions, and the unit of values that is column g (DC 64: half
// units): chosen so that lanes which read together meet all banks.  They read keys as units c .. c + 3 of
// columns 2p and 2p + 1, values as two units of columns 0, 2, 4, 6 or 1, 3, 5, 7.
template <int DC>
__device__ __forceinline__ int token_of(int n) {
  constexpr uint32_t order = DC == 64 ? 0x65742130u : DC == 128 ? 0x73625140u : 0x53427160u;
  return order >> 4 * n & 7;
}
template <int DC>
__device__ __forceinline__ int column_of(int token) {
  constexpr uint32_t order = DC == 64 ? 0x57641320u : DC == 128 ? 0x75316420u : 0x31756420u;
  return order >> 4 * token & 7;
}
template <int DC>
__device__ __forceinline__ int value_unit(int g) {
  return DC == 128 ? (g >> 1) | (g & 1) << 2 : g;
}

// ------------------------------------------------------------------ small pieces
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
__device__ __forceinline__ void mma0(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.0f));
}

// 2^x to two units, results below 2^-126 as zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Constants that the conversion wants in registers: with immediates it takes five instructions a word, not
// three (the inner loop's arithmetic units were busy 56% of the time with them).
struct Magic {
  uint32_t mask, turn;
  __device__ __forceinline__ Magic() {
    asm volatile("mov.b32 %0, 0x00ff00ff;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x64806480;" : "=r"(turn));
  }
};

__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// A word's four codes as two pairs of f16: bytes 0 and kSecond, and the others.  i8: 1024 + (code + 128) is an
// f16 whose low byte is the code's with its top bit turned, less 1152.
template <int FMT>
constexpr int kSecond = FMT == 0 ? 2 : 1;
template <int FMT>
__device__ __forceinline__ void pairs_of(const Magic& k, uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == 0) {
    lo = h2_sub(and_xor(w, k.mask, k.turn), k.turn);
    hi = h2_sub(and_xor(w >> 8, k.mask, k.turn), k.turn);
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(w >> 16)));
  }
}
// Dims 0, 1 (and 2, 3) of two tokens' words as such a word: the pairs are then a dim's two tokens.
template <int FMT>
__device__ __forceinline__ uint32_t weave(uint32_t a, uint32_t b, bool upper) {
  return FMT == 0 ? __byte_perm(a, b, upper ? 0x7632 : 0x5410) : __byte_perm(a, b, upper ? 0x7362 : 0x5140);
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// f16 high and low parts of two values, as pairs.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const float2 r = fsub2(make_float2(a, b), f);
  const __half2 l = __floats2half2_rn(r.x, r.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// ------------------------------------------------------------------ items
struct Item {
  int64_t begin;   // its first unit, among all items'
  int t0, n;       // tokens
  int seq;
  int lo, hi;      // keys [lo, hi) that its tokens see together
  int chunks;      // of one (head, part) of it
  int hs;          // head * subs + part
};

// Keys that token t sees, [lo, hi); none: hi = 0.
__device__ __forceinline__ void keys_of(const AttendArgs& a, int t, int& seq, int& lo, int& hi) {
  seq = a.seq ? a.seq[t] : t;
  lo = hi = 0;
  if (seq < 0 || seq >= a.c.n_seqs) {
    seq = -1;
    return;
  }
  const int64_t most = a.c.table_ld << a.c.page_log2;
  const int p = a.pos[t];
  if (p < 0) {
    seq = -1;
    return;
  }
  hi = static_cast<int>(static_cast<int64_t>(p) + 1 < most ? p + 1 : most);
  const int64_t first = a.window > 0 ? static_cast<int64_t>(p) + 1 - a.window : 0;
  lo = static_cast<int>(first < 0 ? 0 : first < hi ? first : hi);
}

// The item that begins with token t, if one does: neighbouring tokens of one sequence up to the next edge.  `run`
// tokens of a sequence are expected next to each other, and fall into items of `tokens`: an item may begin at their
// edges wherever the sequences lie.
template <int CT>
__device__ __forceinline__ bool item_at(const AttendArgs& a, int t, Item& it) {
  int seq, lo, hi;
  keys_of(a, t, seq, lo, hi);
  it.t0 = t;
  it.n = 1;
  it.seq = seq;
  if (a.tokens > 1 && seq >= 0) {
    const int in_run = t % a.run, in_item = in_run % a.tokens;
    if (in_item > 0) {
      int s, l, h;
      keys_of(a, t - 1, s, l, h);
      if (s == seq) return false;
    }
    const int most = min(min(a.tokens - in_item, a.run - in_run), a.T - t);
    bool same = true;
#pragma unroll 4
    for (int i = 1; i < most; ++i) {  // (no way out: the loads do not wait for one another)
      int s, l, h;
      keys_of(a, t + i, s, l, h);
      same &= s == seq;
      if (same) {
        lo = l < lo ? l : lo;
        hi = h > hi ? h : hi;
        ++it.n;
      }
    }
  }
  it.lo = lo;
  it.hi = hi;
  const int c = (hi + CT - 1) / CT - lo / CT;
  it.chunks = c > 0 ? c : 1;
  return true;
}

// Workspace: a header, a record of each CTA's first item, each CTA's two parts, each warp's first part.
struct AttHeader {
  int64_t ctas;
  int64_t each, more;  // units of a CTA; the first `more` take one more
};
struct AttSpan {       // an item as the joining needs it
  int64_t begin, end;  // units
  int t0, n, hs, pad;
};
constexpr int kAttHead = 64;
__host__ __device__ constexpr int64_t att_parts_at(int ctas) { return kAttHead + static_cast<int64_t>(ctas) * 32; }

// Unit at which CTA i begins.
__device__ __forceinline__ int64_t share(const AttHeader& h, int64_t i) {
  return i * h.each + (i < h.more ? i : h.more);
}

__device__ __forceinline__ AttSpan span_of(const Item& it) {
  return AttSpan{it.begin, it.begin + it.chunks + kItemUnits, it.t0, it.n, it.hs, 0};
}

template <int CT>
__device__ __forceinline__ uint32_t units_at(const AttendArgs& a, int t) {
  Item it;
  return t < a.T && item_at<CT>(a, t, it) ? it.chunks + kItemUnits : 0;
}

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

__device__ __forceinline__ void write_out(const AttendArgs& a, int64_t at, float4 v) {
  if (a.type == 0) {
    float* p = static_cast<float*>(a.dst) + at;
    if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
      store4(p, v.x, v.y, v.z, v.w);
    } else {
      p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
    }
  } else {
    __half* p = static_cast<__half*>(a.dst) + at;
    if ((reinterpret_cast<uintptr_t>(p) & 7) == 0) {
      store4(p, v.x, v.y, v.z, v.w);
    } else {
      store1(p, v.x), store1(p + 1, v.y), store1(p + 2, v.z), store1(p + 3, v.w);
    }
  }
}

// Token and query head of row r of an item; false where it has none.
__device__ __forceinline__ bool row_of(const AttendArgs& a, int t0, int n, int hs, int r, int& t, int& head) {
  const int i = r / a.rows, h = r - i * a.rows, sub = hs % a.subs;
  t = t0 + i;
  const int in_group = sub * a.rows + h;
  head = hs / a.subs * a.group + in_group;
  return i < n && in_group < a.group;
}

// A part's place (maximum, sum of weights, four sums) added to a running one.
__device__ __forceinline__ void join_part(float m, float l, float4 x, float& top, float& z, float4& v) {
  const float now = fmaxf(top, m), e0 = exp2_fast(top - now), e = exp2_fast(m - now);
  top = now;
  z = fmaf(l, e, z * e0);
  v.x = fmaf(x.x, e, v.x * e0), v.y = fmaf(x.y, e, v.y * e0);
  v.z = fmaf(x.z, e, v.z * e0), v.w = fmaf(x.w, e, v.w * e0);
}

// A slice's place of a joined item as output.
template <int DC, int NM>
__device__ __forceinline__ void join_out(const AttendArgs& a, const AttSpan& s, int slice, int lane, float top, float z,
                                         float4 v) {
  using S = AttShape<DC, NM>;
  constexpr int UB = kUnitBytes<DC>, PER = S::kSlices / NM;  // slices of eight rows: unit, column parity, four dims
  static_assert((DC == 256 ? 2 : 1) * 2 * (UB / 4) == PER, "as the parts are laid out");
  const int k = slice % PER, r = 8 * (slice / PER) + (lane >> 2);
  const int d = (value_unit<DC>(2 * (lane & 3) + k / (UB / 4) % 2) + 8 * (k / (UB / 2))) * UB + k % (UB / 4) * 4;
  int t, head;
  if (!row_of(a, s.t0, s.n, s.hs, r, t, head)) return;
  const float inv = z == 0.0f ? 0.0f : 1.0f / kPartScale / z;  // no keys: zeros
  if (d < a.c.dim)
    write_out(a, t * a.ld_dst + static_cast<int64_t>(head) * a.c.dim + d,
              make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
  if (d == 0 && a.lse)
    a.lse[static_cast<int64_t>(t) * a.q_heads + head] = z == 0.0f ? -INFINITY : (top + log2f(z)) * 0.693147181f;
}

// ------------------------------------------------------------------ the kernel
// EXACT: heads of DC elements, else of fewer (a multiple of 16).
template <int DC, bool EXACT, int FMT, int NM>
__global__ void __launch_bounds__(32 * AttShape<DC, NM>::kWarps, 2) attend_kernel(const __grid_constant__ AttendArgs a) {
  using S = AttShape<DC, NM>;
  constexpr int CT = S::kTokens, W = S::kWarps, KS = S::kSteps, NT = CT / 8, KG = CT / 16;
  constexpr int UC = DC == 256 ? 2 : 1;       // units of a value row that a lane holds
  constexpr int UB = kUnitBytes<DC>;
  constexpr int NO = DC / 8;                  // column tiles of the output
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t group_units[kAttMaxTokens / 32];  // of 32 tokens each, for one (head, part)
  __shared__ AttSpan spans[W][2];                       // the items of the warps' parts: first, last
  __shared__ float2 part_rows[W][2][S::kRows];          // maxima and sums of weights of their rows
  __shared__ float2 rooms[W][NM][32];                   // a lane's rows: see `unit`
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c4 = lane & 3;
  const Magic magic;
  const int HS = a.c.heads * a.subs;
  const int D = EXACT ? DC : a.c.dim, U16 = D / 16;

  // ---- this warp's stretch of units
  const int groups = (a.T + 31) / 32;
  for (int k = warp; k < groups; k += W) {
    const uint32_t n = __reduce_add_sync(0xffffffffu, units_at<CT>(a, k * 32 + lane));
    if (lane == 0) group_units[k] = n;
  }
  __syncthreads();
  int64_t total = 0;
  for (int k = lane; k < groups; k += 32) total += group_units[k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= HS;
  // a CTA takes one unit a warp at least
  AttHeader head;
  head.ctas = min(static_cast<int64_t>(a.ctas), (total + W - 1) / W);
  if (blockIdx.x >= head.ctas) return;
  head.each = total >> 32 ? total / head.ctas : static_cast<uint32_t>(total) / static_cast<uint32_t>(head.ctas);
  head.more = total - head.each * head.ctas;
  const int64_t cta_start = share(head, blockIdx.x), cta_units = share(head, blockIdx.x + 1) - cta_start;
  const int64_t start = cta_start + cta_units * warp / W, stop = cta_start + cta_units * (warp + 1) / W;
  float* cta_parts = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.workspace) + att_parts_at(a.ctas)) +
                     static_cast<int64_t>(blockIdx.x) * 2 * S::kPart;
  float* warp_part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.workspace) + att_parts_at(a.ctas)) +
                     (static_cast<int64_t>(a.ctas) * 2 + static_cast<int64_t>(blockIdx.x) * W + warp) * S::kPart;
  bool kept = false;  // a part lies there
  if (lane < 2) spans[warp][lane].end = 0;  // no part
  __syncwarp();
  if (start < stop) {
    Item item;
    {
      int64_t before = 0;  // units of one (head, part) ahead of the group
      int k = 0;
      for (; k < groups; k += 32) {
        const int64_t n = k + lane < groups ? group_units[k + lane] : 0;
        const int64_t incl = warp_scan(n, lane) + before;
        const uint32_t past = __ballot_sync(0xffffffffu, incl * HS > start);
        if (past) {
          const int l = __ffs(past) - 1;
          before = __shfl_sync(0xffffffffu, incl - n, l);
          k += l;
          break;
        }
        before = __shfl_sync(0xffffffffu, incl, 31);
      }
      const int64_t n = units_at<CT>(a, k * 32 + lane);
      const int64_t incl = warp_scan(n, lane) + before;
      const int l = __ffs(__ballot_sync(0xffffffffu, incl * HS > start)) - 1;
      item_at<CT>(a, k * 32 + l, item);
      const int64_t b = __shfl_sync(0xffffffffu, incl - n, l) * HS;
      item.hs = static_cast<int>((start - b) / (item.chunks + kItemUnits));
      item.begin = b + static_cast<int64_t>(item.hs) * (item.chunks + kItemUnits);
    }
    if (start == cta_start && lane == 0) {
      if (blockIdx.x == 0) *reinterpret_cast<AttHeader*>(a.workspace) = head;
      reinterpret_cast<AttSpan*>(reinterpret_cast<uint8_t*>(a.workspace) + kAttHead)[blockIdx.x] = span_of(item);
    }
    uint8_t* ring = smem + warp * 4 * S::kStage;
    static_assert(S::kRows * DC * 4 <= 2 * S::kStage, "a warp's two parts fit its stages");
    const uint32_t ring_at = smem_u32(ring);
    float* ring_scales = reinterpret_cast<float*>(smem + S::kScalesAt) + warp * 2 * CT;
    uint8_t* qs = smem + S::kQueriesAt + warp * NM * KS * 512;

    const int page_log2 = a.c.page_log2, page_mask = (1 << page_log2) - 1, table_ld = static_cast<int>(a.c.table_ld);
    const int64_t page_bytes = static_cast<int64_t>(a.c.heads * D) << page_log2;
    const int64_t page_scales = static_cast<int64_t>(a.c.heads) << (page_log2 - a.c.block_log2);
    const bool one_page = CT == 16 || page_log2 >= 5;  // a chunk never crosses a page's end
    const int scale_lane = (lane & ~7) + column_of<DC>(lane & 7);  // scales lie in the order of the columns
    // where a lane's copies go, less 512 bytes a copy: repeating after kPlaces
    constexpr int kPlaces = DC == 256 ? 4 : 2;
    uint32_t copy_to[kPlaces];
#pragma unroll
    for (int k = 0; k < kPlaces; ++k)
      copy_to[k] = ring_at + smem_place<DC>(lane / (DC / 16) + k * (512 / DC), lane % (DC / 16)) - k * 512;

    const bool lane_on = lane % (DC / 16) < U16;  // a lane copies 16 bytes of every (512 / DC)th token
    const int lane_at = lane / (DC / 16) * D + lane % (DC / 16) * 16, copy_step = 512 / DC * D;

    // What a chunk's copies need of its item.
    struct Source {
      int seq, first, lo, hi, head;  // first: of the item's chunks, among those of its sequence
    };
    auto source_of = [&](const Item& it) {
      return Source{it.seq, it.lo / CT, it.lo, it.hi, it.hs / a.subs};
    };
    struct Pages {
      int id[KG];
    };
    // The pages of a chunk's 16-token halves, as the table has them (-1: outside the table).
    auto pages_of = [&](const Source& s, int chunk) {
      Pages p;
      const int i = (s.first + chunk) * CT >> page_log2;
      const int32_t* row = a.c.table + s.seq * a.c.table_ld;
      p.id[0] = s.hi > 0 && i < table_ld ? row[i] : -1;
      if (KG == 2) p.id[KG - 1] = one_page ? p.id[0] : s.hi > 0 && i + 1 < table_ld ? row[i + 1] : -1;
      return p;
    };
    float key_scale = 0.0f, value_scale = 0.0f;  // of token `lane` of the chunk fetched last, on their way
    // Copies a chunk's keys and values into stage chunk % 2.  Tokens outside [lo, hi) or without a page: zeros,
    // scales and codes.  Returns which tokens of the chunk those are.
    auto fetch = [&](const Source& s, int chunk, const Pages& pages) {
      const int p0 = (s.first + chunk) * CT, slot = p0 & page_mask;
      const uint32_t stage = (chunk & 1) * 2 * S::kStage;
      const int64_t head_at = (static_cast<int64_t>(s.head * D) << page_log2) + lane_at, n_pages = a.c.n_pages;
      const int64_t head_scales = static_cast<int64_t>(s.head) << (page_log2 - a.c.block_log2);
      bool held[KG], all = true;
#pragma unroll
      for (int h = 0; h < KG; ++h) all &= held[h] = static_cast<uint32_t>(pages.id[h]) < n_pages;
      uint32_t hidden = 0;
      key_scale = value_scale = 0.0f;
      // Whole chunks, by halves (a page may hold 16 tokens): one address for each, its copies at fixed steps.  With
      // an address for each copy instead, 64 sequences of 6000 keys in pages of 16 took 195 us where 168, heads of
      // 96 took 192 where 175.
      if (all && p0 >= s.lo && p0 + CT <= s.hi) {
#pragma unroll
        for (int h = 0; h < KG; ++h) {
          const int64_t at = pages.id[h] * page_bytes + (head_at + ((slot + 16 * h) & page_mask) * D);
          const uint8_t* k = a.c.k + at;
          const uint8_t* v = a.c.v + at;
#pragma unroll
          for (int i = 0; i < DC / 32; ++i) {
            const uint32_t to = copy_to[(h * (DC / 32) + i) % kPlaces] + stage + (h * (DC / 32) + i) * 512;
            if (EXACT || lane_on) {
              cp_async16(to, k + i * copy_step, true);
              cp_async16(to + S::kStage, v + i * copy_step, true);
            }
          }
        }
        const int j = lane & (CT - 1);
        const int64_t sc = (KG == 2 && j >= 16 ? pages.id[KG - 1] : pages.id[0]) * page_scales +
                           (head_scales + (((slot + j) & page_mask) >> a.c.block_log2));
        key_scale = a.c.k_scale[sc];
        value_scale = a.c.v_scale[sc];
      } else {
#pragma unroll 1
        for (int i = 0; i < CT * DC / 512; ++i) {
          const int row = lane / (DC / 16) + i * (512 / DC);
          if (EXACT || lane_on) {
            const bool up = KG == 2 && row >= 16;
            const bool on = (up ? held[KG - 1] : held[0]) && p0 + row >= s.lo && p0 + row < s.hi;
            const int64_t at = (up ? pages.id[KG - 1] : pages.id[0]) * page_bytes +
                               (head_at + ((slot + i * (512 / DC)) & page_mask) * D);
            const uint32_t to = ring_at + stage + smem_place<DC>(row, lane % (DC / 16));
            cp_async16(to, a.c.k + (on ? at : 0), on);
            cp_async16(to + S::kStage, a.c.v + (on ? at : 0), on);
          }
        }
        const int j = lane & (CT - 1);
        const bool up = KG == 2 && j >= 16;
        const bool on = (up ? held[KG - 1] : held[0]) && p0 + j >= s.lo && p0 + j < s.hi;
        hidden = __ballot_sync(0xffffffffu, !on);
        if (on) {
          const int64_t sc = (up ? pages.id[KG - 1] : pages.id[0]) * page_scales +
                             (head_scales + (((slot + j) & page_mask) >> a.c.block_log2));
          key_scale = a.c.k_scale[sc];
          value_scale = a.c.v_scale[sc];
        }
      }
      cp_commit();
      return hidden;
    };
    // The item's chunks [c0, c1) of this warp's stretch.
    auto stretch = [&](const Item& it, int& c0, int& c1) {
      const int64_t from = start - it.begin - kItemUnits, to = stop - it.begin - kItemUnits;
      c0 = from < 0 ? 0 : static_cast<int>(from);
      c1 = to < it.chunks ? static_cast<int>(to) : it.chunks;
    };

    int c0, c1;
    stretch(item, c0, c1);
    Source src = source_of(item);
    uint32_t hidden_next = c0 < c1 ? fetch(src, c0, pages_of(src, c0)) : 0;
    Pages pages = pages_of(src, c0 + 1);  // of the chunk that is fetched next: looked up a chunk ahead

    while (stop > item.begin + kItemUnits) {  // (a first item without a chunk of its own is the next warp's)
      // ---- the item's queries, hi and lo parts in the order of the instructions' rows: of row g, lane (g, c4)
      // takes units c4, c4 + 4, .. as it does of a key
      uint4 qr[S::kQRegs ? KS : 1];
      float f[NM];  // of the products: the query's power of two, scale and log2(e)
      int lo[NM], hi[NM];
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        int t, head;
        const bool live = row_of(a, item.t0, item.n, item.hs, 8 * i + g, t, head);
        const int64_t row = t * a.ldq + static_cast<int64_t>(head) * D;
        float4 v[KS];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int d = (k / 4) * 64 + c4 * 16 + (k % 4) * 4;
          v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (live && d < D) {
            const int64_t at = row + d;
            if (a.type == 0) {
              const float* p = static_cast<const float*>(a.q) + at;
              v[k] = a.vec ? load4(p) : make_float4(p[0], p[1], p[2], p[3]);
            } else {
              const __half* p = static_cast<const __half*>(a.q) + at;
              v[k] = a.vec ? load4(p) : make_float4(load1(p), load1(p + 1), load1(p + 2), load1(p + 3));
            }
          }
          top = max(top, max(max(__float_as_uint(v[k].x) & 0x7fffffffu, __float_as_uint(v[k].y) & 0x7fffffffu),
                             max(__float_as_uint(v[k].z) & 0x7fffffffu, __float_as_uint(v[k].w) & 0x7fffffffu)));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // |q| 2^-x lies in [2^14, 2^15) for the largest
        int x = static_cast<int>(top >> 23) - 127 - 14;
        x = x < -110 ? -110 : x;
        const bool number = top < 0x7f800000u;
        const float w = __uint_as_float(static_cast<uint32_t>(127 - x) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint4 h;
          const float e[4] = {number ? v[k].x * w : 0.0f, number ? v[k].y * w : 0.0f, number ? v[k].z * w : 0.0f,
                              number ? v[k].w * w : 0.0f};
          split2(e[0], e[kSecond<FMT>], h.x, h.y);
          split2(e[3 - kSecond<FMT>], e[3], h.z, h.w);
          if constexpr (S::kQRegs)
            qr[k] = h;
          else
            *reinterpret_cast<uint4*>(qs + ((i * KS + k) * 32 + lane) * 16) = h;  // read back by this lane alone
        }
        f[i] = number ? a.scale * __uint_as_float(static_cast<uint32_t>(127 + x) << 23) : __uint_as_float(0x7fffffffu);
        lo[i] = hi[i] = 0;
        int s;
        if (live) keys_of(a, t, s, lo[i], hi[i]);
      }

      float2 o[NM][NO];
      float m[NM], l[NM];
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        m[i] = kNoMax;
        l[i] = 0.0f;
#pragma unroll
        for (int n = 0; n < NO; ++n) o[i][n] = make_float2(0.0f, 0.0f);
      }
      // Biased exponent of each row's unit, at least that of the format's smallest scale.  Beside it, when it was last
      // looked at: how far above (or, after chunks without weight, below) it the sums' own lay, the largest weight times
      // scale that went in, and the maximum then.
      int unit[NM];
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        unit[i] = 127 - 111;
        rooms[warp][i][lane] = make_float2(0.0f, kNoMax);
      }
      const int t0 = token_of<DC>(2 * c4), t1 = token_of<DC>(2 * c4 + 1);  // this lane's columns

      for (int c = c0; c < c1; ++c) {
        const uint32_t hidden = hidden_next;
        if (CT == 32 || lane < CT) {
          ring_scales[scale_lane] = key_scale;
          ring_scales[CT + scale_lane] = value_scale;
        }
        // The chunk's largest and smallest scale.  (One that is not finite makes its own rows NaN, and is no measure
        // for the others; nor is zero, which tokens without a place have.)
        const uint32_t vbits = __float_as_uint(value_scale) & 0x7fffffffu;
        const int vtop = static_cast<int>(__reduce_max_sync(0xffffffffu, vbits < 0x7f800000u ? vbits : 0u) >> 23) + 1;
        const int vlow = static_cast<int>(__reduce_min_sync(0xffffffffu, vbits - 1u) >> 23) + 1;
        if (c + 1 < c1) {
          hidden_next = fetch(src, c + 1, pages);
          pages = pages_of(src, c + 2);
          cp_wait<1>();
        } else {
          cp_wait<0>();
        }
        __syncwarp();
        const uint8_t* kt = ring + (c & 1) * 2 * S::kStage;
        const uint8_t* vt = kt + S::kStage;
        const float* ks = ring_scales;
        const float* vs = ks + CT;
        const int p0 = (src.first + c) * CT;

        // ---- scores (powers of two)
        float2 x[NM][NT];
        {
          float s[NM][NT][4];
#pragma unroll
          for (int u = 0; u < DC / 64; ++u) {
            uint4 q[NM][4];
#pragma unroll
            for (int i = 0; i < NM; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if constexpr (S::kQRegs)
                  q[i][j] = qr[u * 4 + j];
                else
                  q[i][j] = *reinterpret_cast<const uint4*>(qs + ((i * KS + u * 4 + j) * 32 + lane) * 16);
              }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint4 w = make_uint4(0, 0, 0, 0);  // a unit that the head does not have
              if (EXACT || c4 + 4 * u < U16)
                w = *reinterpret_cast<const uint4*>(kt + further<DC>(smem_place<DC>(token_of<DC>(g), c4 + 4 * u), n));
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t b0, b1;
                pairs_of<FMT>(magic, ww[j], b0, b1);
#pragma unroll
                for (int i = 0; i < NM; ++i) u + j == 0 ? mma0(s[i][n], q[i][j], b0, b1) : mma(s[i][n], q[i][j], b0, b1);
              }
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float2 k2 = *reinterpret_cast<const float2*>(ks + 8 * n + 2 * c4);
#pragma unroll
            for (int i = 0; i < NM; ++i)
              x[i][n] = fmul2(fadd2(make_float2(s[i][n][0], s[i][n][1]), make_float2(s[i][n][2], s[i][n][3])),
                              fmul2(k2, make_float2(f[i], f[i])));
          }
        }

        // ---- softmax; the weights, times the values' scales, as instructions' rows
        bool other = false;  // a row's unit does not serve this chunk
#pragma unroll
        for (int i = 0; i < NM; ++i) other |= vtop > unit[i] || vlow < unit[i] - kScaleSpread;
        other = __any_sync(0xffffffffu, other);
        uint4 pf[NM][KG];
        float alpha[NM];
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          const bool whole = hidden == 0 && p0 >= lo[i] && p0 + CT <= hi[i];
          if (!whole) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int j0 = 8 * n + t0, j1 = 8 * n + t1;
              if ((hidden >> j0 & 1) || p0 + j0 < lo[i] || p0 + j0 >= hi[i]) x[i][n].x = -INFINITY;
              if ((hidden >> j1 & 1) || p0 + j1 < lo[i] || p0 + j1 >= hi[i]) x[i][n].y = -INFINITY;
            }
          }
          float top = kNoMax;
#pragma unroll
          for (int n = 0; n < NT; ++n) top = fmaxf(top, fmaxf(x[i][n].x, x[i][n].y));
          top = fmaxf(m[i], quad_max(top));
          const float before = m[i], down = before - top, keep = exp2_fast(down);
          alpha[i] = keep;
          m[i] = top;
          if (__builtin_expect(other, 0)) {
            // A unit for this chunk.  Above its scales, unless those lie far apart, or far above both the sums' own and
            // what this chunk's weights make of them: then above the largest weight times scale among the keys that the row
            // sees, and the unit stays if that is what it serves.  A block of large values that the softmax gives no weight,
            // or that only other rows see, so takes no bits from the others (with a unit above every scale so far, 2^20
            // between scales left errors of 1e-3 of the row, 2^34 zeros; it took 545 us where 556 in the case above).
            float most = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float2 v2 = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * c4);
              const float a = fabsf(exp2_fast(x[i][n].x - top) * v2.x), b = fabsf(exp2_fast(x[i][n].y - top) * v2.y);
              most = fmaxf(most, fmaxf(a < INFINITY ? a : 0.0f, b < INFINITY ? b : 0.0f));
            }
            const int fit = static_cast<int>(__float_as_uint(quad_max(most)) >> 23) + 1;  // (1: no weight at all)
            // The sums' own: as it was and this chunk's; a maximum since then came with a weight of 1 and a scale that the
            // unit served.
            const float2 was = rooms[warp][i][lane];
            float own = fmaxf(static_cast<float>(unit[i]) + was.x + (was.y - top), static_cast<float>(fit));
            if (before > was.y) own = fmaxf(own, static_cast<float>(unit[i] - kScaleSpread) + down);
            const bool alike = vlow >= vtop - kScaleSpread;
            int now = unit[i];
            if (hi[i] == 0 || (alike && static_cast<float>(vtop - kScaleSpread) <= own))
              now = vtop;
            else if (fit > unit[i] || (!alike && fit > 1 && fit < unit[i] - kScaleSpread))
              now = fit;
            const float most_own = fmaxf(fmaxf(own, static_cast<float>(unit[i]) + down), 0.0f);
            now = max(max(now, 127 - 111), static_cast<int>(ceilf(most_own - kUnitFall)));
            const int step = unit[i] - now, half = step / 2;
            alpha[i] = keep * __uint_as_float((127 + half) << 23) * __uint_as_float((127 + step - half) << 23);
            unit[i] = now;
            rooms[warp][i][lane] = make_float2(own - static_cast<float>(now), top);
          }
          // 2^kWeightBits a unit
          const float vinv = __uint_as_float((254 + kWeightBits - unit[i]) << 23);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float2 v2 = *reinterpret_cast<const float2*>(vs + 8 * n + 2 * c4);
            const float2 e = fsub2(x[i][n], make_float2(top, top));
            const float2 p = make_float2(exp2_fast(e.x), exp2_fast(e.y));
            sum = fadd2(sum, p);
            float2 y = fmul2(fmul2(p, v2), make_float2(vinv, vinv));
            if (!whole) {  // a masked token's weight is zero whatever lies in its scale
              if (x[i][n].x == -INFINITY) y.x = 0.0f;
              if (x[i][n].y == -INFINITY) y.y = 0.0f;
            }
            uint32_t h, w;
            split2(y.x, y.y, h, w);
            if (n % 2 == 0) {
              pf[i][n / 2].x = h;
              pf[i][n / 2].y = w;
            } else {
              pf[i][n / 2].z = h;
              pf[i][n / 2].w = w;
            }
          }
          l[i] = l[i] * keep + (sum.x + sum.y);
        }

        // ---- values
#pragma unroll
        for (int u = 0; u < UC; ++u) {
          uint32_t raw[KG][4][UB / 4];
#pragma unroll
          for (int k = 0; k < KG; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // this lane's unit of the tokens that are its k indices: columns 2 c4 and 2 c4 + 1 of two eights
              const int t = i % 2 ? t1 : t0;
              const uint8_t* at = vt + further<DC>(DC == 64 ? smem_place<DC>(t, g >> 1) + (g & 1) * 8
                                                            : smem_place<DC>(t, value_unit<DC>(g) + 8 * u), 2 * k + i / 2);
              if constexpr (UB == 16) {
                const uint4 w = *reinterpret_cast<const uint4*>(at);
                raw[k][i][0] = w.x, raw[k][i][1] = w.y, raw[k][i][2] = w.z, raw[k][i][3] = w.w;
              } else {
                const uint2 w = *reinterpret_cast<const uint2*>(at);
                raw[k][i][0] = w.x, raw[k][i][1] = w.y;
              }
            }
#pragma unroll
          for (int w = 0; w < UB / 4; ++w) {
            float acc[NM][4][4];
#pragma unroll
            for (int k = 0; k < KG; ++k) {
              uint32_t b0[4], b1[4];
              pairs_of<FMT>(magic, weave<FMT>(raw[k][0][w], raw[k][1][w], false), b0[0], b0[1]);
              pairs_of<FMT>(magic, weave<FMT>(raw[k][0][w], raw[k][1][w], true), b0[2], b0[3]);
              pairs_of<FMT>(magic, weave<FMT>(raw[k][2][w], raw[k][3][w], false), b1[0], b1[1]);
              pairs_of<FMT>(magic, weave<FMT>(raw[k][2][w], raw[k][3][w], true), b1[2], b1[3]);
#pragma unroll
              for (int i = 0; i < NM; ++i)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                  k == 0 ? mma0(acc[i][d], pf[i][k], b0[d], b1[d]) : mma(acc[i][d], pf[i][k], b0[d], b1[d]);
            }
#pragma unroll
            for (int i = 0; i < NM; ++i)
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                float2& at = o[i][(u * UB / 4 + w) * 4 + d];
                at = ffma2(at, make_float2(alpha[i], alpha[i]),
                           fadd2(make_float2(acc[i][d][0], acc[i][d][1]), make_float2(acc[i][d][2], acc[i][d][3])));
              }
          }
        }
        __syncwarp();  // the stage and the scales may be written again
      }

      // ---- the next item's first chunk starts on its way
      const int64_t end = item.begin + item.chunks + kItemUnits;
      const bool last = end + kItemUnits >= stop;
      Item next = item;
      if (!last) {
        if (item.hs + 1 < HS) {
          ++next.hs;
        } else {
          next.hs = 0;
          int t = item.t0 + item.n;
          while (!item_at<CT>(a, t, next) && t < a.T - 1) ++t;  // (the token behind an item begins one)
        }
        next.begin = end;
        stretch(next, c0, c1);
        src = source_of(next);
        if (c0 < c1) hidden_next = fetch(src, c0, pages_of(src, c0));
        pages = pages_of(src, c0 + 1);
      }

      // ---- results, or a part to be joined: the warp's last one into its stages, which nothing comes into any
      // more, one before into the workspace
      auto give = [&](auto put_sums, auto put_row, bool divide) {
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          const float back = __uint_as_float((unit[i] - kWeightBits) << 23), z = quad_sum(l[i]);
          const float inv = !divide ? back * kPartScale : z == 0.0f ? 0.0f : back / z;  // no keys: zeros
          int t, head;
          const bool live = row_of(a, item.t0, item.n, item.hs, 8 * i + g, t, head);
          const int64_t row = live ? t * a.ld_dst + static_cast<int64_t>(head) * D : -1;
#pragma unroll
          for (int u = 0; u < UC; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int n = 0; n < UB; n += 4) {
                const float2* x = &o[i][u * UB + n];
                const float4 v = e == 0 ? make_float4(x[0].x * inv, x[1].x * inv, x[2].x * inv, x[3].x * inv)
                                        : make_float4(x[0].y * inv, x[1].y * inv, x[2].y * inv, x[3].y * inv);
                put_sums((((i * UC + u) * 2 + e) * (UB / 4) + n / 4) * 128 + lane * 4, row,
                         (value_unit<DC>(2 * c4 + e) + 8 * u) * UB + n, v);
              }
          if (c4 == 0) put_row(8 * i + g, row >= 0, t, head, m[i], z);
        }
      };
      if (start > item.begin + kItemUnits || end > stop) {
        const int slot = start >= item.begin ? 0 : 1;
        auto put_row = [&](int r, bool, int, int, float top, float z) {
          part_rows[warp][slot][r] = make_float2(top, z);
        };
        if (last) {
          float* part = reinterpret_cast<float*>(ring + slot * 2 * S::kStage);
          give([&](int at, int64_t, int, float4 v) { *reinterpret_cast<float4*>(part + at) = v; }, put_row, false);
        } else {
          give([&](int at, int64_t, int, float4 v) { *reinterpret_cast<float4*>(warp_part + at) = v; }, put_row, false);
          kept = true;
        }
        if (lane == 0) spans[warp][slot] = span_of(item);
      } else {
        give([&](int, int64_t row, int d, float4 v) {
               if (row >= 0 && d < D) write_out(a, row + d, v);
             },
             [&](int, bool live, int t, int head, float top, float z) {
               if (live && a.lse)
                 a.lse[static_cast<int64_t>(t) * a.q_heads + head] = z == 0.0f ? -INFINITY : (top + log2f(z)) * 0.693147181f;
             },
             true);
      }
      if (last) break;
      item = next;
    }
    if (kept) {  // back from the workspace: each lane what it wrote
      float4 v[S::kSlices];
#pragma unroll
      for (int k = 0; k < S::kSlices; ++k) v[k] = *reinterpret_cast<const float4*>(warp_part + k * 128 + lane * 4);
#pragma unroll
      for (int k = 0; k < S::kSlices; ++k) *reinterpret_cast<float4*>(ring + k * 512 + lane * 16) = v[k];
    }
  }

  // ---- the CTA's parts together: neighbours of one item, a warp a slice of them.  Lane k looks at place k.
  __syncthreads();
  AttSpan mine = {};
  if (lane < 2 * W) mine = spans[lane / 2][lane % 2];
  const uint32_t there = __ballot_sync(0xffffffffu, mine.end != 0);
  const uint32_t below = there & ((1u << lane) - 1);
  const int64_t before = __shfl_sync(0xffffffffu, mine.begin, below ? 31 - __clz(below) : 0);
  uint32_t firsts = __ballot_sync(0xffffffffu, mine.end != 0 && (below == 0 || before != mine.begin));
  int task = 0;
  for (; firsts; firsts &= firsts - 1) {
    const int e = __ffs(firsts) - 1;
    const uint32_t behind = firsts & (firsts - 1);
    const uint32_t members = there & ~((1u << e) - 1) & (behind ? (behind & -behind) - 1 : 0xffffffffu);
    const AttSpan s = spans[e / 2][e % 2];
    const bool done = s.begin + kItemUnits >= cta_start && s.end <= cta_start + cta_units;
    float* out = cta_parts + (s.begin <= cta_start ? 0 : S::kPart);
    for (int k = 0; k < S::kSlices; ++k) {
      if (task++ % W != warp) continue;
      const int r = 8 * (k / (S::kSlices / NM)) + g;
      float top = kNoMax, z = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (uint32_t left = members; left; left &= left - 1) {
        const int p = __ffs(left) - 1;
        const float2 ml = part_rows[p / 2][p % 2][r];
        join_part(ml.x, ml.y, *reinterpret_cast<const float4*>(smem + p * 2 * S::kStage + k * 512 + lane * 16), top, z, v);
      }
      if (done) {
        join_out<DC, NM>(a, s, k, lane, top, z, v);
      } else {
        *reinterpret_cast<float4*>(out + k * 128 + lane * 4) = v;
        if (c4 == 0 && k % (S::kSlices / NM) == 0) {
          out[S::kRows * DC + r] = top;
          out[S::kRows * DC + S::kRows + r] = z;
        }
      }
    }
  }
}

// An item that reaches over CTAs' stretches: the first CTA's part, and n - 1 others' two parts apart.
struct Split {
  const float* first;
  const float* rest;
  int n;
};

// Whether CTA i's record is of an item whose first chunk is in the stretch before.
__device__ __forceinline__ bool split_at(const AttendArgs& a, const AttHeader& h, int64_t i, AttSpan& s) {
  if (i >= a.ctas) return false;
  s = reinterpret_cast<const AttSpan*>(reinterpret_cast<const uint8_t*>(a.workspace) + kAttHead)[i];
  return i < h.ctas && share(h, i) > s.begin + kItemUnits && share(h, i - 1) <= s.begin + kItemUnits;
}

// Its parts, by a whole warp.
template <int DC, int NM>
__device__ __forceinline__ Split split_of(const AttendArgs& a, const AttHeader& h, int64_t i, const AttSpan& s, int lane) {
  constexpr int64_t kPart = AttShape<DC, NM>::kPart;
  Split p;
  for (int64_t k = i + 1;; k += 32) {  // the first CTA that begins behind the item
    const uint32_t past = __ballot_sync(0xffffffffu, k + lane >= h.ctas || share(h, k + lane) >= s.end);
    if (past) {
      p.n = static_cast<int>(k - i) + __ffs(past);
      break;
    }
  }
  const float* parts = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(a.workspace) + att_parts_at(a.ctas));
  // CTA i - 1 holds its part second, unless its stretch begins with the item
  p.first = parts + ((i - 1) * 2 + (share(h, i - 1) < s.begin ? 1 : 0)) * kPart;
  p.rest = parts + (i - 1) * 2 * kPart;
  return p;
}

// Parts from, from + STEP, .. of a slice's place, B on their way together.
template <int DC, int NM, int STEP, int B>
__device__ __forceinline__ void join_parts(const Split& p, int slice, int lane, int from, float& top, float& z, float4& v) {
  using S = AttShape<DC, NM>;
  const int r = S::kRows * DC + 8 * (slice / (S::kSlices / NM)) + (lane >> 2), at = slice * 128 + lane * 4;
  top = kNoMax;
  z = 0.0f;
  v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j0 = from; j0 < p.n; j0 += STEP * B) {
    float m[B], l[B];
    float4 x[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int j = j0 + b * STEP;
      const float* part = j == 0 ? p.first : p.rest + j * (2 * S::kPart);
      m[b] = kNoMax;
      l[b] = 0.0f;
      x[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (j < p.n) {
        m[b] = part[r];
        l[b] = part[r + S::kRows];
        x[b] = *reinterpret_cast<const float4*>(part + at);
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) join_part(m[b], l[b], x[b], top, z, v);
  }
}

// Many items, few parts each: CTA (i, y) looks at record i + 1; a warp a slice.
constexpr int kJoinWarps = 4;
template <int DC, int NM>
__global__ void __launch_bounds__(32 * kJoinWarps) attend_join_kernel(const __grid_constant__ AttendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = static_cast<int64_t>(blockIdx.x) + 1;
  const AttHeader h = *reinterpret_cast<const AttHeader*>(a.workspace);
  AttSpan s;
  if (!split_at(a, h, i, s)) return;
  const int lane = threadIdx.x & 31;
  const Split p = split_of<DC, NM>(a, h, i, s, lane);
  for (int k = threadIdx.x / 32 + kJoinWarps * blockIdx.y; k < AttShape<DC, NM>::kSlices; k += kJoinWarps * gridDim.y) {
    float top, z;
    float4 v;
    join_parts<DC, NM, 1, 4>(p, k, lane, 0, top, z, v);
    join_out<DC, NM>(a, s, k, lane, top, z, v);
  }
}

// Few items, many parts: CTA (i, slice) looks at kFewRecords; its warps share the parts.  (A CTA to every record and
// slice took 2 us to find that most have nothing to do.)  Whole calls with this kernel and with the one above: 8 items of
// 16000 keys 30 and 42 us, of 1000 20 and 21; 24 44 and 48, 24 and 24; 40 59 and 59, 26 and 25; 64 77 and 77, 28 and 26.
constexpr int kFewWarps = 8, kFewRecords = 8, kFewItems = 40;
template <int DC, int NM>
__global__ void __launch_bounds__(32 * kFewWarps) attend_join_few_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ float4 sums[kFewWarps][32];
  __shared__ float2 tops[kFewWarps][32];
  pdl_wait();
  pdl_trigger();
  const AttHeader h = *reinterpret_cast<const AttHeader*>(a.workspace);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slice = blockIdx.y;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kFewRecords + 1;
  AttSpan s;
  uint32_t todo = __ballot_sync(0xffffffffu, lane < kFewRecords && split_at(a, h, i0 + lane, s));
  for (; todo; todo &= todo - 1) {
    const int64_t i = i0 + __ffs(todo) - 1;
    split_at(a, h, i, s);
    const Split p = split_of<DC, NM>(a, h, i, s, lane);
    float top, z;
    float4 v;
    join_parts<DC, NM, kFewWarps, 5>(p, slice, lane, warp, top, z, v);
    sums[warp][lane] = v;
    tops[warp][lane] = make_float2(top, z);
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 1; w < kFewWarps; ++w) join_part(tops[w][lane].x, tops[w][lane].y, sums[w][lane], top, z, v);
      join_out<DC, NM>(a, s, slice, lane, top, z, v);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host
int64_t attend_workspace_bytes(int dim, int tiles, int ctas) {
  const int dc = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  return att_parts_at(ctas) + static_cast<int64_t>(ctas) * (2 + att_warps(dc, tiles)) * 8 * tiles * (dc + 2) * 4;
}

int attend_ctas(int sms) { return 2 * sms; }

template <int DC, bool EXACT, int FMT, int NM>
static int launch_part(cudaLaunchConfig_t& cfg, const AttendArgs& a) {
  using S = AttShape<DC, NM>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(reinterpret_cast<const void*>(attend_kernel<DC, EXACT, FMT, NM>));
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
  cfg.blockDim = dim3(32 * S::kWarps);
  cfg.dynamicSmemBytes = S::kSmem;
  return cudaLaunchKernelEx(&cfg, attend_kernel<DC, EXACT, FMT, NM>, a);
}

template <int DC, int NM>
static int launch_attend_t(const AttendArgs& a, cudaStream_t st, bool pdl) {
  using S = AttShape<DC, NM>;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (a.phase == ATT_PART) {
    if (a.c.dim == DC)
      return a.c.format == 0 ? launch_part<DC, true, 0, NM>(cfg, a) : launch_part<DC, true, 1, NM>(cfg, a);
    return a.c.format == 0 ? launch_part<DC, false, 0, NM>(cfg, a) : launch_part<DC, false, 1, NM>(cfg, a);
  }
  if (static_cast<int64_t>(a.T) * a.c.heads * a.subs <= kFewItems) {
    cfg.gridDim = dim3(static_cast<unsigned>((a.ctas - 2) / kFewRecords + 1), S::kSlices);
    cfg.blockDim = dim3(32 * kFewWarps);
    return cudaLaunchKernelEx(&cfg, attend_join_few_kernel<DC, NM>, a);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(a.ctas - 1), 2);
  cfg.blockDim = dim3(32 * kJoinWarps);
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<DC, NM>, a);
}

int launch_attend(const AttendArgs& a, cudaStream_t st, bool pdl) {
  if (a.c.dim <= 64) return a.tiles == 1 ? launch_attend_t<64, 1>(a, st, pdl) : launch_attend_t<64, 2>(a, st, pdl);
  if (a.c.dim <= 128) return a.tiles == 1 ? launch_attend_t<128, 1>(a, st, pdl) : launch_attend_t<128, 2>(a, st, pdl);
  return launch_attend_t<256, 1>(a, st, pdl);
}

}  // namespace gf
