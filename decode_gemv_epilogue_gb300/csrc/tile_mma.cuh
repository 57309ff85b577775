// Tiled products of block-format weights with several columns on the tensor cores: the
// device code shared by the chosen experts' kernels and the shared projection of a wide
// batch with adapters.
//
// x is "packed" first: every 32 elements of a column become 32 pairs of f16,
//     x * 2^s = hi + lo,   hi = f16(x 2^s),   lo = f16(x 2^s - hi)
// with a power of two 2^s that puts the largest magnitude into [2^14, 2^15): hi + lo carries
// x to 2^-22 of itself (2^-39 of the largest where lo is subnormal), less than the rounding
// of a 32-bit sum.  The codes of the weights are exact in f16, the products of f16 are exact
// in the 32-bit accumulators, and the blocks' scales multiply the accumulated sum of a block
// in 32 bits: the only roundings are those of 32-bit sums.
//
// Why mma.sync and not the asynchronous matrix unit: a block format's scale belongs to 32
// weights of one row, so the accumulator of every 32 columns of K has to pass through
// registers to be scaled (folding the scale into f16 weights would round them); with
// accumulators in tensor memory that is one read-back per two instructions.
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

__device__ __forceinline__ uint32_t hadd2u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// (w & mask) | 0x64006400: two f16 of 1024 plus a code each.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t mask) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(0x64006400u));
  return d;
}

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
// The 32-bit word at a 2-byte aligned address, from the two aligned words around it (may
// read up to 3 bytes past it; stages keep slack).
__device__ __forceinline__ uint32_t lds32_half_aligned(uint32_t a) {
  const uint32_t b = a & ~3u;
  return __funnelshift_r(lds32(b), lds32(b + 4u), (a & 3u) * 8u);
}

// ------------------------------------------------------------------ packing x
// Packed columns lie in the order in which the matrix instruction takes them.  Eight columns
// form a column tile, and for every 32 elements a column tile has one record:
//   [step s of 2][column of cp][thread t of 4] 16 bytes {hi, hi, hi, hi, lo, lo, lo, lo},
//   then per column {2^-s, the sum of x 2^s over the 32 elements};
// cp = min(8, columns of the call) columns are stored, so that a single column does not move
// eight.  A warp's 16-byte reads of a step are then consecutive, and the records of a K chunk
// are one piece of memory for one bulk copy.  Which four elements (s, t) holds is the
// weights' choice: 16 s + 4 t + .. in the order 0, 2, 1, 3 for the nibble formats (two masks
// take a code word apart in that order), 16 s + 4 t + 0..3 for Q8_0, and 8 t + 4 s + 0..3
// for F16 (a thread then reads 16 bytes of a row at once).
enum { ORDER_NIBBLE = 0, ORDER_BYTE = 1, ORDER_F16 = 2 };
__host__ __device__ constexpr int pack_order(int wt) {
  return wt == WT_F16 ? ORDER_F16 : wt == WT_Q8_0 ? ORDER_BYTE : ORDER_NIBBLE;
}
__host__ __device__ constexpr int record_bytes(int cp) { return cp * 128 + (cp * 8 + 15) / 16 * 16; }
// Byte offset in a record of the four elements 4q .. 4q + 3 of column c.
__device__ __forceinline__ uint32_t record_offset(uint32_t q, uint32_t c, uint32_t cp, int order) {
  const uint32_t s = order == ORDER_F16 ? (q & 1u) : (q >> 2), t = order == ORDER_F16 ? (q >> 1) : (q & 3u);
  return (s * cp + c) * 64u + t * 16u;
}

// 2^s for the largest magnitude m (finite), s in [-112, 126]; 1 for m = 0.
__device__ __forceinline__ float pack_scale(float m) {
  const int e = static_cast<int>((__float_as_uint(m) >> 23) & 0xFFu);  // m in [2^(e-127), 2^(e-126))
  const int s = m == 0.0f ? 0 : max(-126, min(126, 14 + 127 - e));
  return __uint_as_float(static_cast<uint32_t>(s + 127) << 23);
}
// The inverse of a power of two in [2^-126, 2^126].
__device__ __forceinline__ float pow2_inverse(float p) {
  return __uint_as_float((254u << 23) - __float_as_uint(p));
}

struct HiLo {
  __half hi, lo;
};
// x must be scaled already.  An infinite or NaN x stays so in hi, with lo = 0.
__device__ __forceinline__ HiLo split_hi_lo(float v) {
  HiLo r;
  r.hi = __float2half_rn(v);
  const float rest = v - __half2float(r.hi);
  r.lo = __float2half_rn(fabsf(v) <= 65504.0f ? rest : 0.0f);
  return r;
}

__device__ __forceinline__ uint32_t half_pair(__half a, __half b) {
  return static_cast<uint32_t>(__half_as_ushort(a)) | (static_cast<uint32_t>(__half_as_ushort(b)) << 16);
}

// Four consecutive scaled elements as the 16 bytes of a packed group.
__device__ __forceinline__ uint4 pack_group(float4 v, bool swapped) {
  const HiLo a = split_hi_lo(v.x), b = split_hi_lo(v.y), c = split_hi_lo(v.z), d = split_hi_lo(v.w);
  return swapped ? make_uint4(half_pair(a.hi, c.hi), half_pair(b.hi, d.hi), half_pair(a.lo, c.lo), half_pair(b.lo, d.lo))
                 : make_uint4(half_pair(a.hi, b.hi), half_pair(c.hi, d.hi), half_pair(a.lo, b.lo), half_pair(c.lo, d.lo));
}
__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? a : 0.0f;  // Inf and NaN do not set the scale
}

// ------------------------------------------------------------------ A fragments
// One 32-element block of rows g and g + 8 of a 16-row tile as the A operands of two
// m16n8k16 steps: a[s] = {row g k-slots 2t, 2t+1; row g+8 the same; row g slots 2t+8, 2t+9;
// row g+8 the same}, thread (g, t) = (lane / 4, lane % 4).  Which element sits in which
// k-slot is free as long as the packed x has the same one (see pack_order).  d: the rows'
// block scales (unused for F16).
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

template <int WT>
__device__ __forceinline__ void load_block_row(uint32_t row, uint32_t blk, uint32_t t, uint32_t (&a0)[2],
                                               uint32_t (&a1)[2], float& d) {
  if constexpr (WT == WT_F16) {  // the thread's 16 bytes, swizzled: see tile_kernel
    const uint4 u = lds128(row);
    a0[0] = u.x; a0[1] = u.y;
    a1[0] = u.z; a1[1] = u.w;
    d = 1.0f;
  } else if constexpr (WT == WT_Q8_0) {
    const uint32_t p = row + blk * 34u;
    d = h2f(lds16(p));
    const uint32_t u = lds32_half_aligned(p + 2u + 4u * t) ^ 0x80808080u;
    const uint32_t v = lds32_half_aligned(p + 18u + 4u * t) ^ 0x80808080u;
    constexpr uint32_t kBias = 0xE480E480u;  // -(1024 + 128) twice
    a0[0] = hadd2u(__byte_perm(u, 0x64646464u, 0x4140), kBias);
    a0[1] = hadd2u(__byte_perm(u, 0x64646464u, 0x4342), kBias);
    a1[0] = hadd2u(__byte_perm(v, 0x64646464u, 0x4140), kBias);
    a1[1] = hadd2u(__byte_perm(v, 0x64646464u, 0x4342), kBias);
  } else if constexpr (WT == WT_Q4_K) {  // the scale and min come apart elsewhere
    const uint32_t p = row + (blk >> 3) * kQ4kBytes + 16u + ((blk >> 1) & 3u) * 32u + 4u * t;
    const uint32_t sh = 4u * (blk & 1u), w = lds32(p) >> sh, v = lds32(p + 16u) >> sh;
    constexpr uint32_t kLow = 0xE400E400u;              // -1024
    a0[0] = hadd2u(code_pair(w, 0x000F000Fu), kLow);
    a0[1] = hadd2u(code_pair(w >> 8, 0x000F000Fu), kLow);
    a1[0] = hadd2u(code_pair(v, 0x000F000Fu), kLow);
    a1[1] = hadd2u(code_pair(v >> 8, 0x000F000Fu), kLow);
  } else {  // Q4_0
    const uint32_t p = row + blk * 18u;
    d = h2f(lds16(p));
    const uint32_t w = lds32_half_aligned(p + 2u + 4u * t), w8 = w >> 8;
    constexpr uint32_t kLow = 0xE408E408u;              // -(1024 + 8)
    constexpr uint32_t kSixteenth = 0x2C002C00u;        // 1/16
    constexpr uint32_t kHigh = 0xD480D480u;             // -(64 + 8)
    a0[0] = hadd2u(code_pair(w, 0x000F000Fu), kLow);    // elements 4t, 4t+2
    a0[1] = hadd2u(code_pair(w8, 0x000F000Fu), kLow);   // 4t+1, 4t+3
    a1[0] = hfma2u(code_pair(w, 0x00F000F0u), kSixteenth, kHigh);
    a1[1] = hfma2u(code_pair(w8, 0x00F000F0u), kSixteenth, kHigh);
  }
}

// ------------------------------------------------------------------ the tiled kernel
// A work item is (column group, row tile): up to 8 NT columns that share one matrix, and
// 64 rows of it (gated: 32 gate rows and the same up rows).  Warp 0 streams the item's K
// chunks of 256 -- the rows' weights by tensor-map copies of 32 rows, the columns' records
// by one bulk copy per column tile -- through a ring of shared-memory stages.  The eight
// consumer warps share the K axis: a warp takes one 32-element block of the chunk for all 64
// rows (four 16-row matrix tiles), so that a packed x fragment, once loaded, serves four
// matrix tiles.  At the end of an item the warps' accumulators are added through shared
// memory in warp order (deterministic) and the tail is applied.
//
// (A first version copied every row of a chunk by its own bulk copy: each took about 90
// cycles of an SM's copy engine whatever its size, three to ten times the time of the bytes.)
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
constexpr int kTileK = 256;
constexpr int kTileWarps = 8;           // consumer warps, sharing K
constexpr int kTileThreads = 32 * (1 + kTileWarps);
constexpr int kTileMaxStages = 8;
constexpr int kTileBarBytes = 256;
constexpr int kRedPitch = kTileRows + 4;
constexpr int kTileRedBytes = kTileWarps * 8 * kRedPitch * 4;  // the warps' sums of eight columns
enum { TILE_GLU = 0, TILE_DOWN = 1 };

template <int WT>
__host__ __device__ constexpr int tile_seg() {  // bytes of a row and chunk
  return WT == WT_F16 ? 2 * kTileK : WT == WT_Q8_0 ? kTileK / 32 * 34 : 144;
}
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
  return WT == WT_F16 ? kTileRows * kTileK * 2 : 2 * period * tile_part<WT>(period);
}
template <int WT>
__host__ __device__ constexpr int tile_stage_bytes(int period, int nt, int cp) {
  return (tile_weight_bytes<WT>(period) + 16 + nt * (kTileK / 32) * record_bytes(cp) + 1023) / 1024 * 1024;
}

struct TileArgs {
  int rows, K, row_bytes;   // rows of one matrix (outputs), columns
  int period;
  const int4* groups;       // {matrix, first entry, columns, first column tile}
  const int32_t* n_groups;
  const int32_t* slots;     // slot of each entry
  const uint8_t* records;   // [column tile][K / 32] records of x
  int cp;
  int NS;
  unsigned* err;
  // tails
  uint8_t* out_records;     // gated: records of the next product's x
  int out_order;
  const float* weights;     // down: factor of a slot
  float* y;                 // down: [slot][rows]
};

template <int WT, int MODE, int NT>
__global__ void __launch_bounds__(kTileThreads, NT <= 2 ? 2 : 1)
    tile_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                const __grid_constant__ TileArgs a) {
  constexpr bool kMeta = MODE == TILE_DOWN || WT == WT_Q4_K;  // per-block scales or sums are read in the loop
  constexpr int kOutRows = MODE == TILE_GLU ? 32 : kTileRows;
  constexpr int kBlocks = kTileK / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem), full0 = sbase, empty0 = sbase + 8u * kTileMaxStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kTileBarBytes - 8);
  float* red = reinterpret_cast<float*>(smem + kTileBarBytes);
  const uint32_t ring = (sbase + kTileBarBytes + kTileRedBytes + 1023u) & ~1023u;
  const uint32_t rec = static_cast<uint32_t>(record_bytes(a.cp));
  const uint32_t stage_bytes = tile_stage_bytes<WT>(a.period, NT, a.cp);
  const uint32_t xoff = tile_weight_bytes<WT>(a.period) + 16;  // slack: words are read up to 3 bytes past a row
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < a.NS; ++i) {
      mbar_init(full0 + 8u * i, 1);
      mbar_init(empty0 + 8u * i, kTileWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&map0);
    if (MODE == TILE_GLU) prefetch_tmap(&map1);
  }
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  const int tiles = (a.rows + kOutRows - 1) / kOutRows;
  const int64_t items = static_cast<int64_t>(*a.n_groups) * tiles;
  const int64_t lo = items * blockIdx.x / gridDim.x, hi = items * (blockIdx.x + 1) / gridDim.x;
  const int n_kc = (a.K + kTileK - 1) / kTileK, nblk = a.K / 32;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int slot = 0, issued = 0;
      uint32_t phase = 1u;
      bool ok = true;
      const uint32_t box = 32u / a.period * static_cast<uint32_t>(tile_pitch<WT>(a.period));
      for (int64_t it = lo; it < hi && ok; ++it) {
        const int gi = static_cast<int>(it / tiles);
        const int row0 = static_cast<int>(it - static_cast<int64_t>(gi) * tiles) * kOutRows;
        const int4 g = a.groups[gi];
        const int halves = MODE == TILE_GLU || row0 + 32 < a.rows ? 2 : 1;
        const int nt = (g.z + 7) / 8;
        const int64_t first = static_cast<int64_t>(g.x) * a.rows + row0;
        for (int kc = 0; kc < n_kc; ++kc) {
          if (issued >= a.NS && !mbar_wait_or_abort(empty0 + 8u * slot, phase, abort_flag, a.err)) {
            ok = false;
            break;
          }
          const uint32_t st = ring + static_cast<uint32_t>(slot) * stage_bytes, full = full0 + 8u * slot;
          const uint32_t xlen = static_cast<uint32_t>(min(kBlocks, nblk - kc * kBlocks)) * rec;
          const uint32_t wlen = WT == WT_F16 ? 32u * kTileK * 2u : box * a.period;
          mbar_arrive_expect_tx(full, halves * wlen + nt * xlen);
          for (int h = 0; h < halves; ++h) {
            const CUtensorMap* map = MODE == TILE_GLU && h ? &map1 : &map0;
            const int64_t row = first + (MODE == TILE_GLU ? 0 : 32 * h);
            if constexpr (WT == WT_F16) {
              for (int q = 0; q < 4; ++q)
                tma_load_2d(st + static_cast<uint32_t>((2 * q + h) * 4096), map, kc * kTileK + 64 * q,
                            static_cast<int>(row), full);
            } else {
              for (int i = 0; i < a.period; ++i)
                tma_load_2d(st + static_cast<uint32_t>((h * a.period + i) * tile_part<WT>(a.period)), map,
                            ((i * a.row_bytes + kc * tile_seg<WT>()) & ~15) / 2, static_cast<int>(row / a.period), full);
            }
          }
          for (int n = 0; n < nt; ++n)
            bulk_g2s(st + xoff + static_cast<uint32_t>(n) * kBlocks * rec,
                     a.records + (static_cast<int64_t>(g.w + n) * nblk + kc * kBlocks) * rec, xlen, full);
          ++issued;
          if (++slot == a.NS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      // Drain after an abort: every copy this thread issued lands before the CTA leaves.
      if (!ok)
        for (int i = max(0, issued - a.NS); i < issued; ++i)
          (void)mbar_wait(full0 + 8u * (i % a.NS), static_cast<uint32_t>((i / a.NS) & 1));
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int wk = warp - 1;
    const uint32_t g4 = static_cast<uint32_t>(lane) >> 2, t4 = static_cast<uint32_t>(lane) & 3u;
    // the row of eight that this lane takes
    const uint32_t row8 = WT == WT_F16 ? ((g4 >> 1) | ((g4 & 1u) << 2)) : g4;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    // stage address of rows row8 (+ 8) of a 16-row tile, and the distances of rows 8 and 16
    // apart and of the halves
    const uint32_t P = tile_pitch<WT>(a.period), per = static_cast<uint32_t>(a.period);
    uint32_t rowbase, step8, step16, half;
    if constexpr (WT == WT_F16) {
      rowbase = row8 * 128u;
      step8 = 1024u;
      step16 = 2048u;
      half = 4096u;
    } else {
      const uint32_t res = row8 % per;
      rowbase = res * tile_part<WT>(a.period) + row8 / per * P + ((res * static_cast<uint32_t>(a.row_bytes)) & 15u);
      step8 = 8u / per * P;
      step16 = 16u / per * P;
      half = per * tile_part<WT>(a.period);
    }
    const uint32_t cp = static_cast<uint32_t>(a.cp);
    const uint32_t xlane = min(g4, cp - 1u) * 64u + t4 * 16u;  // lanes past the columns read the last one
    const uint32_t m0 = cp * 128u + min(2u * t4, cp - 1u) * 8u, m1 = cp * 128u + min(2u * t4 + 1u, cp - 1u) * 8u;
    auto group_bar = [&]() { named_bar_sync(1u, 32u * kTileWarps); };
    for (int64_t it = lo; it < hi; ++it) {
      const int gi = static_cast<int>(it / tiles);
      const int row0 = static_cast<int>(it - static_cast<int64_t>(gi) * tiles) * kOutRows;
      const int4 g = a.groups[gi];
      const int ncol = g.z;
      float acc[4][NT][4];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
      for (int kc = 0; kc < n_kc; ++kc) {
        ok = ok && mbar_wait_or_abort(full0 + 8u * slot, phase, abort_flag, a.err);
        const uint32_t st = ring + static_cast<uint32_t>(slot) * stage_bytes;
        const uint32_t blk = static_cast<uint32_t>(wk);  // this warp's block of the chunk
        if (ok && kc * kBlocks + wk < nblk) {
          uint4 b[NT][2];
          float2 meta[NT][2];  // of columns 2t and 2t + 1 of each column tile
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (8 * n < ncol) {
              const uint32_t xa = st + xoff + (static_cast<uint32_t>(n) * kBlocks + blk) * rec;
              b[n][0] = lds128(xa + xlane);
              b[n][1] = lds128(xa + xlane + cp * 64u);
              if constexpr (kMeta) {
                const uint2 u = lds64(xa + m0), v = lds64(xa + m1);
                meta[n][0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
                meta[n][1] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
              }
            }
          }
          // Q4_K: taking a row's 6-bit scale and min apart costs as much as its codes; the four
          // lanes of a row would all do it, so lane t does it for matrix tile t only
          float qd[2], qm[2];
          if constexpr (WT == WT_Q4_K) {
            const uint32_t mine = st + rowbase + (t4 & 1u) * step16 + (t4 >> 1) * half;
            q4k_scale_of(lds128(mine), blk, qd[0], qm[0]);
            q4k_scale_of(lds128(mine + step8), blk, qd[1], qm[1]);
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t a0[2][2], a1[2][2];
            float d[2], dm[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t row = st + rowbase + (m & 1) * step16 + (m >> 1) * half + h * step8;
              if constexpr (WT == WT_F16)  // box blk / 2, 16-byte word 4 (blk % 2) + t of the 128, swizzled by the row
                row += (blk >> 1) * 8192u + ((((blk & 1u) * 4u + t4) ^ row8) << 4);
              load_block_row<WT>(row, blk, t4, a0[h], a1[h], d[h]);
              dm[h] = 0.0f;
              if constexpr (WT == WT_Q4_K) {
                d[h] = __shfl_sync(0xffffffffu, qd[h], m, 4);
                dm[h] = __shfl_sync(0xffffffffu, qm[h], m, 4);
              }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (8 * n < ncol) {
                if constexpr (WT == WT_F16 && MODE != TILE_DOWN) {  // one scale per column: no block scale at all
                  float (&s)[4] = acc[m][n];
                  mma_f16(s, a0[0][0], a0[1][0], a0[0][1], a0[1][1], b[n][0].x, b[n][0].y);
                  mma_f16(s, a1[0][0], a1[1][0], a1[0][1], a1[1][1], b[n][1].x, b[n][1].y);
                  mma_f16(s, a0[0][0], a0[1][0], a0[0][1], a0[1][1], b[n][0].z, b[n][0].w);
                  mma_f16(s, a1[0][0], a1[1][0], a1[0][1], a1[1][1], b[n][1].z, b[n][1].w);
                } else {
                  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma_f16(s, a0[0][0], a0[1][0], a0[0][1], a0[1][1], b[n][0].x, b[n][0].y);
                  mma_f16(s, a1[0][0], a1[1][0], a1[0][1], a1[1][1], b[n][1].x, b[n][1].y);
                  mma_f16(s, a0[0][0], a0[1][0], a0[0][1], a0[1][1], b[n][0].z, b[n][0].w);
                  mma_f16(s, a1[0][0], a1[1][0], a1[0][1], a1[1][1], b[n][1].z, b[n][1].w);
                  // i: row row8 (0, 1) or row8 + 8 (2, 3), column 2t + (i & 1)
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int h = i >> 1, c = i & 1;
                    if constexpr (MODE == TILE_DOWN) {
                      float v = WT == WT_F16 ? s[i] : d[h] * s[i];
                      if constexpr (WT == WT_Q4_K) v = fmaf(-dm[h], meta[n][c].y, v);
                      acc[m][n][i] = fmaf(meta[n][c].x, v, acc[m][n][i]);
                    } else {
                      acc[m][n][i] = fmaf(d[h], s[i], acc[m][n][i]);
                      if constexpr (WT == WT_Q4_K) acc[m][n][i] = fmaf(-dm[h], meta[n][c].y, acc[m][n][i]);
                    }
                  }
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + 8u * slot);
        if (++slot == a.NS) {
          slot = 0;
          phase ^= 1u;
        }
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
            red[(wk * 8 + 2 * t4 + (i & 1)) * kRedPitch + 16 * m + row8 + 8 * (i >> 1)] = acc[m][n][i];
        group_bar();
        const int c = 8 * n + wk;
        if (c < ncol && ok && !*abort_flag) {
          float v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kTileWarps; ++w) s += red[(w * 8 + wk) * kRedPitch + 32 * h + lane];
            v[h] = s;
          }
          if constexpr (MODE == TILE_GLU) {
            // 32 output rows of the gated product (rows are a multiple of 32): one record's column
            const int64_t tile = g.w + n;
            const float sx =
                *reinterpret_cast<const float*>(a.records + tile * nblk * rec + cp * 128u + static_cast<uint32_t>(wk) * 8u);
            const float h = tail_silu(v[0] * sx) * (v[1] * sx);
            const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(finite_abs(h))));
            const float sc = pack_scale(m), hs = h * sc;
            float sum = hs;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const HiLo p = split_hi_lo(hs);
            uint8_t* q = a.out_records + (tile * (a.rows / 32) + row0 / 32) * rec;
            const uint32_t i = static_cast<uint32_t>(lane) & 3u;
            const uint32_t at = record_offset(static_cast<uint32_t>(lane) >> 2, static_cast<uint32_t>(wk), cp, a.out_order) +
                                2u * (a.out_order == ORDER_NIBBLE ? ((i & 1u) << 1) | (i >> 1) : i);
            *reinterpret_cast<__half*>(q + at) = p.hi;
            *reinterpret_cast<__half*>(q + at + 8) = p.lo;
            if (lane == 0)
              *reinterpret_cast<float2*>(q + cp * 128u + static_cast<uint32_t>(wk) * 8u) = make_float2(pow2_inverse(sc), sum);
          } else {
            const int sl = a.slots[g.y + c];
            const float w = a.weights[sl];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = row0 + 32 * h + lane;
              if (r < a.rows) a.y[static_cast<int64_t>(sl) * a.rows + r] = w * v[h];
            }
          }
        }
      }
    }
  }
  __syncthreads();
}

}  // namespace gf
