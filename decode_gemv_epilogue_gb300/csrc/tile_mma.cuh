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

#include "gf_device.cuh"
#include "gf_internal.h"

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
// A packed column: per 32 elements 128 bytes, per four elements 4q .. 4q+3 the 16 bytes
// {hi, hi, hi, hi, lo, lo, lo, lo}.  For the nibble formats the four are in the order
// 0, 2, 1, 3, the order in which two masks take the nibbles of a code word apart.
// Beside it per 32 elements {2^-s, the sum of x 2^s}.
__host__ __device__ constexpr bool pack_swapped(int wt) { return wt == WT_Q4_0 || wt == WT_Q4_K; }

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
// Byte offset in a packed 32-element block of the hi half of element i (lo: 8 further).
__device__ __forceinline__ uint32_t packed_offset(uint32_t i, bool swapped) {
  const uint32_t p = i & 3u, slot = swapped ? ((p & 1u) << 1) | (p >> 1) : p;
  return (i >> 2) * 16u + slot * 2u;
}

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? a : 0.0f;  // Inf and NaN do not set the scale
}

// ------------------------------------------------------------------ A fragments
// One 32-element block of rows g and g + 8 of a 16-row tile as the A operands of two
// m16n8k16 steps: a[s] = {row g k-slots 2t, 2t+1; row g+8 the same; row g slots 2t+8, 2t+9;
// row g+8 the same}, thread (g, t) = (lane / 4, lane % 4).  Which element sits in which
// k-slot is free as long as the packed x has the same one; step s, thread t holds elements
// 16 s + 4 t .. + 3 of the block.  d: the rows' block scales (unused for F16).
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
  if constexpr (WT == WT_F16) {
    const uint2 u = lds64(row + blk * 64u + t * 8u), v = lds64(row + blk * 64u + 32u + t * 8u);
    a0[0] = u.x; a0[1] = u.y;
    a1[0] = v.x; a1[1] = v.y;
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
// 64 WR rows of it (gated: 32 WR gate rows and the same up rows).  Warp 0 streams the
// item's K chunks -- the rows' weights, one bulk copy per row, and the columns' packed x --
// through a ring of shared-memory stages.  8 WR consumer warps: row group wr takes 64 rows
// (four 16-row matrix tiles), and the 8 warps of a row group share the K axis block by
// block, so that each packed x fragment that a warp loads serves four matrix tiles.  At the
// end of an item the warps' accumulators are added through shared memory in warp order
// (deterministic) and the tail is applied.
//
// Rows lie in a stage `pitch` bytes apart, an odd multiple of 16 (of 32 for F16): the eight
// rows that a warp reads together then fall on distinct banks.  Bulk copies want 16-byte
// boundaries: a row that starts or ends off one is copied with the bytes around it, cut at
// the end of the matrices (the last bytes are then copied by hand), and read from the
// offset.
//
// Every wait is bounded; a timeout sets the device error word, and the kernel returns after
// draining its own copies.
constexpr int kTileRows = 64;           // rows of a row group
constexpr int kTileWarpsK = 8;          // warps sharing K in a row group
constexpr int kTileMaxStages = 8;
constexpr int kRedPitch = kTileRows + 4;
enum { TILE_GLU = 0, TILE_DOWN = 1, TILE_LIN = 2 };

// K elements of a stage: two 32-element blocks per warp for the 4-bit formats, one for the
// others and for wide groups, whose packed x fills the stage.
template <int WT, int NT>
__host__ __device__ constexpr int tile_kc() {
  return ((WT == WT_Q4_0 || WT == WT_Q4_K) && NT <= 2) ? 512 : 256;
}
template <int WT>
__host__ __device__ constexpr int tile_seg(int k) {
  return WT == WT_F16 ? 2 * k : WT == WT_Q8_0 ? (k / 32) * 34 : WT == WT_Q4_0 ? (k / 32) * 18 : (k / 256) * 144;
}
// Bytes between the rows of a stage: room for the chunk and up to 30 bytes around it, and
// an odd multiple of 16 (32 for F16, whose rows are always whole 16-byte words).
template <int WT, int NT>
__host__ __device__ constexpr int tile_pitch() {
  constexpr int seg = tile_seg<WT>(tile_kc<WT, NT>());
  if constexpr (WT == WT_F16) return seg + 32;
  constexpr int need = (seg + (WT == WT_Q4_K ? 0 : 30) + 15) / 16;
  return 16 * (need % 2 ? need : need + 1);
}
constexpr int kXPitchPad = 64;     // packed columns half a bank row apart
constexpr int kMetaPitchPad = 16;
template <int WT, int NT>
__host__ __device__ constexpr int tile_xpitch() { return tile_kc<WT, NT>() * 4 + kXPitchPad; }
template <int WT, int NT>
__host__ __device__ constexpr int tile_mpitch() { return tile_kc<WT, NT>() / 4 + kMetaPitchPad; }
template <int WT, int NT>
__host__ __device__ constexpr int tile_stage_bytes(int wr, int cols) {
  return (kTileRows * wr * tile_pitch<WT, NT>() + cols * (tile_xpitch<WT, NT>() + tile_mpitch<WT, NT>()) + 16 + 127) / 128 * 128;
}
constexpr int kTileBarBytes = 256;
// The warps' sums of eight columns at a time.
__host__ __device__ constexpr int tile_red_bytes(int wr) { return wr * kTileWarpsK * 8 * kRedPitch * 4; }

struct TileArgs {
  const uint8_t* W;       // matrices one after another
  const uint8_t* W2;      // gated: the up matrices
  int64_t total_bytes;    // of all matrices of W (of W2 the same)
  int rows, K, row_bytes; // rows of one matrix (outputs), columns
  const int4* groups;     // {matrix, first slot entry, columns, 0}
  const int32_t* n_groups;
  const int32_t* slots;   // slot of each entry
  int slot_div;           // packed column of a slot: slot / slot_div
  const uint8_t* xpack;
  const float2* xmeta;
  int cols;               // columns a stage has room for (<= 8 NT)
  int NS;
  unsigned* err;
  // tails
  uint8_t* hpack;         // gated: packed output columns, by slot
  float2* hmeta;
  int h_swapped;
  const float* weights;   // down: factor of a slot
  float* y;               // down: [slot][rows]
};

struct TileRing {
  uint32_t base, full0, empty0;
};

// The rows and columns of an item.
struct TileItem {
  int4 g;
  int row0;      // first output row
};

template <int WT, int MODE, int NT, int WR>
__global__ void __launch_bounds__(32 * (1 + kTileWarpsK * WR), (WR == 1 && NT <= 2) ? 2 : 1)
    tile_kernel(const __grid_constant__ TileArgs a) {
  constexpr int KC = tile_kc<WT, NT>(), P = tile_pitch<WT, NT>(), XP = tile_xpitch<WT, NT>(), MP = tile_mpitch<WT, NT>();
  constexpr bool kMeta = MODE == TILE_DOWN || WT == WT_Q4_K;  // per-block scales or sums are read in the loop
  constexpr int kOutRows = MODE == TILE_GLU ? 32 * WR : kTileRows * WR;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem), full0 = sbase, empty0 = sbase + 8u * kTileMaxStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kTileBarBytes - 8);
  float* red = reinterpret_cast<float*>(smem + kTileBarBytes);
  const uint32_t ring = sbase + kTileBarBytes + tile_red_bytes(WR);
  const uint32_t stage_bytes = tile_stage_bytes<WT, NT>(WR, a.cols);
  const uint32_t xoff = kTileRows * WR * P + 16, moff = xoff + a.cols * XP;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < a.NS; ++i) {
      mbar_init(full0 + 8u * i, 1);
      mbar_init(empty0 + 8u * i, kTileWarpsK * WR);
    }
    fence_mbar_init();
  }
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  const int tiles = (a.rows + kOutRows - 1) / kOutRows;
  const int64_t items = static_cast<int64_t>(*a.n_groups) * tiles;
  const int64_t lo = items * blockIdx.x / gridDim.x, hi = items * (blockIdx.x + 1) / gridDim.x;
  const int n_kc = (a.K + KC - 1) / KC;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = l2_policy_evict_first();
    int slot = 0, issued = 0;
    uint32_t phase = 1u;
    bool ok = true;
    for (int64_t it = lo; it < hi && ok; ++it) {
      const int gi = static_cast<int>(it / tiles);
      const int row0 = static_cast<int>(it - static_cast<int64_t>(gi) * tiles) * kOutRows;
      const int4 g = a.groups[gi];
      // lane c holds the packed column of the group's column c
      const int64_t col = lane < g.z ? a.slots[g.y + lane] / a.slot_div : 0;
      for (int kc = 0; kc < n_kc; ++kc) {
        if (issued >= a.NS) ok = mbar_wait_or_abort(empty0 + 8u * slot, phase, abort_flag, a.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int klen = min(KC, a.K - kc * KC);
        const int seg = tile_seg<WT>(klen), segoff = tile_seg<WT>(kc * KC);
        const uint32_t st = ring + static_cast<uint32_t>(slot) * stage_bytes, full = full0 + 8u * slot;
        // rows lane, lane + 32, ... of the stage
        uint32_t bytes = 0;
        uint32_t len[2 * WR];
        int64_t src[2 * WR];
#pragma unroll
        for (int q = 0; q < 2 * WR; ++q) {
          // gated: 32-row halves alternate between gate and up
          const int out = MODE == TILE_GLU ? row0 + 32 * (q >> 1) + lane : row0 + 32 * q + lane;
          len[q] = 0;
          if (out < a.rows) {
            const int64_t off = (static_cast<int64_t>(g.x) * a.rows + out) * a.row_bytes + segoff;
            src[q] = off & ~15ll;
            len[q] = static_cast<uint32_t>(((off + seg + 15) & ~15ll) - src[q]);
            if (src[q] + len[q] > a.total_bytes) {  // the end of the last matrix, copied by hand
              len[q] -= 16;
              const uint8_t* W = (MODE == TILE_GLU && (q & 1)) ? a.W2 : a.W;
              for (int64_t b = src[q] + len[q]; b < a.total_bytes; b += 2) {
                const uint16_t v = *reinterpret_cast<const uint16_t*>(W + b);
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(st + (32 * q + lane) * P + static_cast<uint32_t>(b - src[q])),
                             "h"(v)
                             : "memory");
              }
              fence_proxy_async_smem();
            }
            bytes += len[q];
          }
        }
        const uint32_t xlen = static_cast<uint32_t>(klen) * 4u;
        const uint32_t mlen = (static_cast<uint32_t>(klen) / 4u + 15u) & ~15u;
        if (lane < g.z) bytes += xlen + (kMeta ? mlen : 0u);
        bytes = __reduce_add_sync(0xffffffffu, bytes);
        if (lane == 0) mbar_arrive_expect_tx(full, bytes);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 2 * WR; ++q) {
          const uint8_t* W = (MODE == TILE_GLU && (q & 1)) ? a.W2 : a.W;
          if (len[q]) bulk_g2s(st + (32 * q + lane) * P, W + src[q], len[q], full, pol);
        }
        if (lane < g.z) {
          bulk_g2s(st + xoff + lane * XP, a.xpack + (col * a.K + static_cast<int64_t>(kc) * KC) * 4, xlen, full);
          if constexpr (kMeta)
            bulk_g2s(st + moff + lane * MP, a.xmeta + col * expert_meta_stride(a.K) + kc * (KC / 32), mlen, full);
        }
        ++issued;
        if (++slot == a.NS) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    // Drain after an abort: every copy this warp issued lands before the CTA leaves.
    if (!ok) {
      for (int i = max(0, issued - a.NS); i < issued; ++i)
        (void)mbar_wait(full0 + 8u * (i % a.NS), static_cast<uint32_t>((i / a.NS) & 1));
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int cw = warp - 1, wr = cw / kTileWarpsK, wk = cw % kTileWarpsK;
    const uint32_t g4 = static_cast<uint32_t>(lane) >> 2, t4 = static_cast<uint32_t>(lane) & 3u;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    float* myred = red + wr * (kTileWarpsK * 8 * kRedPitch);
    auto group_bar = [&]() { named_bar_sync(1u + static_cast<uint32_t>(wr), 32u * kTileWarpsK); };
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
      // Stage rows g and g + 8 of the row group's first matrix tile (the others lie 16 rows
      // apart).  A row's first byte sits at (its offset in the matrices) mod 16, the same for
      // rows 16 apart, and so for the gate row and the up row 32 stage rows apart.
      uint32_t rowaddr[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * h + static_cast<int>(g4);
        uint32_t shift = 0;
        if constexpr (WT != WT_F16 && WT != WT_Q4_K)
          shift = (static_cast<uint32_t>(g.x * a.rows + row0 + kOutRows / WR * wr + r) *
                   static_cast<uint32_t>(a.row_bytes)) & 15u;
        rowaddr[h] = static_cast<uint32_t>((kTileRows * wr + r) * P) + shift;
      }
      for (int kc = 0; kc < n_kc; ++kc) {
        ok = ok && mbar_wait_or_abort(full0 + 8u * slot, phase, abort_flag, a.err);
        const uint32_t st = ring + static_cast<uint32_t>(slot) * stage_bytes;
        const int units = min(KC, a.K - kc * KC) / 32;
        if (ok) {
#pragma unroll 1
          for (int u = wk; u < units; u += kTileWarpsK) {
            const uint32_t blk = static_cast<uint32_t>(u);
            uint4 b[NT][2];
            float2 meta[NT][2];  // of columns 2t and 2t + 1 of each column tile
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (8 * n < ncol) {
                // lanes past the group's columns read its last column; their sums are dropped
                const uint32_t c = static_cast<uint32_t>(min(8 * n + static_cast<int>(g4), ncol - 1));
                const uint32_t xa = st + xoff + c * XP + blk * 128u + t4 * 16u;
                b[n][0] = lds128(xa);
                b[n][1] = lds128(xa + 64u);
                if constexpr (kMeta) {
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const uint32_t mc = static_cast<uint32_t>(min(8 * n + 2 * static_cast<int>(t4) + h, ncol - 1));
                    const uint2 v = lds64(st + moff + mc * MP + blk * 8u);
                    meta[n][h] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
                  }
                }
              }
            }
            // Q4_K: taking a row's 6-bit scale and min apart costs as much as its codes; the four
            // lanes of a row would all do it, so lane t does it for matrix tile t only
            float qd[2], qm[2];
            if constexpr (WT == WT_Q4_K) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                q4k_scale_of(lds128(st + rowaddr[h] + t4 * (16u * P) + (blk >> 3) * kQ4kBytes), blk & 7u, qd[h], qm[h]);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              uint32_t a0[2][2], a1[2][2];
              float d[2], dm[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t row = st + rowaddr[h] + m * (16u * P);
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
                    // i: row g (0, 1) or g + 8 (2, 3), column 2t + (i & 1)
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
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + 8u * slot);
        if (++slot == a.NS) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // the warps' sums of the row group through shared memory, eight columns at a time:
      // red[warp][column][row]; then warp wk takes column 8n + wk
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= ncol) break;
        group_bar();  // everyone has read the previous sums
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            myred[(wk * 8 + 2 * t4 + (i & 1)) * kRedPitch + 16 * m + g4 + 8 * (i >> 1)] = acc[m][n][i];
        group_bar();
        const int c = 8 * n + wk;
        if (c < ncol && ok && !*abort_flag) {
          const int sl = a.slots[g.y + c];
          float v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kTileWarpsK; ++w) s += myred[(w * 8 + wk) * kRedPitch + 32 * h + lane];
            v[h] = s;
          }
          if constexpr (MODE == TILE_GLU) {
            // 32 output rows of the gated product: one packed block of the slot's column
            const float sx = a.xmeta[static_cast<int64_t>(sl / a.slot_div) * expert_meta_stride(a.K)].x;
            const int r0 = row0 + 32 * wr;
            if (r0 < a.rows) {  // rows are a multiple of 32
              const float h = tail_silu(v[0] * sx) * (v[1] * sx);
              const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(finite_abs(h))));
              const float sc = pack_scale(m), hs = h * sc;
              float sum = hs;
#pragma unroll
              for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              const HiLo p = split_hi_lo(hs);
              uint8_t* q = a.hpack + (static_cast<int64_t>(sl) * a.rows + r0) * 4 +
                           packed_offset(static_cast<uint32_t>(lane), a.h_swapped != 0);
              *reinterpret_cast<__half*>(q) = p.hi;
              *reinterpret_cast<__half*>(q + 8) = p.lo;
              if (lane == 0)
                a.hmeta[static_cast<int64_t>(sl) * expert_meta_stride(a.rows) + r0 / 32] =
                    make_float2(pow2_inverse(sc), sum);
            }
          } else {
            const float w = a.weights[sl];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = row0 + kTileRows * wr + 32 * h + lane;
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
