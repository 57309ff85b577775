// The tiled product for wide column groups (up to 16 columns, block formats in rows of whole
// 16-byte words): the same operands, stages and records as tile_mma.cuh, cut the other way.
//
// With two column tiles the matrix instructions outweigh the decode, and what the K-sharing
// kernel pays per chunk and item (records as large as the weights beside them, a wait per
// block, the sums of eight warps through shared memory) is no longer hidden: it reached a
// quarter of the matrix unit's rate.  Here each of a CTA's consumer warps takes 32 rows for
// all of K (gated: 16 gate rows and their up rows): a chunk's records serve all the warps'
// rows, a warp runs eight blocks between two waits, and nothing is added across warps.
// Gated, the gated value forms in the thread that holds both sums; two warps make one packed
// block of 32 and exchange its largest value and its sum.
//
// Sixteen warps, four a scheduler (eight for Q8_0, whose rows leave no room for two stages of
// sixteen warps' rows).  Measured on 256 tokens, 128 experts, 8 choices, 768 x 2048 Q4_K,
// gate and up: eight warps with three column tiles 166 us, twelve (spilling) 178, sixteen
// with two 153 (141 with items handed out, below); 64 columns of 14336 x 4096 Q4_0: 77, 101, 67.
//
// An item is a large piece of a launch (a quarter of a CTA's share, in that case), and column
// groups differ in size: the experts' items are handed out one by one, large groups first,
// instead of in equal ranges, which left the SMs idle for a fifth of the time.  What bounds it
// now: the matrix unit, 39% busy on average while its four warps collide on it (throttled for
// as long as they issue), and one issue slot in two.
#pragma once

#include "tile_mma.cuh"

namespace gf {

constexpr int kWideNT = 2;  // column tiles
// Consumer warps, 32 rows each.
template <int WT>
__host__ __device__ constexpr int wide_warps() { return WT == WT_Q8_0 ? 8 : 16; }
template <int WT>
__host__ __device__ constexpr int wide_xchg() {  // [item parity][warp][column] {largest, sum}, then counts
  return 2 * wide_warps<WT>() * 8 * kWideNT * 12;
}
template <int WT>
__host__ __device__ constexpr int wide_weight_bytes() { return wide_warps<WT>() * tile_part<WT>(1); }
template <int WT>
__host__ __device__ constexpr int wide_stage_bytes() {
  return (wide_weight_bytes<WT>() + 16 + kWideNT * kTileBlocks * record_bytes(8) + 1023) / 1024 * 1024;
}

// A warp's walk over one pair of blocks (2 b, 2 b + 1) of a chunk: its 32 rows, NTA column tiles.
// row: stage address of row g of matrix tile 0; rows 8 further and matrix tile 1 lie constant
// distances on.
template <int WT, int MODE, int NTA>
__device__ __forceinline__ void wide_pair(const TileLane& l, uint32_t row, uint32_t xs, uint32_t pair,
                                          float (&acc)[2][kWideNT][4]) {
  constexpr uint32_t kP = tile_pitch<WT>(1);
  constexpr uint32_t kM = MODE == TILE_GLU ? wide_warps<WT>() / 2 * tile_part<WT>(1) : 16u * kP;  // matrix tiles apart
  const uint32_t t4 = l.t4;
  constexpr uint32_t kBlock = WT == WT_Q8_0 ? 34u : WT == WT_Q4_0 ? 18u : 0u;
  // the code words: of one block at a time, except Q4_K, whose two blocks are the low and the
  // high nibbles of the same words
  uint32_t kw[2][2], kv[2][2];
  float qd[2], qm[2];  // Q4_K: scale and min of the two blocks, of the row (t4 / 2, t4 % 2)
  if constexpr (WT == WT_Q4_K) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        kw[m][h] = lds32(row + m * kM + h * 8u * kP + 16u + pair * 32u + 4u * t4);
        kv[m][h] = lds32(row + m * kM + h * 8u * kP + 32u + pair * 32u + 4u * t4);
      }
    const uint4 hd = lds128(row + (t4 >> 1) * kM + (t4 & 1u) * (8u * kP));
    q4k_scale_of(hd, 2u * pair, qd[0], qm[0]);
    q4k_scale_of(hd, 2u * pair + 1u, qd[1], qm[1]);
  }
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const uint32_t xo = xs + (2u * pair + o) * l.rec;
    uint32_t a0[2][2][2], a1[2][2][2];
    float d[2][2], dm[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        dm[m][h] = 0.0f;
        if constexpr (WT == WT_Q4_K) {
          a0[m][h][0] = (kw[m][h] << (o ? 2 : 6)) & kNibbles;
          a0[m][h][1] = (kw[m][h] >> (o ? 6 : 2)) & kNibbles;
          a1[m][h][0] = (kv[m][h] << (o ? 2 : 6)) & kNibbles;
          a1[m][h][1] = (kv[m][h] >> (o ? 6 : 2)) & kNibbles;
          d[m][h] = __shfl_sync(0xffffffffu, qd[o], 2 * m + h, 4);
          dm[m][h] = __shfl_sync(0xffffffffu, qm[o], 2 * m + h, 4);
        } else {
          // even blocks start on a word, their codes two bytes later; odd ones the other way
          RowPlace p;
          p.scale = row + m * kM + h * 8u * kP + 2u * kBlock * pair + o * kBlock;
          p.code = p.scale + (o ? 2u : 0u) + 4u * t4;
          p.shift = 16u;
          p.left = p.right = 0u;
          if (o)
            load_block_row<WT, true>(p, 0u, a0[m][h], a1[m][h], d[m][h]);
          else
            load_block_row<WT, false>(p, 0u, a0[m][h], a1[m][h], d[m][h]);
        }
      }
    // column tile by column tile: few registers, so that four warps a scheduler hide the latency
#pragma unroll
    for (int n = 0; n < NTA; ++n) {
      const uint32_t xa = xo + static_cast<uint32_t>(n) * l.xtile;
      const uint4 b0 = lds128(xa + l.xlane), b1 = lds128(xa + l.xlane + l.cp * 64u);
      float sx[2] = {0.0f, 0.0f}, xsum[2] = {0.0f, 0.0f};  // 2^-s and sum of columns 2t and 2t + 1
      if constexpr (MODE == TILE_DOWN || pack_sums(WT)) {
        const uint2 u = lds64(xa + l.m0), v = lds64(xa + l.m1);
        sx[0] = __uint_as_float(u.x); sx[1] = __uint_as_float(v.x);
        xsum[0] = __uint_as_float(u.y); xsum[1] = __uint_as_float(v.y);
      }
      float s[2][4];
      auto step = [&](int i) {  // lo of both k-steps, then hi (see tile_block)
        const uint32_t p = i == 0 ? b0.z : i == 1 ? b1.z : i == 2 ? b0.x : b1.x;
        const uint32_t q = i == 0 ? b0.w : i == 1 ? b1.w : i == 2 ? b0.y : b1.y;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint32_t (&x)[2][2] = (i & 1) ? a1[m] : a0[m];
          if (i == 0)
            mma_f16_first(s[m], x[0][0], x[1][0], x[0][1], x[1][1], p, q);
          else
            mma_f16(s[m], x[0][0], x[1][0], x[0][1], x[1][1], p, q);
        }
      };
      step(0);
      step(1);
      step(2);
      step(3);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // row g + 8 (i / 2), column 2t + i % 2
          const int h = i >> 1, c = i & 1;
          float& r = acc[m][n][i];
          if constexpr (MODE == TILE_DOWN) {
            float y = d[m][h] * s[m][i];
            if constexpr (WT == WT_Q4_K) y = fmaf(-dm[m][h], xsum[c], y);
            r = fmaf(sx[c], y, r);
          } else {
            r = fmaf(d[m][h], s[m][i], r);
            if constexpr (WT == WT_Q4_K) r = fmaf(-dm[m][h], xsum[c], r);
          }
        }
    }
  }
}

// A barrier of nthreads threads that tells them all whether p holds for every one of them.
__device__ __forceinline__ bool named_bar_all(uint32_t id, uint32_t nthreads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %3, 0;\n\t"
      "barrier.cta.red.and.pred b, %1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"(p ? 1u : 0u)
      : "memory");
  return r != 0u;
}

template <int WT, int MODE>
__global__ void __launch_bounds__(32 * (1 + wide_warps<WT>()), 1)
    wide_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                const __grid_constant__ TileArgs a) {
  constexpr int NT = kWideNT;
  constexpr int kWarps = wide_warps<WT>(), kThreads = 32 * (1 + kWarps);
  constexpr int kOutRows = MODE == TILE_GLU ? 16 * kWarps : 32 * kWarps;
  constexpr uint32_t P = tile_pitch<WT>(1), kPart = tile_part<WT>(1), kRec = record_bytes(8);
  constexpr uint32_t kStage = wide_stage_bytes<WT>(), kXoff = wide_weight_bytes<WT>() + 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem), full0 = sbase, empty0 = sbase + 8u * kTileMaxStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 248);
  volatile int* item_of = reinterpret_cast<volatile int*>(smem + 128);  // per stage: item whose first chunk it holds
  float2* xchg = reinterpret_cast<float2*>(smem + kTileHeadBytes);
  const uint32_t ring = (sbase + kTileHeadBytes + wide_xchg<WT>() + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < a.NS; ++i) {
      mbar_init(full0 + 8u * i, 1);
      mbar_init(empty0 + 8u * i, kWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&map0);
    if (MODE == TILE_GLU) prefetch_tmap(&map1);
  }
  pdl_trigger();
  pdl_wait();
  const int out_rows = MODE == TILE_LIN ? min(a.item_rows, kOutRows) : kOutRows;  // of an item; the warps beyond idle
  const int tiles = (a.rows + out_rows - 1) / out_rows;
  const int n_groups = MODE == TILE_LIN ? (a.ncols + a.group_cols - 1) / a.group_cols : *a.n_groups;
  const int items = n_groups * tiles;  // groups <= 2048, tiles <= 2^12
  auto group_of = [&](int gi) -> int4 {
    return MODE == TILE_LIN ? make_int4(0, 0, min(a.group_cols, a.ncols - gi * a.group_cols), gi * ((a.group_cols + 7) / 8))
                            : a.groups[gi];
  };
  __syncthreads();
  const int n_kc = (a.K + kTileK - 1) / kTileK, nblk = a.K / 32;
  const int64_t tile_stride = static_cast<int64_t>(nblk) * kRec;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int slot = 0, issued = 0;
      uint32_t phase = 1u;
      bool ok = true;
      // a batch's items are alike: every grid-th; the experts' as they come
      for (int it = MODE == TILE_LIN ? static_cast<int>(blockIdx.x) : static_cast<int>(atomicAdd(a.next, 1u)); ok;
           it = MODE == TILE_LIN ? it + static_cast<int>(gridDim.x) : static_cast<int>(atomicAdd(a.next, 1u))) {
        if (it >= items) {  // the end: a stage without data
          if (issued >= a.NS && !mbar_wait_or_abort(empty0 + 8u * slot, phase, abort_flag, a.err)) ok = false;
          if (ok) {
            item_of[slot] = -1;
            mbar_arrive(full0 + 8u * slot);
          }
          break;
        }
        const int4 g = group_of(it / tiles);
        const int row0 = (it % tiles) * out_rows;
        const int boxes = min(out_rows / 32, (a.rows - row0 + 31) / 32);  // of each matrix
        const int nt = (g.z + 7) / 8;
        const uint32_t rec = static_cast<uint32_t>(record_bytes(min(8, g.z)));
        const uint8_t* xsrc = a.records + g.w * tile_stride;
        for (int kc = 0; kc < n_kc; ++kc) {
          if (issued >= a.NS && !mbar_wait_or_abort(empty0 + 8u * slot, phase, abort_flag, a.err)) {
            ok = false;
            break;
          }
          const uint32_t st = ring + static_cast<uint32_t>(slot) * kStage, full = full0 + 8u * slot;
          const uint32_t xlen = static_cast<uint32_t>(min(kTileBlocks, nblk - kc * kTileBlocks)) * rec;
          if (kc == 0) item_of[slot] = it;
          mbar_arrive_expect_tx(full, (MODE == TILE_GLU ? 2u : 1u) * boxes * 32u * P + nt * xlen);
          for (int i = 0; i < boxes; ++i) {
            tma_load_2d(st + i * kPart, &map0, kc * (tile_seg<WT>() / 2), g.x * a.rows + row0 + 32 * i, full);
            if constexpr (MODE == TILE_GLU)
              tma_load_2d(st + (kWarps / 2 + i) * kPart, &map1, kc * (tile_seg<WT>() / 2), g.x * a.rows + row0 + 32 * i, full);
          }
          for (int n = 0; n < nt; ++n)
            bulk_g2s(st + kXoff + static_cast<uint32_t>(n) * kTileBlocks * rec,
                     xsrc + n * tile_stride + static_cast<uint32_t>(kc * kTileBlocks) * rec, xlen, full);
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
    const int w = warp - 1;
    const uint32_t g4 = static_cast<uint32_t>(lane) >> 2, t4 = static_cast<uint32_t>(lane) & 3u;
    const uint32_t place = MODE == TILE_GLU ? static_cast<uint32_t>(w >> 1) * kPart + (16u * (w & 1) + g4) * P
                                            : static_cast<uint32_t>(w) * kPart + g4 * P;
    TileLane l = {};
    l.t4 = t4;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true, raw = false;  // raw: a column was
    for (uint32_t round = 0;; ++round) {
      // the item's first chunk, or the end
      ok = __all_sync(0xffffffffu, ok && mbar_wait_or_abort(full0 + 8u * slot, phase, abort_flag, a.err));
      const int it = ok ? item_of[slot] : -1;
      // gated, two warps meet at a barrier below: they go on, or stop, together
      if (!(MODE == TILE_GLU ? named_bar_all(1u + static_cast<uint32_t>(w >> 1), 64u, it >= 0) : it >= 0)) break;
      const int4 g = group_of(it / tiles);
      const int row0 = (it % tiles) * out_rows;
      const int ncol = g.z;
      l.cp = static_cast<uint32_t>(min(8, ncol));
      l.rec = static_cast<uint32_t>(record_bytes(static_cast<int>(l.cp)));
      l.xtile = kTileBlocks * l.rec;
      l.xlane = min(g4, l.cp - 1u) * 64u + t4 * 16u;  // lanes past the columns read the last one
      l.m0 = l.cp * 128u + min(2u * t4, l.cp - 1u) * 8u;
      l.m1 = l.cp * 128u + min(2u * t4 + 1u, l.cp - 1u) * 8u;
      const uint32_t cp = l.cp, rec = l.rec;
      const int at = MODE == TILE_GLU ? 16 * w : 32 * w;  // the warp's rows in the item
      const bool mine = at < out_rows && row0 + at < a.rows;
      float acc[2][NT][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
      auto walk = [&](auto nta) {
        constexpr int NTA = decltype(nta)::value;
#pragma unroll 1
        for (int kc = 0; kc < n_kc; ++kc) {
          if (kc > 0) ok = __all_sync(0xffffffffu, ok && mbar_wait_or_abort(full0 + 8u * slot, phase, abort_flag, a.err));
          const uint32_t st = ring + static_cast<uint32_t>(slot) * kStage;
          if (ok && mine) {
            // rows of whole 16-byte words have whole chunks
#pragma unroll 1
            for (uint32_t p = 0; p < kTileBlocks / 2; ++p) wide_pair<WT, MODE, NTA>(l, st + place, st + kXoff, p, acc);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty0 + 8u * slot);
          if (++slot == a.NS) {
            slot = 0;
            phase ^= 1u;
          }
        }
      };
      if (ncol > 8) walk(TileConst<2>());
      else walk(TileConst<1>());
      // the tail's factors of columns 8n + 2t + c
      float factor[NT][2];
      int sl[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = 8 * n + 2 * static_cast<int>(t4) + c;
          factor[n][c] = 0.0f;
          sl[n][c] = 0;
          if (col < ncol) {
            if constexpr (MODE != TILE_DOWN) {
              factor[n][c] = *reinterpret_cast<const float*>(a.records + (g.w + n) * tile_stride + cp * 128u +
                                                             (2u * t4 + c) * 8u);
            } else {
              sl[n][c] = a.slots[g.y + col];
              factor[n][c] = a.factors[sl[n][c]];
            }
          }
        }
      if constexpr (MODE == TILE_LIN)
#pragma unroll
        for (int n = 0; n < NT; ++n) raw |= __float_as_uint(factor[n][0]) == kRawBlock || __float_as_uint(factor[n][1]) == kRawBlock;
      if constexpr (MODE == TILE_GLU) {
        // the gated values of rows 8h + g (of the warp's 16) and columns 2t + c, in place of the
        // gate sums; two warps make a block: they exchange its largest value, then how many values
        // lie how far below it and, for Q4_K's mins, the sum of what they pack
        float2* mx = xchg + (round & 1u) * (kWarps * 8 * NT);
        int* mc = reinterpret_cast<int*>(xchg + 2 * kWarps * 8 * NT) + (round & 1u) * (kWarps * 8 * NT);
        const uint32_t pair = 1u + static_cast<uint32_t>(w >> 1);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int i = 2 * h + c;
              const float f = tile_unit(WT) * factor[n][c];
              const float v = tail_silu(acc[0][n][i] * f) * (acc[1][n][i] * f);
              acc[0][n][i] = v;
              top = fmaxf(top, fabsf(v));  // (not a NaN)
            }
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (g4 == 0) mx[w * 8 * NT + 8 * n + 2 * t4 + c].x = top;
          }
        named_bar_sync(pair, 64u);
        const int r0 = row0 + 32 * (w >> 1);
        const bool write = r0 < a.rows && ok && !*abort_flag;
        auto is_raw = [&](int n, int c) { return __float_as_uint(factor[n][c]) == kRawBlock; };
        const int order = pack_order(a.out_format);
        const bool sums = pack_sums(a.out_format);
        auto record = [&](int n) {
          return a.out_records + static_cast<int64_t>(g.w + n) * (a.rows / 32) * kRec + static_cast<int64_t>(r0 / 32) * rec;
        };
        auto top_of = [&](int col) { return fmaxf(mx[(w & ~1) * 8 * NT + col].x, mx[(w | 1) * 8 * NT + col].x); };
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t col = 2u * t4 + c;
            const bool in = write && 8 * n + static_cast<int>(col) < ncol && !is_raw(n, c);
            const float top = top_of(8 * n + static_cast<int>(col));
            const float sc = pack_scale(is_finite(top) ? top : 0.0f);
            float sum = 0.0f;
            int counts = 0;  // values of at least kCarryBlock of the largest; tiny ones (x 256); NaN (x 65536)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t rr = 16u * (w & 1) + 8u * h + g4, i = rr & 3u;
              const float v = acc[0][n][2 * h + c];
              const HiLo p = split_hi_lo(v * sc);
              sum += value_of(p);
              counts += (fabsf(v) >= top * kCarryBlock ? 1 : 0) + (v != 0.0f && fabsf(v) < top * kCarryTiny ? 256 : 0) +
                        (v != v ? 65536 : 0);
              if (in) {
                uint8_t* q = record(n) + record_offset(rr >> 2, col, cp, order) +
                             2u * (order == ORDER_NIBBLE ? ((i & 1u) << 1) | (i >> 1) : i);
                *reinterpret_cast<__half*>(q) = p.hi;
                *reinterpret_cast<__half*>(q + 8) = p.lo;
              }
            }
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
              if (sums) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              counts += __shfl_xor_sync(0xffffffffu, counts, o);
            }
            if (g4 == 0) {
              mx[w * 8 * NT + 8 * n + col].y = sum;
              mc[w * 8 * NT + 8 * n + col] = counts;
            }
          }
        named_bar_sync(pair, 64u);
        if (write) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = 8 * n + 2 * static_cast<int>(t4) + c;
              if (col >= ncol || is_raw(n, c)) continue;
              const float top = top_of(col);
              const int counts = mc[(w & ~1) * 8 * NT + col] + mc[(w | 1) * 8 * NT + col];
              const bool carried = counts >= 65536 || (is_finite(top) && ((counts & 255) >= 4 || counts < 256));
              if (!carried)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t rr = 16u * (w & 1) + 8u * h + g4;
                  *reinterpret_cast<float*>(record(n) + record_offset(rr >> 2, 2u * t4 + c, cp, order) + 4u * (rr & 3u)) =
                      acc[0][n][2 * h + c];
                }
              if (g4 != 0 || (w & 1)) continue;
              const float sum = sums ? (mx[w * 8 * NT + col].y + mx[(w + 1) * 8 * NT + col].y) / tile_unit(WT_Q4_K) : 0.0f;
              *reinterpret_cast<float2*>(record(n) + cp * 128u + (2u * t4 + c) * 8u) =
                  carried ? make_float2(pow2_inverse(pack_scale(is_finite(top) ? top : 0.0f)), sum) : make_float2(__uint_as_float(kRawBlock), 1.0f);
            }
        }
      } else if (ok && mine && !*abort_flag) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = 8 * n + 2 * static_cast<int>(t4) + c;
            if (col >= ncol || (MODE == TILE_LIN && __float_as_uint(factor[n][c]) == kRawBlock)) continue;
            const int64_t base = (MODE == TILE_LIN ? static_cast<int64_t>(g.w) * 8 + col : sl[n][c]) * a.out_ld;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int r = row0 + 32 * w + 16 * m + 8 * h + static_cast<int>(g4);
                if (r < a.rows) {
                  const float y = factor[n][c] * (acc[m][n][2 * h + c] * tile_unit(WT));
                  if constexpr (MODE == TILE_LIN)
                    a.out[base + r] = apply_tail(a.epi, y, epi_takes_aux(a.epi) ? a.aux[base + r] : 0.0f);
                  else
                    a.out[base + r] = y;
                }
              }
          }
      }
    }
    // a batch's raw columns: this CTA's items again
    if (MODE == TILE_LIN && __any_sync(0xffffffffu, raw) && ok && !*abort_flag)
      for (int it = static_cast<int>(blockIdx.x); it < items; it += static_cast<int>(gridDim.x)) {
        const int4 g = group_of(it / tiles);
        const int row0 = (it % tiles) * out_rows + 32 * w;
        if (32 * w >= out_rows || row0 >= a.rows) continue;
        for (int c = 0; c < g.z; ++c)
          if (raw_column(a, g, c)) exact_rows<WT>(a, g, c, row0);
      }
  }
  __syncthreads();
}

}  // namespace gf
