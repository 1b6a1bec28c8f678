// Backward pass on tcgen05 tensor cores with TMEM accumulators (sm_100a).
//
// One CTA owns a tile of 128 X rows and walks over blocks of BN Y rows:
//   key tiles    X = keys:  X1 = K, X2 = V,  Y1 = Q, Y2 = dO:  dK and/or dV
//   query tiles  X = rows:  X1 = Q, X2 = dO, Y1 = K, Y2 = V:   dQ
// and in both S = X1 Y1^T, dP = X2 Y2^T, then
//   out1 += dS Y1 (dK or dQ),  out2 += P Y2 (dV).
// With X in the M dimension the rows of S sit in TMEM lanes, so P and dS are
// written back over the scores as packed 16-bit values and become the TMEM A
// operand of the second products: neither passes through shared memory, and a
// Y block, staged once, is the K-major B operand of the first product and the
// MN-major one of the second.  Computing S and dP in both kinds of tile costs
// 7 products where one pass with a shared dQ would need 5, but no gradient is
// ever added across CTAs: no atomics, no fp32 dQ in memory, the same bits every
// time.
//
// Warp roles (10 warps):
//   0-7  softmax.  Phase E: P = 2^(S c + nlse); phase F: dS = P (dP + ndelta) gain,
//        with P kept in registers.  With two score buffers (ST = 2) warps 0-3
//        take the even blocks and 4-7 the odd ones, a row per thread; with one,
//        warps w and w + 4 share TMEM lanes 32 (w % 4) .. +31 and take one half of
//        a block's columns each, packed over their own half only, so that the
//        two need no exchange.
//   8    TMA producer: X once, then Y1 and Y2 blocks through two rings, the row
//        terms of a query block with its Y1.  It alone walks over the block list
//        and tells the others with each Y1 slot which block it holds and whether
//        the block needs its mask tested (a taken branch costs a warp about 25
//        cycles: walking took the softmax warps 400 to 700 cycles a block)
//   9    MMA issuer (the whole warp, one elected lane), in the order
//            out2_n, S_{n+ST}   after P_n
//            out1_n, dP_{n+ST}  after dS_n
//        One warp's MMAs run in issue order, so S_{n+ST} may overwrite P_n once
//        out2_n is issued.
//
// With TWO, P and dS go in as two terms, the 16-bit value and the 16-bit value of
// what its rounding left, in the two halves of the columns they came from: twice
// the second products, and the gradients' own rounding is the only one that shows.
//
// What bounds it.  P_n -> out2_n, S_{n+1} -> P_{n+1} is a chain through one score
// buffer: with ST = 1 it took 4300 cycles per 128 x 128 pairs of a key tile at
// every head dim (E 1900 until the slower of an SM sub-partition's two warps is
// through, then the two products and their hand-overs), against 2048 of tensor
// work at head dim 128.  Two buffers let one warp group's chain run under the
// other's.  Their cost is operand traffic: a 128 x 64 x 16 product with both
// operands in shared memory reads 6 KB (48 cycles) for 32 cycles of math.  So X,
// constant over a tile, is copied to TMEM where columns are left and read from
// there (2 KB, 16 cycles).
// What a block costs now, of the tensor work (cycles per block of 64, from CTA
// times): head dim 128 key tiles 1370 of 1280, query tiles 1000 of 768; 256 dK and
// dQ 2000 of 1792, dV 1270 of 1024.  At 128 and above the chip is at its power
// limit under it (1000 W, 1.5 to 1.7 GHz of 1.96).  At 64 and 80 a block takes
// about 1150 cycles of hand-overs whatever it computes (leaving out the
// exponentials, or three quarters of one product, changed at most 6 %), so
// those take blocks of 96 and 80 instead (6 % faster).
//
// TMEM (512 columns): ST stages of S and dP, out1, out2, X1, X2 where they fit:
// BwdTcRoles below lists what each head-dim pair takes.  Head dims from 192/192
// leave no room for dK and dV together: those take a CTA each.
#pragma once

#include <type_traits>

#include "bwd_blocks.h"
#include "bwd_params.cuh"

namespace sdpa {

constexpr int kBwdTcSoftmaxWarps = 8;
constexpr int kBwdTcThreads = (kBwdTcSoftmaxWarps + 2) * 32;

// One kind of tile.  ST: score buffers; N1 / N2: ring slots of Y1 and Y2;
// XT1 / XT2: X1 / X2 are read from TMEM; W: gradient columns of a CTA where several
// share a tile (0: all); ALIAS: X1 passes through the last Y1
// slots on its way there.
template <int D1_, int D2_, int BN_, int ST_, int N1_, int N2_, bool KEYS_, bool OUT1_, bool OUT2_, bool XT1_, bool XT2_,
          bool ALIAS_ = false, int W_ = 0>
struct BwdTcRole {
  static constexpr int D1 = D1_, D2 = D2_, BN = BN_, ST = ST_, N1 = N1_, N2 = N2_;
  static constexpr bool KEYS = KEYS_, OUT1 = OUT1_, OUT2 = OUT2_, XT1 = XT1_, XT2 = XT2_, ALIAS = ALIAS_;
  static constexpr int kBoxes1 = (D1 + 63) / 64, kBoxes2 = (D2 + 63) / 64;
  static constexpr int W1 = W_ ? W_ : D1, W2 = W_ ? W_ : D2;  // columns of out1, out2
  static constexpr bool PARTED = W_ != 0;
  static constexpr int kBoxRows = 64;  // of the tensor maps of X
  static constexpr uint32_t kX1Bytes = kBoxes1 * 128 * 128;
  static constexpr uint32_t kX2Bytes = OUT1 ? kBoxes2 * 128 * 128 : 0;  // dP only
  static constexpr uint32_t kY1Bytes = kBoxes1 * BN * 128;
  // (without dP, only the columns of out2 are needed of Y2)
  static constexpr int kY2Boxes = OUT1 ? kBoxes2 : (W2 + 63) / 64;
  static constexpr uint32_t kY2Bytes = kY2Boxes * BN * 128;
  // X1 goes through the rings in one pass, or (both rings being smaller) in two
  static constexpr int kXFirst = ALIAS && N1 * kY1Bytes + N2 * kY2Bytes < kX1Bytes
                                     ? (N1 * kY1Bytes + N2 * kY2Bytes) / (128 * 128) : kBoxes1;
  static constexpr bool TWICE = kXFirst < kBoxes1;
  static constexpr int kAliasSlots = !ALIAS ? 0 : TWICE ? N1 : (kX1Bytes + kY1Bytes - 1) / kY1Bytes;
  static constexpr uint32_t kX2Off = ALIAS ? 0 : kX1Bytes;
  static constexpr uint32_t kY1Off = kX2Off + kX2Bytes;
  static constexpr uint32_t kX1Off = ALIAS ? kY1Off + (N1 - kAliasSlots) * kY1Bytes : 0;
  static constexpr uint32_t kY2Off = kY1Off + N1 * kY1Bytes;
  static constexpr uint32_t kTermOff = kY2Off + N2 * kY2Bytes;  // [NT][2][BN] row terms
  // row terms and block notes: behind Y1's slot where that is held until the block
  // is done, else (released before P_n) ST more, so that block n's stay until P_n
  static constexpr int NT = OUT1 ? N1 : N1 + ST;
  static constexpr uint32_t kTermBytes = KEYS ? NT * 2 * BN * 4 : 0;
  static constexpr uint32_t kInfoOff = kTermOff + kTermBytes;  // [NT] BwdBlockInfo
  static constexpr uint32_t kBarOff = kInfoOff + NT * 16;
  static constexpr int kNumBars = 2 * N1 + 2 * N2 + 4 * ST + 6;
  static constexpr uint32_t kSmemBytes = kBarOff + kNumBars * 8 + 16;
  static constexpr int kStageCols = OUT1 ? 2 * BN : BN;  // S and dP of one stage
  static constexpr int kOut1Col = ST * kStageCols;
  static constexpr int kOut2Col = kOut1Col + (OUT1 ? W1 : 0);
  static constexpr int kX1Col = kOut2Col + (OUT2 ? W2 : 0);
  static constexpr int kX2Col = kX1Col + (XT1 ? D1 / 2 : 0);
  static constexpr int kColsUsed = kX2Col + (XT2 ? D2 / 2 : 0);
  static constexpr int kParts = ST == 1 ? 2 : 1;  // softmax warps sharing a row
  static constexpr int kH = BN / kParts;          // columns per softmax thread
  // the finished tile is staged in the X tiles' memory: out1 where X1 was (X2
  // where that is ring slots now), out2 where X2 was (X1 as the only output)
  static constexpr uint32_t kStage1Off = 0;
  static constexpr uint32_t kStage2Off = OUT1 ? kX2Off : 0;
  static_assert(OUT1 || OUT2, "");
  static_assert(KEYS || (OUT1 && !OUT2), "query tiles give dQ");
  static_assert(ST == 1 || ST == 2, "");
  static_assert(kColsUsed <= 512, "TMEM columns");
  // Y1_n is held until out1_n, issued after S_{n+ST} (without out1, until S_n and
  // until the softmax warps of block n have seen it)
  static_assert(N1 >= ST + 1 && N2 >= (OUT1 && OUT2 ? ST : 1), "ring slots");
  static_assert(!ALIAS || (XT1 && OUT1 != OUT2 && N1 >= kAliasSlots && kXFirst >= kBoxes1 - kXFirst), "");
  static_assert(W1 % 16 == 0 && W2 % 16 == 0 && (!PARTED || W1 % 64 == 0), "");
  static_assert(OUT1 || kY2Boxes <= kBoxes1, "out2's staging");
  static_assert(!XT2 || OUT1, "");
  static_assert(kH % 16 == 0 && BN % 16 == 0, "");
  static_assert(kSmemBytes <= 232448, "shared memory");
};

struct BwdTcMaps {
  CUtensorMap q, k, v, dout;  // boxes of 64 rows: X tiles
  CUtensorMap qb, doutb;      // boxes of a key tile's blocks
  CUtensorMap kb, vb;         // boxes of a query tile's blocks
  CUtensorMap dq, dk, dv;     // boxes of 128 rows
};

// Tiles of one kind within the grid.
struct BwdTcSpan {
  int tiles;   // per slab
  int splits;  // most parts that a block list is cut into, `per` blocks each
  int per;
  int *parts;            // splits > 1: [slab][tile] parts of each tile, and where that
  float *part1, *part2;  // is above 1 their fp32 sums [split][slab][X rows][D]
};

// Untiled copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// What the producer says about the block in a Y1 slot.
struct __align__(16) BwdBlockInfo {
  int row0;    // first Y row (behind the last block: the number of blocks)
  int query0;  // key tiles: query index of packed row row0 (behind the last: the tile's parts)
  int masked;  // some pair of tile and block needs its own test
  int valid;   // 0 behind the last block
};

// N consecutive TMEM columns of this thread's lane (N a multiple of 16).
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, float *v) {
#pragma unroll
  for (int c = 0; c + 32 <= N; c += 32) tmem_ld32(taddr + c, v + c);
  if constexpr (N % 32 != 0) {
    float t[16];
    tmem_ld16(taddr + N / 32 * 32, t);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[N / 32 * 32 + i] = t[i];
  }
}

// What rounding the pair (a, b) to 16 bits, to w, left of it, rounded itself.
template <bool kBF16>
__device__ __forceinline__ uint32_t rest2(float a, float b, uint32_t w) {
  const float2 r = unpack2<kBF16>(w);
  return pack2<kBF16>(a - r.x, b - r.y);
}

// X (boxes of 128 rows x 64 columns, 128-byte swizzled) to TMEM as the A operand of
// a first product: 16-bit pairs, a row per lane.  Four warps, one row per thread.
// Columns [16 C0, 16 C1); x holds the boxes from column 16 C0 on.
template <int C0, int C1>
__device__ __forceinline__ void bwd_x_to_tmem(const uint8_t *x, uint32_t taddr, int r) {
  static_assert(C0 % 4 == 0, "whole boxes");
#pragma unroll
  for (int c = C0; c < C1; ++c) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int chunk = (c - C0) * 2 + i;
      const uint4 t = *reinterpret_cast<const uint4 *>(x + (chunk >> 3) * (128 * 128) + sw128_offset(r, chunk & 7));
      v[4 * i] = t.x;
      v[4 * i + 1] = t.y;
      v[4 * i + 2] = t.z;
      v[4 * i + 3] = t.w;
    }
    tmem_st_u8x(taddr + c * 8, v);
  }
  tmem_wait_st();
}

template <bool kBF16, bool TWO, class Role>
__device__ __forceinline__ void bwd_tc_tile(const BwdParams &p, const CUtensorMap *tm_x1,
                                            const CUtensorMap *tm_x2, const CUtensorMap *tm_y1,
                                            const CUtensorMap *tm_y2, const CUtensorMap *tm_o1,
                                            const CUtensorMap *tm_o2, const BwdTcSpan &span, int id,
                                            uint8_t *smem) {
  constexpr int BN = Role::BN, ST = Role::ST, N1 = Role::N1, N2 = Role::N2, NT = Role::NT, kH = Role::kH;
  constexpr bool OUT1 = Role::OUT1, OUT2 = Role::OUT2, KEYS = Role::KEYS;
  const AttnParams &a = p.a;
  uint8_t *sX1 = smem + Role::kX1Off, *sX2 = smem + Role::kX2Off;
  uint8_t *sY1 = smem + Role::kY1Off, *sY2 = smem + Role::kY2Off;
  float *terms = reinterpret_cast<float *>(smem + Role::kTermOff);
  BwdBlockInfo *info = reinterpret_cast<BwdBlockInfo *>(smem + Role::kInfoOff);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Role::kBarOff);
  uint64_t *y1_full = bars, *y1_empty = y1_full + N1;
  uint64_t *y2_full = y1_empty + N1, *y2_empty = y2_full + N2;
  uint64_t *s_full = y2_empty + N2;  // [ST] S_n complete (MMA -> softmax)
  uint64_t *p_full = s_full + ST;    // [ST] P_n in TMEM, or S_n read (softmax -> MMA)
  uint64_t *dp_full = p_full + ST;   // [ST] dP_n complete
  uint64_t *ds_full = dp_full + ST;  // [ST] dS_n in TMEM
  uint64_t *x_full = ds_full + ST;
  uint64_t *xt_full = x_full + 1;   // X copied to TMEM
  uint64_t *o_final = xt_full + 1;  // every product has completed
  uint64_t *fin_bar = o_final + 1;  // teardown drain of the MMA warp
  uint64_t *xh_empty = fin_bar + 1;  // X1 in two passes: the first one copied ...
  uint64_t *xh_full = xh_empty + 1;  // ... the second one there
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(xh_full + 1);
  constexpr int kProducerWarp = kBwdTcSoftmaxWarps, kMmaWarp = kBwdTcSoftmaxWarps + 1;
  constexpr bool XT = Role::XT1 || Role::XT2;
  // (through a shuffle, which tells the compiler that the roles' branches are
  // warp-uniform)
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  // --- work item.  Key tiles: tile fastest (a slab's query blocks stay in L2
  // while its tiles run), then split, then slab.  Query tiles, which run last and
  // read the smaller K and V: slab fastest, so that the grid ends with the tiles
  // of fewest blocks.  The tiles that visit most blocks come first in both ---
  int tile, split, bh, col_part = 0;
  if constexpr (Role::PARTED) {  // the parts of a tile next to each other
    const int parts = ((OUT1 ? a.Dqk : a.Dv) + Role::W1 - 1) / Role::W1;
    col_part = id % parts;
    id /= parts;
  }
  if (KEYS) {
    tile = id % span.tiles;
    id /= span.tiles;
    split = id % span.splits;
    bh = id / span.splits;
  } else {
    const int slabs = a.B * a.Hkv;
    bh = id % slabs;
    id /= slabs;
    split = id % span.splits;
    tile = span.tiles - 1 - id / span.splits;
  }
  const int x0 = tile * kBwdTcRows;
  const int xrows = KEYS ? a.S : a.R;

  // box `bx` of an X tile (128 rows of 64 columns) into the place of box bx - first
  auto load_x = [&](uint8_t *dst, const CUtensorMap *map, uint64_t *bar, int bx, int first) {
#pragma unroll
    for (int row = 0; row < 128; row += Role::kBoxRows)
      tma_load_3d(dst + (bx - first) * (128 * 128) + row * 128, map, bar, bx * 64, x0 + row, bh);
  };
  // The producer sets up the barriers and requests X while the MMA warp takes its
  // tensor memory.  (Launched as a programmatic dependent of the row-term kernel:
  // nothing before the wait touches global memory.)
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(tm_x1);
    tma_prefetch_desc(tm_y1);
    tma_prefetch_desc(tm_y2);
    for (int s = 0; s < N1; ++s) {
      mbar_init(&y1_full[s], 1);
      mbar_init(&y1_empty[s], 1 + (OUT1 ? 0 : kBwdTcSoftmaxWarps / ST));
    }
    for (int s = 0; s < N2; ++s) {
      mbar_init(&y2_full[s], 1);
      mbar_init(&y2_empty[s], 1);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], kBwdTcSoftmaxWarps / ST);
      mbar_init(&dp_full[s], 1);
      mbar_init(&ds_full[s], kBwdTcSoftmaxWarps / ST);
    }
    mbar_init(x_full, 1);
    mbar_init(xt_full, 4 * ((Role::XT1 ? 1 : 0) + (Role::XT2 ? 1 : 0)) + (XT ? 0 : 1));
    mbar_init(o_final, 1);
    mbar_init(fin_bar, 1);
    mbar_init(xh_empty, 4);
    mbar_init(xh_full, 1);
    fence_barrier_init();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    mbar_arrive_expect_tx(x_full, Role::kXFirst * (128 * 128) + Role::kX2Bytes);
#pragma unroll
    for (int bx = 0; bx < Role::kXFirst; ++bx) load_x(sX1, tm_x1, x_full, bx, 0);
    if constexpr (OUT1) {
#pragma unroll
      for (int bx = 0; bx < Role::kBoxes2; ++bx) load_x(sX2, tm_x2, x_full, bx, 0);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == kProducerWarp) {
    // ============================ TMA producer ============================
    if (lane == 0) {
      const float *nlse = p.nlse + (long long)bh * p.rpad;
      const float *ndelta = p.ndelta + (long long)bh * p.rpad;
      // the block list of this CTA: `count` visited blocks from `begin`
      int begin, count = 0x7fffffff, parts = 1;
      BwdBlocks<KEYS, BN> walk = bwd_blocks<KEYS, BN>(a, x0);
      if (span.splits > 1) {
        int total;
        begin = walk.seek(split * span.per, total);
        // (the last part takes what an estimate of `per` may have left)
        parts = min(span.splits, max(1, (total + span.per - 1) / span.per));
        count = total - split * span.per;
        if (split < span.splits - 1) count = min(span.per, count);
        if (split == 0) span.parts[bh * span.tiles + tile] = parts;
      } else {
        begin = walk.at_or_after(walk.first);
      }
      int pos_min = 0, pos_max = 0;  // query tiles: the tile's positions
      if constexpr (!KEYS) packed_positions(a, x0, min(kBwdTcRows, a.R - x0), pos_min, pos_max);
      bool x_twice = false;  // the second pass of X1 was requested
      if constexpr (Role::TWICE) {
        if (mbar_wait(xh_empty, 0, a.wd, kWdTmaEmpty)) {
          x_twice = true;
          mbar_arrive_expect_tx(xh_full, (Role::kBoxes1 - Role::kXFirst) * (128 * 128));
#pragma unroll
          for (int bx = Role::kXFirst; bx < Role::kBoxes1; ++bx) load_x(sX1, tm_x1, xh_full, bx, Role::kXFirst);
        }
      }
      // Y1 and Y2 are loaded as their slots come free, whichever is first: in one
      // fixed order a full Y2 ring would hold back the Y1 that the next scores
      // wait for.  u1 / u2: blocks loaded; behind the last block, one more Y1 slot
      // per score buffer says that there is none.
      int u1 = 0, u2 = 0, last = 0, b = begin < 0 || count <= 0 ? -1 : begin, idle = 0;
      bool alias_free = !Role::ALIAS;
      uint64_t since = 0;
      while (last < ST || u2 < u1) {
        bool moved = false;
        const int n = u1 + last, s1 = n % N1, nt = n % NT;
        if (!alias_free && n >= N1 - Role::kAliasSlots) alias_free = mbar_test(xt_full, 0);  // X1 has left the slot
        if (last < ST && n - u2 < NT && (alias_free || n < N1 - Role::kAliasSlots) &&
            mbar_test(&y1_empty[s1], ((uint32_t)(n / N1) & 1u) ^ 1u)) {
          moved = true;
          BwdBlockInfo in = {u1, parts, 0, 0};
          if (b < 0) {
            info[nt] = in;
            mbar_arrive(&y1_full[s1]);
            ++last;
          } else {
            in.row0 = b * BN;
            in.valid = 1;
            // Does any pair of the tile and the block need its own mask test?  (Rows
            // past the slab have nlse = -inf; keys past S matter as Y only: their dS
            // would meet zero-filled rows, but P of a zero score may overflow.)
            if constexpr (KEYS) {
              in.query0 = walk.query(in.row0);
              const bool wraps = in.query0 + BN > a.L;
              const int qmin = (wraps ? 0 : in.query0) + a.off, qmax = (wraps ? a.L : in.query0 + BN) - 1 + a.off;
              in.masked = a.causal && (min(x0 + kBwdTcRows, a.S) - 1 > qmin || (a.window > 0 && qmax - x0 >= a.window));
            } else {
              in.masked = in.row0 + BN > a.S || (a.causal && in.row0 + BN - 1 > pos_min) ||
                          (a.window > 0 && pos_max - in.row0 >= a.window);
            }
            info[nt] = in;
            mbar_arrive_expect_tx(&y1_full[s1], Role::kY1Bytes + (KEYS ? 2 * BN * 4 : 0));
            uint8_t *d1 = sY1 + s1 * Role::kY1Bytes;
#pragma unroll
            for (int bx = 0; bx < Role::kBoxes1; ++bx)
              tma_load_3d(d1 + bx * (BN * 128), tm_y1, &y1_full[s1], bx * 64, in.row0, bh);
            if constexpr (KEYS) {  // row0 + BN <= rpad
              bulk_load(terms + nt * 2 * BN, nlse + in.row0, BN * 4, &y1_full[s1]);
              bulk_load(terms + nt * 2 * BN + BN, ndelta + in.row0, BN * 4, &y1_full[s1]);
            }
            ++u1;
            b = u1 < count ? walk.at_or_after(b + 1) : -1;
          }
        }
        const int s2 = u2 % N2;
        if (u2 < u1 && (!Role::TWICE || alias_free) && mbar_test(&y2_empty[s2], ((uint32_t)(u2 / N2) & 1u) ^ 1u)) {
          moved = true;
          const int row0 = info[u2 % NT].row0;
          mbar_arrive_expect_tx(&y2_full[s2], Role::kY2Bytes);
          uint8_t *d2 = sY2 + s2 * Role::kY2Bytes;
          const int col0 = OUT1 ? 0 : col_part * Role::W2;  // (zeros past the head dim)
#pragma unroll
          for (int bx = 0; bx < Role::kY2Boxes; ++bx)
            tma_load_3d(d2 + bx * (BN * 128), tm_y2, &y2_full[s2], col0 + bx * 64, row0, bh);
          ++u2;
        }
        if (moved) {
          idle = 0;
        } else if ((++idle & 31) == 0) {  // bounded, as every wait
          const uint64_t now = globaltimer_ns();
          if (idle == 32) since = now;
          if (wd_tripped(a.wd)) break;
          if (now - since > a.wd.limit_ns) {
            wd_record(a.wd, kWdTmaEmpty);
            break;
          }
        }
      }
      // drain copies still landing (only ever waits after an abort)
      mbar_wait_drain(x_full, 0, a.wd);
      if (x_twice) mbar_wait_drain(xh_full, 0, a.wd);
      for (int v = max(u1 + last - N1, 0); v < u1; ++v)  // (not the slots used once more)
        mbar_wait_drain(&y1_full[v % N1], (uint32_t)(v / N1) & 1u, a.wd);
      for (int v = max(u2 - N2, 0); v < u2; ++v)
        mbar_wait_drain(&y2_full[v % N2], (uint32_t)(v / N2) & 1u, a.wd);
    }
  } else if (warp == kMmaWarp) {
    // ========== MMA issuer: the whole warp, converged (see elect_leader) ==========
    const uint32_t leader = elect_leader();
    constexpr uint32_t kIdescS = umma_idesc_f16(kBF16, 128, BN, false, false);
    // (the last part of a parted tile may be narrower: D1 = D2 there)
    const int cols = Role::PARTED ? min(Role::W1, Role::D1 - col_part * Role::W1) : 0;
    const uint32_t idesc1 = umma_idesc_f16(kBF16, 128, Role::PARTED ? cols : Role::D1, false, true);
    const uint32_t idesc2 = umma_idesc_f16(kBF16, 128, Role::PARTED ? cols : Role::D2, false, true);
    const uint32_t y1_cols = Role::PARTED ? col_part * (Role::W1 / 64) * (BN * 128) : 0;
    const uint32_t x1 = smem_u32(sX1), x2 = smem_u32(sX2), y1 = smem_u32(sY1), y2 = smem_u32(sY2);
    auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t code) -> bool {
      return mbar_wait_warp(bar, parity, a.wd, code);
    };
    // first products: 128 x BN scores over the head dim; Y K-major, X K-major in
    // shared memory or in TMEM
    auto first = [&](auto in_tmem, auto dim, uint32_t x, uint32_t y, uint32_t col) {
      tc_fence_after();
      const uint64_t a0 = umma_desc_sw128(x, 16, 1024);
      const uint64_t b0 = umma_desc_sw128(y, 16, 1024);
#pragma unroll
      for (int ks = 0; ks < decltype(dim)::value / 16; ++ks) {
        const uint64_t bd = umma_desc_advance(b0, (ks >> 2) * (BN * 128) + (ks & 3) * 32);
        if constexpr (decltype(in_tmem)::value)
          tc_mma_ts_warp(leader, tmem + col, tmem + x + ks * 8, bd, kIdescS, ks > 0 ? 1u : 0u);
        else
          tc_mma_ss_warp(leader, tmem + col, umma_desc_advance(a0, (ks >> 2) * (128 * 128) + (ks & 3) * 32), bd, kIdescS,
                         ks > 0 ? 1u : 0u);
      }
    };
    // second products: weights from TMEM (each part of the columns packed at the
    // start of its own columns) times the same Y block, MN-major
    auto second = [&](uint32_t wcol, uint32_t y, uint32_t out, uint32_t idesc, bool fresh) {
      tc_fence_after();
      const uint64_t b0 = umma_desc_sw128_mn(y, BN * 128, 1024);
#pragma unroll
      for (int term = 0; term < (TWO ? 2 : 1); ++term)
#pragma unroll
        for (int ks = 0; ks < BN / 16; ++ks) {
          const int part = ks / (kH / 16);
          tc_mma_ts_warp(leader, tmem + out, tmem + wcol + part * kH + term * (kH / 2) + (ks - part * (kH / 16)) * 8,
                         umma_desc_advance(b0, ks * 2048), idesc, fresh && ks == 0 && term == 0 ? 0u : 1u);
        }
    };
    bool ok = wait(x_full, 0, kWdTmaFull);
    if (XT) ok = ok && wait(xt_full, 0, kWdSoftmax);
    // First products of block i (into score buffer st): false behind the last.
    // Slots and parities run along as counters: what is computed between two
    // products, and the latency of a wait, drains the tensor pipe, which holds
    // only about four issued MMAs.
    struct Ring {
      uint32_t slot, parity;
      __device__ __forceinline__ void step(uint32_t n) {
        if (++slot == n) {
          slot = 0;
          parity ^= 1u;
        }
      }
    };
    Ring r1 = {0, 0}, r2 = {0, 0}, rt = {0, 0};  // Y1, Y2 and note of the next block to start
    auto start_s = [&](uint32_t st) {
      first(std::bool_constant<Role::XT1>(), std::integral_constant<int, Role::D1>(), Role::XT1 ? Role::kX1Col : x1,
            y1 + r1.slot * Role::kY1Bytes, st * Role::kStageCols);
      tc_commit_warp(leader, &s_full[st]);
      if constexpr (!OUT1) tc_commit_warp(leader, &y1_empty[r1.slot]);
    };
    auto start_dp = [&](uint32_t st, uint32_t slot) {
      first(std::bool_constant<Role::XT2>(), std::integral_constant<int, Role::D2>(), Role::XT2 ? Role::kX2Col : x2,
            y2 + slot * Role::kY2Bytes, st * Role::kStageCols + BN);
      tc_commit_warp(leader, &dp_full[st]);
      if constexpr (!OUT2) tc_commit_warp(leader, &y2_empty[slot]);
    };
    int started = 0;
    bool more = ok;
    for (uint32_t st = 0; st < ST && more; ++st) {
      if (!(ok = wait(&y1_full[r1.slot], r1.parity, kWdTmaFull))) break;
      if (!(more = __any_sync(0xffffffffu, info[rt.slot].valid))) break;
      start_s(st);
      if constexpr (OUT1) {
        if (!(ok = wait(&y2_full[r2.slot], r2.parity, kWdTmaFull))) break;
        start_dp(st, r2.slot);
      }
      ++started;
      r1.step(N1);
      r2.step(N2);
      rt.step(NT);
    }
    // step n: second products of block n, first ones of block n + ST
    Ring c1 = {0, 0}, c2 = {0, 0}, cs = {0, 0};  // Y1, Y2 and score buffer of block n
    int n = 0;
    bool ready = false;  // P_n (and Y1 of block n + ST) seen complete under the last product
    while (ok && n < started) {
      if (!__all_sync(0xffffffffu, ready)) {
        ok = more ? mbar_wait_warp2(&p_full[cs.slot], cs.parity, kWdSoftmax, &y1_full[r1.slot], r1.parity, kWdTmaFull, a.wd)
                  : wait(&p_full[cs.slot], cs.parity, kWdSoftmax);
        if (!ok) break;
      }
      if constexpr (OUT2) {
        if constexpr (!OUT1)
          if (!(ok = wait(&y2_full[c2.slot], c2.parity, kWdTmaFull))) break;
        second(cs.slot * Role::kStageCols, y2 + c2.slot * Role::kY2Bytes, Role::kOut2Col, idesc2, n == 0);
        tc_commit_warp(leader, &y2_empty[c2.slot]);
      }
      bool ds_ready = false;
      if (more) {
        if constexpr (OUT1)
          ds_ready = mbar_test(&ds_full[cs.slot], cs.parity) && mbar_test(&y2_full[r2.slot], r2.parity);
        more = __any_sync(0xffffffffu, info[rt.slot].valid);
      }
      if (more) {
        start_s(cs.slot);
        ++started;
        r1.step(N1);
        rt.step(NT);
      }
      const uint32_t st = cs.slot, y2_next = r2.slot;
      if constexpr (OUT1) {
        if (!__all_sync(0xffffffffu, ds_ready)) {
          ok = more ? mbar_wait_warp2(&ds_full[st], cs.parity, kWdSoftmax, &y2_full[y2_next], r2.parity, kWdTmaFull, a.wd)
                    : wait(&ds_full[st], cs.parity, kWdSoftmax);
          if (!ok) break;
        }
        second(st * Role::kStageCols + BN, y1 + c1.slot * Role::kY1Bytes + y1_cols, Role::kOut1Col, idesc1, n == 0);
        tc_commit_warp(leader, &y1_empty[c1.slot]);
      }
      ++n;
      c1.step(N1);
      c2.step(N2);
      cs.step(ST);
      if (more) r2.step(N2);
      ready = more && mbar_test(&p_full[cs.slot], cs.parity) && mbar_test(&y1_full[r1.slot], r1.parity);
      if constexpr (OUT1)
        if (more) start_dp(st, y2_next);
    }
    if (ok && n > 0) tc_commit_warp(leader, o_final);
    // all MMAs of this CTA complete before TMEM is released
    tc_commit_warp(leader, fin_bar);
    mbar_wait_drain(fin_bar, 0, a.wd);
  } else {
    // ============ softmax warps: X rows 32 (w % 4) .. +31 ============
    const int group = warp >> 2;
    const int part = Role::kParts == 2 ? group : 0;  // columns [part kH, +kH) of every block
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = a.scale_log2;
    const float gain = bwd_gain<kBF16>(p, bh);
    // query tiles: this row's terms and position
    float x_nlse = 0.f, x_ndelta = 0.f;
    int pos = 0;
    if constexpr (!KEYS) {
      x_nlse = p.nlse[(long long)bh * p.rpad + x0 + r];  // x0 + 127 < rpad
      x_ndelta = p.ndelta[(long long)bh * p.rpad + x0 + r];
      pos = (x0 + r) % a.L + a.off;
    }
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
      // (the waiting loop in line here: with the MMA warp's it took head dims 256
      // 5 % longer)
      bool w = __all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity));
      if (!w) w = __all_sync(0xffffffffu, mbar_wait(bar, parity, a.wd, kWdMma));
      tc_fence_after();
      return w;
    };
    auto arrive = [&](uint64_t *bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    if constexpr (XT) {
      ok = wait(x_full, 0);
      if (Role::XT1 && group == 0) {
        constexpr int kC1 = Role::D1 / 16, kFirst = Role::TWICE ? Role::kXFirst * 4 : kC1;
        if (ok) bwd_x_to_tmem<0, kFirst>(sX1, lanes + Role::kX1Col, r);
        if constexpr (Role::TWICE) {
          arrive(xh_empty);
          ok = ok && wait(xh_full, 0);
          if (ok) bwd_x_to_tmem<kFirst, kC1>(sX1, lanes + Role::kX1Col, r);
        }
        arrive(xt_full);
      }
      if (Role::XT2 && group == 1) {
        if (ok) bwd_x_to_tmem<0, Role::D2 / 16>(sX2, lanes + Role::kX2Col, r);
        arrive(xt_full);
      }
    }
    int blocks = 0, parts = 1;  // of this CTA; of the tile
    for (uint32_t n = ST == 2 ? group : 0; ok; n += ST) {
      constexpr int kStage = Role::kStageCols;
      const uint32_t st = n % ST, ph = (n / ST) & 1u, slot = n % N1, nt = n % NT;
      const uint32_t t_s = lanes + st * kStage + part * kH, t_dp = t_s + BN;
      const float *t_nlse = terms + nt * 2 * BN + part * kH;
      const float *t_ndelta = t_nlse + BN;
      // what the block is, and (key tiles) the row terms came with Y1
      if (!(ok = wait(&y1_full[slot], (n / N1) & 1u))) break;
      const BwdBlockInfo in = info[nt];
      if (!in.valid) {
        blocks = in.row0;
        parts = in.query0;
        break;
      }
      // Without out1, Y1_n's slot waits for no weights of block n.  It must not be
      // filled again before this warp has seen it full: two phases later the
      // barrier's parity reads "not yet" again.
      if constexpr (!OUT1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&y1_empty[slot]);
      }
      // Rows that take no part, among this warp's columns, as bits: masked, since their
      // scores and dP may have overflowed.  (Their Q and dO still enter the second
      // products, with weights of 0.  Zeros in their place, written here or by a warp of
      // its own, took head dims 192/128 5 to 12 % longer, with such rows or without.)
      constexpr int kWords = (kH + 31) / 32;
      uint32_t gone[kWords] = {};
      bool dead = false;
      if constexpr (KEYS) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          gone[j] = __ballot_sync(0xffffffffu, 32 * j + lane < kH && t_nlse[32 * j + lane] == -INFINITY);
          dead |= gone[j] != 0;
        }
      }
      if (!(ok = wait(&s_full[st], ph))) break;
      // ---- phase E ----
      float w[kH];
      tmem_ldn<kH>(t_s, w);
      tmem_wait_ld();
      if constexpr (!OUT2) arrive(&p_full[st]);  // S_n is free
      const float2 c2 = make_float2(c, c);
      // (all on the MUFU: with part of them on the FMA pipe's polynomial head dim 192
      // took 6 to 8 % longer, 64 and 72 1 to 4 %, the others the same to 2 %)
#pragma unroll
      for (int i = 0; i < kH; i += 4) {
        float4 nl = make_float4(x_nlse, x_nlse, x_nlse, x_nlse);
        if constexpr (KEYS) nl = *reinterpret_cast<const float4 *>(t_nlse + i);
        const float2 t = fma2(make_float2(w[i], w[i + 1]), c2, make_float2(nl.x, nl.y));
        const float2 u = fma2(make_float2(w[i + 2], w[i + 3]), c2, make_float2(nl.z, nl.w));
        w[i] = fast_exp2(t.x);
        w[i + 1] = fast_exp2(t.y);
        w[i + 2] = fast_exp2(u.x);
        w[i + 3] = fast_exp2(u.y);
      }
      if (in.masked || dead) {
        // visible columns of this thread as bits
        uint32_t seen[kWords] = {};
        auto see = [&](int from, int to) {  // columns [from, to)
#pragma unroll
          for (int j = 0; j < kWords; ++j) {
            const int lo = max(from - 32 * j, 0), hi = min(to - 32 * j, 32);
            if (hi > lo) seen[j] |= (0xffffffffu >> (32 - (hi - lo))) << lo;
          }
        };
        if constexpr (KEYS) {
          // one interval of queries per head that the block touches
          const int q_lo = a.causal ? x0 + r - a.off : 0;
          const int q_hi = a.window > 0 ? (int)min((long long)a.L, (long long)q_lo + a.window) : a.L;
#pragma unroll 1
          for (int col = -in.query0 - part * kH; col < kH; col += a.L) see(col + max(q_lo, 0), col + q_hi);
#pragma unroll
          for (int j = 0; j < kWords; ++j) seen[j] &= ~gone[j];
        } else {
          const VisibleRange vis = visible_range(a, pos, in.row0 + part * kH);
          see(vis.first, (int)min((long long)kH, (long long)vis.first + vis.span));
        }
#pragma unroll
        for (int e = 0; e < kH; ++e)
          if (!((seen[e / 32] >> (e % 32)) & 1)) w[e] = 0.f;
      }
      if constexpr (OUT2) {
#pragma unroll
        for (int i = 0; i < kH; i += 16) {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) pk[e] = pack2<kBF16>(w[i + 2 * e], w[i + 2 * e + 1]);
          tmem_st_u8x(t_s + i / 2, pk);
          if constexpr (TWO) {
#pragma unroll
            for (int e = 0; e < 8; ++e) pk[e] = rest2<kBF16>(w[i + 2 * e], w[i + 2 * e + 1], pk[e]);
            tmem_st_u8x(t_s + kH / 2 + i / 2, pk);
          }
        }
        tmem_wait_st();
        arrive(&p_full[st]);
      }
      // ---- phase F ----
      if constexpr (OUT1) {
        if (!(ok = wait(&dp_full[st], ph))) break;
        // columns at a time (two terms write past the columns they come from)
        constexpr int kC = TWO ? kH : kH % 48 == 0 ? 48 : kH % 32 == 0 ? 32 : 16;
#pragma unroll
        for (int j0 = 0; j0 < kH; j0 += kC) {
          float d[kC];
          tmem_ldn<kC>(t_dp + j0, d);
          tmem_wait_ld();
          if (in.masked || dead) {  // a masked pair's dP may be anything, also not a number
#pragma unroll
            for (int e = 0; e < kC; ++e)
              if (w[j0 + e] == 0.f) d[e] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < kC; j += 16) {
            uint32_t pk[8], lo[8];
#pragma unroll
            for (int i = j; i < j + 16; i += 4) {
              float4 nd = make_float4(x_ndelta, x_ndelta, x_ndelta, x_ndelta);
              if constexpr (KEYS) nd = *reinterpret_cast<const float4 *>(t_ndelta + j0 + i);
#pragma unroll
              for (int e = i; e < i + 4; e += 2) {
                float2 t = add2(make_float2(d[e], d[e + 1]), e == i ? make_float2(nd.x, nd.y) : make_float2(nd.z, nd.w));
                if constexpr (!kBF16) t = mul2(t, make_float2(gain, gain));
                t = mul2(t, make_float2(w[j0 + e], w[j0 + e + 1]));
                pk[(e - j) / 2] = pack2<kBF16>(t.x, t.y);
                if constexpr (TWO) lo[(e - j) / 2] = rest2<kBF16>(t.x, t.y, pk[(e - j) / 2]);
              }
            }
            tmem_st_u8x(t_dp + (j0 + j) / 2, pk);
            if constexpr (TWO) tmem_st_u8x(t_dp + kH / 2 + (j0 + j) / 2, lo);
          }
        }
        tmem_wait_st();
        arrive(&ds_full[st]);
      }
    }

    // ------------------------------ epilogue ------------------------------
    const bool have = ok && blocks > 0;
    // (without a block, X may still be landing where the zeros are staged)
    ok = wait(have ? o_final : x_full, 0) && ok;
    const bool have_o = have && ok;
    // a row that takes no part has no dQ, whatever its lane of the sums holds
    const bool none = !KEYS && x_nlse == -INFINITY;
    const int nvalid = min(kBwdTcRows, xrows - x0);
    auto finish = [&](int col, int d, int first, int width, float factor, uint8_t *stage, float *out_part) {
      const int chunks = (Role::PARTED ? min(width, d - first) : width) / 16;
      for (int c16 = group * chunks / 2; c16 < (group + 1) * chunks / 2; ++c16) {
        float o[16];
        if (have_o) {
          tmem_ld16(lanes + col + c16 * 16, o);
          tmem_wait_ld();
        }
        if (!have_o || none) {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0.f;
        }
        if (out_part == nullptr) {
          uint32_t w8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w8[e] = pack2<kBF16>(o[2 * e] * factor, o[2 * e + 1] * factor);
          stage_16bit_x16(stage, r, c16, w8);
        } else if (r < nvalid && split < parts) {  // fp32 sums, [split][slab][row][d]
          float4 *dst = reinterpret_cast<float4 *>(
              out_part + ((((long long)split * a.B * a.Hkv + bh) * xrows + x0 + r) * d + first + c16 * 16));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
    };
    const int first1 = col_part * Role::W1, first2 = col_part * Role::W2;  // gradient columns
    const bool split_out = parts > 1;
    if constexpr (OUT1)
      finish(Role::kOut1Col, Role::D1, first1, Role::W1, bwd_ds_factor<kBF16>(p, gain), smem + Role::kStage1Off, split_out ? span.part1 : nullptr);
    if constexpr (OUT2)
      finish(Role::kOut2Col, Role::D2, first2, Role::W2, bwd_dv_factor<kBF16>(), smem + Role::kStage2Off, split_out ? span.part2 : nullptr);
    if (!split_out && split == 0) {
      fence_proxy_async_smem();
      asm volatile("bar.sync 1, %0;" ::"n"(kBwdTcSoftmaxWarps * 32) : "memory");
      // rows past the slab and columns past the head dim are clipped
      if (warp == 0 && lane == 0) {
        if constexpr (OUT1)
          for (int bx = 0; bx * 64 < Role::W1 && first1 + bx * 64 < a.Dqk; ++bx)
            tma_store_3d(tm_o1, smem + Role::kStage1Off + bx * (128 * 128), first1 + bx * 64, x0, bh);
        if constexpr (OUT2)
          for (int bx = 0; bx * 64 < Role::W2 && first2 + bx * 64 < a.Dv; ++bx)
            tma_store_3d(tm_o2, smem + Role::kStage2Off + bx * (128 * 128), first2 + bx * 64, x0, bh);
        bulk_commit_group();
        bulk_wait_group_read0();  // the staging may go; the grid's end completes the writes
      }
    }
  }

  // ------------------------------ teardown ------------------------------
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr uint32_t bwd_max(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The kinds of tile of one head-dim pair: TMEM columns
//   pair      key tiles                          query tiles
//   64/64     2 x 192 + 64 + 64                  2 x 192 + 64  + X 32 + 32
//   80/80     2 x 160 + 80 + 80                  2 x 160 + 80  + X 40 + 40
//   128/128   2 x 128 + 128 + 128                2 x 128 + 128 + X 64 + 64
//   192/128   2 x  96 + 192 + 128                2 x 128 + 192 +   X2 64
//   192/192   128 + 192 + X 96 + 96 (dK)         128 + 192 + X 96 + 96
//             2 x  64 + 192 + X1 96 (dV)
//   256/256   128 + 256 + X1 128    (dK)         128 + 256 + X1 128
//             2 x  64 + 256 + X1 128 (dV)
//   512/512   64 + 192 + X1 256     (dK)         64 + 192 + X1 256, 32-row blocks,
//             2 x  32 + 192 + X1 256 (dV)        192 gradient columns per CTA
template <int DQK, int DV>
struct BwdTcRoles;
template <>
struct BwdTcRoles<64, 64> {
  using Key = BwdTcRole<64, 64, 96, 2, 4, 4, true, true, true, false, false>;
  using Query = BwdTcRole<64, 64, 96, 2, 4, 4, false, true, false, true, true>;
  using KeyV = void;
  // (more than half of an SM's, whatever the tiles need: a CTA takes all of TMEM)
  static constexpr uint32_t kSmem = bwd_max(120 * 1024, bwd_max(Key::kSmemBytes, Query::kSmemBytes));
};
template <>
struct BwdTcRoles<80, 80> {
  using Key = BwdTcRole<80, 80, 80, 2, 4, 4, true, true, true, false, false>;
  using Query = BwdTcRole<80, 80, 80, 2, 4, 4, false, true, false, true, true>;
  using KeyV = void;
  static constexpr uint32_t kSmem = bwd_max(120 * 1024, bwd_max(Key::kSmemBytes, Query::kSmemBytes));
};
template <>
struct BwdTcRoles<128, 128> {
  using Key = BwdTcRole<128, 128, 64, 2, 4, 4, true, true, true, false, false>;
  using Query = BwdTcRole<128, 128, 64, 2, 4, 4, false, true, false, true, true>;
  using KeyV = void;
  static constexpr uint32_t kSmem = bwd_max(Key::kSmemBytes, Query::kSmemBytes);
};
template <>
struct BwdTcRoles<192, 128> {
  using Key = BwdTcRole<192, 128, 48, 2, 4, 4, true, true, true, false, false>;
  using Query = BwdTcRole<192, 128, 64, 2, 4, 3, false, true, false, false, true>;
  using KeyV = void;
  static constexpr uint32_t kSmem = bwd_max(Key::kSmemBytes, Query::kSmemBytes);
};
template <>
struct BwdTcRoles<192, 192> {
  using Key = BwdTcRole<192, 192, 64, 1, 3, 2, true, true, false, true, true>;
  using Query = BwdTcRole<192, 192, 64, 1, 3, 2, false, true, false, true, true>;
  using KeyV = BwdTcRole<192, 192, 64, 2, 3, 3, true, false, true, true, false>;
  static constexpr uint32_t kSmem = bwd_max(KeyV::kSmemBytes, bwd_max(Key::kSmemBytes, Query::kSmemBytes));
};
template <>
struct BwdTcRoles<256, 256> {
  using Key = BwdTcRole<256, 256, 64, 1, 3, 2, true, true, false, true, false, true>;
  using Query = BwdTcRole<256, 256, 64, 1, 3, 2, false, true, false, true, false, true>;
  using KeyV = BwdTcRole<256, 256, 64, 2, 3, 2, true, false, true, true, false>;
  static constexpr uint32_t kSmem = bwd_max(KeyV::kSmemBytes, bwd_max(Key::kSmemBytes, Query::kSmemBytes));
};

template <>
struct BwdTcRoles<512, 512> {
  using Key = BwdTcRole<512, 512, 32, 1, 2, 1, true, true, false, true, false, true, 192>;
  using Query = BwdTcRole<512, 512, 32, 1, 2, 1, false, true, false, true, false, true, 192>;
  using KeyV = BwdTcRole<512, 512, 32, 2, 5, 4, true, false, true, true, false, true, 192>;
  static constexpr uint32_t kSmem = bwd_max(KeyV::kSmemBytes, bwd_max(Key::kSmemBytes, Query::kSmemBytes));
};

// CTAs that share a tile, one per W gradient columns.
template <class Role>
__host__ __device__ constexpr int bwd_col_parts(int d) {
  return Role::PARTED ? (d + Role::W1 - 1) / Role::W1 : 1;
}

template <bool kBF16, bool TWO, int DQK, int DV>
__global__ void __launch_bounds__(kBwdTcThreads, 1)
    bwd_tc_kernel(const __grid_constant__ BwdTcMaps tm, const __grid_constant__ BwdParams p,
                  const __grid_constant__ BwdTcSpan keys, const __grid_constant__ BwdTcSpan rows,
                  const int rows_first) {
  using Roles = BwdTcRoles<DQK, DV>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // The 128-byte swizzle atoms need 1024-byte aligned tiles; see tc.cuh.
  if ((smem_u32(smem_raw) & 1023u) != 0u) {
    if (threadIdx.x == 0) wd_record(p.a.wd, kWdSmemAlign);
    return;
  }
  const int slabs = p.a.B * p.a.Hkv;
  using Key = typename Roles::Key;
  using KeyV = typename Roles::KeyV;
  using Query = typename Roles::Query;
  const int key_tiles = slabs * keys.tiles * keys.splits;
  const int key_ctas = key_tiles * bwd_col_parts<Key>(p.a.Dqk);
  const int row_ctas = slabs * rows.tiles * rows.splits * bwd_col_parts<Query>(p.a.Dqk);
  // the kind with the longest block lists first
  int id = blockIdx.x;
  if (rows_first) id = id < row_ctas ? (int)gridDim.x - row_ctas + id : id - row_ctas;
  if (id < key_ctas) {
    bwd_tc_tile<kBF16, TWO, Key>(p, &tm.k, &tm.v, &tm.qb, &tm.doutb, &tm.dk, &tm.dv, keys, id, smem_raw);
    return;
  }
  id -= key_ctas;
  if constexpr (!std::is_void_v<KeyV>) {
    const int v_ctas = key_tiles * bwd_col_parts<KeyV>(p.a.Dv);
    if (id < v_ctas) {
      bwd_tc_tile<kBF16, TWO, KeyV>(p, &tm.k, &tm.v, &tm.qb, &tm.doutb, &tm.dk, &tm.dv, keys, id, smem_raw);
      return;
    }
    id -= v_ctas;
  }
  bwd_tc_tile<kBF16, TWO, Query>(p, &tm.q, &tm.dout, &tm.kb, &tm.vb, &tm.dq, &tm.dq, rows, id, smem_raw);
}

// Sum of a tile's parts, where it has several, times the factor, rounded once: X rows of all
// slabs, d columns (a multiple of 8; the tiles' rows are dpad wide).
template <bool kBF16>
__global__ void __launch_bounds__(256)
    bwd_join_kernel(const BwdParams p, const float *__restrict__ part, uint16_t *__restrict__ out,
                    const int *__restrict__ parts, int tiles, long long rows, int rows_per_slab, int d,
                    int dpad, int is_dv) {
  const int per_row = d / 4;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= rows * per_row) return;
  const long long row = id / per_row;
  const int c = (int)(id - row * per_row) * 4;
  const int slab = (int)(row / rows_per_slab);
  const int n = parts[slab * tiles + (int)(row - (long long)slab * rows_per_slab) / kBwdTcRows];
  if (n <= 1) return;  // written by its one part
  const float4 *src = reinterpret_cast<const float4 *>(part + row * dpad + c);
  const long long stride = rows * dpad / 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float4 x = __ldcs(src + i * stride);
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  const float f = is_dv ? bwd_dv_factor<kBF16>()
                        : bwd_ds_factor<kBF16>(p, bwd_gain<kBF16>(p, slab));
  uint2 w;
  w.x = pack2<kBF16>(s.x * f, s.y * f);
  w.y = pack2<kBF16>(s.z * f, s.w * f);
  *reinterpret_cast<uint2 *>(out + row * d + c) = w;
}

}  // namespace sdpa
