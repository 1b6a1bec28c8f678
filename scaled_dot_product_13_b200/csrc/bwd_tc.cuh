// Backward pass on tcgen05 tensor cores with TMEM accumulators (sm_100a),
// head dims up to 256.
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
//   0-7  softmax: warps w and w + 4 share TMEM lanes 32 (w % 4) .. +31 and take
//        one half of a block's columns each.  Phase E: P = 2^(S c + nlse);
//        phase F: dS = P (dP + ndelta) gain, with P kept in registers.  A half
//        writes its packed values over its own columns only, so the two warps
//        of a lane need no exchange.
//   8    TMA producer (X once, then Y1 and Y2 blocks through two rings, the row
//        terms of a query block with its Y1)
//   9    MMA issuer (the whole warp, one elected lane), in the order
//            out2_j, S_{j+1}   after P_j   (runs under phase F of block j)
//            out1_j, dP_{j+1}  after dS_j  (runs under phase E of block j+1)
//        so the tensor pipe works on one pair while the softmax warps work on
//        the other, with one S and one dP buffer: one thread's MMAs run in
//        issue order, so S_{j+1} may overwrite P_j once out2_j is issued.
//
// TMEM (512 columns): S [0, BN), dP [BN, 2 BN), out1 [2 BN, ..), out2 behind.
// Head dims 256 leave no room for dK and dV together: those take a CTA each.
#pragma once

#include <type_traits>

#include "bwd_params.cuh"

// How many of every four exponential pairs go to the FMA-pipe polynomial
// instead of the MUFU unit (0-4).  Build-time knob for measurement.
#ifndef SDPA_BWD_POLY_OF4
#define SDPA_BWD_POLY_OF4 0
#endif

namespace sdpa {

constexpr int kBwdTcRows = 128;
constexpr int kBwdTcSoftmaxWarps = 8;
constexpr int kBwdTcThreads = (kBwdTcSoftmaxWarps + 2) * 32;

// One kind of tile.  N1 / N2: ring slots of Y1 and Y2.
template <int D1_, int D2_, int BN_, int N1_, int N2_, bool KEYS_, bool OUT1_, bool OUT2_>
struct BwdTcRole {
  static constexpr int D1 = D1_, D2 = D2_, BN = BN_, N1 = N1_, N2 = N2_;
  static constexpr bool KEYS = KEYS_, OUT1 = OUT1_, OUT2 = OUT2_;
  static constexpr int kBoxes1 = (D1 + 63) / 64, kBoxes2 = (D2 + 63) / 64;
  static constexpr uint32_t kX1Bytes = kBoxes1 * 128 * 128;
  static constexpr uint32_t kX2Bytes = OUT1 ? kBoxes2 * 128 * 128 : 0;  // dP only
  static constexpr uint32_t kY1Bytes = kBoxes1 * BN * 128;
  static constexpr uint32_t kY2Bytes = kBoxes2 * BN * 128;
  static constexpr uint32_t kX2Off = kX1Bytes;
  static constexpr uint32_t kY1Off = kX2Off + kX2Bytes;
  static constexpr uint32_t kY2Off = kY1Off + N1 * kY1Bytes;
  static constexpr uint32_t kTermOff = kY2Off + N2 * kY2Bytes;  // [N1][2][BN] row terms
  static constexpr uint32_t kTermBytes = KEYS ? N1 * 2 * BN * 4 : 0;
  static constexpr uint32_t kBarOff = kTermOff + kTermBytes;
  static constexpr int kNumBars = 2 * N1 + 2 * N2 + 7;
  static constexpr uint32_t kSmemBytes = kBarOff + kNumBars * 8 + 16;
  static constexpr int kOut1Col = OUT1 ? 2 * BN : BN;  // without out1 there is no dP
  static constexpr int kOut2Col = kOut1Col + (OUT1 ? D1 : 0);
  static constexpr int kH = BN / 2;  // columns per softmax thread
  // staging of the finished tile: out1 in X1's memory; out2 in X2's, or in X1's
  // where it is the only output
  static constexpr uint32_t kStage2Off = OUT1 ? kX2Off : 0;
  static_assert(OUT1 || OUT2, "");
  static_assert(KEYS || (OUT1 && !OUT2), "query tiles give dQ");
  static_assert(kOut2Col + (OUT2 ? D2 : 0) <= 512, "TMEM columns");
  static_assert(N1 >= 2 || !OUT1, "Y1_j is held while S_{j+1} needs the next");
  static_assert(OUT1 || kBoxes2 <= kBoxes1, "out2's staging");
  static_assert(kH % 16 == 0 && BN % 16 == 0, "");
  static_assert(kSmemBytes <= 232448, "shared memory");
};

struct BwdTcMaps {
  CUtensorMap kx, vx, qy, doy;  // key tiles: X boxes of 128 rows, Y boxes of BN rows
  CUtensorMap qx, dox, ky, vy;  // query tiles
  CUtensorMap dq, dk, dv;       // 128-row boxes
};

// Tiles of one kind within the grid.
struct BwdTcSpan {
  int tiles, splits;  // per slab: row tiles, and parts of each tile's block list
  float *part1, *part2;  // splits > 1: fp32 sums [split][slab][X rows][D]
};

// Untiled copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The blocks of BN Y rows that a tile visits, in rising order.  Query tiles
// see one range of keys.  Key tiles see, of each head's L packed rows, the same
// range of queries [i_lo, i_hi); a block may span two heads.
struct BwdBlocks {
  bool keys;
  int bn, first, end;        // block range
  int L, R, i_lo, i_hi;

  // smallest visited block >= b, or -1
  __device__ __forceinline__ int at_or_after(int b) const {
    if (b >= end) return -1;
    if (!keys || i_hi - i_lo == L) return b;
    for (;;) {
      const int r0 = b * bn;
      if (r0 >= R) return -1;
      const int j = r0 / L;
      int lo = j * L + i_lo;
      if (r0 >= j * L + i_hi) lo += L;  // behind this head's visible rows
      if (lo >= R) return -1;
      if (r0 + bn > lo) return b;
      b = lo / bn;
    }
  }
};

template <class Role>
__device__ __forceinline__ BwdBlocks bwd_blocks(const AttnParams &a, int x0) {
  BwdBlocks w;
  w.keys = Role::KEYS;
  w.bn = Role::BN;
  w.L = a.L;
  w.R = a.R;
  w.i_lo = 0;
  w.i_hi = a.L;
  w.first = 0;
  if constexpr (Role::KEYS) {
    const int key_max = min(x0 + kBwdTcRows, a.S) - 1;
    if (a.causal) w.i_lo = min(max(x0 - a.off, 0), a.L);
    if (a.window > 0) w.i_hi = (int)max(0LL, min((long long)a.L, (long long)key_max + a.window - a.off));
    w.end = w.i_lo < w.i_hi ? (a.R + Role::BN - 1) / Role::BN : 0;
  } else {
    int pos_min, pos_max;
    packed_positions(a, x0, min(kBwdTcRows, a.R - x0), pos_min, pos_max);
    const int kend = a.causal ? min(a.S, pos_max + 1) : a.S;
    const int kbeg = a.window > 0 ? max(0, pos_min - a.window + 1) : 0;
    w.first = kbeg / Role::BN;
    w.end = kend > kbeg ? (kend + Role::BN - 1) / Role::BN : w.first;
  }
  return w;
}

// Does any pair of the tile and the block need its own mask test?  (Rows past
// the slab have nlse = -inf, keys past S only matter as Y: their dS would meet
// zero-filled rows, but P of a zero score may overflow.)
template <class Role>
__device__ __forceinline__ bool bwd_needs_mask(const AttnParams &a, int x0, int blk) {
  int pos_min, pos_max, key_min, key_max;
  if constexpr (Role::KEYS) {
    const int r0 = blk * Role::BN;
    packed_positions(a, r0, min(Role::BN, a.R - r0), pos_min, pos_max);
    key_min = x0;
    key_max = min(x0 + kBwdTcRows, a.S) - 1;
  } else {
    packed_positions(a, x0, min(kBwdTcRows, a.R - x0), pos_min, pos_max);
    key_min = blk * Role::BN;
    key_max = key_min + Role::BN - 1;
    if (key_max >= a.S) return true;
  }
  return (a.causal && key_max > pos_min) || (a.window > 0 && pos_max - key_min >= a.window);
}

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

template <bool kBF16, class Role>
__device__ __forceinline__ void bwd_tc_tile(const BwdParams &p, const CUtensorMap *tm_x1,
                                            const CUtensorMap *tm_x2, const CUtensorMap *tm_y1,
                                            const CUtensorMap *tm_y2, const CUtensorMap *tm_o1,
                                            const CUtensorMap *tm_o2, const BwdTcSpan &span, int id,
                                            uint8_t *smem) {
  constexpr int BN = Role::BN, N1 = Role::N1, N2 = Role::N2, kH = Role::kH;
  constexpr bool OUT1 = Role::OUT1, OUT2 = Role::OUT2, KEYS = Role::KEYS;
  const AttnParams &a = p.a;
  uint8_t *sX1 = smem, *sX2 = smem + Role::kX2Off;
  uint8_t *sY1 = smem + Role::kY1Off, *sY2 = smem + Role::kY2Off;
  float *terms = reinterpret_cast<float *>(smem + Role::kTermOff);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Role::kBarOff);
  uint64_t *y1_full = bars, *y1_empty = y1_full + N1;
  uint64_t *y2_full = y1_empty + N1, *y2_empty = y2_full + N2;
  uint64_t *x_full = y2_empty + N2;
  uint64_t *s_full = x_full + 1;    // S_j complete (MMA -> softmax)
  uint64_t *p_full = s_full + 1;    // P_j in TMEM, or S_j read (softmax -> MMA)
  uint64_t *dp_full = p_full + 1;   // dP_j complete
  uint64_t *ds_full = dp_full + 1;  // dS_j in TMEM
  uint64_t *o_final = ds_full + 1;  // every product has completed
  uint64_t *fin_bar = o_final + 1;  // teardown drain of the MMA warp
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fin_bar + 1);
  constexpr int kProducerWarp = kBwdTcSoftmaxWarps, kMmaWarp = kBwdTcSoftmaxWarps + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // --- work item: tile fastest (a slab's Y blocks stay in L2 while its tiles
  // run), then split, then slab; the tiles that visit most blocks first ---
  int tile = id % span.tiles;
  id /= span.tiles;
  const int split = id % span.splits, bh = id / span.splits;
  if (!KEYS) tile = span.tiles - 1 - tile;
  const int x0 = tile * kBwdTcRows;
  const int xrows = KEYS ? a.S : a.R;

  if (threadIdx.x == 0) {
    for (int s = 0; s < N1; ++s) {
      mbar_init(&y1_full[s], 1);
      mbar_init(&y1_empty[s], 1);
    }
    for (int s = 0; s < N2; ++s) {
      mbar_init(&y2_full[s], 1);
      mbar_init(&y2_empty[s], 1);
    }
    mbar_init(x_full, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, kBwdTcSoftmaxWarps);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, kBwdTcSoftmaxWarps);
    mbar_init(o_final, 1);
    mbar_init(fin_bar, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // launched as a programmatic dependent of the row-term kernel: nothing below
  // touches global memory before that grid has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // the block list of this CTA: [begin, ...) of `count` visited blocks
  const BwdBlocks walk = bwd_blocks<Role>(a, x0);
  int begin = walk.at_or_after(walk.first), count = 0x7fffffff;
  if (span.splits > 1) {
    int total = 0;
    for (int b = begin; b >= 0; b = walk.at_or_after(b + 1)) ++total;
    const int per = (total + span.splits - 1) / span.splits;
    count = min(per, total - split * per);
    for (int s = 0; s < split * per && begin >= 0; ++s) begin = walk.at_or_after(begin + 1);
    if (count <= 0) begin = -1;
  }

  if (warp == kProducerWarp) {
    // ============================ TMA producer ============================
    if (lane == 0) {
      tma_prefetch_desc(tm_x1);
      tma_prefetch_desc(tm_y1);
      tma_prefetch_desc(tm_y2);
      mbar_arrive_expect_tx(x_full, Role::kX1Bytes + Role::kX2Bytes);
#pragma unroll
      for (int bx = 0; bx < Role::kBoxes1; ++bx)
        tma_load_3d(sX1 + bx * (128 * 128), tm_x1, x_full, bx * 64, x0, bh);
      if constexpr (OUT1) {
#pragma unroll
        for (int bx = 0; bx < Role::kBoxes2; ++bx)
          tma_load_3d(sX2 + bx * (128 * 128), tm_x2, x_full, bx * 64, x0, bh);
      }
      const float *nlse = p.nlse + (long long)bh * p.rpad;
      const float *ndelta = p.ndelta + (long long)bh * p.rpad;
      int u1 = 0, u2 = 0;
      int n = 0;
      for (int b = begin; b >= 0 && n < count; b = walk.at_or_after(b + 1), ++n) {
        const int s1 = n % N1, s2 = n % N2;
        if (!mbar_wait(&y1_empty[s1], ((uint32_t)(n / N1) & 1u) ^ 1u, a.wd, kWdTmaEmpty)) break;
        mbar_arrive_expect_tx(&y1_full[s1], Role::kY1Bytes + (KEYS ? 2 * BN * 4 : 0));
        uint8_t *d1 = sY1 + s1 * Role::kY1Bytes;
#pragma unroll
        for (int bx = 0; bx < Role::kBoxes1; ++bx)
          tma_load_3d(d1 + bx * (BN * 128), tm_y1, &y1_full[s1], bx * 64, b * BN, bh);
        if constexpr (KEYS) {  // b BN + BN <= rpad
          bulk_load(terms + s1 * 2 * BN, nlse + b * BN, BN * 4, &y1_full[s1]);
          bulk_load(terms + s1 * 2 * BN + BN, ndelta + b * BN, BN * 4, &y1_full[s1]);
        }
        ++u1;
        if (!mbar_wait(&y2_empty[s2], ((uint32_t)(n / N2) & 1u) ^ 1u, a.wd, kWdTmaEmpty)) break;
        mbar_arrive_expect_tx(&y2_full[s2], Role::kY2Bytes);
        uint8_t *d2 = sY2 + s2 * Role::kY2Bytes;
#pragma unroll
        for (int bx = 0; bx < Role::kBoxes2; ++bx)
          tma_load_3d(d2 + bx * (BN * 128), tm_y2, &y2_full[s2], bx * 64, b * BN, bh);
        ++u2;
      }
      // drain copies still landing (only ever waits after an abort)
      mbar_wait_drain(x_full, 0, a.wd);
      for (int v = max(u1 - N1, 0); v < u1; ++v)
        mbar_wait_drain(&y1_full[v % N1], (uint32_t)(v / N1) & 1u, a.wd);
      for (int v = max(u2 - N2, 0); v < u2; ++v)
        mbar_wait_drain(&y2_full[v % N2], (uint32_t)(v / N2) & 1u, a.wd);
    }
  } else if (warp == kMmaWarp) {
    // ============================ MMA issuer ============================
    // the whole warp, converged: see tc_mma_ss_warp
    {
      constexpr uint32_t kIdescS = umma_idesc_f16(kBF16, 128, BN, false, false);
      constexpr uint32_t kIdesc1 = umma_idesc_f16(kBF16, 128, Role::D1, false, true);
      constexpr uint32_t kIdesc2 = umma_idesc_f16(kBF16, 128, Role::D2, false, true);
      const uint32_t x1 = smem_u32(sX1), x2 = smem_u32(sX2), y1 = smem_u32(sY1), y2 = smem_u32(sY2);
      auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t code) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.wd, code));
      };
      bool ok = wait(x_full, 0, kWdTmaFull);
      // first products: 128 x BN scores over the head dim, both K-major
      auto first = [&](uint32_t x, uint32_t y, int steps, uint32_t col) {
        tc_fence_after();
        const uint64_t a0 = umma_desc_sw128(x, 16, 1024);
        const uint64_t b0 = umma_desc_sw128(y, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < steps; ++ks)
          tc_mma_ss_warp(tmem + col, umma_desc_advance(a0, (ks >> 2) * (128 * 128) + (ks & 3) * 32),
                    umma_desc_advance(b0, (ks >> 2) * (BN * 128) + (ks & 3) * 32), kIdescS,
                    ks > 0 ? 1u : 0u);
      };
      // second products: weights from TMEM (each half of the columns packed at
      // the start of its own half) times the same Y block, MN-major
      auto second = [&](uint32_t wcol, uint32_t y, uint32_t out, uint32_t idesc, bool fresh) {
        tc_fence_after();
        const uint64_t b0 = umma_desc_sw128_mn(y, BN * 128, 1024);
#pragma unroll
        for (int ks = 0; ks < BN / 16; ++ks) {
          const int half = ks / (kH / 16);
          tc_mma_ts_warp(tmem + out, tmem + wcol + half * kH + (ks - half * (kH / 16)) * 8,
                    umma_desc_advance(b0, ks * 2048), idesc, fresh && ks == 0 ? 0u : 1u);
        }
      };
      auto issue_s = [&](int n) -> bool {
        const int s1 = n % N1;
        if (!wait(&y1_full[s1], (uint32_t)(n / N1) & 1u, kWdTmaFull)) return false;
        first(x1, y1 + s1 * Role::kY1Bytes, Role::D1 / 16, 0);
        tc_commit_warp(s_full);
        return true;
      };
      auto issue_dp = [&](int n) -> bool {
        const int s2 = n % N2;
        if (!wait(&y2_full[s2], (uint32_t)(n / N2) & 1u, kWdTmaFull)) return false;
        first(x2, y2 + s2 * Role::kY2Bytes, Role::D2 / 16, BN);
        tc_commit_warp(dp_full);
        if constexpr (!OUT2) tc_commit_warp(&y2_empty[s2]);
        return true;
      };
      int n = 0;
      int b = begin;
      if (ok && b >= 0) {
        ok = issue_s(0);
        if constexpr (OUT1) ok = ok && issue_dp(0);
      }
      while (ok && b >= 0 && n < count) {
        b = walk.at_or_after(b + 1);
        const bool more = b >= 0 && n + 1 < count;
        const int s1 = n % N1, s2 = n % N2;
        if (!(ok = wait(p_full, (uint32_t)n & 1u, kWdSoftmax))) break;
        if constexpr (OUT2) {
          if constexpr (!OUT1)
            if (!(ok = wait(&y2_full[s2], (uint32_t)(n / N2) & 1u, kWdTmaFull))) break;
          second(0, y2 + s2 * Role::kY2Bytes, Role::kOut2Col, kIdesc2, n == 0);
          tc_commit_warp(&y2_empty[s2]);
          // (not after S_j: the softmax warps read the row terms of the slot)
          if constexpr (!OUT1) tc_commit_warp(&y1_empty[s1]);
        }
        if (more && !(ok = issue_s(n + 1))) break;
        if constexpr (OUT1) {
          if (!(ok = wait(ds_full, (uint32_t)n & 1u, kWdSoftmax))) break;
          second(BN, y1 + s1 * Role::kY1Bytes, Role::kOut1Col, kIdesc1, n == 0);
          tc_commit_warp(&y1_empty[s1]);
          if (more && !(ok = issue_dp(n + 1))) break;
        }
        ++n;
        if (!more) break;
      }
      if (ok && n > 0) tc_commit_warp(o_final);
      // all MMAs of this CTA complete before TMEM is released
      tc_commit_warp(fin_bar);
      mbar_wait_drain(fin_bar, 0, a.wd);
    }
  } else {
    // ===== softmax warps: X rows 32 (w % 4) .. +31, block columns half w / 4 =====
    const int quarter = warp & 3, half = warp >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const float c = a.scale_log2;
    const float gain = bwd_gain<kBF16>(p, bh);
    float x_nlse = 0.f, x_ndelta = 0.f;
    int pos = 0;  // query tiles: this row's position
    if constexpr (!KEYS) {
      x_nlse = p.nlse[(long long)bh * p.rpad + x0 + r];  // x0 + 127 < rpad
      x_ndelta = p.ndelta[(long long)bh * p.rpad + x0 + r];
      pos = (x0 + r) % a.L + a.off;
    }
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
      bool w = true;
      if (lane == 0) w = mbar_wait(bar, parity, a.wd, kWdMma);
      w = __shfl_sync(0xffffffffu, (int)w, 0) != 0;
      tc_fence_after();
      return w;
    };
    auto arrive = [&](uint64_t *bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int n = 0;
    for (int b = begin; b >= 0 && n < count; b = walk.at_or_after(b + 1), ++n) {
      const float *t_nlse = terms + (n % N1) * 2 * BN + half * kH;
      const float *t_ndelta = t_nlse + BN;
      if (!(ok = wait(s_full, (uint32_t)n & 1u))) break;
      // the row terms came with Y1 (already complete: S_j was computed from it)
      if constexpr (KEYS)
        if (!(ok = wait(&y1_full[n % N1], (uint32_t)(n / N1) & 1u))) break;
      // ---- phase E ----
      float w[kH];
      tmem_ldn<kH>(tmem + lane_base + half * kH, w);
      tmem_wait_ld();
      if constexpr (!OUT2) arrive(p_full);  // S_j is free
      const bool masked = bwd_needs_mask<Role>(a, x0, b);
      const float2 c2 = make_float2(c, c);
#pragma unroll
      for (int i = 0; i < kH; i += 4) {
        float4 nl = make_float4(x_nlse, x_nlse, x_nlse, x_nlse);
        if constexpr (KEYS) nl = *reinterpret_cast<const float4 *>(t_nlse + i);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          float2 t = fma2(make_float2(w[i + e], w[i + e + 1]), c2,
                          e == 0 ? make_float2(nl.x, nl.y) : make_float2(nl.z, nl.w));
          if ((((i + e) >> 1) & 3) < SDPA_BWD_POLY_OF4) {
            t = exp2_poly2(t);
          } else {
            t.x = fast_exp2(t.x);
            t.y = fast_exp2(t.y);
          }
          w[i + e] = t.x;
          w[i + e + 1] = t.y;
        }
      }
      uint64_t hidden = 0;  // masked columns of this thread
      if (masked) {
        if constexpr (KEYS) {
          const int key = x0 + r;
          const unsigned lim = a.window > 0 ? (unsigned)a.window : 0x80000000u;
          int i = (b * BN + half * kH) % a.L;
#pragma unroll
          for (int e = 0; e < kH; ++e) {
            if ((unsigned)(i + a.off - key) >= lim) {
              hidden |= 1ull << e;
              w[e] = 0.f;
            }
            if (++i == a.L) i = 0;
          }
        } else {
          const VisibleRange vis = visible_range(a, pos, b * BN + half * kH);
#pragma unroll
          for (int e = 0; e < kH; ++e)
            if (!vis(e)) {
              hidden |= 1ull << e;
              w[e] = 0.f;
            }
        }
      }
      if constexpr (OUT2) {
        uint32_t pk[kH / 2];
#pragma unroll
        for (int i = 0; i < kH / 2; ++i) pk[i] = pack2<kBF16>(w[2 * i], w[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < kH / 2; i += 8) tmem_st_u8x(tmem + lane_base + half * kH + i, pk + i);
        tmem_wait_st();
        arrive(p_full);
      }
      // ---- phase F ----
      if constexpr (OUT1) {
        if (!(ok = wait(dp_full, (uint32_t)n & 1u))) break;
        // two copies: a masked pair's dP may be anything, also not a number
        auto phase_f = [&](auto with_mask) {
#pragma unroll
          for (int i0 = 0; i0 < kH; i0 += 16) {
            float d[16];
            tmem_ld16(tmem + lane_base + BN + half * kH + i0, d);
            tmem_wait_ld();
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              float4 nd = make_float4(x_ndelta, x_ndelta, x_ndelta, x_ndelta);
              if constexpr (KEYS) nd = *reinterpret_cast<const float4 *>(t_ndelta + i0 + i);
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                float2 t = add2(make_float2(d[i + e], d[i + e + 1]),
                                e == 0 ? make_float2(nd.x, nd.y) : make_float2(nd.z, nd.w));
                if constexpr (!kBF16) t = mul2(t, make_float2(gain, gain));
                t = mul2(t, make_float2(w[i0 + i + e], w[i0 + i + e + 1]));
                if constexpr (decltype(with_mask)::value) {
                  if ((hidden >> (i0 + i + e)) & 1) t.x = 0.f;
                  if ((hidden >> (i0 + i + e + 1)) & 1) t.y = 0.f;
                }
                pk[(i + e) / 2] = pack2<kBF16>(t.x, t.y);
              }
            }
            tmem_st_u8x(tmem + lane_base + BN + half * kH + i0 / 2, pk);
          }
        };
        if (masked)
          phase_f(std::true_type());
        else
          phase_f(std::false_type());
        tmem_wait_st();
        arrive(ds_full);
      }
    }

    // ------------------------------ epilogue ------------------------------
    const bool have = ok && n > 0;
    // (without a block, X may still be landing where the zeros are staged)
    ok = wait(have ? o_final : x_full, 0) && ok;
    const bool have_o = have && ok;
    const int nvalid = min(kBwdTcRows, xrows - x0);
    auto finish = [&](int col, int d, float factor, uint8_t *stage, float *part) {
      const int chunks = d / 16;
      for (int c16 = half * chunks / 2; c16 < (half + 1) * chunks / 2; ++c16) {
        float o[16];
        if (have_o) {
          tmem_ld16(tmem + lane_base + col + c16 * 16, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0.f;
        }
        if (part == nullptr) {
          uint32_t w8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w8[e] = pack2<kBF16>(o[2 * e] * factor, o[2 * e + 1] * factor);
          stage_16bit_x16(stage, r, c16, w8);
        } else if (r < nvalid) {  // fp32 sums, [split][slab][row][d]
          float4 *dst = reinterpret_cast<float4 *>(
              part + ((((long long)split * a.B * a.Hkv + bh) * xrows + x0 + r) * d + c16 * 16));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
    };
    const bool split_out = span.splits > 1;
    if constexpr (OUT1)
      finish(Role::kOut1Col, Role::D1, bwd_ds_factor<kBF16>(p, gain), sX1, split_out ? span.part1 : nullptr);
    if constexpr (OUT2)
      finish(Role::kOut2Col, Role::D2, bwd_dv_factor<kBF16>(), smem + Role::kStage2Off, split_out ? span.part2 : nullptr);
    if (!split_out) {
      fence_proxy_async_smem();
      asm volatile("bar.sync 1, %0;" ::"n"(kBwdTcSoftmaxWarps * 32) : "memory");
      // rows past the slab and columns past the head dim are clipped
      if (warp == 0 && lane == 0) {
        if constexpr (OUT1)
          for (int bx = 0; bx < Role::kBoxes1 && bx * 64 < a.Dqk; ++bx)
            tma_store_3d(tm_o1, sX1 + bx * (128 * 128), bx * 64, x0, bh);
        if constexpr (OUT2)
          for (int bx = 0; bx < Role::kBoxes2 && bx * 64 < a.Dv; ++bx)
            tma_store_3d(tm_o2, smem + Role::kStage2Off + bx * (128 * 128), bx * 64, x0, bh);
        bulk_commit_group();
        bulk_wait_group0();
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

// The kinds of tile of one head-dim pair, most work per block first.
template <int DQK, int DV>
struct BwdTcRoles {
  // key tiles with dK and dV together: 128-row blocks where TMEM and shared
  // memory have room, 96 or 64 otherwise
  static constexpr int BN = DQK <= 128 ? 128 : DV <= 128 ? 96 : 64;
  using Key = BwdTcRole<DQK, DV, BN, 2, 2, true, true, true>;
  using Query = BwdTcRole<DQK, DV, BN, 2, 2, false, true, false>;
  static constexpr int kKinds = 2;
  // (more than half of an SM's, whatever the tiles need: a CTA takes all of TMEM)
  static constexpr uint32_t kSmem = bwd_max(120 * 1024, bwd_max(Key::kSmemBytes, Query::kSmemBytes));
};
template <>
struct BwdTcRoles<256, 256> {
  using Key = BwdTcRole<256, 256, 64, 2, 1, true, true, false>;    // dK
  using Query = BwdTcRole<256, 256, 64, 2, 1, false, true, false>;
  using KeyV = BwdTcRole<256, 256, 64, 2, 2, true, false, true>;   // dV
  static constexpr int BN = 64;
  static constexpr int kKinds = 3;
  static constexpr uint32_t kSmem = bwd_max(KeyV::kSmemBytes, bwd_max(Key::kSmemBytes, Query::kSmemBytes));
};

template <bool kBF16, int DQK, int DV>
__global__ void __launch_bounds__(kBwdTcThreads, 1)
    bwd_tc_kernel(const __grid_constant__ BwdTcMaps tm, const __grid_constant__ BwdParams p,
                  const __grid_constant__ BwdTcSpan keys, const __grid_constant__ BwdTcSpan rows) {
  using Roles = BwdTcRoles<DQK, DV>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // The 128-byte swizzle atoms need 1024-byte aligned tiles; see tc.cuh.
  if ((smem_u32(smem_raw) & 1023u) != 0u) {
    if (threadIdx.x == 0) wd_record(p.a.wd, kWdSmemAlign);
    return;
  }
  const int slabs = p.a.B * p.a.Hkv;
  const int key_ctas = slabs * keys.tiles * keys.splits, row_ctas = slabs * rows.tiles * rows.splits;
  int id = blockIdx.x;
  if (id < key_ctas) {
    bwd_tc_tile<kBF16, typename Roles::Key>(p, &tm.kx, &tm.vx, &tm.qy, &tm.doy, &tm.dk, &tm.dv, keys, id, smem_raw);
    return;
  }
  id -= key_ctas;
  if (id < row_ctas) {
    bwd_tc_tile<kBF16, typename Roles::Query>(p, &tm.qx, &tm.dox, &tm.ky, &tm.vy, &tm.dq, &tm.dq, rows, id, smem_raw);
    return;
  }
  if constexpr (Roles::kKinds == 3) {
    id -= row_ctas;
    bwd_tc_tile<kBF16, typename Roles::KeyV>(p, &tm.kx, &tm.vx, &tm.qy, &tm.doy, &tm.dk, &tm.dv, keys, id, smem_raw);
  }
}

// Sum of the splits' fp32 tiles, times the factor, rounded once: X rows of all
// slabs, d columns (a multiple of 8; the tiles' rows are dpad wide).
template <bool kBF16>
__global__ void __launch_bounds__(256)
    bwd_join_kernel(const BwdParams p, const float *__restrict__ part, uint16_t *__restrict__ out,
                    long long rows, int rows_per_slab, int d, int dpad, int splits, int is_dv) {
  const int per_row = d / 4;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= rows * per_row) return;
  const long long row = id / per_row;
  const int c = (int)(id - row * per_row) * 4;
  const float4 *src = reinterpret_cast<const float4 *>(part + row * dpad + c);
  const long long stride = rows * dpad / 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < splits; ++i) {
    const float4 x = __ldcs(src + i * stride);
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  const float f = is_dv ? bwd_dv_factor<kBF16>()
                        : bwd_ds_factor<kBF16>(p, bwd_gain<kBF16>(p, (int)(row / rows_per_slab)));
  uint2 w;
  w.x = pack2<kBF16>(s.x * f, s.y * f);
  w.y = pack2<kBF16>(s.z * f, s.w * f);
  *reinterpret_cast<uint2 *>(out + row * d + c) = w;
}

}  // namespace sdpa
