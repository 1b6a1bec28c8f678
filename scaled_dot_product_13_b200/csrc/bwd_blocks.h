// The blocks of BN Y rows that a tile of the backward pass visits, in rising order:
// whole-number arithmetic alone, so that it also compiles for the host (tests).
//
// Query tiles see one range of keys.  Key tiles see, of each head's L packed rows, the
// same range of queries [lo, hi); a block may span several heads.
#pragma once

#ifdef __CUDACC__
#define SDPA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SDPA_HOST_DEVICE inline
#endif

namespace sdpa {

constexpr int kBwdTcRows = 128;  // X rows of a tile

// Positions of packed rows [r0, r0 + n) of a slab (n >= 1 valid rows).
template <class Params>
SDPA_HOST_DEVICE void packed_positions(const Params &a, int r0, int n, int &pos_min, int &pos_max) {
  const int i0 = r0 % a.L;
  const int i1 = (r0 + n - 1) % a.L;
  const bool wraps = n >= a.L || i1 < i0;  // over the end of a head's rows
  pos_min = (wraps ? 0 : i0) + a.off;
  pos_max = (wraps ? a.L - 1 : i1) + a.off;
}

template <bool KEYS, int BN>
struct BwdBlocks {
  int first;      // query tiles: blocks begin here
  int end;        // blocks end here
  int L, R;
  int lo, hi;     // packed rows of the current head that the tile sees
  int base;       // first packed row of that head
  bool all;       // every row is visible: nothing to skip

  // Smallest visited block >= b (rising from call to call), or -1.  Leaves the
  // first head with visible rows at or behind the block's first row as the
  // current one.
  SDPA_HOST_DEVICE int at_or_after(int b) {
    if (b >= end) return -1;
    if constexpr (KEYS) {
      const int r0 = b * BN;
      while (r0 >= hi) {
        lo += L;
        hi += L;
        base += L;
        if (lo >= R) return -1;
      }
      if (!all && r0 + BN <= lo) b = lo / BN;
    }
    return b;
  }

  // Visited block number k (from 0), or -1, and how many there are in all; before any
  // at_or_after, and leaving the current head as that does.  Without walking over the
  // blocks before it: each part of a split list begins somewhere in it.
  SDPA_HOST_DEVICE int seek(int k, int &total) {
    if constexpr (!KEYS) {
      total = end - first;
      return k < total ? first + k : -1;
    } else if (end == 0) {
      total = 0;
      return -1;
    } else if (all || L <= BN) {
      // no block is skipped but behind the last visible row: BN rows in a row hold one
      // of every query index
      total = (R - L + hi - 1) / BN + 1;
      if (k >= total) return -1;
      const int r0 = k * BN;
      int head = r0 / L;
      if (r0 >= head * L + hi) ++head;
      to_head(head);
      return k;
    } else {
      // by heads (fewer than blocks); neighbours may share one
      int found = -1, head = 0, behind = 0;  // behind the last head's blocks
      total = 0;
      for (int h = 0; h < R / L; ++h) {
        const int from = (lo + h * L) / BN, to = (hi + h * L - 1) / BN + 1;
        const int b = from > behind ? from : behind;
        if (found < 0 && k < total + to - b) {
          found = b + k - total;
          head = h;
        }
        total += to - b;
        behind = to;
      }
      if (found >= 0) to_head(head);
      return found;
    }
  }

  SDPA_HOST_DEVICE void to_head(int head) {
    lo += head * L;
    hi += head * L;
    base += head * L;
  }

  // Query index of packed row r0 (the first of the last returned block).
  SDPA_HOST_DEVICE int query(int r0) const { return r0 >= base ? r0 - base : r0 - base + L; }
};

template <bool KEYS, int BN, class Params>
SDPA_HOST_DEVICE BwdBlocks<KEYS, BN> bwd_blocks(const Params &a, int x0) {
  BwdBlocks<KEYS, BN> w;
  w.L = a.L;
  w.R = a.R;
  w.base = 0;
  w.lo = 0;
  w.hi = a.L;
  w.first = 0;
  if constexpr (KEYS) {
    const int key_max = (x0 + kBwdTcRows < a.S ? x0 + kBwdTcRows : a.S) - 1;
    if (a.causal) {
      w.lo = x0 - a.off > 0 ? x0 - a.off : 0;
      if (w.lo > a.L) w.lo = a.L;
    }
    if (a.window > 0) {
      const long long hi = (long long)key_max + a.window - a.off;
      w.hi = hi < 0 ? 0 : hi < a.L ? (int)hi : a.L;
    }
    w.end = w.lo < w.hi ? (a.R + BN - 1) / BN : 0;
  } else {
    int pos_min, pos_max;
    packed_positions(a, x0, kBwdTcRows < a.R - x0 ? kBwdTcRows : a.R - x0, pos_min, pos_max);
    const int kend = a.causal && pos_max + 1 < a.S ? pos_max + 1 : a.S;
    const int kbeg = a.window > 0 && pos_min - a.window + 1 > 0 ? pos_min - a.window + 1 : 0;
    w.first = kbeg / BN;
    w.end = kend > kbeg ? (kend + BN - 1) / BN : w.first;
  }
  w.all = w.hi - w.lo == a.L;
  return w;
}

}  // namespace sdpa
