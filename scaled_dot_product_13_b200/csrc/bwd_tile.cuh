// Backward pass on warp-level tensor-core tiles (mma.sync), any head dims up
// to 512.
//
// One CTA owns 64 X rows and 128 columns of their gradients and walks over
// blocks of 32 Y rows:
//   key tiles    X = keys:  X1 = K, X2 = V,  Y1 = Q, Y2 = dO:  dK, dV
//   query tiles  X = rows:  X1 = Q, X2 = dO, Y1 = K, Y2 = V:   dQ
// S = X1 Y1^T and dP = X2 Y2^T come out as accumulator fragments, and P and dS
// go on as the A operands of acc2 += P Y2 and acc1 += dS Y1 straight from those
// registers.  Four warps, 16 X rows each.  Both kinds of tile run in one grid.
// Head dims above 128 take several CTAs per tile, one per 128 gradient
// columns, each computing S and dP over the whole head dim: at 512 columns the
// accumulators of one row would not fit a warp otherwise.
#pragma once

#include "bwd_params.cuh"

namespace sdpa {

constexpr int kBwdTileX = 64;
constexpr int kBwdTileY = 32;
constexpr int kBwdTileCols = 128;
constexpr int kBwdTileThreads = 128;

// Row pitch in elements: 16 bytes of padding put the eight rows of one
// ldmatrix on distinct banks.
__host__ __device__ constexpr int bwd_tile_pitch(int d) { return (d + 15) / 16 * 16 + 8; }
__host__ __device__ constexpr size_t bwd_tile_smem(int dqk, int dv) {
  return (size_t)(kBwdTileX + kBwdTileY) * (bwd_tile_pitch(dqk) + bwd_tile_pitch(dv)) * 2 +
         kBwdTileY * 12;
}

// Rows [row0, row0 + n) of a [rows][d] slab into shared memory, zero past the
// slab and in the columns that round d up to 16.
__device__ __forceinline__ void bwd_tile_load(uint16_t *dst, const uint16_t *slab, int row0, int n,
                                              int rows, int d) {
  const int pitch = bwd_tile_pitch(d);
  const int chunks = (d + 15) / 16 * 2;
  for (int i = threadIdx.x; i < n * chunks; i += kBwdTileThreads) {
    const int r = i / chunks, c = (i - r * chunks) * 8;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (row0 + r < rows && c < d)
      x = *reinterpret_cast<const uint4 *>(slab + (long long)(row0 + r) * d + c);
    *reinterpret_cast<uint4 *>(dst + r * pitch + c) = x;
  }
}

// acc (16 x 32, four n8 tiles) = X rows of this warp times Y rows, over d.
template <bool kBF16>
__device__ __forceinline__ void bwd_tile_product(float (&acc)[4][4], const uint16_t *x,
                                                 const uint16_t *y, int d) {
  const int pitch = bwd_tile_pitch(d), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
  const uint32_t xa = smem_u32(x + (16 * warp + (lane & 15)) * pitch + (lane >> 4) * 8);
  const uint32_t ya = smem_u32(y + ((lane >> 4) * 8 + (lane & 7)) * pitch + ((lane >> 3) & 1) * 8);
  for (int k = 0; k < d; k += 16) {
    uint32_t a0, a1, a2, a3;
    ldsm_x4(xa + k * 2, a0, a1, a2, a3);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4(ya + (n * 16 * pitch + k) * 2, b0, b1, b2, b3);
      mma_16816<kBF16>(acc[2 * n], a0, a1, a2, a3, b0, b1);
      mma_16816<kBF16>(acc[2 * n + 1], a0, a1, a2, a3, b2, b3);
    }
  }
}

// acc (16 x 128 columns from col0) += W (16 x 32, as accumulator fragments) Y.
template <bool kBF16>
__device__ __forceinline__ void bwd_tile_accumulate(float (&acc)[16][4], const float (&w)[4][4],
                                                    const uint16_t *y, int col0, int d) {
  const int pitch = bwd_tile_pitch(d), lane = threadIdx.x & 31;
  const int dpad = (d + 15) / 16 * 16;
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    const uint32_t a0 = pack2<kBF16>(w[2 * kk][0], w[2 * kk][1]);
    const uint32_t a1 = pack2<kBF16>(w[2 * kk][2], w[2 * kk][3]);
    const uint32_t a2 = pack2<kBF16>(w[2 * kk + 1][0], w[2 * kk + 1][1]);
    const uint32_t a3 = pack2<kBF16>(w[2 * kk + 1][2], w[2 * kk + 1][3]);
    const uint32_t ya = smem_u32(y + (16 * kk + (lane & 15)) * pitch + col0 + (lane >> 4) * 8);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      if (col0 + 16 * n >= dpad) break;
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(ya + n * 32, b0, b1, b2, b3);
      mma_16816<kBF16>(acc[2 * n], a0, a1, a2, a3, b0, b1);
      mma_16816<kBF16>(acc[2 * n + 1], a0, a1, a2, a3, b2, b3);
    }
  }
}

// This warp's 16 rows x 128 columns, times `factor`, to a [rows][d] slab.
template <bool kBF16>
__device__ __forceinline__ void bwd_tile_store(const float (&acc)[16][4], float factor,
                                               uint16_t *slab, int row0, int rows, int col0,
                                               int d) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = row0 + 16 * warp + (lane >> 2) + 8 * half;
    if (r >= rows) continue;
    uint16_t *dst = slab + (long long)r * d;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const int c = col0 + 8 * t + (lane & 3) * 2;
      if (c < d)
        *reinterpret_cast<uint32_t *>(dst + c) =
            pack2<kBF16>(acc[t][2 * half] * factor, acc[t][2 * half + 1] * factor);
    }
  }
}

// grid: key tiles (slab, tile, column part), then query tiles
struct BwdTileGrid {
  int key_tiles, key_parts;  // per slab
  int row_tiles, row_parts;
  long long key_ctas;        // B*Hkv * key_tiles * key_parts
};

template <bool kBF16>
__global__ void __launch_bounds__(kBwdTileThreads)
    bwd_tile_kernel(const BwdParams p, const BwdTileGrid g) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const AttnParams &a = p.a;
  const int Dqk = a.Dqk, Dv = a.Dv;
  uint16_t *x1 = reinterpret_cast<uint16_t *>(smem_raw);
  uint16_t *x2 = x1 + kBwdTileX * bwd_tile_pitch(Dqk);
  uint16_t *y1 = x2 + kBwdTileX * bwd_tile_pitch(Dv);
  uint16_t *y2 = y1 + kBwdTileY * bwd_tile_pitch(Dqk);
  float *col_nlse = reinterpret_cast<float *>(y2 + kBwdTileY * bwd_tile_pitch(Dv));
  float *col_ndelta = col_nlse + kBwdTileY;
  int *col_pos = reinterpret_cast<int *>(col_ndelta + kBwdTileY);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  const bool keys = blockIdx.x < g.key_ctas;  // a key tile: X = keys
  long long id = keys ? blockIdx.x : blockIdx.x - g.key_ctas;
  const int parts = keys ? g.key_parts : g.row_parts;
  const int tiles = keys ? g.key_tiles : g.row_tiles;
  const int part = (int)(id % parts);
  id /= parts;
  // the tiles that see the most rows (first keys) or keys (last rows) first
  const int tile = keys ? (int)(id % tiles) : tiles - 1 - (int)(id % tiles);
  const int bh = (int)(id / tiles);
  const int x0 = tile * kBwdTileX, col0 = part * kBwdTileCols;
  const int xrows = keys ? a.S : a.R, yrows = keys ? a.R : a.S;
  const uint16_t *q = static_cast<const uint16_t *>(p.q) + (long long)bh * a.R * Dqk;
  const uint16_t *dout = static_cast<const uint16_t *>(p.dout) + (long long)bh * a.R * Dv;
  const uint16_t *k = static_cast<const uint16_t *>(p.k) + (long long)bh * a.S * Dqk;
  const uint16_t *v = static_cast<const uint16_t *>(p.v) + (long long)bh * a.S * Dv;
  const float *nlse = p.nlse + (long long)bh * p.rpad;
  const float *ndelta = p.ndelta + (long long)bh * p.rpad;
  const float gain = bwd_gain<kBF16>(p, bh);

  bwd_tile_load(x1, keys ? k : q, x0, kBwdTileX, xrows, Dqk);
  bwd_tile_load(x2, keys ? v : dout, x0, kBwdTileX, xrows, Dv);

  // this thread's two X rows
  int xi[2], xpos[2];
  float xnlse[2], xndelta[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    xi[h] = x0 + 16 * warp + (lane >> 2) + 8 * h;
    if (!keys) {  // x0 + 63 < rpad: rows past the slab carry -inf
      xpos[h] = xi[h] % a.L + a.off;
      xnlse[h] = nlse[xi[h]];
      xndelta[h] = ndelta[xi[h]];
    }
  }
  const int key_lo = x0, key_hi = min(x0 + kBwdTileX, a.S) - 1;
  int rpos_min, rpos_max;
  packed_positions(a, min(x0, a.R - 1), max(1, min(kBwdTileX, a.R - x0)), rpos_min, rpos_max);

  float acc1[16][4], acc2[16][4];
#pragma unroll
  for (int t = 0; t < 16; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc1[t][e] = acc2[t][e] = 0.f;

  for (int y0 = 0; y0 < yrows; y0 += kBwdTileY) {
    // skip a block that no row of the tile sees
    int pos_min = rpos_min, pos_max = rpos_max, klo = y0, khi = min(y0 + kBwdTileY, a.S) - 1;
    if (keys) {
      packed_positions(a, y0, min(kBwdTileY, a.R - y0), pos_min, pos_max);
      klo = key_lo;
      khi = key_hi;
    }
    if (a.causal && klo > pos_max) continue;
    if (a.window > 0 && pos_min - khi >= a.window) continue;
    __syncthreads();  // the previous block's readers are done
    bwd_tile_load(y1, keys ? q : k, y0, kBwdTileY, yrows, Dqk);
    bwd_tile_load(y2, keys ? dout : v, y0, kBwdTileY, yrows, Dv);
    if (keys && threadIdx.x < kBwdTileY) {  // y0 + 31 < rpad
      col_nlse[threadIdx.x] = nlse[y0 + threadIdx.x];
      col_ndelta[threadIdx.x] = ndelta[y0 + threadIdx.x];
      col_pos[threadIdx.x] = (y0 + threadIdx.x) % a.L + a.off;
    }
    __syncthreads();
    float s[4][4], dp[4][4];
    bwd_tile_product<kBF16>(s, x1, y1, Dqk);
    bwd_tile_product<kBF16>(dp, x2, y2, Dv);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = e >> 1, c = 8 * t + (lane & 3) * 2 + (e & 1);
        const int pos = keys ? col_pos[c] : xpos[h];
        const int key = keys ? xi[h] : y0 + c;
        const float nl = keys ? col_nlse[c] : xnlse[h];
        const float nd = keys ? col_ndelta[c] : xndelta[h];
        const bool live = key_visible(a, pos, key) && nl != -INFINITY;
        const float w = live ? exp2f(fmaf(s[t][e], a.scale_log2, nl)) : 0.f;
        s[t][e] = w;
        dp[t][e] = live ? w * ((dp[t][e] + nd) * gain) : 0.f;
      }
    if (keys) bwd_tile_accumulate<kBF16>(acc2, s, y2, col0, Dv);
    bwd_tile_accumulate<kBF16>(acc1, dp, y1, col0, Dqk);
  }
  const float f = bwd_ds_factor<kBF16>(p, gain);
  uint16_t *d1 = static_cast<uint16_t *>(keys ? p.dk : p.dq) + (long long)bh * xrows * Dqk;
  bwd_tile_store<kBF16>(acc1, f, d1, x0, xrows, col0, Dqk);
  if (keys)
    bwd_tile_store<kBF16>(acc2, bwd_dv_factor<kBF16>(),
                          static_cast<uint16_t *>(p.dv) + (long long)bh * a.S * Dv, x0, a.S, col0, Dv);
}

}  // namespace sdpa
