// Row terms of the backward pass: one read of dO and O per query row.
//
//   nlse   = kPExp - lse log2(e)        ndelta = dlse - rowsum(dO O)
// over slabs padded to a multiple of 128 rows.  A row that takes no part (lse = -inf)
// carries nlse = -inf and ndelta = 0 and has no share in the norms, whatever its dO,
// O and dlse hold; padding rows, whose Q and dO are read as zeros, carry the lowest
// finite nlse, so that their P is 0 without a test.  For fp16 also the largest finite
// row norms of dO, O and V and the largest |dlse| of each slab (an order-independent
// maximum over the bits of non-negative floats), from which the gain on dS is taken.
//
// Bound by memory: eight lanes share a row, 128 contiguous bytes per load.
#pragma once

#include <cfloat>

#include "bwd_params.cuh"

namespace sdpa {

constexpr int kBwdRowsThreads = 256;
constexpr int kBwdRowsPerCta = kBwdRowsThreads / 8;

struct BwdRowsParams {
  const void *out, *dout, *v;
  const float *lse, *dlse;
  float *nlse, *ndelta;
  unsigned int *norms;
  int R, rpad, S, Dv;
  long long row_ctas;  // CTAs over query rows; the ones behind them (fp16) go over V
  int v_ctas;          // ... per slab
};

__device__ __forceinline__ float sum8(float x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Block maximum of the sizes of finite values.  (A row that holds an inf or NaN has
// no finite dS to scale; counted, it would take the scale from the other rows'.)
__device__ __forceinline__ void block_max_to(unsigned int *cell, float x, unsigned int *tmp) {
  unsigned int m = __float_as_uint(x) & 0x7fffffffu;
  if (m >= 0x7f800000u) m = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kBwdRowsThreads / 32; ++w) m = max(m, tmp[w]);
    if (m != 0) atomicMax(cell, m);
  }
  __syncthreads();
}

template <bool kBF16>
__global__ void __launch_bounds__(kBwdRowsThreads) bwd_rows_kernel(const BwdRowsParams p) {
  __shared__ unsigned int tmp[kBwdRowsThreads / 32];
  // the main kernel may set up now (it waits for this grid)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int sub = threadIdx.x & 7, local = threadIdx.x >> 3;
  const int chunks = p.Dv / 8;
  if (blockIdx.x < p.row_ctas) {
    const long long prow = (long long)blockIdx.x * kBwdRowsPerCta + local;
    const int bh = (int)(prow / p.rpad);  // one slab per CTA: rpad is a multiple of 128
    const int r = (int)(prow - (long long)bh * p.rpad);
    const bool live = r < p.R;
    const long long row = (long long)bh * p.R + r;
    float part[4] = {0.f, 0.f, 0.f, 0.f}, sq = 0.f, sq_o = 0.f;  // four short sums: less rounding than one
    if (live) {
      const uint4 *o = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.out) + row * p.Dv);
      const uint4 *d = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.dout) + row * p.Dv);
#pragma unroll 2
      for (int c = sub; c < chunks; c += 8) {
        const uint4 ov = __ldg(o + c), dv = __ldg(d + c);
        const uint32_t ow[4] = {ov.x, ov.y, ov.z, ov.w}, dw[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = unpack2<kBF16>(ow[i]), b = unpack2<kBF16>(dw[i]);
          part[i] = fmaf(a.x, b.x, fmaf(a.y, b.y, part[i]));
          if constexpr (!kBF16) {
            sq = fmaf(b.x, b.x, fmaf(b.y, b.y, sq));
            sq_o = fmaf(a.x, a.x, fmaf(a.y, a.y, sq_o));
          }
        }
      }
    }
    const float dot = sum8((part[0] + part[1]) + (part[2] + part[3]));
    const float lse = live ? p.lse[row] : 0.f;
    const bool takes_part = live && lse != -INFINITY;
    float dl = 0.f;
    if (takes_part && p.dlse != nullptr) dl = p.dlse[row];
    if (sub == 0) {
      float nlse = bwd_p_exp<kBF16>() - lse * 1.4426950408889634f;
      if (!live || nlse == -INFINITY) nlse = -FLT_MAX;  // (lse = +inf: exp(s - lse) = 0 as well)
      p.nlse[prow] = lse == -INFINITY ? -INFINITY : nlse;
      p.ndelta[prow] = takes_part ? dl - dot : 0.f;
    }
    if constexpr (!kBF16) {
      if (!takes_part) sq = sq_o = 0.f;  // (the row's eight lanes agree)
      block_max_to(p.norms + 4 * bh, sqrtf(sum8(sq)), tmp);
      block_max_to(p.norms + 4 * bh + 2, dl, tmp);
      block_max_to(p.norms + 4 * bh + 3, sqrtf(sum8(sq_o)), tmp);
    }
  } else if constexpr (!kBF16) {
    const long long id = blockIdx.x - p.row_ctas;
    const int bh = (int)(id / p.v_ctas);
    const int r = (int)(id - (long long)bh * p.v_ctas) * kBwdRowsPerCta + local;
    float sq = 0.f;
    if (r < p.S) {
      const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.v) + ((long long)bh * p.S + r) * p.Dv);
#pragma unroll 2
      for (int c = sub; c < chunks; c += 8) {
        const uint4 x = __ldg(v + c);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = unpack2<kBF16>(w[i]);
          sq = fmaf(a.x, a.x, fmaf(a.y, a.y, sq));
        }
      }
    }
    block_max_to(p.norms + 4 * bh + 1, sqrtf(sum8(sq)), tmp);
  }
}

// dsink_h = -sum over rows of exp(sink_h - lse) delta.  One CTA per query head,
// rows in a fixed order; the terms differ in sign and the sum runs over all
// tokens, so it is kept in 64 bits (a few terms per thread).
constexpr int kBwdSinksThreads = 512;
__global__ void __launch_bounds__(kBwdSinksThreads)
    bwd_sinks_kernel(const float *sinks, const float *lse, const float *ndelta, float *dsinks, int B,
                     int Hq, int Hkv, int L, int rpad) {
  __shared__ double tmp[kBwdSinksThreads / 32];
  const int h = blockIdx.x, g = Hq / Hkv;
  const float sink = sinks[h];
  double sum = 0;
  for (int b = 0; b < B; ++b) {
    const float *ls = lse + ((long long)b * Hq + h) * L;
    const float *nd = ndelta + (long long)(b * Hkv + h / g) * rpad + (long long)(h % g) * L;
    for (int i = threadIdx.x; i < L; i += kBwdSinksThreads)
      if (ls[i] != -INFINITY) sum += exp((double)sink - ls[i]) * nd[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kBwdSinksThreads / 32; ++w) sum += tmp[w];
    dsinks[h] = (float)sum;
  }
}

}  // namespace sdpa
