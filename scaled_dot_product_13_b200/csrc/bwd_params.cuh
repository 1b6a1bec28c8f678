// Parameters and arithmetic shared by the backward kernels.
//
//   S  = scale Q K^T            P  = exp(S - lse)      (0 where masked)
//   dP = dO V^T                 dS = P (dP - delta)    delta = rowsum(dO O) - dlse
//   dQ = scale dS K    dK = scale dS^T Q    dV = P^T dO
//
// P is recomputed from the forward pass's log-sum-exp, so nothing of size L x S
// is stored.  Query rows are the packed slab rows of the forward pass: the g*L
// rows that read one KV head are contiguous, so a product over all rows of a
// slab sums the gradients of a shared KV head by itself, in a fixed order and
// without atomics.
//
// Rounding: P and dS enter their products as 16-bit values (one, or for small
// problems the sum of two), all sums and row terms are fp32, each gradient is
// rounded once.  For fp16 both are scaled by powers of two first (bf16 has fp32's exponents and needs none):
//   - P by 2^14: P <= 1, and a weight of 2^-16 (one of 64K equal keys) would
//     otherwise be a subnormal number;
//   - dS by 2^14 gain: |dP - delta| <= max||dO|| (max||V|| + max||O||) + max|dlse|
//     =: bound (Cauchy-Schwarz), and gain is the power of two that takes bound
//     into [1, 2).  So |dS| stays below 2^15 and cannot overflow, whatever the
//     gradient's scale, and a loss scale is not needed to keep it from
//     underflowing.  (O's own norm, although it is a mean of V's rows: out and
//     lse may be those of more keys than the call's.)
// The output factors take the powers of two back, exactly.
#pragma once

#include "params.cuh"

namespace sdpa {

struct BwdParams {
  AttnParams a;         // geometry, mask, scale_log2, watchdog (as in the forward kernels)
  const float *nlse;    // [B*Hkv][rpad] kPExp - lse log2(e); -inf: the row takes no part
  const float *ndelta;  // [B*Hkv][rpad] -delta
  const unsigned int *norms;  // fp16: [B*Hkv][4] float bits of max||dO||, max||V||, max|dlse|, max||O||
  int rpad;             // R rounded up so that every tile and block stays inside
  float scale;
  const void *q, *k, *v, *dout;
  void *dq, *dk, *dv;
};

// Power of two on P (fp16 only).
template <bool kBF16>
__device__ __forceinline__ constexpr float bwd_p_exp() {
  return kBF16 ? 0.f : 14.f;
}

// Power of two on dP - delta for one KV head's slab (fp16 only).  (Plain loads: the
// grid that writes the norms may still be running when a programmatic dependent
// starts, so they are not read-only for its lifetime.)
template <bool kBF16>
__device__ __forceinline__ float bwd_gain(const BwdParams &p, int bh) {
  if constexpr (kBF16) return 1.f;
  const float n_do = __uint_as_float(p.norms[4 * bh]);
  const float n_v = __uint_as_float(p.norms[4 * bh + 1]);
  const float n_l = __uint_as_float(p.norms[4 * bh + 2]);
  const float n_o = __uint_as_float(p.norms[4 * bh + 3]);
  const float bound = n_do * (n_v + n_o) + n_l;
  if (!(bound > 0.f)) return 1.f;  // nothing to scale
  const int e = min(max(ilogbf(bound), -100), 100);
  return __int_as_float((127 - e) << 23);
}

// Factors of the finished sums: dV, and dQ / dK (gain is a power of two, so
// its reciprocal is exact).
template <bool kBF16>
__device__ __forceinline__ float bwd_dv_factor() {
  return kBF16 ? 1.f : 6.103515625e-05f;  // 2^-14
}
template <bool kBF16>
__device__ __forceinline__ float bwd_ds_factor(const BwdParams &p, float gain) {
  return p.scale * bwd_dv_factor<kBF16>() / gain;
}

}  // namespace sdpa
