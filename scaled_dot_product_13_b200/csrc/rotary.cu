// Rotary positions (forward and gradient): the plan, the checks, the kernel.
//
// Per pair: (a, b) -> m (a cos t - b sin t, a sin t + b cos t), t = position *
// frequency.  The work is one read and one write of every element, so the
// kernel is bound by memory traffic; what it must avoid is (1) paying for the
// angles per head and (2) losing them at far positions.  8192 tokens of 16 + 8
// heads of 256: 36.5 us for 201 MB, 5.5 TB/s, 85 % of a copy's rate; 4095
// tokens of 64 + 8 heads of 192, 64 of them rotated: 41.2 us for 226 MB.
//
// (1) A thread owns V pairs of one token and walks over a group of heads of q or
// of k, so one sine and cosine per pair serves the group; the first heads are
// requested before the angles are computed.
// (2) Frequencies are 64-bit fixed-point turns per position: position * turns
// wraps modulo one turn by itself, exactly; the top 32 bits are the angle in
// 2^-32 turns, converted to half-turns in fp32 (relative error 2^-24, at most 2^-26 of
// a turn) for sincospif.  A float product position * w would be off by 2^-24 * t radians,
// i.e. 0.008 at position 131072 in the first pair.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "launch.h"
#include "ptx.cuh"

namespace sdpa {
namespace {

constexpr int kThreads = 256;
// Heads loaded before the first is computed (loads in flight per thread).
constexpr int kBatch = 4;

struct RotaryTensor {
  const uint16_t *x;
  uint16_t *out;
  long long xb, xh, xt, ob, oh, ot;
};

struct RotaryParams {
  RotaryTensor t[2];
  int heads[2];
  int group;         // heads per grid.y
  int groups0;       // grid.y below it: t[0]
  int L;
  long long tokens;  // B * L
  int tokens_per_cta;
  int rot_items;     // items of V pairs of one head
  int copy_items;    // ... and of up to 2V elements copied behind them
  int dim;           // head_dim
  int half;          // rotary_dim / 2
  const void *positions;
  int position_bits;
  long long position_batch_stride, offset;
  int inverse;
  float magnitude;
  uint64_t turns[256];
};

template <int V>
struct Pack {
  static_assert(V == 1 || V == 2 || V == 4 || V == 8, "");
};
template <>
struct Pack<1> { using type = uint16_t; };
template <>
struct Pack<2> { using type = uint32_t; };
template <>
struct Pack<4> { using type = uint2; };
template <>
struct Pack<8> { using type = uint4; };

template <int V>
union Elems {
  typename Pack<V>::type v;
  uint32_t w[V < 2 ? 1 : V / 2];
};

template <bool kBF16, bool kInterleaved, int V>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(const __grid_constant__ RotaryParams p) {
  using T = typename Pack<V>::type;
  constexpr int W = V < 2 ? 1 : V / 2;  // words of a run
  // the rotated items of the CTA's tokens first, then the copied ones: the few
  // threads with angles of a partly rotated head share their warps
  const int rot_threads = p.tokens_per_cta * p.rot_items;
  const bool rotated = (int)threadIdx.x < rot_threads;
  const int id = rotated ? threadIdx.x : threadIdx.x - rot_threads;
  const int per = rotated ? p.rot_items : p.copy_items;
  if (per == 0) return;
  const int tok = id / per, item = id - tok * per;
  const long long token = (long long)blockIdx.x * p.tokens_per_cta + tok;
  if (tok >= p.tokens_per_cta || token >= p.tokens) return;
  const long long b = token / p.L;
  const long long l = token - b * p.L;
  // the item's two runs of V elements (the last copied item may have one)
  int e0, e1;
  if (rotated) {
    e0 = kInterleaved ? 2 * V * item : V * item;
    e1 = kInterleaved ? e0 + V : e0 + p.half;
  } else {
    e0 = 2 * p.half + 2 * V * item;
    e1 = e0 + V;
  }
  const bool two = e1 < p.dim;
  const bool second = (int)blockIdx.y >= p.groups0;
  const RotaryTensor &t = p.t[second];
  const int h0 = ((int)blockIdx.y - (second ? p.groups0 : 0)) * p.group;
  int left = min(p.group, p.heads[second] - h0);
  const uint16_t *src = t.x + b * t.xb + h0 * t.xh + l * t.xt;
  uint16_t *dst = t.out + b * t.ob + h0 * t.oh + l * t.ot;
  const long long xh = t.xh, oh = t.oh;

  Elems<V> a[kBatch], c[kBatch];
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (u < left) {
        a[u].v = *reinterpret_cast<const T *>(src + u * xh + e0);
        if (two) c[u].v = *reinterpret_cast<const T *>(src + u * xh + e1);
      }
    }
  };
  load();
  float cs[V], sn[V];
  if (rotated) {
    long long pos = l;
    if (p.position_bits == 64)
      pos = static_cast<const long long *>(p.positions)[b * p.position_batch_stride + l];
    else if (p.position_bits == 32)
      pos = static_cast<const int *>(p.positions)[b * p.position_batch_stride + l];
    pos += p.offset;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t turn = (uint64_t)pos * p.turns[V * item + i];
      const float half_turns = (float)(int)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
      sincospif(half_turns, &sn[i], &cs[i]);
      cs[i] *= p.magnitude;
      sn[i] *= p.inverse ? -p.magnitude : p.magnitude;
    }
  }
  for (;;) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (u >= left) break;
      if (rotated) {
        // x[0..V) the first run, x[V..2V) the second
        float x[2 * V], y[2 * V];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float2 f = unpack2<kBF16>(a[u].w[i]), g = unpack2<kBF16>(c[u].w[i]);
          x[2 * i] = f.x;
          if constexpr (V > 1) x[2 * i + 1] = f.y;
          x[V + 2 * i] = g.x;
          if constexpr (V > 1) x[V + 2 * i + 1] = g.y;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          // pair i: neighbours 2i, 2i+1 of the 2V elements, or i of both runs
          const int ia = kInterleaved ? 2 * i : i, ib = kInterleaved ? 2 * i + 1 : V + i;
          y[ia] = x[ia] * cs[i] - x[ib] * sn[i];
          y[ib] = x[ia] * sn[i] + x[ib] * cs[i];
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
          a[u].w[i] = pack2<kBF16>(y[2 * i], V > 1 ? y[2 * i + (V > 1)] : 0.f);
          c[u].w[i] = pack2<kBF16>(y[V + 2 * i], V > 1 ? y[V + 2 * i + (V > 1)] : 0.f);
        }
      }
      *reinterpret_cast<T *>(dst + u * oh + e0) = a[u].v;
      if (two) *reinterpret_cast<T *>(dst + u * oh + e1) = c[u].v;
    }
    left -= kBatch;
    if (left <= 0) break;
    src += kBatch * xh;
    dst += kBatch * oh;
    load();
  }
}

template <bool kBF16, bool kInterleaved>
cudaError_t launch_width(int v, dim3 grid, cudaStream_t stream, const RotaryParams &p) {
  switch (v) {
    case 8: rotary_kernel<kBF16, kInterleaved, 8><<<grid, kThreads, 0, stream>>>(p); break;
    case 4: rotary_kernel<kBF16, kInterleaved, 4><<<grid, kThreads, 0, stream>>>(p); break;
    case 2: rotary_kernel<kBF16, kInterleaved, 2><<<grid, kThreads, 0, stream>>>(p); break;
    default: rotary_kernel<kBF16, kInterleaved, 1><<<grid, kThreads, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

sdpa_status bad(const char *fmt, double a = 0, double b = 0) {
  char buf[256];
  snprintf(buf, sizeof(buf), fmt, a, b);
  return set_error(SDPA_ERR_INVALID_ARG, buf);
}

// Elements from the first to one past the last of a view, and whether strides
// keep its elements apart (each stride, in rising order, at least the extent
// of the dimensions below it).
long long extent(const sdpa_strides &s, int B, int heads, int L, int D) {
  return (long long)(B - 1) * s.batch + (long long)(heads - 1) * s.head +
         (long long)(L - 1) * s.token + D;
}
bool apart(const sdpa_strides &s, int B, int heads, int L, int D) {
  struct Dim { long long stride, size; } d[3] = {{s.batch, B}, {s.head, heads}, {s.token, L}};
  std::sort(d, d + 3, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
  long long span = D;
  for (const Dim &x : d) {
    if (x.size == 1) continue;
    if (x.stride < span) return false;
    span = (x.size - 1) * x.stride + span;
  }
  return true;
}

// One view of a tensor: what a call reads or writes.
struct View {
  const void *p;
  sdpa_strides s;
  int heads;
};

// Multiples lo .. hi of a stride.
struct Term {
  long long stride, lo, hi;
};

// Whether `at` plus one multiple of each of n terms (falling strides) can come within
// less than D of 0.  What the terms behind the first can add bounds its multiples: two or
// three of them where the strides nest, as in every dense layout and its slices.
// Gives up, with true, after `steps`.
bool reaches(const Term *t, int n, long long at, int D, int *steps) {
  if (n == 0) return at > -D && at < D;
  long long lo = 0, hi = 0;  // of the terms behind
  for (int i = 1; i < n; ++i) {
    lo += t[i].stride * t[i].lo;
    hi += t[i].stride * t[i].hi;
  }
  // stride m in (-D - at - hi, D - at - lo)
  const long long s = t[0].stride, from = 1 - D - at - hi, to = D - 1 - at - lo;
  const long long first = std::max(t[0].lo, from >= 0 ? (from + s - 1) / s : -(-from / s));
  const long long last = std::min(t[0].hi, to >= 0 ? to / s : -((-to + s - 1) / s));
  for (long long m = first; m <= last; ++m) {
    if (--*steps < 0) return true;
    if (reaches(t + 1, n - 1, at + s * m, D, steps)) return true;
  }
  return false;
}

// Whether two views share no element: extents that do not meet, or else no pair of rows
// whose distance is below D (rows of views whose strides are in no relation may take
// too many steps: those count as sharing).
bool disjoint(const View &x, const View &y, int B, int L, int D) {
  if (!extents_meet(x.p, 2 * extent(x.s, B, x.heads, L, D), y.p, 2 * extent(y.s, B, y.heads, L, D))) return true;
  Term t[6];
  int n = 0;
  auto add = [&](long long stride, long long lo, long long hi) {
    if (stride == 0 || lo == hi) return;
    int i = 0;
    while (i < n && t[i].stride > stride) ++i;
    if (i < n && t[i].stride == stride) {
      t[i].lo += lo;
      t[i].hi += hi;
      return;
    }
    for (int j = n++; j > i; --j) t[j] = t[j - 1];
    t[i] = {stride, lo, hi};
  };
  add(y.s.batch, 0, B - 1);
  add(y.s.head, 0, y.heads - 1);
  add(y.s.token, 0, L - 1);
  add(x.s.batch, 1 - B, 0);
  add(x.s.head, 1 - x.heads, 0);
  add(x.s.token, 1 - L, 0);
  const long long bytes = static_cast<const char *>(y.p) - static_cast<const char *>(x.p);
  int steps = 10000;
  return !reaches(t, n, bytes / 2, D, &steps);  // (both are 2-byte aligned)
}

}  // namespace
}  // namespace sdpa

using namespace sdpa;

extern "C" SDPA_API sdpa_status sdpa_rotary_init(const sdpa_rotary_config *c,
                                                 sdpa_rotary_plan *plan) {
  set_error(SDPA_OK, "");
  if (!c || !plan) return bad("config and plan must be non-NULL");
  const int R = c->rotary_dim == 0 ? c->head_dim : c->rotary_dim;
  if (c->head_dim < 2 || c->head_dim > 512)
    return bad("head_dim must lie in [2, 512] (got %.0f)", c->head_dim);
  if (R < 2 || R % 2 != 0 || R > c->head_dim)
    return bad("rotary_dim must be even, in [2, head_dim] (got %.0f of %.0f)", R, c->head_dim);
  if (c->interleaved != 0 && c->interleaved != 1)
    return bad("interleaved must be 0 or 1 (got %.0f)", c->interleaved);
  const double base = c->base == 0 ? 10000.0 : c->base;
  if (!(base > 1.0) || !std::isfinite(base)) return bad("base must be above 1 (got %g)", base);
  if (c->scaling < SDPA_ROPE_PLAIN || c->scaling > SDPA_ROPE_BANDED)
    return bad("unknown scaling %.0f", c->scaling);
  const bool by_turns = c->scaling == SDPA_ROPE_YARN || c->scaling == SDPA_ROPE_BANDED;
  if (c->scaling != SDPA_ROPE_PLAIN && !(c->factor > 0 && std::isfinite(c->factor)))
    return bad("factor must be positive (got %g)", c->factor);
  if (c->scaling == SDPA_ROPE_NTK && R < 4) return bad("ntk scaling needs rotary_dim >= 4");
  const double fast = c->beta_fast != 0 ? c->beta_fast : c->scaling == SDPA_ROPE_BANDED ? 4.0 : 32.0;
  const double slow = c->beta_slow != 0 ? c->beta_slow : 1.0;
  if (by_turns && c->original_length < 1)
    return bad("original_length must be >= 1 (got %.0f)", c->original_length);
  if (by_turns && !(slow > 0 && fast > slow && std::isfinite(fast)))
    return bad("beta_fast (%g) must be above beta_slow (%g), both positive", fast, slow);
  if (!std::isfinite(c->magnitude) || c->magnitude < 0)
    return bad("magnitude must be finite and not negative (got %g)", c->magnitude);

  // In extended precision: a frequency, below a sixth of a turn, is off by about 2^-64,
  // its angle by less than 2^-32 of a turn at positions up to 2^30.
  const long double kTwoPi = 6.283185307179586476925286766559L;
  long double b = base;
  const long double f = c->scaling == SDPA_ROPE_PLAIN ? 1.0L : (long double)c->factor;
  if (c->scaling == SDPA_ROPE_NTK) b = b * powl(f, (long double)R / (R - 2));
  long double lo = 0, hi = 0;  // yarn: pair indices of beta_fast and beta_slow turns
  if (c->scaling == SDPA_ROPE_YARN) {
    lo = floorl(R * logl(c->original_length / (fast * kTwoPi)) / (2 * logl(b)));
    hi = ceill(R * logl(c->original_length / (slow * kTwoPi)) / (2 * logl(b)));
    lo = std::max(lo, 0.0L);
    hi = std::min(hi, (long double)(R - 1));
  }
  memset(plan, 0, sizeof(*plan));
  for (int i = 0; i < R / 2; ++i) {
    long double w = powl(b, -2.0L * i / R);
    long double keep = 1;
    switch (c->scaling) {
      case SDPA_ROPE_LINEAR: keep = 0; break;
      case SDPA_ROPE_YARN: keep = 1 - std::min(std::max((i - lo) / std::max(hi - lo, 0.001L), 0.0L), 1.0L); break;
      case SDPA_ROPE_BANDED:
        keep = std::min(std::max((c->original_length * w / kTwoPi - slow) / (fast - slow), 0.0L), 1.0L);
        break;
    }
    w = w * keep + w / f * (1 - keep);
    long double turns = w / kTwoPi;
    turns -= floorl(turns);
    // to the nearest 2^-64 of a turn; a whole turn is none
    const long double fixed = roundl(ldexpl(turns, 64));
    plan->turns[i] = fixed >= ldexpl(1.0L, 64) ? 0 : (uint64_t)fixed;
  }
  plan->head_dim = c->head_dim;
  plan->rotary_dim = R;
  plan->interleaved = c->interleaved;
  plan->magnitude = c->magnitude != 0                ? (float)c->magnitude
                    : c->scaling == SDPA_ROPE_YARN && f > 1 ? (float)(0.1L * logl(f) + 1)
                                                     : 1.0f;
  return SDPA_OK;
}

extern "C" SDPA_API sdpa_status sdpa_rotary(const sdpa_rotary_plan *plan,
                                            const sdpa_rotary_tensor *tensors, int count, int B,
                                            int L, const void *positions, int position_bits,
                                            long long position_batch_stride, long long offset,
                                            int inverse, sdpa_dtype dtype, sdpa_stream_t stream) {
  set_error(SDPA_OK, "");
  if (!plan || !tensors) return bad("plan and tensors must be non-NULL");
  if (count != 1 && count != 2) return bad("count must be 1 or 2 (got %.0f)", count);
  const int D = plan->head_dim, R = plan->rotary_dim;
  if (D < 2 || D > 512 || R < 2 || R > D || R % 2 != 0 ||
      (plan->interleaved != 0 && plan->interleaved != 1))
    return bad("the plan was not filled by sdpa_rotary_init");
  if (dtype != SDPA_BF16 && dtype != SDPA_F16)
    return set_error(SDPA_ERR_UNSUPPORTED, "dtype is not supported (bf16 = 0, f16 = 1)");
  if (B < 1 || L < 1) return bad("B and L must be >= 1 (got B=%.0f L=%.0f)", B, L);
  if ((long long)B * L > 0x7fffffffLL)
    return set_error(SDPA_ERR_UNSUPPORTED, "B*L must stay below 2^31");
  if (inverse != 0 && inverse != 1) return bad("inverse must be 0 or 1 (got %.0f)", inverse);
  if (positions ? (position_bits != 32 && position_bits != 64) : position_bits != 0)
    return bad("position_bits must be 32 or 64 with positions, 0 without (got %.0f)", position_bits);
  if (positions && ((reinterpret_cast<uintptr_t>(positions) & (position_bits / 8 - 1)) != 0 ||
                    position_batch_stride < 0))
    return bad("positions must be aligned to their type, with a batch stride >= 0");

  RotaryParams p;
  memset(&p, 0, sizeof(p));
  // Widest run of elements that every row, run and pitch is a multiple of:
  // 16-byte accesses for the common head dims, down to 2 bytes for odd pitches.
  int v = 8;
  auto fit = [&v](unsigned long long x) {
    while (x % v != 0) v >>= 1;
  };
  fit(R / 2);
  fit(D);
  View reads[2], writes[2];
  for (int i = 0; i < count; ++i) {
    const sdpa_rotary_tensor &t = tensors[i];
    if (!t.x || !t.out) return bad("x and out must be non-NULL device pointers");
    if (t.heads < 1) return bad("heads must be >= 1 (got %.0f)", t.heads);
    if ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.out)) & 1u)
      return bad("x and out must be 2-byte aligned");
    // the stride of a dimension of one element is never used
    auto used = [&](sdpa_strides s) {
      if (B == 1) s.batch = 0;
      if (t.heads == 1) s.head = 0;
      if (L == 1) s.token = 0;
      return s;
    };
    const sdpa_strides xs = used(t.x_strides), os = used(t.out_strides);
    for (long long st : {xs.batch, xs.head, xs.token, os.batch, os.head, os.token})
      if (st < 0 || st > (1LL << 40)) return bad("strides must lie in [0, 2^40] (got %.0f)", (double)st);
    for (const sdpa_strides &st : {xs, os})  // (later sums of them stay in 64 bits)
      if ((__int128)(B - 1) * st.batch + (__int128)(t.heads - 1) * st.head + (__int128)(L - 1) * st.token > (1LL << 48))
        return bad("strides must keep a tensor within 2^48 elements");
    if (!apart(os, B, t.heads, L, D))
      return bad("out strides must keep the rows of head_dim elements apart");
    const bool same = t.x == t.out && xs.batch == os.batch && xs.head == os.head && xs.token == os.token;
    if (!same && !disjoint({t.x, xs, t.heads}, {t.out, os, t.heads}, B, L, D))
      return bad("out must be x itself or not overlap it");
    fit(reinterpret_cast<uintptr_t>(t.x) / 2);
    fit(reinterpret_cast<uintptr_t>(t.out) / 2);
    for (long long st : {xs.batch, xs.head, xs.token, os.batch, os.head, os.token}) fit((unsigned long long)st);
    p.t[i] = {static_cast<const uint16_t *>(t.x), static_cast<uint16_t *>(t.out),
              xs.batch, xs.head, xs.token, os.batch, os.head, os.token};
    p.heads[i] = t.heads;
    reads[i] = {t.x, xs, t.heads};
    writes[i] = {t.out, os, t.heads};
    if (p.heads[0] + p.heads[1] > 0xffff) return set_error(SDPA_ERR_UNSUPPORTED, "more than 65535 heads in one call");
  }
  if (count == 2 && !(disjoint(writes[0], writes[1], B, L, D) && disjoint(writes[0], reads[1], B, L, D) &&
                      disjoint(writes[1], reads[0], B, L, D)))
    return bad("out must not overlap x or out of another tensor of the call");
  int sms;
  unsigned int *wd;
  uint64_t limit;
  sdpa_status st = device_info(&sms, &wd, &limit);
  if (st != SDPA_OK) return st;

  p.L = L;
  p.tokens = (long long)B * L;
  p.rot_items = R / 2 / v;
  p.copy_items = (D - R + 2 * v - 1) / (2 * v);
  p.dim = D;
  p.tokens_per_cta = kThreads / (p.rot_items + p.copy_items);  // at least 1: D <= 512
  p.half = R / 2;
  p.positions = positions;
  p.position_bits = position_bits;
  p.position_batch_stride = position_batch_stride;
  p.offset = offset;
  p.inverse = inverse;
  p.magnitude = plan->magnitude;
  memcpy(p.turns, plan->turns, sizeof(p.turns));
  // Heads per thread: as many as leave three threads for each of the device's
  // resident slots at half occupancy, so that the angles are shared, in whole
  // batches of kBatch; fewer only where the tokens are too few to give every SM
  // two CTAs otherwise (decode: a head per thread).
  const long long threads = p.tokens * (p.rot_items + p.copy_items), heads = p.heads[0] + p.heads[1];
  const int most = std::max(p.heads[0], p.heads[1]);
  long long group = heads * threads / (3LL * sms * 1024);
  if (group < kBatch && heads * threads >= (long long)kBatch * sms * 2 * kThreads) group = kBatch;
  if (group > kBatch) group = (group + kBatch - 1) / kBatch * kBatch;
  p.group = (int)std::min<long long>(most, std::max<long long>(1, group));
  p.groups0 = (p.heads[0] + p.group - 1) / p.group;
  const int groups = p.groups0 + (p.heads[1] + p.group - 1) / p.group;
  const long long ctas = (p.tokens + p.tokens_per_cta - 1) / p.tokens_per_cta;
  if (ctas > 0x7fffffffLL) return set_error(SDPA_ERR_UNSUPPORTED, "too many tokens for one launch");
  const dim3 grid((unsigned)ctas, (unsigned)groups);
  const cudaStream_t cs = (cudaStream_t)stream;
  const bool il = plan->interleaved != 0;
  cudaError_t e = dtype == SDPA_BF16 ? (il ? launch_width<true, true>(v, grid, cs, p) : launch_width<true, false>(v, grid, cs, p))
                                     : (il ? launch_width<false, true>(v, grid, cs, p) : launch_width<false, false>(v, grid, cs, p));
  if (e != cudaSuccess)
    return set_error(SDPA_ERR_CUDA, std::string("rotary_kernel launch failed: ") + cudaGetErrorString(e));
  return SDPA_OK;
}
