// C ABI of the backward pass: checks, the choice of path, workspace, launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "bwd_rows.cuh"
#include "launch_bwd.h"

namespace sdpa {
namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

sdpa_status refuse(sdpa_status st, const char *msg) { return set_error(st, msg); }

// Up to this many pairs of row and key, P and dS enter their products as two
// 16-bit terms unless the caller says otherwise.  What it steadies is the error of the
// results as a whole: one term's is 1.41 times that of exact weights on average at any
// size, up to 1.8 times where the whole call has a handful of rows, 1.45 at most above
// 2^20 pairs.  (A single row's error is no smaller for the other rows of a call.)  What
// it costs below the limit, on the device, one term against two: 8.3 and 8.3 us at 16 x
// 16, 9.3 and 12.2 at 4 heads of 128 x 128, 10.3 and 12.4 at 8 of 362 x 362 (head dim
// 64), 26.5 and 26.7 at 4 of 512 x 512 (256), 158 and 167 at 16 rows over 60000 keys;
// above it 50 and 54 at 2^22 pairs of head dim 256, 62 and 86 at 2^25 of 64.
constexpr long long kTwoTermPairs = 1 << 20;

// Blocks each part of a split tile keeps at least: below that its operand
// loads and its share of the join cost more than the parallelism gives.
constexpr int kMinBlocksPerPart = 4;
// ... and lists are only split when the longest is this much longer than an SM's
// share; then every list of more than `per` blocks is cut.  Limits of 1.0 to 1.2 cut the
// causal 192/128 case, whose longest list is 1.3 shares, at half of that, and most of
// its lists with it: 2 to 6 % slower (a ragged chunk 18 %; no gain elsewhere).  Cutting
// the few longest alone was not tried.
constexpr double kSplitOver = 1.5;

sdpa_status make_bwd_plan(const Problem &pb, int sms, int weight_terms, BwdPlan *out) {
  BwdPlan pl;
  memset(&pl, 0, sizeof(pl));
  const long long rows = (long long)pb.Hq / pb.Hkv * pb.L;
  if (rows > (1 << 30) || pb.S > (1 << 30))  // tile and block ends stay in 32 bits
    return refuse(SDPA_ERR_UNSUPPORTED, "more than 2^30 packed query rows per KV head, or keys");
  pl.rows = (int)rows;
  if (weight_terms < 0 || weight_terms > 2) return refuse(SDPA_ERR_INVALID_ARG, "weight_terms must be 0, 1 or 2");
  pl.weight_terms = weight_terms != 0                                             ? weight_terms
                    : (double)pb.B * pb.Hq * pb.L * pb.S <= (double)kTwoTermPairs ? 2
                                                                                  : 1;
  pl.pair = 0;
  while (kDimPairs[pl.pair].dqk < pb.Dqk || kDimPairs[pl.pair].dv < pb.Dv) ++pl.pair;  // (512/512 covers all)
  pl.rpad = (pl.rows + 127) / 128 * 128;
  pl.key_splits = pl.row_splits = 1;
  const size_t slabs = (size_t)pb.B * pb.Hkv;
  const DimPair dp = kDimPairs[pl.pair];
  const int bk = bwd_tc_key_block(dp.dqk, dp.dv), bq = bwd_tc_query_block(dp.dqk, dp.dv);
  if (128 % bk != 0) pl.rpad += 128;  // a last block may end behind the padding
  // Split a tile's block list where one tile would outlast the whole grid's
  // work spread over the SMs (few tiles with long lists: few query rows over
  // many keys, one KV head under many rows, the first keys of a causal call).
  // Work in pairs of row and key, times 4 products in a key tile, 3 in a query tile:
  // an SM's share by the pairs that the mask leaves, a list by its whole tiles, so that
  // a few rows, which fill little of a tile, are cut into more parts than they need.
  const int g = pb.Hq / pb.Hkv;
  const double first = pb.causal ? std::min<double>(pb.S, pb.q_offset + 1.0) : pb.S;
  const double last = pb.causal ? std::min<double>(pb.S, (double)pb.q_offset + pb.L) : pb.S;
  double per_row = 0.5 * (first + last);  // keys that a row sees, on average
  if (pb.window > 0) per_row = std::min<double>(per_row, pb.window);
  const double ideal = (double)slabs * g * pb.L * per_row * 7 / sms;
  // the longest lists: of the first keys, and of the last rows (whose tile
  // spans all positions where it runs over the end of a head)
  const long long seen_rows = pb.window > 0 ? std::min<long long>(pb.L, (long long)pb.window + 128) : pb.L;
  const long long span = g > 1 && pb.L % 128 != 0 ? pb.L : std::min(pb.L, 128);
  const long long row_keys = pb.window > 0 ? std::min<long long>(last, pb.window + span) : (long long)last;
  const long long kb = (g * seen_rows + bk - 1) / bk, rb = (row_keys + bq - 1) / bq;
  auto parts = [&](long long blocks, int pairs, int *per) {
    const double over = (double)blocks * pairs * 128 / ideal;
    int n = 1;
    if (over > kSplitOver) n = (int)std::max(1.0, std::min(std::ceil(over), (double)(blocks / kMinBlocksPerPart)));
    *per = (int)((blocks + n - 1) / n);
    return n;
  };
  pl.key_splits = parts(kb, 4 * bk, &pl.key_per);
  pl.row_splits = parts(rb, 3 * bq, &pl.row_per);
  pl.rows_first = (long long)pl.row_per * bq * 3 > (long long)pl.key_per * bk * 4;
  if (pl.key_splits > 1) {
    pl.key_part1_bytes = align256((size_t)pl.key_splits * slabs * pb.S * dp.dqk * sizeof(float));
    pl.key_part2_bytes = align256((size_t)pl.key_splits * slabs * pb.S * dp.dv * sizeof(float));
  }
  if (pl.row_splits > 1)
    pl.row_part_bytes = align256((size_t)pl.row_splits * slabs * pl.rows * dp.dqk * sizeof(float));
  if (pl.key_splits > 1 || pl.row_splits > 1)
    pl.count_bytes = align256(slabs * ((pb.S + 127) / 128 + (pl.rows + 127) / 128) * sizeof(int));
  pl.row_bytes = align256(slabs * pl.rpad * sizeof(float));
  pl.norm_bytes = align256(slabs * 16);
  pl.ws_bytes = 2 * pl.row_bytes + pl.norm_bytes + pl.count_bytes + pl.key_part1_bytes + pl.key_part2_bytes + pl.row_part_bytes;
  *out = pl;
  return SDPA_OK;
}

struct Range {
  const void *p;
  size_t n;
};

}  // namespace
}  // namespace sdpa

using namespace sdpa;

static Problem bwd_problem(int B, int Hq, int Hkv, int L, int S, int Dqk, int Dv, float scale,
                           int causal, int window, sdpa_dtype dtype,
                           const sdpa_backward_options *opt) {
  Problem p;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.L = L; p.S = S; p.Dqk = Dqk; p.Dv = Dv;
  p.scale = scale; p.causal = causal; p.window = window; p.dtype = dtype;
  p.has_q_offset = opt != nullptr && opt->has_q_offset ? 1 : 0;
  p.q_offset = p.has_q_offset ? opt->q_offset : S - L;
  return p;
}

extern "C" SDPA_API size_t sdpa_backward_workspace_bytes(int B, int Hq, int Hkv, int L, int S,
                                                         int Dqk, int Dv, int causal,
                                                         int window_size, sdpa_dtype dtype,
                                                         const sdpa_backward_options *opt) {
  set_error(SDPA_OK, "");
  const Problem pb = bwd_problem(B, Hq, Hkv, L, S, Dqk, Dv, 1.f, causal, window_size, dtype, opt);
  if (validate_problem(pb) != SDPA_OK) return 0;
  int sms;
  unsigned int *wd;
  uint64_t limit;
  if (device_info(&sms, &wd, &limit) != SDPA_OK) return 0;
  BwdPlan pl;
  if (make_bwd_plan(pb, sms, opt ? opt->weight_terms : 0, &pl) != SDPA_OK) return 0;
  return pl.ws_bytes;
}

extern "C" SDPA_API sdpa_status sdpa_backward(
    const void *q, const void *k, const void *v, const void *out, const float *lse,
    const void *dout, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int L, int S, int Dqk,
    int Dv, float scale, int causal, int window_size, sdpa_dtype dtype,
    const sdpa_backward_options *opt, void *workspace, size_t workspace_bytes,
    sdpa_stream_t stream) {
  set_error(SDPA_OK, "");
  const Problem pb = bwd_problem(B, Hq, Hkv, L, S, Dqk, Dv, scale, causal, window_size, dtype, opt);
  sdpa_status st = validate_problem(pb);
  if (st != SDPA_OK) return st;
  const float *sinks = opt ? opt->sinks : nullptr, *dlse = opt ? opt->dlse : nullptr;
  float *dsinks = opt ? opt->dsinks : nullptr;
  if (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv)
    return refuse(SDPA_ERR_INVALID_ARG, "q, k, v, out, lse, dout, dq, dk and dv must be non-NULL device pointers");
  for (const void *p : {q, k, v, out, dout, (const void *)dq, (const void *)dk, (const void *)dv})
    if (reinterpret_cast<uintptr_t>(p) & 15u)
      return refuse(SDPA_ERR_INVALID_ARG, "q, k, v, out, dout, dq, dk and dv must be 16-byte aligned");
  for (const float *p : {lse, sinks, dlse, (const float *)dsinks})
    if (reinterpret_cast<uintptr_t>(p) & 3u)
      return refuse(SDPA_ERR_INVALID_ARG, "lse, sinks, dlse and dsinks must be 4-byte aligned");
  if (dsinks && !sinks) return refuse(SDPA_ERR_INVALID_ARG, "dsinks needs sinks");
  const size_t rows = (size_t)B * Hq * L, keys = (size_t)B * Hkv * S;
  const Range in[] = {{q, rows * Dqk * 2}, {k, keys * Dqk * 2},  {v, keys * Dv * 2}, {out, rows * Dv * 2},
                      {dout, rows * Dv * 2}, {lse, rows * 4}, {sinks, sinks ? (size_t)Hq * 4 : 0}, {dlse, dlse ? rows * 4 : 0}};
  const Range to[] = {{dq, rows * Dqk * 2}, {dk, keys * Dqk * 2}, {dv, keys * Dv * 2}, {dsinks, dsinks ? (size_t)Hq * 4 : 0}};
  for (int i = 0; i < 4; ++i) {
    if (to[i].n == 0) continue;
    for (const Range &r : in)
      if (r.n && extents_meet(to[i].p, to[i].n, r.p, r.n))
        return refuse(SDPA_ERR_INVALID_ARG, "a gradient must not overlap an input");
    for (int j = 0; j < i; ++j)
      if (to[j].n && extents_meet(to[i].p, to[i].n, to[j].p, to[j].n))
        return refuse(SDPA_ERR_INVALID_ARG, "the gradients must not overlap each other");
  }
  const bool own_ws = workspace == nullptr && workspace_bytes == 0;
  if (!own_ws && (reinterpret_cast<uintptr_t>(workspace) & 15u))
    return refuse(SDPA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");

  BwdLaunch ln;
  memset(&ln, 0, sizeof(ln));
  st = device_info(&ln.sms, &ln.wd_word, &ln.wd_limit_ns);
  if (st != SDPA_OK) return st;
  st = make_bwd_plan(pb, ln.sms, opt ? opt->weight_terms : 0, &ln.plan);
  if (st != SDPA_OK) return st;
  const BwdPlan &pl = ln.plan;
  const cudaStream_t cs = (cudaStream_t)stream;
  if (own_ws) {
    st = pool_alloc(&workspace, pl.ws_bytes, cs, "backward");
    if (st != SDPA_OK) return st;
  } else if (workspace == nullptr || workspace_bytes < pl.ws_bytes) {
    char buf[128];
    snprintf(buf, sizeof(buf), "workspace of %zu bytes needed, %zu given", pl.ws_bytes,
             workspace == nullptr ? (size_t)0 : workspace_bytes);
    return refuse(SDPA_ERR_RESOURCES, buf);
  }
  for (const Range &r : in)
    if (!own_ws && r.n && extents_meet(workspace, pl.ws_bytes, r.p, r.n))
      return refuse(SDPA_ERR_INVALID_ARG, "workspace must not overlap a tensor of the call");
  for (const Range &r : to)
    if (!own_ws && r.n && extents_meet(workspace, pl.ws_bytes, r.p, r.n))
      return refuse(SDPA_ERR_INVALID_ARG, "workspace must not overlap a tensor of the call");
  ln.pb = pb;
  ln.q = q; ln.k = k; ln.v = v; ln.out = out; ln.dout = dout;
  ln.dq = dq; ln.dk = dk; ln.dv = dv;
  ln.lse = lse; ln.dlse = dlse;
  char *ws = static_cast<char *>(workspace);
  ln.nlse = reinterpret_cast<float *>(ws);
  ln.ndelta = reinterpret_cast<float *>(ws + pl.row_bytes);
  ln.norms = reinterpret_cast<unsigned int *>(ws + 2 * pl.row_bytes);
  ws += 2 * pl.row_bytes + pl.norm_bytes;
  ln.key_parts = reinterpret_cast<int *>(ws);
  ln.row_parts = ln.key_parts + (size_t)B * Hkv * ((S + 127) / 128);
  ws += pl.count_bytes;
  ln.key_part1 = reinterpret_cast<float *>(ws);
  ln.key_part2 = reinterpret_cast<float *>(ws + pl.key_part1_bytes);
  ln.row_part = reinterpret_cast<float *>(ws + pl.key_part1_bytes + pl.key_part2_bytes);
  ln.stream = cs;

  std::string err;
  st = dtype == SDPA_BF16 ? launch_bwd_bf16(ln, &err) : launch_bwd_f16(ln, &err);
  if (st == SDPA_OK && dsinks) {
    bwd_sinks_kernel<<<Hq, kBwdSinksThreads, 0, cs>>>(sinks, lse, ln.ndelta, dsinks, B, Hq, Hkv, L, pl.rpad);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
      err = std::string("bwd_sinks_kernel launch failed: ") + cudaGetErrorString(e);
      st = SDPA_ERR_CUDA;
    }
  }
  if (own_ws) {
    cudaError_t e = cudaFreeAsync(workspace, cs);
    if (st == SDPA_OK && e != cudaSuccess) {
      err = std::string("cudaFreeAsync: ") + cudaGetErrorString(e);
      st = SDPA_ERR_CUDA;
    }
  }
  return st == SDPA_OK ? SDPA_OK : set_error(st, err);
}

namespace sdpa {

sdpa_status launch_bwd_rows(const BwdLaunch &ln, std::string *err) {
  const Problem &pb = ln.pb;
  const long long slabs = (long long)pb.B * pb.Hkv;
  const bool bf16 = pb.dtype == SDPA_BF16;
  BwdRowsParams p;
  p.out = ln.out; p.dout = ln.dout; p.v = ln.v;
  p.lse = ln.lse; p.dlse = ln.dlse;
  p.nlse = ln.nlse; p.ndelta = ln.ndelta; p.norms = ln.norms;
  p.R = ln.plan.rows; p.rpad = ln.plan.rpad; p.S = pb.S; p.Dv = pb.Dv;
  p.row_ctas = slabs * p.rpad / kBwdRowsPerCta;
  p.v_ctas = bf16 ? 0 : (pb.S + kBwdRowsPerCta - 1) / kBwdRowsPerCta;
  const long long ctas = p.row_ctas + slabs * p.v_ctas;
  if (ctas > 0x7fffffffLL) {  // (the first launch of a call: nothing is enqueued yet)
    *err = "problem needs more than 2^31 CTAs for its row terms";
    return SDPA_ERR_UNSUPPORTED;
  }
  cudaError_t e = cudaSuccess;
  if (!bf16) e = cudaMemsetAsync(ln.norms, 0, slabs * 16, ln.stream);
  if (e == cudaSuccess) {
    if (bf16)
      bwd_rows_kernel<true><<<(unsigned)ctas, kBwdRowsThreads, 0, ln.stream>>>(p);
    else
      bwd_rows_kernel<false><<<(unsigned)ctas, kBwdRowsThreads, 0, ln.stream>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    *err = std::string("bwd_rows_kernel launch failed: ") + cudaGetErrorString(e);
    return SDPA_ERR_CUDA;
  }
  return SDPA_OK;
}

void fill_bwd_params(const BwdLaunch &ln, BwdParams *p) {
  const Problem &pb = ln.pb;
  memset(p, 0, sizeof(*p));
  AttnParams &a = p->a;
  a.B = pb.B; a.Hq = pb.Hq; a.Hkv = pb.Hkv; a.L = pb.L; a.S = pb.S; a.Dqk = pb.Dqk; a.Dv = pb.Dv;
  a.R = ln.plan.rows;
  a.off = pb.q_offset;
  a.causal = pb.causal;
  a.window = pb.window;
  a.scale_log2 = pb.scale * 1.4426950408889634f;
  a.splits = 1;
  a.wd.word = ln.wd_word;
  a.wd.limit_ns = ln.wd_limit_ns;
  p->nlse = ln.nlse; p->ndelta = ln.ndelta; p->norms = ln.norms;
  p->rpad = ln.plan.rpad;
  p->scale = pb.scale;
  p->q = ln.q; p->k = ln.k; p->v = ln.v; p->dout = ln.dout;
  p->dq = ln.dq; p->dk = ln.dk; p->dv = ln.dv;
}

}  // namespace sdpa
