// Launches of the tcgen05 backward kernel and its join; included by one unit per
// type.
#include "bwd_tc.cuh"
#include "launch_bwd.h"

namespace sdpa {

namespace {

template <bool kBF16>
cudaError_t join(const BwdLaunch &ln, const BwdParams &p, const BwdTcSpan &span, const float *part, void *out,
                 int rows_per_slab, int d, int dpad, int is_dv) {
  const long long rows = (long long)ln.pb.B * ln.pb.Hkv * rows_per_slab;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows * (d / 4) + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = ln.stream;
  return cudaLaunchKernelEx(&cfg, bwd_join_kernel<kBF16>, p, part, (uint16_t *)out, (const int *)span.parts,
                            span.tiles, rows, rows_per_slab, d, dpad, is_dv);
}

template <bool kBF16, bool TWO, int DQK, int DV>
sdpa_status run(const BwdLaunch &ln, std::string *err) {
  using Roles = BwdTcRoles<DQK, DV>;
  static_assert(Roles::Key::BN == bwd_tc_key_block(DQK, DV) && Roles::Query::BN == bwd_tc_query_block(DQK, DV),
                "the plan counts the kernel's blocks");
  if constexpr (!std::is_void_v<typename Roles::KeyV>)
    static_assert(Roles::KeyV::BN == Roles::Key::BN, "both read the same boxes of Q and dO");
  auto kern = bwd_tc_kernel<kBF16, TWO, DQK, DV>;
  sdpa_status st = prepare_kernel((const void *)kern, kBwdTcThreads, Roles::kSmem, "bwd_tc_kernel", err);
  if (st != SDPA_OK) return st;
  const Problem &pb = ln.pb;
  const BwdPlan &pl = ln.plan;
  BwdParams p;
  fill_bwd_params(ln, &p);
  const long long slabs = (long long)pb.B * pb.Hkv;
  BwdTcSpan keys = {(pb.S + 127) / 128, pl.key_splits, pl.key_per, ln.key_parts, ln.key_part1, ln.key_part2};
  BwdTcSpan rows = {(pl.rows + 127) / 128, pl.row_splits, pl.row_per, ln.row_parts, ln.row_part, nullptr};
  const long long key_ctas = slabs * keys.tiles * keys.splits, row_ctas = slabs * rows.tiles * rows.splits;
  long long ctas = key_ctas * bwd_col_parts<typename Roles::Key>(pb.Dqk) + row_ctas * bwd_col_parts<typename Roles::Query>(pb.Dqk);
  if constexpr (!std::is_void_v<typename Roles::KeyV>) ctas += key_ctas * bwd_col_parts<typename Roles::KeyV>(pb.Dv);
  const long long join_ctas = slabs * (pb.S > pl.rows ? (long long)pb.S : pl.rows) * 128 / 256;
  if (ctas > 0x7fffffffLL || join_ctas > 0x7fffffffLL) {
    *err = "problem needs more than 2^31 CTAs";
    return SDPA_ERR_UNSUPPORTED;
  }
  auto map = [&](CUtensorMap *m, const void *base, int d, int n, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)d, (uint64_t)n, (uint64_t)slabs};
    const uint64_t strides[2] = {(uint64_t)d * 2, (uint64_t)n * d * 2};
    const uint32_t box[3] = {64, (uint32_t)box_rows, 1};
    return encode_tma(m, pb.dtype, 3, base, dims, strides, box, err);
  };
  constexpr int BK = Roles::Key::BN, BQ = Roles::Query::BN, BX = Roles::Key::kBoxRows;
  const int R = pl.rows, S = pb.S, Dqk = pb.Dqk, Dv = pb.Dv;
  BwdTcMaps tm;
  if (!map(&tm.q, ln.q, Dqk, R, BX) || !map(&tm.k, ln.k, Dqk, S, BX) || !map(&tm.v, ln.v, Dv, S, BX) ||
      !map(&tm.dout, ln.dout, Dv, R, BX) || !map(&tm.dq, ln.dq, Dqk, R, 128) ||
      !map(&tm.dk, ln.dk, Dqk, S, 128) || !map(&tm.dv, ln.dv, Dv, S, 128))
    return SDPA_ERR_CUDA;
  tm.qb = tm.q;
  tm.doutb = tm.dout;
  tm.kb = tm.k;
  tm.vb = tm.v;
  if (BK != BX && (!map(&tm.qb, ln.q, Dqk, R, BK) || !map(&tm.doutb, ln.dout, Dv, R, BK))) return SDPA_ERR_CUDA;
  if (BQ != BX && (!map(&tm.kb, ln.k, Dqk, S, BQ) || !map(&tm.vb, ln.v, Dv, S, BQ))) return SDPA_ERR_CUDA;

  // (behind every check that may still refuse the call)
  st = launch_bwd_rows(ln, err);
  if (st != SDPA_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kBwdTcThreads);
  cfg.dynamicSmemBytes = Roles::kSmem;
  cfg.stream = ln.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tm, p, keys, rows, pl.rows_first);
  if (e == cudaSuccess && pl.key_splits > 1)
    e = join<kBF16>(ln, p, keys, keys.part1, ln.dk, S, Dqk, DQK, 0);
  if (e == cudaSuccess && pl.key_splits > 1)
    e = join<kBF16>(ln, p, keys, keys.part2, ln.dv, S, Dv, DV, 1);
  if (e == cudaSuccess && pl.row_splits > 1)
    e = join<kBF16>(ln, p, rows, rows.part1, ln.dq, R, Dqk, DQK, 0);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    *err = std::string("bwd_tc_kernel launch failed: ") + cudaGetErrorString(e);
    return SDPA_ERR_CUDA;
  }
  return SDPA_OK;
}

template <bool kBF16, bool TWO>
sdpa_status run_pair(const BwdLaunch &ln, std::string *err) {
  switch (ln.plan.pair) {
    case 0: return run<kBF16, TWO, 64, 64>(ln, err);
    case 1: return run<kBF16, TWO, 80, 80>(ln, err);
    case 2: return run<kBF16, TWO, 128, 128>(ln, err);
    case 3: return run<kBF16, TWO, 192, 128>(ln, err);
    case 4: return run<kBF16, TWO, 192, 192>(ln, err);
    case 5: return run<kBF16, TWO, 256, 256>(ln, err);
    case 6: return run<kBF16, TWO, 512, 512>(ln, err);
  }
  *err = "internal: no tcgen05 backward instance for this head-dim pair";
  return SDPA_ERR_UNSUPPORTED;
}

template <bool kBF16>
sdpa_status run_dtype(const BwdLaunch &ln, std::string *err) {
  return ln.plan.weight_terms == 2 ? run_pair<kBF16, true>(ln, err) : run_pair<kBF16, false>(ln, err);
}

}  // namespace

// (the bf16 and fp16 instances are compiled in two units, to build in parallel)
#if SDPA_BWD_BF16
sdpa_status launch_bwd_bf16(const BwdLaunch &ln, std::string *err) { return run_dtype<true>(ln, err); }
#else
sdpa_status launch_bwd_f16(const BwdLaunch &ln, std::string *err) { return run_dtype<false>(ln, err); }
#endif

}  // namespace sdpa
