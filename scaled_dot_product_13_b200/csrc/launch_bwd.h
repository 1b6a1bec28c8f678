// Host-side declarations of the backward pass.
#pragma once

#include "launch.h"

namespace sdpa {

struct BwdParams;

struct BwdPlan {
  int weight_terms;  // 16-bit terms of P and dS: 1 or 2
  int rows;   // packed query rows per (batch, KV head)
  int rpad;   // ... rounded up so that every tile and block stays inside
  int pair;   // index into kDimPairs
  int key_splits, row_splits;  // parts of the longest block list of a key / query tile
  int key_per, row_per;        // blocks of a part
  int rows_first;              // the query tiles have the longer lists: first in the grid
  size_t row_bytes, norm_bytes;
  size_t count_bytes;  // parts of each tile
  size_t key_part1_bytes, key_part2_bytes, row_part_bytes;  // their fp32 sums
  size_t ws_bytes;
};

struct BwdLaunch {
  Problem pb;
  BwdPlan plan;
  const void *q, *k, *v, *out, *dout;
  void *dq, *dk, *dv;
  const float *lse, *dlse;
  float *nlse, *ndelta;
  unsigned int *norms;
  int *key_parts, *row_parts;
  float *key_part1, *key_part2, *row_part;
  int sms;
  unsigned int *wd_word;
  uint64_t wd_limit_ns;
  cudaStream_t stream;
};

// Kernel parameters.
void fill_bwd_params(const BwdLaunch &ln, BwdParams *p);

sdpa_status launch_bwd_rows(const BwdLaunch &ln, std::string *err);  // row terms
// ... and all products
sdpa_status launch_bwd_bf16(const BwdLaunch &ln, std::string *err);
sdpa_status launch_bwd_f16(const BwdLaunch &ln, std::string *err);

// Rows per block: query rows of a key tile's block, keys of
// a query tile's.
constexpr int bwd_tc_key_block(int dqk, int dv) {
  return dqk == 64 ? 96 : dqk == 80 ? 80 : dqk == 512 ? 32 : dqk == 192 && dv == 128 ? 48 : 64;
}
constexpr int bwd_tc_query_block(int dqk, int dv) { return dqk == 64 ? 96 : dqk == 80 ? 80 : dqk == 512 ? 32 : 64; }

}  // namespace sdpa
