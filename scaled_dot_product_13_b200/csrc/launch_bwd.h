// Host-side declarations of the backward pass.
#pragma once

#include "launch.h"

namespace sdpa {

struct BwdParams;

struct BwdPlan {
  int path;   // an sdpa_backward_path value other than AUTO
  int rows;   // packed query rows per (batch, KV head)
  int rpad;   // ... rounded up to 128
  size_t row_bytes, norm_bytes, ws_bytes;
};

struct BwdLaunch {
  Problem pb;
  BwdPlan plan;
  const void *q, *k, *v, *out, *dout;
  void *dq, *dk, *dv;
  const float *lse, *dlse;
  float *nlse, *ndelta;
  unsigned int *norms;
  int sms;
  unsigned int *wd_word;
  uint64_t wd_limit_ns;
  cudaStream_t stream;
};

// Kernel parameters common to the paths.
void fill_bwd_params(const BwdLaunch &ln, BwdParams *p);

sdpa_status launch_bwd_rows(const BwdLaunch &ln, std::string *err);
sdpa_status launch_bwd_tile(const BwdLaunch &ln, std::string *err);

}  // namespace sdpa
