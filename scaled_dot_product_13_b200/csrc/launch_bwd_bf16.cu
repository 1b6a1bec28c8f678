// Launch unit of the backward kernels, bf16.
#define SDPA_BWD_BF16 1
#include "launch_bwd_tc.inl"
