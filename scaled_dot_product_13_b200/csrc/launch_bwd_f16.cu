// Launch unit of the backward kernels, fp16.
#define SDPA_BWD_BF16 0
#include "launch_bwd_tc.inl"
