// Instantiation of the varlen forward kernel with sinks and trees for d_qk = 64, d_v = 64.
#include "varlen_fwd_kernel.cuh"
FA_DEFINE_MASKED_LAUNCHER(64, 64)
