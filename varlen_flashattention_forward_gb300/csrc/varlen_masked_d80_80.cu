// Instantiation of the varlen forward kernel with sinks and trees for d_qk = 80, d_v = 80.
#include "varlen_fwd_kernel.cuh"
FA_DEFINE_MASKED_LAUNCHER(80, 80)
