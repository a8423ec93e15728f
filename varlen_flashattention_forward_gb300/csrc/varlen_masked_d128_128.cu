// Instantiation of the varlen forward kernel with sinks and trees for d_qk = 128, d_v = 128.
#include "varlen_fwd_kernel.cuh"
FA_DEFINE_MASKED_LAUNCHER(128, 128)
