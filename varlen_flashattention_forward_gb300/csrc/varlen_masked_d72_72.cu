// Instantiation of the varlen forward kernel with sinks and trees for d_qk = 72, d_v = 72.
#include "varlen_fwd_kernel.cuh"
FA_DEFINE_MASKED_LAUNCHER(72, 72)
