// fa_cache_ops.cu -- host side of the entry points around drafted trees and
// the eviction from the paged cache.  Argument checks, launch shapes,
// launches; nothing here copies data, synchronises or allocates.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "draft_tree_kernel.cuh"
#include "host_common.h"

using fa::is_aligned;

namespace {

fa_status launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH; }

}  // namespace

extern "C" fa_status fa_draft_tree(const int* parents, const int* cu_seqlens, const int* seq_lens,
                                   int batch, int total, int tree_words, int* tree_mask,
                                   int* positions, fa_stream_t stream) {
  if (!cu_seqlens || !seq_lens || (total > 0 && (!parents || !tree_mask))) return FA_ERR_INVALID_ARG;
  if (batch < 1 || total < 0 || tree_words < 1) return FA_ERR_INVALID_ARG;
  if (!is_aligned(parents, 4) || !is_aligned(cu_seqlens, 4) || !is_aligned(seq_lens, 4) ||
      !is_aligned(tree_mask, 4) || !is_aligned(positions, 4))
    return FA_ERR_INVALID_ARG;
  if ((int64_t)total * tree_words > INT32_MAX) return FA_ERR_UNSUPPORTED;
  fa::DeviceFacts dev;
  const fa_status st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  if (total == 0) return FA_OK;
  // Blocks for the mean number of nodes; a longer tree's go round.
  const int mean = (int)(((int64_t)total + batch - 1) / batch);
  const int blocks = std::min((mean + fa::kTreeThreads - 1) / fa::kTreeThreads, 1024);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // (A grid has at most 65535 blocks in y.)
  for (int b0 = 0; b0 < batch; b0 += 65535) {
    const fa::DraftTreeArgs a = {parents,    cu_seqlens + b0, seq_lens + b0, total,
                                 tree_words, tree_mask,       positions};
    fa::draft_tree_kernel<<<dim3(blocks, std::min(batch - b0, 65535)), fa::kTreeThreads, 0, s>>>(a);
  }
  return launched();
}
