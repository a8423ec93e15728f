// fa_cache_ops.cu -- host side of the entry points around drafted trees and
// the eviction from the paged cache.  Argument checks, launch shapes,
// launches; nothing here copies data, synchronises or allocates.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "draft_tree_kernel.cuh"
#include "host_common.h"
#include "key_weights_kernel.cuh"
#include "kv_evict_kernels.cuh"
#include "paged_host.h"

using fa::is_aligned;

namespace {

template <int D, int N>
cudaError_t launch_weights(const CUtensorMap& map, const fa::KeyWeightsArgs& a, int sm_count,
                           cudaStream_t stream) {
  // Set once per device; concurrent first calls may both set it (the call is
  // idempotent), the flag itself is atomic.
  static std::atomic<bool> attr_done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const int smem = (int)fa::weights_smem<D, N>();
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(fa::key_weights_kernel<D, N>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_done[dev].store(true, std::memory_order_release);
  }
  fa::key_weights_kernel<D, N>
      <<<sm_count * fa::WeightsCfg<D, N>::kResident, fa::WeightsCfg<D, N>::kThreads, smem, stream>>>(map, a);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_weights_rows(const CUtensorMap& map, const fa::KeyWeightsArgs& a, int sm_count,
                                cudaStream_t stream) {
  switch (a.shape.rows) {
    case 16: return launch_weights<D, 16>(map, a, sm_count, stream);
    case 32: return launch_weights<D, 32>(map, a, sm_count, stream);
    case 64: return launch_weights<D, 64>(map, a, sm_count, stream);
    default: return launch_weights<D, 128>(map, a, sm_count, stream);
  }
}

fa_status launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH; }

}  // namespace

extern "C" fa_status fa_draft_tree(const int* parents, const int* cu_seqlens, const int* seq_lens,
                                   int batch, int total, int tree_words, int* tree_mask,
                                   int* positions, fa_stream_t stream) {
  return fa_draft_tree_windowed(parents, cu_seqlens, seq_lens, batch, total, tree_words, -1, 0,
                                tree_mask, positions, stream);
}

extern "C" fa_status fa_draft_tree_windowed(const int* parents, const int* cu_seqlens,
                                            const int* seq_lens, int batch, int total,
                                            int tree_words, int window_left, int sink_tokens,
                                            int* tree_mask, int* positions, fa_stream_t stream) {
  if (!cu_seqlens || !seq_lens || (total > 0 && (!parents || !tree_mask))) return FA_ERR_INVALID_ARG;
  if (batch < 1 || total < 0 || tree_words < 1 || window_left < -1 || sink_tokens < 0)
    return FA_ERR_INVALID_ARG;
  if (!is_aligned(parents, 4) || !is_aligned(cu_seqlens, 4) || !is_aligned(seq_lens, 4) ||
      !is_aligned(tree_mask, 4) || !is_aligned(positions, 4))
    return FA_ERR_INVALID_ARG;
  // (A sequence's threads step over its nodes together: a node's number passes the last
  // by as many at most.)
  constexpr int kMostNodes = INT32_MAX - fa::kTreeBlocks * fa::kTreeThreads;
  if ((int64_t)total * tree_words > INT32_MAX || total > kMostNodes) return FA_ERR_UNSUPPORTED;
  fa::DeviceFacts dev;
  const fa_status st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  if (total == 0) return FA_OK;
  // Blocks for the mean number of nodes; a longer tree's go round.
  const int mean = (int)(((int64_t)total + batch - 1) / batch);
  const int blocks = std::min((mean + fa::kTreeThreads - 1) / fa::kTreeThreads, fa::kTreeBlocks);
  const int window = window_left < 0 ? INT32_MAX : window_left;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // (A grid has at most 65535 blocks in y.)
  for (int b0 = 0; b0 < batch; b0 += 65535) {
    const fa::DraftTreeArgs a = {parents, cu_seqlens + b0, seq_lens + b0, total,    tree_words,
                                 window,  sink_tokens,     tree_mask,     positions};
    fa::draft_tree_kernel<<<dim3(blocks, std::min(batch - b0, 65535)), fa::kTreeThreads, 0, s>>>(a);
  }
  return launched();
}

extern "C" fa_status fa_paged_key_weights(
    const void* q, long long q_row_stride, long long q_head_stride, const float* lse,
    const void* k_cache, const float* k_scale, const int* cu_seqlens_q, const int* seq_lens,
    const int* page_table, int batch, int total_q, int num_heads, int num_heads_k, int head_dim,
    int num_pages, int max_pages_per_seq, float softmax_scale, int causal, int window_left,
    int sink_tokens, float decay, float* weights, int capacity, fa_stream_t stream) {
  if ((total_q > 0 && (!q || !lse)) || !seq_lens || !weights) return FA_ERR_INVALID_ARG;
  fa_status st = fa::check_cache(k_cache, k_cache, k_scale, k_scale, cu_seqlens_q, page_table, batch,
                                 total_q, num_heads_k, head_dim, num_pages, max_pages_per_seq);
  if (st != FA_OK) return st;
  if (num_heads < 1 || num_heads % num_heads_k != 0 || window_left < -1 || sink_tokens < 0 ||
      capacity < 1 || !(softmax_scale > 0.f) || !std::isfinite(softmax_scale) ||
      !(decay >= 0.f && decay <= 1.f))
    return FA_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(lse, 4) || !is_aligned(seq_lens, 4) ||
      !is_aligned(weights, 4))
    return FA_ERR_INVALID_ARG;
  if (total_q > 0 && !fa::settle_view(total_q, num_heads, head_dim, &q_row_stride, &q_head_stride))
    return FA_ERR_INVALID_ARG;
  if ((int64_t)total_q * num_heads > INT32_MAX || num_heads > 65535) return FA_ERR_UNSUPPORTED;
  fa::DeviceFacts dev;
  st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  if (total_q == 0) return FA_OK;
  CUtensorMap map;
  const int dim = head_dim <= 64 ? 64 : 128;
  if (!fa::encode_cache(&map, k_cache, head_dim, num_pages * num_heads_k, dim)) return FA_ERR_LAUNCH;
  // Rows of a chunk: what holds the mean sequence's, at most 128.
  const int group = num_heads / num_heads_k;
  const long long rows = (((int64_t)total_q + batch - 1) / batch) * group;
  const int n = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  fa::KeyWeightsArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.lse = lse;
  a.k_scale = k_scale;
  a.total_q = total_q;
  a.dim = head_dim;
  a.max_pages = max_pages_per_seq;
  a.num_pages = num_pages;
  a.keys = std::min(max_pages_per_seq * fa::kPageTokens, capacity);
  a.shape = {num_heads_k, group, n, causal != 0, window_left, a.keys, sink_tokens, 0};
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  const double log2e = (double)a.scale_log2 / softmax_scale;
  a.lse_log2 = (float)log2e;
  a.lse_log2_rest = (float)(log2e - a.lse_log2);
  a.decay = decay;
  a.capacity = capacity;
  a.status = dev.status;
  a.wait_limit_ns = dev.wait_limit_ns;
  // Costs of a launch are counted in 32 bits (see fa_paged_attn).
  const long long most = (long long)num_heads_k * (a.keys / fa::kTileKeys + 1 + fa::kUnitCost);
  if (most > fa::kMaxCost) return FA_ERR_UNSUPPORTED;
  const int step = (int)std::min<long long>(fa::kWeightMaxBatch, fa::kMaxCost / most);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  for (int b0 = 0; b0 < batch; b0 += step) {
    a.batch = std::min(batch - b0, step);
    a.cu = cu_seqlens_q + b0;
    a.seq_lens = seq_lens + b0;
    a.page_table = page_table + (size_t)b0 * max_pages_per_seq;
    a.weights = weights + (size_t)b0 * num_heads_k * capacity;
    const cudaError_t e = dim == 64 ? launch_weights_rows<64>(map, a, dev.sm_count, s)
                                    : launch_weights_rows<128>(map, a, dev.sm_count, s);
    if (e != cudaSuccess) return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

extern "C" fa_status fa_paged_kv_select(const float* weights, const int* seq_lens, int batch,
                                        int num_heads_k, int capacity, int budget, int sink_tokens,
                                        int recent_tokens, int* keep, int* new_lens,
                                        fa_stream_t stream) {
  if (!weights || !seq_lens || !keep || !new_lens) return FA_ERR_INVALID_ARG;
  if (batch < 1 || num_heads_k < 1 || capacity < 1 || budget < 1 || sink_tokens < 0 ||
      recent_tokens < 0 || (int64_t)sink_tokens + recent_tokens > budget)
    return FA_ERR_INVALID_ARG;
  if (!is_aligned(weights, 4) || !is_aligned(seq_lens, 4) || !is_aligned(keep, 4) ||
      !is_aligned(new_lens, 4))
    return FA_ERR_INVALID_ARG;
  // (A cluster's threads step over keys and budget together: an index passes the end
  // by as many at most.)
  constexpr int kMostKeys = INT32_MAX - fa::kSelectThreads * fa::kSelectCtas;
  if ((int64_t)batch * num_heads_k > INT32_MAX || capacity > kMostKeys || budget > kMostKeys)
    return FA_ERR_UNSUPPORTED;
  fa::DeviceFacts dev;
  const fa_status st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  const fa::KvSelectArgs a = {weights, seq_lens,    num_heads_k,   capacity,
                              budget,  sink_tokens, recent_tokens, keep, new_lens};
  // CTAs of a cluster: what holds a row's keys in registers, and more while each
  // keeps 2048 and all are resident at once.
  const int64_t units = (int64_t)batch * num_heads_k;
  constexpr int kHeld = fa::kSelectThreads * fa::kSelectItems;
  int ctas = 1;
  while (ctas < fa::kSelectCtas && ((int64_t)ctas * kHeld < capacity ||
                      (units * ctas <= dev.sm_count && capacity / ctas > 2048)))
    ctas *= 2;
  if (units * ctas > INT32_MAX) return FA_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3((unsigned)(units * ctas));
  cfg.blockDim = dim3(fa::kSelectThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = (int64_t)ctas * kHeld >= capacity
                            ? cudaLaunchKernelEx(&cfg, fa::kv_select_kernel<fa::kSelectItems>, a)
                            : cudaLaunchKernelEx(&cfg, fa::kv_select_kernel<0>, a);
  return e == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

extern "C" fa_status fa_paged_kv_compact(void* k_cache, void* v_cache, float* k_scale,
                                         float* v_scale, const int* page_table, const int* keep,
                                         const int* first, const int* counts, int batch,
                                         int num_heads_k, int keep_heads, int keep_row, int head_dim,
                                         int num_pages, int max_pages_per_seq, float* weights,
                                         int capacity, fa_stream_t stream) {
  if ((keep_row > 0 && !keep) || !counts) return FA_ERR_INVALID_ARG;
  fa_status st = fa::check_cache(k_cache, v_cache, k_scale, v_scale, counts, page_table, batch, 0,
                                 num_heads_k, head_dim, num_pages, max_pages_per_seq);
  if (st != FA_OK) return st;
  if (keep_row < 0 || (keep_heads != 1 && keep_heads != num_heads_k) || (weights && capacity < 1))
    return FA_ERR_INVALID_ARG;
  if (!is_aligned(keep, 4) || !is_aligned(first, 4) || !is_aligned(weights, 4))
    return FA_ERR_INVALID_ARG;
  const int64_t units = 2ll * batch * num_heads_k;
  if (units * 8 > INT32_MAX) return FA_ERR_UNSUPPORTED;
  fa::DeviceFacts dev;
  st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  if (keep_row == 0) return FA_OK;
  fa::KvCompactArgs a;
  a.page_table = page_table;
  a.keep = keep;
  a.first = first;
  a.counts = counts;
  a.batch = batch;
  a.heads = num_heads_k;
  a.keep_heads = keep_heads;
  a.keep_row = keep_row;
  a.dim = head_dim;
  a.max_pages = max_pages_per_seq;
  a.num_pages = num_pages;
  a.cache[0] = static_cast<uint8_t*>(k_cache);
  a.cache[1] = static_cast<uint8_t*>(v_cache);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.weights = weights;
  a.capacity = weights ? capacity : 0;
  // CTAs of a cluster: more while all units' are resident at once (four an SM)
  // and have pages of their own.
  const int64_t pages = std::min<int64_t>(((int64_t)keep_row + 126) / 64, max_pages_per_seq);
  int ctas = 8;
  while (ctas > 1 && (units * ctas > 4ll * dev.sm_count || ctas / 2 * fa::kCompactPages >= pages))
    ctas /= 2;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3((unsigned)(units * ctas));
  cfg.blockDim = dim3(fa::kCompactThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa::kv_compact_kernel, a) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}
