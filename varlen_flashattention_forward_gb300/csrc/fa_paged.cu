// fa_paged.cu -- host side of the serving entry points around the attention
// forward: q/k norm with rotation, and the paged 8-bit cache (append, gather,
// attention).  Argument checks, launch shapes, launches; nothing here copies
// data, synchronises or allocates.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "host_common.h"
#include "paged_host.h"
#include "paged_kv_kernels.cuh"
#include "paged_launch.cuh"
#include "paged_wide_kernel.cuh"
#include "qk_norm_rope_kernel.cuh"

using fa::cache_dim;
using fa::check_cache;
using fa::encode_cache;
using fa::is_aligned;
using fa::settle_view;

namespace {

// Launch shape of fa_paged_attn.  Rows of a tile: 16 where they hold a
// sequence's rows (the max_seqlen_q hint, else the mean, times the heads of a
// group), else 32.  (4 rows a sequence, 32 of 32768 keys, 8 heads of 128 dims:
// 16 rows 319 us, 32: 364.  8 to 28 rows, 24 sequences, windows of 4096 keys, 8
// heads of 64 dims: 53.6 and 48.7.  Tiles of 64 rows, which read the keys of
// more rows once, lost to 32 for want of registers and buffers: 52 rows, 24
// sequences of 2500 to 5000 keys, 8 heads of 128 dims 137 against 114 us, 64 rows
// and 1 head, 64 sequences of 2000 to 4096 keys 75 against 52.)
struct AttnLaunch {
  int grid, rows, dim;  // CTAs, rows of a tile, padded head dim
  size_t o_bytes, lse_bytes, meta_bytes;
  size_t bytes() const { return o_bytes + lse_bytes + meta_bytes; }
};
// masked: under sinks or a tree, where more than 16 rows go 256 to a tile
// (paged_wide_kernel): trees of 5 and 8 nodes, 4 heads of a group (20 and 32 rows),
// 24 sequences of 517 to 5000 keys, 8 kv heads of 128 dims 64 and 65 us, 32 to a
// tile 70 and 76; 4 nodes (16 rows) 16 to a tile 54 us; 64 nodes 82 against 384.  A
// step behind sinks, windows of 4095 keys, 17, 32 and 64 heads of 128 dims on one kv
// head: 64 sequences of 100 to 16384 keys 38, 38 and 38 us, 16 to a tile 47, 49 and 77; but
// 4 sequences of 8000 to 16384 keys 28, 28 and 29 against 20, 20 and 22 (the change of
// unit, where a CTA has one).
AttnLaunch attn_launch(int sm_count, int batch, int total_q, int group, int head_dim,
                       int max_seqlen_q, bool masked) {
  AttnLaunch l;
  const long long tokens =
      max_seqlen_q > 0 ? max_seqlen_q : ((long long)total_q + batch - 1) / batch;
  const long long rows = tokens * group;
  l.rows = rows <= 16 ? 16 : masked ? fa::kWideRows : 32;
  l.dim = head_dim <= 64 ? 64 : 128;
  l.grid = std::min(sm_count, fa::kPagedMaxGrid);
  l.o_bytes = (size_t)2 * l.grid * l.rows * l.dim * sizeof(float);
  l.lse_bytes = (size_t)2 * l.grid * l.rows * sizeof(float);
  l.meta_bytes = (size_t)2 * l.grid * sizeof(int4);
  return l;
}

// fa_qk_norm_rope takes kNormRopeRows heads of a token together where an SM has
// kNormRopeWide threads' work (8 dims of a row each), else one.  64 tokens x 40
// heads of 128 dims: one 2.25 us, four 2.83; 8192 tokens: 49.2 against 30.1;
// 5003 tokens x 32 heads of 96 dims: 24.7 against 14.6.
constexpr int kNormRopeWide = 8192;
constexpr int kNormRopeRows = 4;
// Blocks of it that an SM gets; they take their units in turn.
constexpr int kNormRopeBlocks = 4;

// Blocks of 256 threads of the prompt append for an SM (three are resident):
// 4 x 2048 tokens x 8 heads of 128 dims 3: 20.5, 4 and 6: 16.7, 8: 18.0,
// 14 (a head each): 21.9 us.
constexpr int kAppendWave = 4;

fa_status launched() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_LAUNCH; }

// Checks that the rotation arguments share.
bool valid_rope(const float* cos_sin, int rot_dim, int max_pos, int head_dim) {
  if (rot_dim < 0 || rot_dim % 16 != 0 || rot_dim > head_dim || max_pos < 0) return false;
  return rot_dim == 0 || (cos_sin != nullptr && is_aligned(cos_sin, 16) && max_pos > 0);
}

}  // namespace

extern "C" fa_status fa_qk_norm_rope(const void* q, long long q_row_stride,
                                     long long q_head_stride, const void* k,
                                     long long k_row_stride, long long k_head_stride,
                                     const int* positions, const float* cos_sin,
                                     const float* q_weight, const float* k_weight, int num_tokens,
                                     int num_heads, int num_heads_k, int head_dim, int rot_dim,
                                     int max_pos, int interleaved, float eps, void* q_out,
                                     long long q_out_row_stride, long long q_out_head_stride,
                                     void* k_out, long long k_out_row_stride,
                                     long long k_out_head_stride, fa_stream_t stream) {
  if (num_tokens < 0 || num_heads < 0 || num_heads_k < 0 || num_heads + num_heads_k < 1)
    return FA_ERR_INVALID_ARG;
  if (num_tokens > 0 && ((num_heads > 0 && (!q || !q_out)) || (num_heads_k > 0 && (!k || !k_out))))
    return FA_ERR_INVALID_ARG;
  if (head_dim < 8 || !valid_rope(cos_sin, rot_dim, max_pos, head_dim)) return FA_ERR_INVALID_ARG;
  if (rot_dim > 0 && num_tokens > 0 && !positions) return FA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return FA_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(k, 16) || !is_aligned(q_out, 16) ||
      !is_aligned(k_out, 16) || !is_aligned(positions, 4) || !is_aligned(q_weight, 16) ||
      !is_aligned(k_weight, 16))
    return FA_ERR_INVALID_ARG;
  if (head_dim % 8 != 0 || head_dim > 256) return FA_ERR_UNSUPPORTED;
  if ((num_heads > 0 &&
       (!settle_view(num_tokens, num_heads, head_dim, &q_row_stride, &q_head_stride) ||
        !settle_view(num_tokens, num_heads, head_dim, &q_out_row_stride, &q_out_head_stride))) ||
      (num_heads_k > 0 &&
       (!settle_view(num_tokens, num_heads_k, head_dim, &k_row_stride, &k_head_stride) ||
        !settle_view(num_tokens, num_heads_k, head_dim, &k_out_row_stride, &k_out_head_stride))))
    return FA_ERR_INVALID_ARG;
  if ((int64_t)num_tokens * ((int64_t)num_heads + num_heads_k) > INT32_MAX)
    return FA_ERR_UNSUPPORTED;
  fa::DeviceFacts dev;
  const fa_status st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  if (num_tokens == 0) return FA_OK;

  fa::QkNormRopeArgs a;
  a.q = {static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_row_stride,
         q_head_stride, q_out_row_stride, q_out_head_stride, q_weight};
  a.k = {static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_out), k_row_stride,
         k_head_stride, k_out_row_stride, k_out_head_stride, k_weight};
  a.heads = num_heads;
  a.heads_k = num_heads_k;
  a.dim = head_dim;
  a.inv_dim = 1.f / (float)head_dim;
  a.eps = eps;
  a.rope = {cos_sin, rot_dim, interleaved != 0};
  a.positions = rot_dim > 0 ? positions : nullptr;
  a.max_pos = max_pos;
  const int lanes = head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32;
  // Heads of a token together load its table row and the weights once; one at
  // a time where that would leave SMs idle.
  const long long all = (long long)num_tokens * (num_heads + num_heads_k);
  const int rows = all * lanes >= (long long)kNormRopeWide * dev.sm_count ? kNormRopeRows : 1;
  a.groups_q = (num_heads + rows - 1) / rows;
  a.groups = a.groups_q + (num_heads_k + rows - 1) / rows;
  a.units = (unsigned)((long long)num_tokens * a.groups);
  const unsigned grid = (unsigned)std::min<long long>(((long long)a.units * lanes + 255) / 256,
                                                      kNormRopeBlocks * (long long)dev.sm_count);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 1) {
    if (lanes == 8) fa::qk_norm_rope_kernel<8, 1><<<grid, 256, 0, s>>>(a);
    else if (lanes == 16) fa::qk_norm_rope_kernel<16, 1><<<grid, 256, 0, s>>>(a);
    else fa::qk_norm_rope_kernel<32, 1><<<grid, 256, 0, s>>>(a);
  } else {
    if (lanes == 8) fa::qk_norm_rope_kernel<8, kNormRopeRows><<<grid, 256, 0, s>>>(a);
    else if (lanes == 16) fa::qk_norm_rope_kernel<16, kNormRopeRows><<<grid, 256, 0, s>>>(a);
    else fa::qk_norm_rope_kernel<32, kNormRopeRows><<<grid, 256, 0, s>>>(a);
  }
  return launched();
}

extern "C" fa_status fa_paged_kv_append(
    const void* k, long long k_row_stride, long long k_head_stride, const void* v,
    long long v_row_stride, long long v_head_stride, const int* cu_seqlens, const int* seq_lens,
    const int* page_table, int batch, int total_new, int num_heads_k, int head_dim, int num_pages,
    int max_pages_per_seq, const float* k_weight, float eps, const float* cos_sin, int rot_dim,
    int max_pos, int interleaved, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
    fa_stream_t stream) {
  if (!seq_lens || !is_aligned(seq_lens, 4)) return FA_ERR_INVALID_ARG;
  if (total_new > 0 && (!k || !v)) return FA_ERR_INVALID_ARG;
  fa_status st = check_cache(k_cache, v_cache, k_scale, v_scale, cu_seqlens, page_table, batch,
                             total_new, num_heads_k, head_dim, num_pages, max_pages_per_seq);
  if (st != FA_OK) return st;
  if (!valid_rope(cos_sin, rot_dim, max_pos, head_dim) || !(eps >= 0.f) || !std::isfinite(eps))
    return FA_ERR_INVALID_ARG;
  if (!is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(k_weight, 16))
    return FA_ERR_INVALID_ARG;
  if (total_new > 0 &&
      (!settle_view(total_new, num_heads_k, head_dim, &k_row_stride, &k_head_stride) ||
       !settle_view(total_new, num_heads_k, head_dim, &v_row_stride, &v_head_stride)))
    return FA_ERR_INVALID_ARG;
  fa::DeviceFacts dev;
  st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  if (total_new == 0) return FA_OK;

  fa::KvAppendArgs a;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_row = k_row_stride;
  a.k_head = k_head_stride;
  a.v_row = v_row_stride;
  a.v_head = v_head_stride;
  a.cu = cu_seqlens;
  a.seq_lens = seq_lens;
  a.page_table = page_table;
  a.batch = batch;
  a.total = total_new;
  a.heads = num_heads_k;
  a.dim = head_dim;
  a.max_pages = max_pages_per_seq;
  a.num_pages = num_pages;
  a.limit = max_pages_per_seq * fa::kPageTokens;
  if (rot_dim > 0) a.limit = std::min(a.limit, max_pos);
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_weight = k_weight;
  a.inv_dim = 1.f / (float)head_dim;
  a.eps = eps;
  a.rope = {cos_sin, rot_dim, interleaved != 0};
  // n new tokens of a sequence touch at most (n + 62) / 64 + 1 pages, and n.
  const long long chunks =
      std::min<long long>(total_new, total_new / fa::kPageTokens + 2ll * batch);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool step = (long long)total_new < 16ll * batch;
  if (step) {
    const unsigned grid = (unsigned)chunks;
    if (head_dim <= 64) fa::kv_append_step_kernel<8><<<grid, fa::kStepThreads, 0, s>>>(a);
    else fa::kv_append_step_kernel<16><<<grid, fa::kStepThreads, 0, s>>>(a);
  } else {
    // Blocks of 256 threads, or of 128 at 64 dims; heads each for about
    // kAppendWave blocks an SM.
    const int threads = head_dim <= 64 ? 128 : 256;
    const long long slots = kAppendWave * 256ll / threads * dev.sm_count;
    const long long blocks =
        std::max<long long>(1, std::min<long long>(num_heads_k, slots / (2 * chunks)));
    a.per_block = (int)((num_heads_k + blocks - 1) / blocks);
    a.key_blocks = (num_heads_k + a.per_block - 1) / a.per_block;
    const dim3 grid((unsigned)chunks, 2 * a.key_blocks);
    const size_t table = (size_t)fa::kPageTokens * rot_dim * sizeof(float);
    if (head_dim <= 64) fa::kv_append_prompt_kernel<8><<<grid, threads, table, s>>>(a);
    else fa::kv_append_prompt_kernel<16><<<grid, threads, table, s>>>(a);
  }
  return launched();
}

extern "C" fa_status fa_paged_kv_gather(const void* k_cache, const void* v_cache,
                                        const float* k_scale, const float* v_scale,
                                        const int* cu_seqlens, const int* page_table, int batch,
                                        int total_k, int num_heads_k, int head_dim, int num_pages,
                                        int max_pages_per_seq, void* k_out, void* v_out,
                                        fa_stream_t stream) {
  if (total_k > 0 && (!k_out || !v_out)) return FA_ERR_INVALID_ARG;
  if (!is_aligned(k_out, 16) || !is_aligned(v_out, 16)) return FA_ERR_INVALID_ARG;
  fa_status st = check_cache(k_cache, v_cache, k_scale, v_scale, cu_seqlens, page_table, batch,
                             total_k, num_heads_k, head_dim, num_pages, max_pages_per_seq);
  if (st != FA_OK) return st;
  fa::DeviceFacts dev;
  st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  if (total_k == 0) return FA_OK;
  fa::KvGatherArgs a;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.cu = cu_seqlens;
  a.page_table = page_table;
  a.batch = batch;
  a.total = total_k;
  a.heads = num_heads_k;
  a.dim = head_dim;
  a.max_pages = max_pages_per_seq;
  a.num_pages = num_pages;
  a.k = static_cast<uint16_t*>(k_out);
  a.v = static_cast<uint16_t*>(v_out);
  a.wide_stores = is_aligned(k_out, 32) && is_aligned(v_out, 32);
  const long long pages =
      std::min<long long>(total_k, total_k / fa::kPageTokens + (long long)batch);
  // Blocks of 128 threads where there are enough of them for every SM, else of
  // 256 (2 x 32768 tokens: 64.4 against 66.4 us; 21 contexts of 1 to 1300
  // tokens, 500 blocks: 8.3 against 7.9 us).
  const int threads = 2 * pages >= 8ll * dev.sm_count ? 128 : 256;
  fa::kv_gather_kernel<<<dim3((unsigned)pages, 2), threads, 0,
                         reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

namespace {

fa_status plan_attn(int batch, int total_q, int num_heads, int num_heads_k, int head_dim,
                    int max_seqlen_q, bool masked, int* grid, int* rows_per_tile,
                    size_t* workspace_bytes) {
  if (!grid || !rows_per_tile || !workspace_bytes) return FA_ERR_INVALID_ARG;
  if (batch < 1 || total_q < 0 || num_heads < 1 || num_heads_k < 1 ||
      num_heads % num_heads_k != 0 || max_seqlen_q < 0)
    return FA_ERR_INVALID_ARG;
  if (!cache_dim(head_dim)) return FA_ERR_UNSUPPORTED;
  fa::DeviceFacts dev;
  const fa_status st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  const AttnLaunch l =
      attn_launch(dev.sm_count, batch, total_q, num_heads / num_heads_k, head_dim, max_seqlen_q,
                  masked);
  *grid = total_q > 0 ? l.grid : 0;
  *rows_per_tile = l.rows;
  *workspace_bytes = total_q > 0 ? l.bytes() : 0;
  return FA_OK;
}

}  // namespace

extern "C" fa_status fa_paged_attn_plan(int batch, int total_q, int num_heads, int num_heads_k,
                                        int head_dim, int max_seqlen_q, int* grid,
                                        int* rows_per_tile, size_t* workspace_bytes) {
  return plan_attn(batch, total_q, num_heads, num_heads_k, head_dim, max_seqlen_q, false, grid,
                   rows_per_tile, workspace_bytes);
}

extern "C" fa_status fa_paged_attn_masked_plan(int batch, int total_q, int num_heads,
                                               int num_heads_k, int head_dim, int max_seqlen_q,
                                               int* grid, int* rows_per_tile,
                                               size_t* workspace_bytes) {
  return plan_attn(batch, total_q, num_heads, num_heads_k, head_dim, max_seqlen_q, true, grid,
                   rows_per_tile, workspace_bytes);
}

extern "C" fa_status fa_paged_attn(const void* q, long long q_row_stride, long long q_head_stride,
                                   const void* k_cache, const void* v_cache, const float* k_scale,
                                   const float* v_scale, const int* cu_seqlens_q,
                                   const int* seq_lens, const int* page_table, int batch,
                                   int total_q, int num_heads, int num_heads_k, int head_dim,
                                   int num_pages, int max_pages_per_seq, int max_seqlen_q,
                                   int max_seqlen_k, float softmax_scale, int causal,
                                   int window_left, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, fa_stream_t stream) {
  return fa_paged_attn_masked(q, q_row_stride, q_head_stride, k_cache, v_cache, k_scale, v_scale,
                              cu_seqlens_q, seq_lens, page_table, batch, total_q, num_heads,
                              num_heads_k, head_dim, num_pages, max_pages_per_seq, max_seqlen_q,
                              max_seqlen_k, softmax_scale, causal, window_left, 0, nullptr, 0, out,
                              lse, workspace, workspace_bytes, stream);
}

extern "C" fa_status fa_paged_attn_masked(
    const void* q, long long q_row_stride, long long q_head_stride, const void* k_cache,
    const void* v_cache, const float* k_scale, const float* v_scale, const int* cu_seqlens_q,
    const int* seq_lens, const int* page_table, int batch, int total_q, int num_heads,
    int num_heads_k, int head_dim, int num_pages, int max_pages_per_seq, int max_seqlen_q,
    int max_seqlen_k, float softmax_scale, int causal, int window_left, int sink_tokens,
    const int* tree_mask, int tree_words, void* out, float* lse, void* workspace,
    size_t workspace_bytes, fa_stream_t stream) {
  if ((total_q > 0 && (!q || !out)) || !seq_lens) return FA_ERR_INVALID_ARG;
  fa_status st = check_cache(k_cache, v_cache, k_scale, v_scale, cu_seqlens_q, page_table, batch,
                             total_q, num_heads_k, head_dim, num_pages, max_pages_per_seq);
  if (st != FA_OK) return st;
  if (num_heads < 1 || num_heads % num_heads_k != 0 || max_seqlen_q < 0 || max_seqlen_k < 0 ||
      window_left < -1 || !(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return FA_ERR_INVALID_ARG;
  if (sink_tokens < 0 || tree_words < 0 || !is_aligned(tree_mask, 4) ||
      (tree_words > 0 && total_q > 0 && !tree_mask))
    return FA_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(out, 16) || !is_aligned(lse, 4) ||
      !is_aligned(seq_lens, 4) || !is_aligned(workspace, 16))
    return FA_ERR_INVALID_ARG;
  if (total_q > 0 && !settle_view(total_q, num_heads, head_dim, &q_row_stride, &q_head_stride))
    return FA_ERR_INVALID_ARG;
  if ((int64_t)total_q * num_heads > INT32_MAX || num_heads > 65535 ||
      (int64_t)total_q * tree_words > INT32_MAX)
    return FA_ERR_UNSUPPORTED;
  fa::DeviceFacts dev;
  st = fa::device_facts(&dev);
  if (st != FA_OK) return st;
  if (total_q == 0) return FA_OK;
  const int group = num_heads / num_heads_k;
  // (Sinks say nothing without a window.)
  const bool sinks = sink_tokens > 0 && window_left >= 0, masked = sinks || tree_words > 0;
  const AttnLaunch l =
      attn_launch(dev.sm_count, batch, total_q, group, head_dim, max_seqlen_q, masked);
  if (!workspace || workspace_bytes < l.bytes()) return FA_ERR_INVALID_ARG;
  CUtensorMap k_map, v_map;
  if (!encode_cache(&k_map, k_cache, head_dim, num_pages * num_heads_k, l.dim) ||
      !encode_cache(&v_map, v_cache, head_dim, num_pages * num_heads_k, l.dim))
    return FA_ERR_LAUNCH;
  fa::PagedAttnArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.total_q = total_q;
  a.heads = num_heads;
  a.dim = head_dim;
  a.max_pages = max_pages_per_seq;
  a.num_pages = num_pages;
  a.shape = {num_heads_k, group, l.rows, causal != 0, window_left,
             max_pages_per_seq * fa::kPageTokens, sink_tokens, tree_words > 0};
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_lse = reinterpret_cast<float*>(ws + l.o_bytes);
  a.meta = reinterpret_cast<int4*>(ws + l.o_bytes + l.lse_bytes);
  a.tree_mask = tree_mask;
  a.tree_words = tree_words;
  a.status = dev.status;
  a.wait_limit_ns = dev.wait_limit_ns;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // A launch holds the costs of kPagedMaxBatch sequences in shared
  // memory and counts them in 32 bits; a larger batch runs as
  // consecutive launches, which share the workspace in stream order.
  const long long per_row_tile =
      (long long)num_heads_k *
      ((long long)max_pages_per_seq * fa::kPageTokens / fa::kTileKeys + 1 + fa::kUnitCost);
  const long long row_tiles = (long long)total_q * group / l.rows;
  const long long fit = fa::kMaxCost / per_row_tile - row_tiles;
  if (fit < 1) return FA_ERR_UNSUPPORTED;
  const int step = (int)std::min<long long>(fa::kPagedMaxBatch, fit);
  for (int b0 = 0; b0 < batch; b0 += step) {
    a.batch = std::min(batch - b0, step);
    a.cu = cu_seqlens_q + b0;
    a.seq_lens = seq_lens + b0;
    a.page_table = page_table + (size_t)b0 * max_pages_per_seq;
    const cudaError_t e =
        l.rows == fa::kWideRows ? fa::launch_attn_wide(l.dim, k_map, v_map, a, l.grid, s)
        : tree_words > 0 ? fa::launch_attn_tree(l.dim, l.rows, k_map, v_map, a, l.grid, s)
        : sinks        ? fa::launch_attn_sinks(l.dim, l.rows, k_map, v_map, a, l.grid, s)
                       : fa::launch_attn_shape<fa::kNoMask>(l.dim, l.rows, k_map, v_map, a, l.grid, s);
    if (e != cudaSuccess) return FA_ERR_LAUNCH;
  }
  return FA_OK;
}
