// kv_evict_kernels.cuh -- which keys of the paged cache to keep, and the cache
// moved together in place.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "paged_index.h"
#include "sm103_ptx.cuh"

namespace fa {

// ------------------------------------------------------------------ select
struct KvSelectArgs {
  const float* weights;  // [batch, heads, capacity]
  const int* seq_lens;
  int heads, capacity, budget, sinks, recent;
  int *keep, *new_lens;  // [batch, heads, budget], [batch]
};

// The order of weights as unsigned numbers: NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t weight_order(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelectThreads = 1024;
constexpr int kSelectBins = 2048;

// A block chooses for one (sequence, head): the m-th largest weight by three
// radix passes (11, 11, 10 bits) over the weights between sinks and the recent
// keys, then all above it and its first ties, in order.
__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const KvSelectArgs a) {
  __shared__ int bins[kSelectBins];
  __shared__ int warp_sum[2][32];
  __shared__ int s_digit, s_above;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.heads, h = blockIdx.x - b * a.heads;
  const int n = imin(imax(__ldg(a.seq_lens + b), 0), a.capacity);
  const float* w = a.weights + (size_t)blockIdx.x * a.capacity;
  int* keep = a.keep + (size_t)blockIdx.x * a.budget;
  if (h == 0 && tid == 0) a.new_lens[b] = imin(n, a.budget);
  if (n <= a.budget) {
    for (int j = tid; j < a.budget; j += kSelectThreads) keep[j] = j < n ? j : -1;
    return;
  }
  // (sinks + recent <= budget < n)
  const int lo = a.sinks, hi = n - a.recent;
  int need = a.budget - a.sinks - a.recent;
  for (int j = tid; j < lo; j += kSelectThreads) keep[j] = j;
  for (int j = tid; j < a.recent; j += kSelectThreads) keep[a.budget - a.recent + j] = hi + j;
  if (need == 0) return;
  // Inclusive sum over the block of one number a thread.
  int turn = 0;
  auto block_scan = [&](int x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += v;
    }
    int* sums = warp_sum[turn];
    turn ^= 1;
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int s = lane < warp ? sums[lane] : 0;
    return x + __reduce_add_sync(0xffffffffu, s);
  };
  uint32_t prefix = 0;
  const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = shifts[pass], count = 1 << widths[pass];
    for (int k = tid; k < count; k += kSelectThreads) bins[k] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += kSelectThreads) {
      const uint32_t u = weight_order(w[j]);
      if (pass == 0 || (u >> (shift + widths[pass])) == prefix)
        atomicAdd(bins + ((u >> shift) & (count - 1)), 1);
    }
    __syncthreads();
    // Bins from the largest down, count / 1024 of them a thread.
    const int per = count / kSelectThreads;
    const int top = count - 1 - tid * per;
    const int c0 = bins[top], c1 = per > 1 ? bins[top - 1] : 0;
    const int upto = block_scan(c0 + c1), above = upto - c0 - c1;
    if (above < need && need <= upto) {
      const bool second = above + c0 < need;
      s_digit = second ? top - 1 : top;
      s_above = second ? above + c0 : above;
    }
    __syncthreads();
    prefix = (prefix << widths[pass]) | (uint32_t)s_digit;
    need -= s_above;
  }
  // All above the threshold, and its first `need` ties.
  int done_above = 0, done_ties = 0;
  for (int j0 = lo; j0 < hi; j0 += kSelectThreads) {
    const int j = j0 + tid;
    const uint32_t u = j < hi ? weight_order(w[j]) : 0u;
    const bool in = j < hi;
    const int above = in && u > prefix, tie = in && u == prefix;
    const int upto = block_scan(above << 16 | tie);
    const int all = warp_sum[turn ^ 1][lane];
    const int n_above = done_above + (upto >> 16) - above;
    const int n_ties = done_ties + (upto & 0xffff) - tie;
    if (above || (tie && n_ties < need)) keep[lo + n_above + imin(n_ties, need)] = j;
    const int sum = __reduce_add_sync(0xffffffffu, all);
    done_above += sum >> 16;
    done_ties += sum & 0xffff;
  }
}

// ----------------------------------------------------------------- compact
struct KvCompactArgs {
  const int *page_table, *keep, *first, *counts;  // first: or null (0)
  int batch, heads, keep_heads, keep_row, dim, max_pages, num_pages;
  uint8_t* cache[2];  // K, V
  float* scale[2];
  float* weights;  // [batch, heads, capacity] or null
  int capacity;
};

constexpr int kCompactThreads = 256;

// Where a row comes from: its cell (-1: a row of zeros), slot and scale.
struct RowSource {
  int cell, slot;
  float scale;
};

// A cluster of CTAs takes K or V of one (sequence, head) in rounds of one page
// for each CTA.  A row's source is at its own slot or behind it, so what a
// round reads is only written in that round or a later one: every CTA has
// loaded its page's rows before any of them writes (the cluster's barrier), and
// the next round's loads need not wait for the writes.  Between them the
// page's new scale is found, from the codes.
__global__ void __launch_bounds__(kCompactThreads) kv_compact_kernel(const KvCompactArgs a) {
  // (Three, as a slow warp may still write round r - 1 while r + 1 is noted.)
  __shared__ RowSource s_row[3][kPageTokens];
  __shared__ float s_amax[2][kCompactThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank, ctas;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const unsigned unit = blockIdx.x / ctas;
  const int kv = unit & 1, h = (int)(unit >> 1) % a.heads, b = (int)(unit >> 1) / a.heads;
  const long long slots = (long long)a.max_pages * kPageTokens;
  const int first = a.first ? imax(__ldg(a.first + b), 0) : 0;
  int count = imin(imax(__ldg(a.counts + b), 0), a.keep_row);
  if (first + (long long)count > slots) count = first < slots ? (int)(slots - first) : 0;
  const int pages = pages_touched(first, count), page0 = first / kPageTokens;
  const int* keep = a.keep + ((size_t)b * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.keep_row;
  const int* table = a.page_table + (size_t)b * a.max_pages;
  uint8_t* cache = a.cache[kv];
  float* scales = a.scale[kv];
  float* weights = kv == 0 && a.weights ? a.weights + ((size_t)b * a.heads + h) * a.capacity
                                        : nullptr;
  const int per_row = a.dim / 16, chunks = kPageTokens * per_row;  // 16-byte chunks

  const int rounds = (pages + (int)ctas - 1) / (int)ctas;
  // The source of this thread's row (threads 0 .. 63) in round r; whether it moves.
  float weight = 0.f;
  bool moves = false;
  auto find_row = [&](int r, RowSource* src) {
    *src = {-1, 0, 0.f};
    moves = false;
    const int p = r * (int)ctas + (int)rank;
    if (p >= pages || tid >= kPageTokens) return;
    const PageSpan sp = page_span(first, count, page0 + p);
    if (tid >= sp.count) return;
    const int dst = (page0 + p) * kPageTokens + sp.slot + tid;
    const int from = __ldg(keep + sp.row + tid);
    moves = from != dst;
    if (from < dst || from >= slots) return;
    const int id = checked_page(__ldg(table + from / kPageTokens), a.num_pages);
    if (id < 0) return;
    src->cell = id * a.heads + h;
    src->slot = from % kPageTokens;
    src->scale = scales[src->cell];
    if (weights && from < a.capacity) weight = weights[from];
  };
  RowSource mine;
  find_row(0, &mine);
  if (tid < kPageTokens) s_row[0][tid] = mine;
  bool moved = __syncthreads_or(moves);
  for (int r = 0; r < rounds; ++r) {
    const int p = r * (int)ctas + (int)rank;
    const bool live = p < pages && moved;
    const PageSpan sp = page_span(first, count, page0 + (p < pages ? p : 0));
    const RowSource* row = s_row[r % 3];
    const float my_weight = weight;
    uint4 code[2];
    float amax = 0.f;
    if (live) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = tid + k * kCompactThreads, i = e / per_row;
        code[k] = make_uint4(0u, 0u, 0u, 0u);
        if (e < chunks && i < sp.count && row[i].cell >= 0)
          code[k] = *reinterpret_cast<const uint4*>(
              cache + ((size_t)row[i].cell * kPageTokens + row[i].slot) * a.dim +
              (e - i * per_row) * 16);
      }
    }
    // The next round's sources under way.
    weight = 0.f;
    if (r + 1 < rounds) find_row(r + 1, &mine); else moves = false;
    if (live) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = tid + k * kCompactThreads, i = e / per_row;
        if (e >= chunks || i >= sp.count) continue;
        // The largest finite code, sign apart (0x7f is NaN).
        uint32_t top = 0;
        const uint32_t w[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t m = w[q] & 0x7f7f7f7fu;
          top = __vmaxu4(top, m & ~__vcmpeq4(m, 0x7f7f7f7fu));
        }
        top = __vmaxu4(top, top >> 16);
        top = __vmaxu4(top, top >> 8) & 0xffu;
        amax = fmaxf(amax, f16x2_floats(unpack_e4m3x2(top)).x * row[i].scale);
      }
    }
    if (r + 1 < rounds && tid < kPageTokens) s_row[(r + 1) % 3][tid] = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_amax[r & 1][warp] = amax;
    const bool next_moved = __syncthreads_or(moves);
    if (ctas > 1) {
      ptx::cluster_arrive_release();
      ptx::cluster_wait_acquire();
    }
    if (live) {
      const int id = checked_page(__ldg(table + page0 + p), a.num_pages);
      if (id >= 0) {
        const size_t cell = (size_t)id * a.heads + h;
#pragma unroll
        for (int i = 0; i < kCompactThreads / 32; ++i) amax = fmaxf(amax, s_amax[r & 1][i]);
        const float old = sp.slot > 0 ? scales[cell] : 0.f;
        const float s = fmaxf(scale_for(amax), old);
        const float inv = 1.f / s;
        uint8_t* codes = cache + cell * kPageTokens * a.dim;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int e = tid + k * kCompactThreads, i = e / per_row;
          if (e >= chunks || i >= sp.count) continue;
          const float f = row[i].scale * inv;
          uint32_t w[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
          if (f != 1.f) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 lo = f16x2_floats(unpack_e4m3x2(w[q]));
              const float2 hi = f16x2_floats(unpack_e4m3x2(w[q] >> 16));
              w[q] = pack_e4m3x2(lo.x * f, lo.y * f) | pack_e4m3x2(hi.x * f, hi.y * f) << 16;
            }
          }
          *reinterpret_cast<uint4*>(codes + (size_t)(sp.slot + i) * a.dim +
                                    (e - i * per_row) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // Tokens before the first slot follow a scale that has grown.
        if (s > old && sp.slot > 0) {
          const float f = old * inv;
          uint32_t* c = reinterpret_cast<uint32_t*>(codes);
          for (int i = tid; i < sp.slot * a.dim / 4; i += kCompactThreads) {
            const uint32_t u = c[i];
            const float2 lo = f16x2_floats(unpack_e4m3x2(u));
            const float2 hi = f16x2_floats(unpack_e4m3x2(u >> 16));
            c[i] = pack_e4m3x2(lo.x * f, lo.y * f) | pack_e4m3x2(hi.x * f, hi.y * f) << 16;
          }
          __syncthreads();  // (every thread has read the old scale)
        } else if (sp.slot > 0) {
          __syncthreads();
        }
        if (tid == 0) scales[cell] = s;
      }
      const int dst = (page0 + p) * kPageTokens + sp.slot + tid;
      if (weights && tid < sp.count && dst < a.capacity) weights[dst] = my_weight;
    }
    moved = next_moved;
  }
}

}  // namespace fa
