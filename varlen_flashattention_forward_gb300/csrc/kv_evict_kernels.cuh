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

constexpr int kSelectThreads = 256;
constexpr int kSelectItems = 32;   // keys of a thread that stay in registers
constexpr int kSelectBins = 256;   // a thread has one
constexpr int kSelectCtas = 8;     // of a cluster, at most

// A cluster of CTAs chooses for one (sequence, head): the m-th largest weight by
// four radix passes of eight bits over the weights between sinks and the recent
// keys, then all above it and its first ties, in order.  (Passes of 11, 11 and 10
// bits: each took some 7 us of the single row below, most of it reading the other
// CTAs' 2048 bins; one block of 1024 threads without a cluster 26 us.)  The CTAs
// count bins for themselves and add up each other's through distributed shared memory; all
// find the same digit.  A CTA has a stretch of the keys and a warp
// a stretch of that, 32 at a time, so that the last step needs two sums over the
// warps and CTAs before.  ITEMS: keys of a thread in registers (0: read again
// each time).
//
// 512 rows of up to 8192 weights 16 us (the loads alone 8), 8 rows of 32768 12 us.
//
template <int ITEMS>
__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const KvSelectArgs a) {
  constexpr unsigned kFull = 0xffffffffu;
  constexpr int kWarps = kSelectThreads / 32;
  __shared__ int bins[2][kSelectBins];  // by turns of the passes
  __shared__ int warp_sum[2][kWarps];
  __shared__ __align__(8) float2 cta_sum;  // above and ties of the CTA (as ints)
  __shared__ int s_digit, s_above, s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t rank, ctas;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const unsigned unit = blockIdx.x / ctas;
  const int b = (int)unit / a.heads, h = (int)unit - b * a.heads;
  const int n = imin(imax(__ldg(a.seq_lens + b), 0), a.capacity);
  const float* w = a.weights + (size_t)unit * a.capacity;
  int* keep = a.keep + (size_t)unit * a.budget;
  const int t0 = (int)rank * kSelectThreads + tid, threads = (int)ctas * kSelectThreads;
  if (h == 0 && t0 == 0) a.new_lens[b] = imin(n, a.budget);
  if (n <= a.budget) {
    for (int j = t0; j < a.budget; j += threads) keep[j] = j < n ? j : -1;
    return;
  }
  // (sinks + recent <= budget < n)
  const int lo = a.sinks, hi = n - a.recent;
  int need = a.budget - a.sinks - a.recent;
  const int steps = (hi - lo + threads - 1) / threads;  // of 32 keys, of each warp
  // This thread's first key, and how many of every 32nd there are.  (Keys are
  // 32-bit; the stretches past the end are not.)
  const long long from = lo + ((long long)rank * kWarps + warp) * steps * 32 + lane;
  const int at = (int)(from < hi ? from : hi);
  const int mine = imin(steps, (hi - at + 31) / 32);
  uint32_t held[ITEMS > 0 ? ITEMS : 1];
  if constexpr (ITEMS > 0) {
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
      held[k] = k < mine ? weight_order(__ldg(w + at + 32 * k)) : 0u;
  }
  for (int j = t0; j < lo; j += threads) keep[j] = j;
  for (int j = t0; j < a.recent; j += threads) keep[a.budget - a.recent + j] = hi + j;
  if (need == 0) return;
  // f(step, order of the key, whether there is one), step by step.
  auto each = [&](auto f) {
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) {
        if (k >= steps) break;
        f(k, held[k], k < mine);
      }
    } else {
#pragma unroll 4
      for (int k = 0; k < steps; ++k) {
        f(k, k < mine ? weight_order(__ldg(w + at + 32 * k)) : 0u, k < mine);
      }
    }
  };
  auto cluster_sync = [&]() {
    if (ctas > 1) {
      ptx::cluster_arrive_release();
      ptx::cluster_wait_acquire();
    } else {
      __syncthreads();
    }
  };
  uint32_t prefix = 0;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* count = bins[pass & 1];
    count[tid] = 0;
    __syncthreads();
    each([&](int, uint32_t u, bool in) {
      if (in && (pass == 0 || (u >> (shift + 8)) == prefix))
        atomicAdd(count + ((u >> shift) & (kSelectBins - 1)), 1);
    });
    cluster_sync();
    // Bins from the largest down, one a thread.
    const int bin = kSelectBins - 1 - tid;
    int c = 0;
    if (ctas > 1) {
      int of[kSelectCtas];
      const uint32_t place = ptx::smem_u32(count + bin);
#pragma unroll
      for (uint32_t k = 0; k < kSelectCtas; ++k)
        of[k] = k < ctas ? ptx::ld_shared_cluster_s32(ptx::mapa_shared(place, k)) : 0;
#pragma unroll
      for (int k = 0; k < kSelectCtas; ++k) c += of[k];
    } else {
      c = count[bin];
    }
    int upto = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) warp_sum[0][warp] = upto;
    __syncthreads();
    upto += __reduce_add_sync(kFull, lane < warp ? warp_sum[0][lane] : 0);
    if (upto - c < need && need <= upto) {
      s_digit = bin;
      s_above = upto - c;
      s_count = c;
    }
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)s_digit;
    need -= s_above;
    // All with this prefix are needed (mostly so by the third pass): the weights above
    // the largest below them, and no ties.  (The smallest prefix has none below.)
    if (need == s_count && prefix != 0u) {
      prefix = (prefix << shift) - 1u;
      need = 0;
      break;
    }
  }
  // All above the threshold, and its first `need` ties.
  int above = 0, ties = 0;
  each([&](int, uint32_t u, bool in) {
    above += in && u > prefix;
    ties += in && u == prefix;
  });
  above = __reduce_add_sync(kFull, above);
  ties = __reduce_add_sync(kFull, ties);
  if (lane == 0) {
    warp_sum[0][warp] = above;
    warp_sum[1][warp] = ties;
  }
  __syncthreads();
  const int warp_above = lane < kWarps ? warp_sum[0][lane] : 0;
  const int warp_ties = lane < kWarps ? warp_sum[1][lane] : 0;
  above = __reduce_add_sync(kFull, lane < warp ? warp_above : 0);
  ties = __reduce_add_sync(kFull, lane < warp ? warp_ties : 0);
  if (ctas > 1) {
    const int all_above = __reduce_add_sync(kFull, warp_above);
    const int all_ties = __reduce_add_sync(kFull, warp_ties);
    if (tid == 0) cta_sum = make_float2(__int_as_float(all_above), __int_as_float(all_ties));
    cluster_sync();
    for (uint32_t k = 0; k < rank; ++k) {
      const float2 v = ptx::ld_shared_cluster_v2(ptx::mapa_shared(ptx::smem_u32(&cta_sum), k));
      above += __float_as_int(v.x);
      ties += __float_as_int(v.y);
    }
    ptx::cluster_arrive_release();  // (this CTA has read the others')
  }
  const unsigned before = (1u << lane) - 1u;
  each([&](int k, uint32_t u, bool in) {
    const unsigned up = __ballot_sync(kFull, in && u > prefix);
    const unsigned eq = __ballot_sync(kFull, in && u == prefix);
    const int my_ties = ties + __popc(eq & before);
    if (((up >> lane) & 1) || (((eq >> lane) & 1) && my_ties < need))
      keep[lo + above + __popc(up & before) + imin(my_ties, need)] = at + 32 * k;
    above += __popc(up);
    ties += __popc(eq);
  });
  if (ctas > 1) ptx::cluster_wait_acquire();  // no CTA leaves while its sums are read
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
constexpr int kCompactPages = kCompactThreads / kPageTokens;  // of a CTA's round: a row a thread
constexpr int kCompactNoted = 1024;  // pages of a sequence noted in shared memory

// Where a row comes from: its cell (-1: a row of zeros), slot and scale.
struct RowSource {
  int cell, slot;
  float scale;
};

// 16 codes times a factor, as codes again.  A power of two within f16's range
// multiplies f16 pairs: a product that matters, from 2^-10 (half e4m3's
// smallest) to 448, is exact there.  Any other goes through fp32.
__device__ __forceinline__ void scale_codes(uint32_t* w, float f) {
  if ((__float_as_uint(f) & 0x007fffffu) == 0u && f <= 32768.f) {
    const uint32_t f2 = ptx::pack_f16x2(f, f);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t lo = unpack_e4m3x2(w[q]), hi = unpack_e4m3x2(w[q] >> 16);
      uint16_t c0, c1;
      asm("mul.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(f2));
      asm("mul.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(f2));
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c0) : "r"(lo));
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c1) : "r"(hi));
      w[q] = (uint32_t)c0 | (uint32_t)c1 << 16;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 lo = f16x2_floats(unpack_e4m3x2(w[q]));
      const float2 hi = f16x2_floats(unpack_e4m3x2(w[q] >> 16));
      w[q] = pack_e4m3x2(lo.x * f, lo.y * f) | pack_e4m3x2(hi.x * f, hi.y * f) << 16;
    }
  }
}
// The largest magnitude of 16 codes but NaN (0x7f), as a code.
__device__ __forceinline__ uint32_t largest_code(const uint4& c) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    top = __vmaxu2(__vmaxu2(top, w[q] & 0x007f007fu), (w[q] >> 8) & 0x007f007fu);
  top = max(top & 0xffffu, top >> 16);
  if (top == 0x7fu) {
    top = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int s = 0; s < 32; s += 8) {
        const uint32_t m = (w[q] >> s) & 0x7fu;
        if (m != 0x7fu) top = max(top, m);
      }
  }
  return top;
}

// A cluster of CTAs takes K or V of one (sequence, head) in rounds of four pages
// for each CTA, one for every 64 threads.  A row's source is at its own slot or
// behind it, so what a round reads is only written in that round or a later
// one: every CTA has loaded its pages' rows before any of them writes (the
// cluster's barrier), and what the next round needs may be read at any time
// before.
//
// The cells and scales of the sequence's pages are noted in shared memory first
// (as they are before the move, which is what every row needs), and a round's
// entries of `keep` loaded two rounds ahead, so that a round waits for its codes
// alone.  A thread looks up one row of its page; then the page's threads take
// its rows 16 bytes at a time, find their largest value and so the new scale,
// and write them under it.
//
// 64 caches of 1000 to 8192 tokens, 8 heads of 128 dims, to 2048 kept rows each:
// 107 us, 5.0 TB/s read and written (a copy 6.8), bound by instruction issue, codes'
// maxima and new scales.  One cache of 32768 to 4097
// rows of 96 dims: 16 us, four rounds of a cluster of eight.  Entries, pages and
// scales looked up round by round made the first 186 us, a page's rows spread over
// the whole block 129, copies through shared memory a round ahead 156.
__global__ void __launch_bounds__(kCompactThreads, 4) kv_compact_kernel(const KvCompactArgs a) {
  // (Two, written between a round's barriers and read behind them.)
  __shared__ RowSource s_row[2][kCompactThreads];
  __shared__ float s_amax[kCompactThreads / 32];
  __shared__ int s_moved[2][kCompactThreads / 32];
  __shared__ int s_cell[kCompactNoted];
  __shared__ float s_scale[kCompactNoted];
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
  const int per_round = (int)ctas * kCompactPages;
  const int rounds = (pages + per_round - 1) / per_round;
  // This thread's place: page of the CTA's four, row to look up, and 16 bytes of
  // every `step`-th row from row0 on (8 lanes a row, or 4 at 64 dims).
  const int page = tid / kPageTokens, my_row = tid % kPageTokens;
  const int lanes = a.dim <= 64 ? 4 : 8, step = kPageTokens / lanes;
  const int row0 = my_row / lanes, byte = (my_row % lanes) * 16;
  auto page_of = [&](int r) { return r * per_round + (int)rank * kCompactPages + page; };

  // Cell and scale of the sequence's page p.
  auto look_up = [&](int p, int* cell, float* scale) {
    const int id = checked_page(__ldg(table + p), a.num_pages);
    *cell = id < 0 ? -1 : id * a.heads + h;
    *scale = id < 0 ? 0.f : scales[*cell];
  };
  // Those noted: [page0, page0 + noted), up to the last entry's (of an ascending
  // list the last page of any).
  int noted = 0;
  if (pages > 0) {
    const int last = __ldg(keep + count - 1);
    noted = imin(imin(last < 0 ? 0 : last / kPageTokens + 1, a.max_pages) - page0, kCompactNoted);
    for (int p = tid; p < noted; p += kCompactThreads) look_up(page0 + p, s_cell + p, s_scale + p);
  }
  // This thread's row of round r: its entry of `keep`, and what that names.
  auto entry = [&](int r) {
    const int p = page_of(r);
    if (p >= pages) return -1;
    const PageSpan sp = page_span(first, count, page0 + p);
    return my_row < sp.count ? __ldg(keep + sp.row + my_row) : -1;
  };
  float weight = 0.f;
  auto publish = [&](int r, int from) {
    RowSource src = {-1, 0, 0.f};
    bool moves = false;
    weight = 0.f;
    const int p = page_of(r);
    if (p < pages) {
      const PageSpan sp = page_span(first, count, page0 + p);
      const int dst = (page0 + p) * kPageTokens + sp.slot + my_row;
      if (my_row < sp.count) {
        moves = from != dst;
        if (from >= dst && from < slots) {
          const int at = from / kPageTokens - page0;
          if (at < noted) {
            src.cell = s_cell[at];
            src.scale = s_scale[at];
          } else {
            look_up(page0 + at, &src.cell, &src.scale);
          }
          src.slot = from % kPageTokens;
          if (weights && src.cell >= 0 && from < a.capacity) weight = weights[from];
        }
      }
    }
    s_row[r & 1][tid] = src;
    const bool any = __any_sync(0xffffffffu, moves);
    if (lane == 0) s_moved[r & 1][warp] = any;
  };
  int from = entry(0), ahead = entry(1);
  __syncthreads();
  publish(0, from);
  __syncthreads();
  for (int r = 0; r < rounds; ++r) {
    const int p = page_of(r);
    const RowSource* row = s_row[r & 1] + page * kPageTokens;
    const float my_weight = weight;
    // (A page none of whose rows moves is left alone.)
    const bool live = p < pages && (s_moved[r & 1][2 * page] | s_moved[r & 1][2 * page + 1]);
    const PageSpan sp = page_span(first, count, page0 + (p < pages ? p : 0));
    uint4 code[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = row0 + k * step;
      code[k] = make_uint4(0u, 0u, 0u, 0u);
      if (live && k < lanes && i < sp.count && byte < a.dim) {
        const RowSource src = row[i];
        if (src.cell >= 0)
          code[k] = *reinterpret_cast<const uint4*>(
              cache + ((size_t)src.cell * kPageTokens + src.slot) * a.dim + byte);
      }
    }
    // The next round's rows under way.
    from = ahead;
    ahead = entry(r + 2);
    if (r + 1 < rounds) publish(r + 1, from);
    // ---- the largest finite value, and so the scale
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t top = largest_code(code[k]);
      if (top != 0)
        amax = fmaxf(amax, f16x2_floats(unpack_e4m3x2(top)).x * row[row0 + k * step].scale);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_amax[warp] = amax;
    const int id = live ? checked_page(__ldg(table + page0 + p), a.num_pages) : -1;
    const size_t cell = (size_t)imax(id, 0) * a.heads + h;
    const float old = id >= 0 && sp.slot > 0 ? scales[cell] : 0.f;
    __syncthreads();
    if (ctas > 1) {
      ptx::cluster_arrive_release();
      ptx::cluster_wait_acquire();
    }
    // ---- the codes under it
    if (id >= 0) {
      const float s = fmaxf(scale_for(fmaxf(s_amax[2 * page], s_amax[2 * page + 1])), old);
      const float inv = 1.f / s;
      uint8_t* codes = cache + cell * kPageTokens * a.dim;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = row0 + k * step;
        if (k >= lanes || i >= sp.count || byte >= a.dim) continue;
        // (A code that is not 0 has f <= 2^18; a row of zeros may have any.)
        const float f = fminf(row[i].scale * inv, 1e38f);
        uint32_t w[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
        if (f != 1.f) scale_codes(w, f);
        *reinterpret_cast<uint4*>(codes + (size_t)(sp.slot + i) * a.dim + byte) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      // Tokens before the first slot follow a scale that has grown.
      if (sp.slot > 0 && s > old) {
        const float f = old * inv;
        uint4* c = reinterpret_cast<uint4*>(codes);
        for (int i = my_row; i < sp.slot * a.dim / 16; i += kPageTokens) {
          uint4 u = c[i];
          uint32_t w[4] = {u.x, u.y, u.z, u.w};
          scale_codes(w, f);
          c[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (my_row == 0) scales[cell] = s;
    }
    if (weights && live) {
      const int dst = (page0 + p) * kPageTokens + sp.slot + my_row;
      if (my_row < sp.count && dst < a.capacity) weights[dst] = my_weight;
    }
    // (The maxima and rows that the next round writes over are read.)
    __syncthreads();
  }
}

}  // namespace fa
