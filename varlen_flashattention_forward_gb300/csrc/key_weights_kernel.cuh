// key_weights_kernel.cuh -- attention weights that each cached key has got,
// for sm_103a:
//
//   W[b, h, j] = decay * W[b, h, j] + sum over the rows i of sequence b and the
//                heads of group h of exp(scale q_i k_j - LSE_i)
//
// over the keys that a row sees (a key that is among the rows' own starts from
// 0).  The LSE is that of the rows' attention, so the weights are final as they
// come: no maximum, no V and no second pass.
//
// The transposed form of paged_attn_kernel: St[key, row] = K[key, d] Q[row, d]t
// as products of K as it lies in the cache and Q as three terms, one in e4m3 and two in
// e5m2, off by 2^-24 of a row's largest value (split_three; two e4m3 terms, 2^-17 off, gave
// sums an error of 4e-6 instead of 1e-6).  A thread has a key:
// its weights' sum over the rows stays in the thread, in a fixed order, and no two
// threads write the same place.
//
// Work: every (sequence, kv head) has its 128-key tiles; their costs are cut
// into equal contiguous ranges (paged_index.h), one for each CTA, so a tile is
// one CTA's alone.  More rows than N go in chunks, tile by tile again.
//
//   producer   walks the CTA's segments of key tiles and publishes them, 16 tiles
//              at a time with their pages' scales, then loads the pages by TMA
//              into a ring of K tiles
//   issuer     S MMAs into two buffers of N columns
//   the rest   stage the rows of Q, then a thread for each key: exp2, sum, the
//              weight's update (with what stood there loaded a tile ahead).
//              Where a tile has 64 or 128 rows, whose exponentials take longer
//              than its bytes, two warpgroups take pairs of tiles by turns: a
//              row's factor and LSE come from shared memory, 4 cycles of its
//              path for two rows, once for both.
//
// One row of 64 sequences with 100 to 8192 keys, 32 and 4 heads of 128 dims: 34 us,
// 4.2 TB/s; without any load of keys and weights it would take 24, launch, search,
// rows and first tile of each CTA.  The last 32 rows of 4 prompts of 20001 to 32768
// tokens, 8 kv heads (128 rows a unit): 46 us, of which 13 are the exponentials and
// 17 the tensor core's, and 9 the way to the first tile.  A pair's products and its
// sums follow each other (four buffers fill TMEM), so that no part is hidden well:
// without the rows' factors 6 us less, without exponentials 5, without two of three
// products 4, without all of them 34 us.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "cost_scan.cuh"
#include "e4m3.cuh"
#include "named_bar.cuh"
#include "paged_attn_kernel.cuh"  // bounded waits
#include "paged_index.h"
#include "rope_row.cuh"
#include "sm103_ptx.cuh"

namespace fa {

constexpr int kWeightMaxBatch = 256;  // sequences of a launch

struct KeyWeightsArgs {
  const uint16_t* q;
  long long q_row, q_head;
  const float* lse;  // [heads, total_q], natural
  const float* k_scale;
  const int *cu, *seq_lens, *page_table;
  int batch, total_q, dim, max_pages, num_pages;
  AttnShape shape;   // rows: N
  int keys;          // positions of a sequence that have a page and a weight
  // The scores' factor, and the LSE's in two terms: log2(e) as scale_log2, once
  // rounded, holds it.  (Large scores and LSE cancel: with a factor 6e-8 off in one of
  // them, a weight of a score of 40 would be 2e-6 off.  What is left at 128 dims, 1.1e-6
  // of a sum, is mostly the products' sums, which the tensor core cuts: 7e-7 too small;
  // 4e-7 at 64 dims, half as many steps.)
  float scale_log2, lse_log2, lse_log2_rest, decay;
  float* weights;    // [batch, kv heads, capacity]
  long long capacity;
  unsigned int* status;
  uint64_t wait_limit_ns;
};

template <int D, int N>
struct WeightsCfg {
  static constexpr uint32_t kSwK = D == 128 ? ptx::kLayoutSw128 : ptx::kLayoutSw64;
  static constexpr int kTileBytes = kTileKeys * D;
  static constexpr int kPageBytes = kPageTokens * D;
  static constexpr int kTiles = N >= 64 ? 2 : 1;  // of a key thread at once
  static constexpr int kBuffers = 2 * kTiles;     // of St
  // Columns of a buffer: the products with Q's e5m2 terms side by side, so that the
  // tensor core reads K once for both, or, where there are many rows, in one sum.
  static constexpr bool kApart = N <= 32;
  static constexpr int kCols = kApart ? 2 * N : N;
  static constexpr int kSlots = N == 16 ? 4 : N == 32 ? 3 : N == 64 ? 5 : 6;
  static constexpr int kQBytes = 3 * N * D;  // terms of the rows, one behind the other
  static constexpr uint32_t kTmemCols = kBuffers * kCols;
  static constexpr int kQ = kSlots * kTileBytes;
  static constexpr int kCtl = kQ + kQBytes;
  static constexpr int kKeyThreads = 128 * kTiles;
  static constexpr int kThreads = kKeyThreads + 64;
  // Resident CTAs (by shared memory, 64 to 149 KB at 128 dims, and columns).
  static constexpr int kResident = N <= 32 ? 3 : N == 64 ? 2 : 1;
};

// A chunk of a sequence's rows against its keys.
struct WeightChunk {
  KeyRange keys;
  int span;        // from its first row's token to its last row's
  long long at0;   // position of its first row's token
  // Whether some row may see a key of the tile; of the tiles [j0, j1).
  __device__ __forceinline__ bool seen(int j0) const { return any(j0, (long long)j0 + kTileKeys); }
  __device__ __forceinline__ bool any(int j0, long long j1) const {
    return (keys.hi > keys.lo && j0 < keys.hi && j1 > keys.lo) || j0 < keys.sink;
  }
  // Whether every row sees every key of the tile.
  __device__ __forceinline__ bool whole(int j0, const AttnShape& s) const {
    return (!s.causal || (long long)j0 + kTileKeys - 1 <= at0) &&
           (s.window < 0 || (long long)j0 >= at0 + span - s.window ||
            (long long)j0 + kTileKeys <= s.sinks);
  }
};
__device__ __forceinline__ WeightChunk weight_chunk(const AttnShape& s, int c, int n, int len) {
  WeightChunk w;
  w.keys = tile_keys<true>(s, c, n, len);
  const unsigned r0 = (unsigned)c * s.rows;
  unsigned r1 = r0 + s.rows;
  if (r1 > (unsigned)n * s.group) r1 = (unsigned)n * s.group;
  const int t0 = token_of(s, r0);
  w.at0 = (long long)len - n + t0;
  w.span = token_of(s, r1 - 1) - t0;
  return w;
}

// Up to 16 tiles of a segment for one chunk of its rows; count = 0 ends the range.
struct alignas(16) WeightPlan {
  float scale[32];      // of the tiles' pages, NaN where there is none
  WeightChunk chunk;
  int seq, head, len, keys_hi;
  int row0, rows, c;    // the sequence's first row and rows, number of the chunk
  int tile0, count;
  int first, any;       // it begins the chunk; some tile of the segment is seen in it
};
constexpr int kWeightPlans = 4;

template <int N>
struct alignas(16) WeightsCtl {
  uint64_t plan_full[kWeightPlans], plan_free[kWeightPlans];  // published / read by every warp
  uint64_t scale_full[kWeightPlans];                          // its pages' scales are there
  uint64_t k_full[6], k_free[6];  // K slot landed / read
  uint64_t s_full[4], s_free[4];  // St computed / loaded (128)
  uint64_t q_full;                // rows of a chunk staged (all key threads)
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
  alignas(16) float4 row[N / 2];  // of two rows: score factors, then -LSE log2(e)
  alignas(16) int token[N];       // of a row, from the chunk's first; -1: no row
  WeightPlan plan[kWeightPlans];
  long long warp_sum[4];
  int before[kWeightMaxBatch + 1];
};
template <int D, int N>
constexpr size_t weights_smem() {
  return 1024 + WeightsCfg<D, N>::kCtl + sizeof(WeightsCtl<N>);
}
// (Of an SM's 228 KB, each CTA takes 1 KB more than its own.)
template <int N>
constexpr bool weights_fit() {
  return WeightsCfg<128, N>::kResident * (weights_smem<128, N>() + 1024) <= 228 * 1024;
}
static_assert(weights_fit<16>() && weights_fit<32>() && weights_fit<64>() && weights_fit<128>(),
              "resident CTAs");

template <int D, int N>
__global__ void __launch_bounds__(WeightsCfg<D, N>::kThreads, WeightsCfg<D, N>::kResident)
    key_weights_kernel(const __grid_constant__ CUtensorMap k_map, const KeyWeightsArgs a) {
  using C = WeightsCfg<D, N>;
  constexpr int kIssuer = C::kKeyThreads / 32, kProducer = kIssuer + 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  WeightsCtl<N>* cb = reinterpret_cast<WeightsCtl<N>*>(smem + C::kCtl);
  volatile int* abort_flag = &cb->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const AttnShape& sh = a.shape;
  // The split sees one unit for each (sequence with rows, head), of all its keys.
  const AttnShape whole = {sh.heads_k, 1, 1, 0, -1, a.keys, 0, 0};
  auto seq_of = [&](int b, RowRange* q, int* len) {
    *q = row_range(__ldg(a.cu + b), __ldg(a.cu + b + 1), a.total_q);
    q->n = q->n > 0 ? 1 : 0;
    *len = __ldg(a.seq_lens + b);
  };

  if (tid == C::kKeyThreads) {
    auto init = [&](uint64_t& b, uint32_t n) { ptx::mbar_init(ptx::smem_u32(&b), n); };
    for (int s = 0; s < kWeightPlans; ++s) {
      init(cb->plan_full[s], 1);
      init(cb->plan_free[s], kProducer);  // the warps before it
      init(cb->scale_full[s], 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      init(cb->k_full[s], 1);
      init(cb->k_free[s], 1);
    }
    for (int s = 0; s < C::kBuffers; ++s) {
      init(cb->s_full[s], 1);
      init(cb->s_free[s], 128);
    }
    init(cb->q_full, C::kKeyThreads);
    init(cb->drain, 1);
    cb->abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&k_map);
  }
  if (warp == kProducer) {
    ptx::tmem_alloc(ptx::smem_u32(&cb->tmem_base), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp < 4) {
    scan_costs<128>(cb->before, cb->warp_sum, a.batch, [&](int b) {
      RowRange q;
      int len;
      seq_of(b, &q, &len);
      return (long long)capped_cost(sh.heads_k * head_cost(whole, q.n, len));
    });
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = cb->tmem_base;
  auto before = [&](int b) { return cb->before[b]; };
  const int total = cb->before[a.batch];
  auto wait = [&](uint64_t& b, int parity) {
    return paged_wait(ptx::smem_u32(&b), (uint32_t)parity, abort_flag, a.status, a.wait_limit_ns);
  };
  // Batch number b; every warp but the producer's reads it and lets it go.
  auto plan_of = [&](int b, bool* ok) -> const WeightPlan& {
    *ok = wait(cb->plan_full[b % kWeightPlans], (b / kWeightPlans) & 1);
    return cb->plan[b % kWeightPlans];
  };
  auto plan_done = [&](int b) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->plan_free[b % kWeightPlans]));
  };
  bool ok = true;

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    test_load_delay(a.wait_limit_ns);
    SegmentWalk walk;
    walk_begin(&walk, range_start(total, gridDim.x, blockIdx.x),
               range_start(total, gridDim.x, blockIdx.x + 1), a.batch, before);
    Segment g = {};
    int rows = 0, row0 = 0;       // of the segment's sequence
    int c = 0, chunks = 0, t0 = 0;  // of the batch at hand
    auto next_segment = [&]() {
      if (!walk_next(&walk, whole, before, seq_of, &g)) return false;
      const RowRange r = row_range(__ldg(a.cu + g.seq), __ldg(a.cu + g.seq + 1), a.total_q);
      row0 = r.lo;
      rows = r.n;
      chunks = row_tiles(sh, rows);
      c = 0;
      t0 = 0;
      return true;
    };
    bool more = next_segment();
    int loads = 0;
    for (int b = 0;; ++b) {
      const int slot = b % kWeightPlans;
      WeightPlan& plan = cb->plan[slot];
      // Lane l: page l of the batch's tiles, as its cell, or -1.
      int id = -1;
      int tile0 = 0, count = 0;
      WeightChunk wc = {};
      if (more) {
        tile0 = g.tile0 + t0;
        count = imin(16, g.count - t0);
        const long long p = (long long)tile0 * 2 + lane;
        if (lane / 2 < count && p * kPageTokens < g.keys.hi)
          id = __ldg(a.page_table + (size_t)g.seq * a.max_pages + p);
        wc = weight_chunk(sh, c, rows, g.len);
      }
      if (b >= kWeightPlans) ok = wait(cb->plan_free[slot], (b / kWeightPlans - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        plan.count = count;
        plan.chunk = wc;
        plan.seq = g.seq;
        plan.head = g.head;
        plan.len = g.len;
        plan.keys_hi = g.keys.hi;
        plan.row0 = row0;
        plan.rows = rows;
        plan.c = c;
        plan.tile0 = tile0;
        plan.first = t0 == 0;
        plan.any = wc.any(g.tile0 * kTileKeys, (g.tile0 + g.count) * (long long)kTileKeys);
        ptx::mbar_arrive(ptx::smem_u32(&cb->plan_full[slot]));
      }
      __syncwarp();
      if (!more) break;
      // (The rows of Q are on their way now; the scales follow the first tile.)
      id = checked_page(id, a.num_pages);
      const int cell = id >= 0 ? id * sh.heads_k + g.head : -1;
      const float scale = cell >= 0 ? __ldg(a.k_scale + cell) : __int_as_float(0x7fffffff);
#pragma unroll 1
      for (int t = 0; ok && t < count; ++t) {
        if (wc.seen((tile0 + t) * kTileKeys)) {
          const int mine = __shfl_sync(0xffffffffu, cell, 2 * t + (lane & 1));
          const unsigned held = __ballot_sync(0xffffffffu, mine >= 0) & 3;
          const int s = loads % C::kSlots;
          if (loads >= C::kSlots) ok = wait(cb->k_free[s], (loads / C::kSlots - 1) & 1);
          if (!ok) break;
          const uint32_t bar = ptx::smem_u32(&cb->k_full[s]);
          if (lane == 0)
            ptx::mbar_arrive_expect_tx(bar, ((held & 1) + (held >> 1)) * C::kPageBytes);
          __syncwarp();
          if (lane < 2 && mine >= 0)
            ptx::tma_load_3d(ptx::smem_u32(smem + s * C::kTileBytes) + lane * C::kPageBytes, &k_map,
                             bar, 0, 0, mine);
          ++loads;
        }
        if (t == 0) {
          plan.scale[lane] = scale;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->scale_full[slot]));
        }
      }
      if (!ok) break;
      t0 += 16;
      if (t0 >= g.count) {
        t0 = 0;
        if (++c == chunks) more = next_segment();
      }
    }
    // Every copy this CTA started lands before it exits.
    for (int s = 0; s < C::kSlots && s < loads; ++s)
      wait_drain_warp(ptx::smem_u32(&cb->k_full[s]), ((loads - 1 - s) / C::kSlots) & 1, a.status);
  } else if (warp == kIssuer) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, N);
    constexpr uint32_t idesc_e5m2 = ptx::idesc_e4m3_e5m2_f32(128, C::kCols);
    const uint64_t q_hi = ptx::smem_desc(ptx::smem_u32(smem + C::kQ), 16, 8 * D, C::kSwK);
    const uint64_t q_mid = ptx::smem_desc(ptx::smem_u32(smem + C::kQ + N * D), 16, 8 * D, C::kSwK);
    const uint64_t q_rest =
        ptx::smem_desc(ptx::smem_u32(smem + C::kQ + 2 * N * D), 16, 8 * D, C::kSwK);
    int i = 0, staged = 0;
    for (int b = 0; ok; ++b) {
      const WeightPlan& plan = plan_of(b, &ok);
      if (!ok || plan.count == 0) break;
      const int count = plan.count, tile0 = plan.tile0;
      const WeightChunk wc = plan.chunk;
      const bool stage = plan.first && plan.any;
      plan_done(b);
      if (stage) ok = wait(cb->q_full, staged++ & 1);
#pragma unroll 1
      for (int t = 0; ok && t < count; ++t) {
        if (!wc.seen((tile0 + t) * kTileKeys)) continue;
        const int s = i % C::kSlots, sb = i % C::kBuffers;
        ok = wait(cb->k_full[s], (i / C::kSlots) & 1);
        if (ok && i >= C::kBuffers) ok = wait(cb->s_free[sb], (i / C::kBuffers - 1) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t kd =
            ptx::smem_desc(ptx::smem_u32(smem + s * C::kTileBytes), 16, 8 * D, C::kSwK);
        // (The small terms first: each step rounds at the sum's size so far.)
        const uint32_t d = tmem + sb * C::kCols;
        if constexpr (C::kApart) {
          ptx::mma_f8_elect<D / 32>(d, kd, q_mid, idesc_e5m2);  // and q_rest, N columns on
          ptx::mma_f8_elect<D / 32, true>(d, kd, q_hi, idesc);
        } else {
          ptx::mma_f8_elect<D / 32>(d, kd, q_rest, idesc_e5m2);
          ptx::mma_f8_elect<D / 32, true>(d, kd, q_mid, idesc_e5m2);
          ptx::mma_f8_elect<D / 32, true>(d, kd, q_hi, idesc);
        }
        ptx::mma_commit_elect(ptx::smem_u32(&cb->s_full[sb]));
        ptx::mma_commit_elect(ptx::smem_u32(&cb->k_free[s]));
        ++i;
      }
    }
    ptx::mma_commit_elect(ptx::smem_u32(&cb->drain));
    wait_drain_warp(ptx::smem_u32(&cb->drain), 0, a.status);
  } else {
    // ------------------------------------------------------------- weights
    const float neg_inf = -__int_as_float(0x7f800000);
    constexpr int kLanes = D / 16;  // lanes of a row of Q, 16 dims each
    const uint32_t s_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int key = tid & 127, group = tid >> 7;  // key of a tile; warpgroup
    int i = 0, turn = 0;
    for (int b = 0;; ++b) {
      // (A warp whose wait has given up joins the others here, and all leave.  So
      // does every chunk's last tile before the next one's rows are staged.)
      bool got;
      const WeightPlan& plan = plan_of(b, &got);
      ok = named_bar_and(1, C::kKeyThreads, ok && got);
      if (!ok || plan.count == 0) break;
      if (plan.first && plan.any) {
        // ---- the chunk's rows of Q.  (The last chunk's MMAs are done: every thread
        // has waited for them.  So the issuer has taken each staging before the
        // next one.)
        const int rows = plan.rows, row0 = plan.row0, c = plan.c, head = plan.head;
        const int n_rows = imin(N, rows * sh.group - c * N);
        {
          // A warp's kEach rows: as bf16 into the place of their first two terms, a
          // half of the dims each; then kLanes lanes take a row at a time, 16 dims
          // each.  (In a short loop: its code is fetched anew for each unit.)
          constexpr int kEach = N / (C::kKeyThreads / 32), kAtOnce = 32 / kLanes;
          constexpr int kTurns = (kEach + kAtOnce - 1) / kAtOnce;
          const int sub = lane % kLanes, dim0 = sub * 16;
          uint8_t* warp_q = smem + C::kQ + warp * kEach * D;
          uint8_t* raw0 = warp_q + (sub >= kLanes / 2 ? N * D : 0) + (sub % (kLanes / 2)) * 32;
          float lse_of[kTurns];
#pragma unroll
          for (int k = 0; k < kTurns; ++k) {
            const int i = k * kAtOnce + lane / kLanes, n = warp * kEach + i, row = c * N + n;
            const int tok = token_of(sh, row), h = head * sh.group + row - tok * sh.group;
            const bool some = i < kEach && n < n_rows;
            const uint16_t* from =
                a.q + (some ? (long long)(row0 + tok) * a.q_row + (long long)h * a.q_head + dim0 : 0);
            if (i < kEach) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const bool in = some && dim0 + 8 * u < a.dim;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 ptx::smem_u32(raw0 + i * D + 16 * u)),
                             "l"(in ? from + 8 * u : a.q), "r"(in ? 16 : 0)
                             : "memory");
              }
            }
            // (A row that sees nothing, LSE -inf, or that is none, adds 0.)
            lse_of[k] = some ? __ldg(a.lse + (size_t)h * a.total_q + row0 + tok) : neg_inf;
            if (sub == 0 && i < kEach) cb->token[n] = some ? tok - token_of(sh, c * N) : -1;
          }
#pragma unroll
          for (int k = 0; k < kTurns; ++k) {
            const int i = k * kAtOnce + lane / kLanes, n = warp * kEach + i;
            if (sub == 0 && i < kEach)
              reinterpret_cast<float*>(cb->row + n / 2)[2 + (n & 1)] =
                  lse_of[k] == neg_inf
                      ? neg_inf
                      : -fmaf(lse_of[k], a.lse_log2, lse_of[k] * a.lse_log2_rest);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
#pragma unroll 1
          for (int k = 0; k < kTurns; ++k) {
            const int i = k * kAtOnce + lane / kLanes, n = warp * kEach + i;
            uint4 r0 = make_uint4(0u, 0u, 0u, 0u), r1 = r0;
            // (A row that adds nothing is zeros: a NaN of its would stay one times 0.)
            if (i < kEach && reinterpret_cast<const float*>(cb->row + n / 2)[2 + (n & 1)] != neg_inf) {
              r0 = *reinterpret_cast<const uint4*>(raw0 + i * D);
              r1 = *reinterpret_cast<const uint4*>(raw0 + i * D + 16);
            }
            // The largest magnitude, as bits of bf16 (those past infinity's are NaN).
            const uint32_t w[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
            uint32_t top = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) top = __vmaxu2(top, w[u] & 0x7fff7fffu);
            top = max(top & 0xffffu, top >> 16);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
              top = max(top, __shfl_xor_sync(0xffffffffu, top, o));  // (the row is read)
            const float mx = __uint_as_float(min(top, 0x7f80u) << 16);
            const int e = terms_exponent(mx);
            float x[8];
            uint32_t hi[8], mid[8], rest[8];
            unpack_bf16x8(r0, x);
            split_three(x, e, hi, mid, rest);
            unpack_bf16x8(r1, x);
            split_three(x, e, hi + 4, mid + 4, rest + 4);
            const int us = D == 128 ? (sub ^ (n & 7)) : (sub ^ ((n >> 1) & 3));
            uint8_t* at = warp_q + i * D + us * 16;
            auto put = [&](int term, const uint32_t* v) {
              *reinterpret_cast<uint4*>(at + term * N * D) =
                  make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16,
                             v[6] | v[7] << 16);
            };
            if (i < kEach) {
              put(0, hi);
              put(1, mid);
              put(2, rest);
              if (sub == 0) {
                float* r = reinterpret_cast<float*>(cb->row + n / 2) + (n & 1);
                r[0] = r[2] == neg_inf ? 0.f : terms_scale(mx, e, a.scale_log2);
              }
            }
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(ptx::smem_u32(&cb->q_full));
          named_bar_sync(1, C::kKeyThreads);
        }
      }
      // ---- the tiles
      const int count = plan.count, tile0 = plan.tile0, keys_hi = plan.keys_hi;
      const bool first_chunk = plan.c == 0;
      float* out = a.weights + ((long long)plan.seq * sh.heads_k + plan.head) * a.capacity;
      // The rows' own keys have no weight yet.
      const long long fresh = (long long)plan.len - plan.rows;
      const WeightChunk& wc = plan.chunk;
      ok = wait(cb->scale_full[b % kWeightPlans], (b / kWeightPlans) & 1);
      // Sums of the rows' weights for this thread's key in kCount tiles from t on,
      // whose St are in the buffers from tile i on.
      auto add_up = [&](auto tiles, int t, float* sum) {
        constexpr int kCount = decltype(tiles)::value;
        bool all = true;
        int lo[kCount], hi[kCount];
        uint64_t ks2[kCount], acc[kCount][2];
        uint32_t col[kCount];
#pragma unroll
        for (int k = 0; k < kCount; ++k) {
          const int sb = (i + k) % C::kBuffers, j0 = (tile0 + t + k) * kTileKeys, j = j0 + key;
          if (ok) ok = wait(cb->s_full[sb], ((i + k) / C::kBuffers) & 1);
          col[k] = s_lane + sb * C::kCols;
          const float ks = plan.scale[2 * (t + k) + ((warp >> 1) & 1)];
          ks2[k] = ptx::f2_pack(ks, ks);
          acc[k][0] = acc[k][1] = 0ull;
          // Rows that see the key: tokens [lo, hi].
          lo[k] = 0;
          hi[k] = 0x7fffffff;
          if (!wc.whole(j0, sh)) {
            all = false;
            const long long r = (long long)j - wc.at0;
            if (sh.causal) lo[k] = (int)(r > 0 ? (r < 0x7fffffff ? r : 0x7fffffff) : 0);
            if (sh.window >= 0 && j >= sh.sinks) {
              const long long w = r + sh.window;
              hi[k] = (int)(w < 0x7fffffff ? (w > -1 ? w : -1) : 0x7fffffff);
            }
          }
        }
        if (!ok) return;
        ptx::tc_fence_after();
        // (Twice: whole tiles without a test for each row.)
        auto rows_of = [&](auto masked) {
#pragma unroll 1
          for (int n0 = 0; n0 < N; n0 += 16) {
            uint32_t now[kCount][16], low[C::kApart ? kCount : 1][16];
#pragma unroll
            for (int k = 0; k < kCount; ++k) {
              ptx::tmem_ld16(col[k] + n0, now[k]);
              if constexpr (C::kApart) ptx::tmem_ld16(col[k] + N + n0, low[k]);
            }
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < kCount; ++k) {
              ptx::reg_fence16(now[k]);
              if constexpr (C::kApart) ptx::reg_fence16(low[k]);
            }
            if (n0 + 16 == N) {
              ptx::tc_fence_before();
#pragma unroll
              for (int k = 0; k < kCount; ++k)
                ptx::mbar_arrive(ptx::smem_u32(&cb->s_free[(i + k) % C::kBuffers]));
            }
#pragma unroll
            for (int n = 0; n < 16; n += 2) {
              const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(cb->row + (n0 + n) / 2);
#pragma unroll
              for (int k = 0; k < kCount; ++k) {
                uint64_t s2 =
                    ptx::f2_pack(__uint_as_float(now[k][n]), __uint_as_float(now[k][n + 1]));
                if constexpr (C::kApart)
                  s2 = ptx::add2(s2, ptx::f2_pack(__uint_as_float(low[k][n]),
                                                  __uint_as_float(low[k][n + 1])));
                float u, v;
                ptx::f2_unpack(ptx::fma2(s2, ptx::mul2(f.x, ks2[k]), f.y), u, v);
                if constexpr (decltype(masked)::value != 0) {
                  const int2 tok = *reinterpret_cast<const int2*>(cb->token + n0 + n);
                  u = tok.x >= lo[k] && tok.x <= hi[k] ? u : neg_inf;
                  v = tok.y >= lo[k] && tok.y <= hi[k] ? v : neg_inf;
                }
                acc[k][(n >> 1) & 1] =
                    ptx::add2(acc[k][(n >> 1) & 1], ptx::f2_pack(ptx::ex2(u), ptx::ex2(v)));
              }
            }
          }
        };
        if (all) rows_of(IntTag<0>{});
        else rows_of(IntTag<1>{});
#pragma unroll
        for (int k = 0; k < kCount; ++k) {
          float u, v;
          ptx::f2_unpack(ptx::add2(acc[k][0], acc[k][1]), u, v);
          // (No page: no weight.)
          sum[k] = __isnanf(plan.scale[2 * (t + k) + ((warp >> 1) & 1)]) ? 0.f : u + v;
        }
      };
      // What stands at this thread's key of tile t already, where it counts.
      auto held = [&](int t) {
        const int j = (tile0 + t) * kTileKeys + key;
        const bool add = !first_chunk || (a.decay != 0.f && j < fresh);
        return t < count && j < keys_hi && add ? out[j] : 0.f;
      };
      // (One tile at a time: the next one's is under way while this is summed.)
      float ahead = C::kTiles == 1 ? held(0) : 0.f;
#pragma unroll 1
      for (int t = 0; ok && t < count;) {
        const bool seen = wc.seen((tile0 + t) * kTileKeys);
        // Two neighbours that are seen go together.
        const int n_tiles = C::kTiles == 2 && seen && t + 1 < count &&
                                    wc.seen((tile0 + t + 1) * kTileKeys) ? 2 : 1;
        // (Two groups: by turns.  What a chunk writes, the next may read in the
        // other group, behind the barrier between them.)
        if (C::kTiles == 2 && (turn++ & 1) != group) {
          i += seen ? n_tiles : 0;
          t += n_tiles;
          continue;
        }
        // What stands there already, and whether it changes.
        float old[C::kTiles], sum[C::kTiles];
        if constexpr (C::kTiles == 1) {
          old[0] = ahead;
          ahead = held(t + 1);
        } else {
          old[0] = held(t);
          old[1] = n_tiles == 2 ? held(t + 1) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < C::kTiles; ++k) sum[k] = 0.f;
        const bool change = seen || (first_chunk && !(a.decay == 1.f &&
                                                      (tile0 + t) * kTileKeys + key < fresh));
        if (seen) {
          if (n_tiles == C::kTiles) add_up(IntTag<C::kTiles>{}, t, sum);
          else add_up(IntTag<1>{}, t, sum);
          if (!ok) break;
          i += n_tiles;
        }
#pragma unroll
        for (int k = 0; k < C::kTiles; ++k) {
          const int j = (tile0 + t + k) * kTileKeys + key;
          if (change && k < n_tiles && j < keys_hi)
            out[j] = (first_chunk ? old[k] * a.decay : old[k]) + sum[k];
        }
        t += n_tiles;
      }
      plan_done(b);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kProducer) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace fa
