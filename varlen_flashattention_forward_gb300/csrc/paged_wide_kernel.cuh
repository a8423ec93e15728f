// paged_wide_kernel.cuh -- attention of many query rows per sequence over the
// paged 8-bit cache under the masks (drafted trees, sinks), for sm_103a.
//
// paged_attn_kernel puts the keys on the tensor core's M side and few rows on the
// other, and reads and converts the keys again for every 16 or 32 of them.  A
// tree of 64 nodes with 4 heads of a group has 256 rows.  Here the rows are on
// the M side, two tiles of 128 of them (row = token * group + head) against each
// tile of 128 keys:
//
//   S_t[row, key] = Q_t[row, d] . K[key, d]t   e4m3 x e4m3, M = N = 128
//   O_t[row, d]  += P_t[row, key] . V[key, d]  f16 x f16,   P_t from TMEM
//
// K is multiplied as it lies in the cache.  A row of Q is the sum of two e4m3
// terms (split_terms), whose products add up in one accumulator.  V goes through
// registers to f16 (exact).  A thread has a row, so that a mask is a word of
// bits for 32 keys, and nothing is reduced between threads:
//
//   x = scale q.k, x' = x + log2(vs): m is the maximum of x' so far (taken anew
//   when a tile passes it by 2^8), P' = 2^(x - m + 7) vs as f16, the row sum adds
//   2^(x - m + 7) (see paged_attn_kernel for the ranges).
//
//   planner warp     walks the CTA's segments of key tiles (paged_index.h) and
//                    publishes them, 16 tiles at a time, with the places and
//                    scales of their pages
//   producer warp    TMA of K and V pages into two rings
//   converter warps  V to f16, rows nobody sees as zeros
//   two issuers      of a row tile each: S_t of a page (64 keys) into one half of
//                    its columns while the softmax has the other, O_t once P_t
//                    and V are there
//   two softmax      warpgroups, of a row tile each: its rows of Q in two terms
//                    at a segment's start, the softmax page by page, the output
//                    at its end
//
// TMEM: S_0 / P_0, S_1 / P_1 (two pages each), O_0, O_1, 128 columns each.
//
// 24 trees of 33 to 64 nodes over 517 to 5000 keys, 32 and 8 heads of 128 dims: 82
// us with the merge, 610 TFLOP/s (384 us 32 rows to a tile, 157 us through the
// gather and the packed forward).  Of some 135 000 cycles of a CTA, 28 tiles take
// 3500 each: softmax 2700 (exponentials 1330, masks and maxima 370, rescaling 450,
// TMEM 450), waiting for S 500; the tensor core's own share is 2150.  A whole tile
// of scores at once, with P in its place, took 4200 to 5000, the chain S, softmax,
// P V of each row tile.  A change of unit takes some 13 000: rows of Q 8000, bound by
// the conversions to e4m3, output 3000 (7000 to 10 000 with parts copied by the lanes).
// One tree of 16 nodes over 4096 keys: 22 us, of 24 000 cycles in the longest CTA 2400
// up to the split, 3200 for its first unit, 7000 for the rows, 7000 for three tiles.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "cost_scan.cuh"
#include "paged_attn_kernel.cuh"  // arguments, waits

namespace fa {

constexpr int kWideRows = 256;  // of a unit's row tile
constexpr int kWideThreads = 512;
constexpr int kWideConvertWarp = 8, kWideIssueWarp = 12, kWideLoadWarp = 14, kWidePlanWarp = 15;
// Register split (launch: 128 x 512 = 65536): softmax 256 x 192, converters and
// control 128 x 64 each = 65536.
constexpr uint32_t kWideSoftmaxRegs = 192;
constexpr uint32_t kWideOtherRegs = 64;

// Up to kPlanTiles tiles of one segment; count = 0 ends the range.
struct alignas(16) WidePlan {
  PagePlan page[2 * kPlanTiles];
  int cell[2 * kPlanTiles];
  int count, tile0, gap_at, gap;  // tile t: tile0 + t, and gap more from gap_at on
  int first, last;                // it begins, ends the segment
  int lo, hi, sink;               // keys that some row of the unit sees
  int head, q0, n, len;           // of the sequence: first q row, rows, keys
  int row0, rows;                 // of the unit's row tile
  int whole, unit_end;            // see BatchPlan
};

template <int D>
struct WideCfg {
  static constexpr uint32_t kSwK = D == 128 ? ptx::kLayoutSw128 : ptx::kLayoutSw64;
  static constexpr int kTileBytes = kTileKeys * D;  // K or V slot
  static constexpr int kPageBytes = kPageTokens * D;
  static constexpr int kVhBytes = kTileKeys * D * 2;
  static constexpr int kTermBytes = 128 * D;        // one term of a row tile of Q
  static constexpr int NK = D == 64 ? 6 : 3;
  static constexpr int NV = D == 64 ? 4 : 2;
  static constexpr int kK = 0;
  static constexpr int kV = kK + NK * kTileBytes;
  static constexpr int kVh = kV + NV * kTileBytes;
  static constexpr int kQ = kVh + 2 * kVhBytes;     // [tile][hi, lo][row]
  static constexpr int kCtl = kQ + 4 * kTermBytes;
  static constexpr uint32_t kOt = 256;              // TMEM column of O_0
};

struct alignas(16) WideCtl {
  uint64_t plan_full[kPagedPlans], plan_free[kPagedPlans];  // batch published / read (15)
  uint64_t cell_full[kPagedPlans], scale_full[kPagedPlans];  // its pages, their scales there
  uint64_t k_full[6], k_free[6];      // K slot landed / read by both issuers' S
  uint64_t v_full[4], v_free[4];      // V slot landed / converted (128)
  uint64_t vh_full[2], vh_free[2];    // f16 V written (128) / read by both issuers' P V
  uint64_t q_full[2];                 // rows of Q staged (128)
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // of a row tile and half: S_t
                                      // computed, P_t written (128), P V complete
  uint64_t o_full[2], o_free[2];      // O_t complete / read out (128)
  uint64_t drain;
  uint32_t tmem_base;
  volatile int abort_flag;
  WidePlan plan[kPagedPlans];
  long long warp_sum[8];
  int before[kPagedMaxBatch + 1];
};
template <int D>
constexpr size_t wide_smem() {
  return 1024 + WideCfg<D>::kCtl + sizeof(WideCtl);
}
static_assert(wide_smem<128>() <= 232448, "shared memory exceeds the per-CTA limit");

template <int D>
__global__ void __launch_bounds__(kWideThreads, 1)
    paged_wide_kernel(const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map, const PagedAttnArgs a) {
  using C = WideCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  WideCtl* cb = reinterpret_cast<WideCtl*>(smem + C::kCtl);
  volatile int* abort_flag = &cb->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const AttnShape& sh = a.shape;
  auto seq_of = [&](int b, RowRange* q, int* len) {
    *q = row_range(__ldg(a.cu + b), __ldg(a.cu + b + 1), a.total_q);
    *len = __ldg(a.seq_lens + b);
  };

  ptx::grid_launch_dependents();
  if (warp == kWideLoadWarp && lane == 0) {
    auto init = [&](uint64_t& b, uint32_t n) { ptx::mbar_init(ptx::smem_u32(&b), n); };
    for (int s = 0; s < kPagedPlans; ++s) {
      init(cb->plan_full[s], 1);
      init(cb->plan_free[s], kPlanReaders);
      init(cb->cell_full[s], 1);
      init(cb->scale_full[s], 1);
    }
    for (int s = 0; s < C::NK; ++s) {
      init(cb->k_full[s], 1);
      init(cb->k_free[s], 2);
    }
    for (int s = 0; s < C::NV; ++s) {
      init(cb->v_full[s], 1);
      init(cb->v_free[s], 128);
    }
    for (int s = 0; s < 2; ++s) {
      init(cb->vh_full[s], 128);
      init(cb->vh_free[s], 2);
      init(cb->q_full[s], 128);
      for (int h = 0; h < 2; ++h) {
        init(cb->s_full[s][h], 1);
        init(cb->p_full[s][h], 128);
        init(cb->pv_done[s][h], 1);
      }
      init(cb->o_full[s], 1);
      init(cb->o_free[s], 128);
    }
    init(cb->drain, 2);
    cb->abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&k_map);
    ptx::prefetch_tmap(&v_map);
  }
  if (warp == kWideIssueWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&cb->tmem_base), 512);
    ptx::tmem_relinquish();
  }
  if (warp < 8) {
    if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    scan_costs<256>(cb->before, cb->warp_sum, a.batch, [&](int b) {
      RowRange q;
      int len;
      seq_of(b, &q, &len);
      return (long long)capped_cost(sh.heads_k * head_cost<true>(sh, q.n, len));
    });
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = cb->tmem_base;
  auto before = [&](int b) { return cb->before[b]; };
  const int total = cb->before[a.batch];
  const int cta = blockIdx.x, ctas = gridDim.x;
  auto wait = [&](uint64_t& b, int parity) {
    return paged_wait(ptx::smem_u32(&b), (uint32_t)parity, abort_flag, a.status, a.wait_limit_ns);
  };
  // Batch number b; every warp that reads it lets it go with plan_done.
  auto plan_of = [&](int b, bool* ok) -> const WidePlan& {
    *ok = wait(cb->plan_full[b % kPagedPlans], (b / kPagedPlans) & 1);
    return cb->plan[b % kPagedPlans];
  };
  auto plan_done = [&](int b) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->plan_free[b % kPagedPlans]));
  };

  if (warp >= kWideConvertWarp && warp < kWideIssueWarp) {
    ptx::regs_dec<kWideOtherRegs>();
    // ------------------------------------------------------------ converters
    // (As in paged_attn_kernel: units of 16 codes, eight lanes on the rows r and
    // r ^ 5, so that loads and stores meet no bank twice.)
    constexpr int kChunks = D / 64;          // 64-dim chunks of an f16 row
    constexpr int kIters = D / 16;           // units of a thread
    constexpr int kStep = 32 / kChunks;      // its rows' distance
    const int t = tid - 32 * kWideConvertWarp;
    const int u4 = t & 3, pair = t >> 3, chunk = pair % kChunks;
    const int even = 2 * (pair / kChunks), r0 = (t & 4) ? even ^ 5 : even;
    const int u = chunk * 4 + u4;
    const int us = D == 128 ? (u ^ (r0 & 7)) : (u ^ ((r0 >> 1) & 3));
    const uint8_t* src0 = smem + C::kV + r0 * D + us * 16;
    const int p0 = (2 * u4) ^ (r0 & 7);
    uint8_t* dst0 = smem + C::kVh + chunk * (kTileKeys * 128) + r0 * 128 + p0 * 16;
    uint8_t* dst1 = smem + C::kVh + chunk * (kTileKeys * 128) + r0 * 128 + (p0 ^ 1) * 16;
    bool ok = true;
    int i = 0;
    for (int b = 0; ok; ++b) {
      const WidePlan& plan = plan_of(b, &ok);
      if (!ok) break;
      const int count = plan.count, tile0 = plan.tile0, gap_at = plan.gap_at, gap = plan.gap;
      const int key_lo = plan.lo, key_hi = plan.hi, sink = plan.sink;
      if (count == 0) break;
      ok = wait(cb->scale_full[b % kPagedPlans], (b / kPagedPlans) & 1);  // (held)
      if (!ok) break;
      const unsigned held = __ballot_sync(0xffffffffu, plan.page[lane].held != 0);
      plan_done(b);
#pragma unroll 1
      for (int n = 0; n < count; ++n, ++i) {
        const int hb = i & 1, slot = i % C::NV;
        ok = wait(cb->v_full[slot], (i / C::NV) & 1);
        if (!ok) break;
        const uint8_t* src = src0 + slot * C::kTileBytes;
        uint4 c[kIters];
#pragma unroll
        for (int k = 0; k < kIters; ++k)
          c[k] = *reinterpret_cast<const uint4*>(src + k * kStep * D);
        const int key0 = (tile0 + n + (n >= gap_at ? gap : 0)) * kTileKeys;
        const int lo = key_lo - key0, hi = key_hi - key0, first = sink - key0;
        const unsigned pages = (held >> (2 * n)) & 3;
        if (__builtin_expect(lo > 0 || hi < kTileKeys || pages != 3, 0)) {
#pragma unroll
          for (int k = 0; k < kIters; ++k) {
            const int r = r0 + k * kStep;
            if ((r < lo && r >= first) || r >= hi || !((pages >> (r >> 6)) & 1))
              c[k] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        if (i >= 2) {
          ok = wait(cb->vh_free[hb], ((i >> 1) - 1) & 1);
          if (!ok) break;
        }
#pragma unroll
        for (int k = 0; k < kIters; ++k) {
          const int at = hb * C::kVhBytes + k * kStep * 128;
          *reinterpret_cast<uint4*>(dst0 + at) =
              make_uint4(unpack_e4m3x2(c[k].x), unpack_e4m3x2(c[k].x >> 16),
                         unpack_e4m3x2(c[k].y), unpack_e4m3x2(c[k].y >> 16));
          *reinterpret_cast<uint4*>(dst1 + at) =
              make_uint4(unpack_e4m3x2(c[k].z), unpack_e4m3x2(c[k].z >> 16),
                         unpack_e4m3x2(c[k].w), unpack_e4m3x2(c[k].w >> 16));
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(ptx::smem_u32(&cb->vh_full[hb]));
        ptx::mbar_arrive(ptx::smem_u32(&cb->v_free[slot]));
      }
    }
  } else if (warp >= kWideIssueWarp) {
    ptx::regs_dec<kWideOtherRegs>();
    if (warp < kWideLoadWarp) {
      // ------------------------------------------------------------- issuers
      const int t = warp - kWideIssueWarp;
      constexpr uint32_t idesc_s = ptx::idesc_e4m3_f32(128, kPageTokens);
      constexpr uint32_t idesc_pv = ptx::idesc_f16_f32(128, D, false, true);
      const uint32_t q_s = ptx::smem_u32(smem + C::kQ + 2 * t * C::kTermBytes);
      const uint64_t q_hi = ptx::smem_desc(q_s, 16, 8 * D, C::kSwK);
      const uint64_t q_lo = ptx::smem_desc(q_s + C::kTermBytes, 16, 8 * D, C::kSwK);
      const uint32_t s_col = tmem + 128 * t, o_col = tmem + C::kOt + 128 * t;
      bool ok = true;
      int i = 0, ki = 0, tiles = 0, seg = 0;  // tiles done and S'ed, tiles and segments of this row tile
      // S of a page of tile `ki`.  (Its columns: P_t of the page two before has been
      // taken by its P V, which this warp issued first.)
      auto issue_s = [&](int half) {
        const int slot = ki % C::NK;
        const uint64_t kd = ptx::smem_desc(
            ptx::smem_u32(smem + C::kK + slot * C::kTileBytes + half * C::kPageBytes), 16, 8 * D,
            C::kSwK);
        ptx::mma_f8_elect<D / 32>(s_col + 64 * half, q_lo, kd, idesc_s);
        ptx::mma_f8_elect<D / 32, true>(s_col + 64 * half, q_hi, kd, idesc_s);
        ptx::mma_commit_elect(ptx::smem_u32(&cb->s_full[t][half]));
        if (half == 1) {
          ptx::mma_commit_elect(ptx::smem_u32(&cb->k_free[slot]));
          ++ki;
        }
      };
      auto wait_k = [&]() {
        const bool landed = wait(cb->k_full[ki % C::NK], (ki / C::NK) & 1);
        ptx::tc_fence_after();
        return landed;
      };
      for (int b = 0; ok; ++b) {
        const WidePlan& plan = plan_of(b, &ok);
        if (!ok) break;
        const int count = plan.count, first = plan.first, last = plan.last;
        const bool mine = plan.rows > 128 * t;
        plan_done(b);
        if (count == 0) break;
        if (!mine) {
          // (A row tile that the unit has not: the slots are let go all the same.)
          for (int n = 0; ok && n < count; ++n, ++i, ++ki) {
            ok = wait_k();
            if (!ok) break;
            ptx::mma_commit_elect(ptx::smem_u32(&cb->k_free[ki % C::NK]));
            ok = wait(cb->vh_full[i & 1], (i >> 1) & 1);
            if (ok) ptx::mma_commit_elect(ptx::smem_u32(&cb->vh_free[i & 1]));
          }
          continue;
        }
        if (first) {
          ok = wait(cb->q_full[t], seg & 1);
          if (ok) ok = wait_k();
          if (!ok) break;
          issue_s(0);
          issue_s(1);
          if (seg > 0) ok = wait(cb->o_free[t], (seg - 1) & 1);
        }
#pragma unroll 1
        for (int n = 0; ok && n < count; ++n, ++i, ++tiles) {
          const int hb = i & 1;
          const bool end = last && n + 1 == count;  // of the segment
          const uint64_t vd = ptx::smem_desc(ptx::smem_u32(smem + C::kVh + hb * C::kVhBytes),
                                             kTileKeys * 128, 1024, ptx::kLayoutSw128);
          ok = wait(cb->vh_full[hb], (i >> 1) & 1);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (ok) ok = wait(cb->p_full[t][half], tiles & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            // (issue_pv_half counts from a 128-key tile's P; this page's is its own.)
            issue_pv_half<128>(o_col, s_col + 64 * half - 32 * half, vd, idesc_pv,
                               first && n == 0 && half == 0 ? 0u : 1u, half);
            ptx::mma_commit_elect(ptx::smem_u32(&cb->pv_done[t][half]));
            if (end && half == 1) ptx::mma_commit_elect(ptx::smem_u32(&cb->o_full[t]));
            if (!end) {
              if (half == 0) ok = wait_k();
              if (ok) issue_s(half);
            }
          }
          if (!ok) break;
          ptx::mma_commit_elect(ptx::smem_u32(&cb->vh_free[hb]));
        }
        if (last) ++seg;
      }
      ptx::mma_commit_elect(ptx::smem_u32(&cb->drain));
      wait_drain_warp(ptx::smem_u32(&cb->drain), 0, a.status);
    } else if (warp == kWideLoadWarp) {
      // ------------------------------------------------------------ producer
      // Lanes 0 and 1 issue the two pages of a tile with one instruction.
      test_load_delay(a.wait_limit_ns);
      bool ok = true;
      int kn = 0, vn = 0;
      for (int b = 0; ok; ++b) {
        const WidePlan& plan = plan_of(b, &ok);
        if (!ok) break;
        const int count = plan.count;
        if (count == 0) break;
        ok = wait(cb->cell_full[b % kPagedPlans], (b / kPagedPlans) & 1);
        if (!ok) break;
        const int cell = plan.cell[lane];
        plan_done(b);
#pragma unroll 1
        for (int n = 0; n < count; ++n) {
          const int mine = __shfl_sync(0xffffffffu, cell, 2 * n + (lane & 1));
          const unsigned held = __ballot_sync(0xffffffffu, mine >= 0) & 3;
          const uint32_t bytes = ((held & 1) + (held >> 1)) * C::kPageBytes;
          auto load = [&](const CUtensorMap* map, uint64_t& full, uint8_t* slot) {
            const uint32_t bar = ptx::smem_u32(&full);
            if (lane == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (lane < 2 && mine >= 0)
              ptx::tma_load_3d(ptx::smem_u32(slot) + lane * C::kPageBytes, map, bar, 0, 0, mine);
          };
          const int sk = kn % C::NK, sv = vn % C::NV;
          if (kn >= C::NK) ok = wait(cb->k_free[sk], (kn / C::NK - 1) & 1);
          if (!ok) break;
          load(&k_map, cb->k_full[sk], smem + C::kK + sk * C::kTileBytes);
          ++kn;
          if (vn >= C::NV) ok = wait(cb->v_free[sv], (vn / C::NV - 1) & 1);
          if (!ok) break;
          load(&v_map, cb->v_full[sv], smem + C::kV + sv * C::kTileBytes);
          ++vn;
        }
      }
      // Every copy this CTA started lands before it exits.
      for (int s = 0; s < C::NK && s < kn; ++s)
        wait_drain_warp(ptx::smem_u32(&cb->k_full[s]), ((kn - 1 - s) / C::NK) & 1, a.status);
      for (int s = 0; s < C::NV && s < vn; ++s)
        wait_drain_warp(ptx::smem_u32(&cb->v_full[s]), ((vn - 1 - s) / C::NV) & 1, a.status);
    } else {
      // ------------------------------------------------------------- planner
      SegmentWalk walk;
      walk_begin(&walk, range_start(total, ctas, cta), range_start(total, ctas, cta + 1), a.batch,
                 before);
      Segment g = {};
      bool ok = true, more = walk_next<true>(&walk, sh, before, seq_of, &g);
      int n0 = 0;  // tiles of the segment in earlier batches
      for (int b = 0;; ++b) {
        const int slot = b % kPagedPlans;
        WidePlan& plan = cb->plan[slot];
        // Lane l: page l of the batch's tiles, or -1 where it is not needed.
        int id = -1;
        if (more && n0 + lane / 2 < g.count) {
          const long long p = tile_of(g.tiles, g.part_lo + n0 + lane / 2) * 2ll + (lane & 1);
          if (p * kPageTokens < g.keys.hi &&
              ((p + 1) * kPageTokens > g.keys.lo || p * kPageTokens < g.keys.sink))
            id = __ldg(a.page_table + (size_t)g.seq * a.max_pages + p);
        }
        if (b >= kPagedPlans) ok = wait(cb->plan_free[slot], (b / kPagedPlans - 1) & 1);
        if (!ok) break;
        if (!more) {
          if (lane == 0) {
            plan.count = 0;
            ptx::mbar_arrive(ptx::smem_u32(&cb->plan_full[slot]));
          }
          break;
        }
        const bool last = g.count - n0 <= kPlanTiles;
        if (lane == 0) {
          const int left = g.tiles.head - (g.part_lo + n0);  // tiles before the gap
          plan.count = imin(g.count - n0, kPlanTiles);
          plan.tile0 = tile_of(g.tiles, g.part_lo + n0);
          plan.gap_at = imax(left, 0);
          plan.gap = left > 0 ? g.tiles.first - g.tiles.head : 0;
          plan.first = n0 == 0;
          plan.last = last;
          plan.lo = g.keys.lo;
          plan.hi = g.keys.hi;
          plan.sink = g.keys.sink;
          plan.head = g.head;
          plan.q0 = g.q.lo;
          plan.n = g.q.n;
          plan.len = g.len;
          plan.row0 = g.row_tile * kWideRows;
          plan.rows = imin(kWideRows, g.q.n * sh.group - g.row_tile * kWideRows);
          plan.whole = g.count == g.unit_count;
          plan.unit_end = g.part_lo == 0 && g.count < g.unit_count ? g.unit_end : -1;
          ptx::mbar_arrive(ptx::smem_u32(&cb->plan_full[slot]));
        }
        __syncwarp();
        // (The rows of Q are on their way now; then the pages, then their scales.)
        id = checked_page(id, a.num_pages);
        const int cell = id >= 0 ? id * sh.heads_k + g.head : -1;
        plan.cell[lane] = cell;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->cell_full[slot]));
        float ks = 0.f, vs = 0.f;
        if (cell >= 0) {
          ks = __ldg(a.k_scale + cell);
          vs = __ldg(a.v_scale + cell);
        }
        plan.page[lane] = PagePlan{ks, vs, fmaxf(log2f(vs), -(float)kScaleExpMax), cell >= 0};
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->scale_full[slot]));
        n0 += kPlanTiles;
        if (last) {
          n0 = 0;
          more = walk_next<true>(&walk, sh, before, seq_of, &g);
        }
      }
    }
  } else {
    ptx::regs_inc<kWideSoftmaxRegs>();
    // -------------------------------------------------------------- softmax
    const float neg_inf = -__int_as_float(0x7f800000);
    const int t = warp >> 2, r = tid & 127;  // row tile, row of it (TMEM lane)
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + 128 * t;
    const uint32_t o_addr = tmem + lane_base + C::kOt + 128 * t;
    uint8_t* q_tile = smem + C::kQ + 2 * t * C::kTermBytes;
    bool ok = true;
    int tiles = 0, seg = 0, segs = 0;  // key tiles and segments of this row tile; segments of the CTA
    // The segment's row: scale of its terms, the keys it sees ([lo, hi), [0,
    // sink) and those its mask names from key ctx on), maximum and sum.
    float qs = 0.f, m_used = neg_inf, l = 0.f;
    int lo_i = 0, hi_i = 0, sink_i = 0, ctx = 0, row_q = 0, row_h = 0;
    const int* mask_row = nullptr;
    for (int b = 0; ok; ++b) {
      const WidePlan& plan = plan_of(b, &ok);
      if (!ok) break;
      const int count = plan.count;
      if (count == 0) break;
      const bool mine = plan.rows > 128 * t;
      if (!mine) {
        segs += plan.last;
        plan_done(b);
        continue;
      }
      const int keys_hi = plan.hi;
      const bool valid = t * 128 + r < plan.rows;
      if (plan.first) {
        // ---- the row of Q, in two terms, and its mask
        const int row = plan.row0 + t * 128 + r, tok = valid ? token_of(sh, row) : 0;
        row_q = plan.q0 + tok;
        row_h = plan.head * sh.group + (valid ? row - tok * sh.group : 0);
        // The warp's 32 rows come together, as bf16 into the place of their two
        // terms, a half of the dims each; then kLanes lanes take a row at a time.
        // (In short loops: the code runs once a segment, and is fetched each time.)
        constexpr int kLanes = D / 16, kAtOnce = 32 / kLanes;
        const int sub = lane % kLanes, dim0 = sub * 16;
        const long long mine_at =
            valid ? (long long)row_q * a.q_row + (long long)row_h * a.q_head : -1;
        // (Raw: 32 bytes of dims dim0 .., in the term of their half.)
        uint8_t* warp_q = q_tile + (warp & 3) * 32 * D;
        uint8_t* raw0 = warp_q + (sub >= kLanes / 2 ? C::kTermBytes : 0) + (sub % (kLanes / 2)) * 32;
#pragma unroll 2
        for (int k = 0; k < kLanes; ++k) {
          const int n = k * kAtOnce + lane / kLanes;
          const long long at = __shfl_sync(0xffffffffu, mine_at, n);
          const uint16_t* from = a.q + (at >= 0 ? at + dim0 : 0);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const bool some = at >= 0 && dim0 + 8 * c < a.dim;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(
                             ptx::smem_u32(raw0 + n * D + 16 * c)),
                         "l"(some ? from + 8 * c : a.q), "r"(some ? 16 : 0)
                         : "memory");
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
#pragma unroll 2
        for (int k = 0; k < kLanes; ++k) {
          const int n = k * kAtOnce + lane / kLanes;
          const uint4 r0 = *reinterpret_cast<const uint4*>(raw0 + n * D);
          const uint4 r1 = *reinterpret_cast<const uint4*>(raw0 + n * D + 16);
          // The largest magnitude, as bits of bf16 (those past infinity's are NaN).
          const uint32_t w[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
          uint32_t top = 0;
#pragma unroll
          for (int c = 0; c < 8; ++c) top = __vmaxu2(top, w[c] & 0x7fff7fffu);
          top = max(top & 0xffffu, top >> 16);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, o));  // (the row is read)
          const float mx = __uint_as_float(min(top, 0x7f80u) << 16);
          const int e = terms_exponent(mx);
          float x[8];
          uint32_t hi[8], lo[8];
          unpack_bf16x8(r0, x);
          split_terms(x, e, hi, lo);
          unpack_bf16x8(r1, x);
          split_terms(x, e, hi + 4, lo + 4);
          // (n and the row's number in the tile agree modulo 32.)
          const int us = D == 128 ? (sub ^ (n & 7)) : (sub ^ ((n >> 1) & 3));
          uint8_t* at = warp_q + n * D + us * 16;
          *reinterpret_cast<uint4*>(at) =
              make_uint4(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, hi[4] | hi[5] << 16,
                         hi[6] | hi[7] << 16);
          *reinterpret_cast<uint4*>(at + C::kTermBytes) =
              make_uint4(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16, lo[4] | lo[5] << 16,
                         lo[6] | lo[7] << 16);
          // Its scale to the row's thread.
          const float scale = __shfl_sync(0xffffffffu, terms_scale(mx, e, a.scale_log2),
                                          (lane % kAtOnce) * kLanes);
          if (lane / kAtOnce == k) qs = scale;
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(ptx::smem_u32(&cb->q_full[t]));
        m_used = neg_inf;
        l = 0.f;
        // Keys in [0, keys_hi]: positions are 64-bit until they are cut to that.
        auto cut = [&](long long j) { return (int)(j < 0 ? 0 : j < keys_hi ? j : keys_hi); };
        const long long first = (long long)plan.len - plan.n;  // of the sequence's rows
        lo_i = 0;
        hi_i = keys_hi;
        mask_row = nullptr;
        // (A context outside 32 bits is far from every key.)
        ctx = (int)(first > -0x40000000ll ? first : -0x40000000ll);
        if (sh.tree) {
          hi_i = cut(first);
          int depth = 0;
          if (valid) {
            mask_row = a.tree_mask + (size_t)row_q * a.tree_words;
            if (sh.window >= 0) {
#pragma unroll 1
              for (int w = 0; w < a.tree_words; ++w) depth += __popc(__ldg(mask_row + w));
              depth = imax(depth - 1, 0);
            }
          }
          if (sh.window >= 0) lo_i = imin(cut(first + depth - sh.window), hi_i);
        } else {
          if (sh.causal) hi_i = cut(first + tok + 1);
          if (sh.window >= 0) lo_i = imin(cut(first + tok - sh.window), hi_i);
        }
        sink_i = imin(sh.sinks, hi_i);
      }
      const int tile0 = plan.tile0, gap_at = plan.gap_at, gap = plan.gap, ends = plan.last;
      ok = wait(cb->scale_full[b % kPagedPlans], (b / kPagedPlans) & 1);
      if (!ok) break;
#pragma unroll 1
      for (int step = 0; step < 2 * count; ++step) {
        const int half = step & 1;
        const PagePlan g = plan.page[step];
        const int k0 = (tile0 + (step >> 1) + ((step >> 1) >= gap_at ? gap : 0)) * kTileKeys +
                       half * kPageTokens;
        const uint32_t s_half = s_addr + 64 * half;
        ok = wait(cb->s_full[t][half], tiles & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        float s[kPageTokens], qmax[2];
        ptx::tmem_ld32_max(s_half, s, qmax[0]);
        ptx::tmem_ld32_max(s_half + 32, s + 32, qmax[1]);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) ptx::reg_fence16f(s + q * 16);
        ptx::reg_fence1f(qmax[0]);
        ptx::reg_fence1f(qmax[1]);
        float f = qs * g.ks;
        float top;
        if ((k0 >= lo_i || k0 + kPageTokens <= sink_i) && k0 + kPageTokens <= hi_i && g.held) {
          top = fmaxf(qmax[0], qmax[1]) * f;
        } else {
          // A word of visible keys for each 32; the scores themselves from here on.
          top = neg_inf;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int at = k0 + 32 * q;
            uint32_t seen = (low_bits(hi_i - at) & ~low_bits(lo_i - at)) | low_bits(sink_i - at);
            const int p = at - ctx;  // node of the first key
            if (mask_row && p > -32 && (p >> 5) < a.tree_words) {
              const int k = p >> 5;
              const uint32_t w0 = k >= 0 ? __ldg(mask_row + k) : 0u;
              const uint32_t w1 = k + 1 < a.tree_words ? __ldg(mask_row + k + 1) : 0u;
              seen |= __funnelshift_r(w0, w1, p & 31) & low_bits(keys_hi - at);
            }
            if (!g.held) seen = 0;
            float m4[4] = {neg_inf, neg_inf, neg_inf, neg_inf};
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float x = (seen >> c) & 1 ? s[32 * q + c] * f : neg_inf;
              s[32 * q + c] = x;
              m4[c & 3] = fmaxf(m4[c & 3], x);
            }
            top = fmaxf(top, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
          }
          f = 1.f;
        }
        const float m_tile = top + g.lv - kPagedBias;
        const bool need = m_tile > m_used + kRescaleLog2;
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = fmaxf(m_used, m_tile);
          const float root = m_used == neg_inf ? 0.f : root_ex2(m_used - m_new);
          if (!plan.first || step > 0) {
            // O_t holds the earlier pages once the last one's P V is complete.  (Its
            // barrier cannot have gone on: that takes this warp's next P.)
            ok = wait(cb->pv_done[t][half ^ 1], (half ? tiles : tiles - 1) & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            const float alpha = root * root;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o[32];
              ptx::tmem_ld16(o_addr + c0, o);
              ptx::tmem_ld16(o_addr + c0 + 16, o + 16);
              ptx::tmem_wait_ld();
              ptx::reg_fence16(o);
              ptx::reg_fence16(o + 16);
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              ptx::tmem_st32(o_addr + c0, o);
            }
          }
          if (m_new != neg_inf) {
            l = l * root * root;
            m_used = m_new;
          }
        }
        const float base = m_used == neg_inf ? 0.f : m_used;
        const uint64_t nb2 = ptx::f2_pack(-base, -base), f2 = ptx::f2_pack(f, f);
        const uint64_t v2 = ptx::f2_pack(g.vs, g.vs);
        uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t pr[kPageTokens / 2];
#pragma unroll
        for (int c = 0; c < kPageTokens; c += 2) {
          float u, v;
          ptx::f2_unpack(ptx::fma2(ptx::f2_pack(s[c], s[c + 1]), f2, nb2), u, v);
          const uint64_t p2 = ptx::f2_pack(ptx::ex2(u), ptx::ex2(v));
          ls[(c >> 1) & 3] = ptx::add2(ls[(c >> 1) & 3], p2);
          ptx::f2_unpack(ptx::mul2(p2, v2), u, v);
          pr[c >> 1] = ptx::pack_f16x2(u, v);
        }
        {
          float a0, a1, b0, b1;
          ptx::f2_unpack(ptx::add2(ls[0], ls[1]), a0, a1);
          ptx::f2_unpack(ptx::add2(ls[2], ls[3]), b0, b1);
          l += (a0 + b0) + (a1 + b1);
        }
        ptx::tmem_st32(s_half, pr);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&cb->p_full[t][half]));
        tiles += half;
      }
      if (!ok) break;
      if (!ends) {
        plan_done(b);
        continue;
      }
      // ---- the segment's output
      const int whole = plan.whole, unit_end = plan.unit_end, rows = plan.rows;
      const int q0 = plan.q0, row0 = plan.row0, head = plan.head;
      plan_done(b);
      const int slot = 2 * cta + (segs == 0 ? 0 : 1);
      ++segs;
      ok = wait(cb->o_full[t], seg & 1);
      ++seg;
      if (!ok) break;
      ptx::tc_fence_after();
      if (unit_end >= 0 && tid == 0) {
        // The unit starts here: tell the merge how many CTAs share it.
        const int parts = imin(range_of(total, ctas, unit_end - 1), ctas - 1) - cta + 1;
        a.meta[2 * cta + 1] = make_int4(rows, slot, 0, 0);
        a.meta[2 * cta] = make_int4(parts, q0, row0, head);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float l2 = l == 0.f ? neg_inf : m_used + log2f(l);
      if (valid) {
        if (!whole)
          a.part_lse[(size_t)slot * kWideRows + t * 128 + r] = l2;
        else if (a.lse)
          a.lse[(size_t)row_h * a.total_q + row_q] = l2 * 0.69314718055994531f;
      }
      // Through the rows' place in shared memory (Q's terms, read by the last S).  A
      // warp's rows are its own, as they are when it stages the next rows of Q, which
      // it may do while the others still have outputs there: so a row's bytes lie
      // where its two terms do, D in each.  (Weight 0: O_t may hold anything.)
      auto unit_at = [&](int row, int term, int v) {  // 16 bytes
        return q_tile + term * C::kTermBytes + row * D +
               (D == 128 ? (v ^ (row & 7)) : (v ^ ((row >> 1) & 3))) * 16;
      };
      auto o_of = [&](int c0, uint32_t* o) {  // 16 dims
        ptx::tmem_ld16(o_addr + c0, o);
        ptx::tmem_wait_ld();
        ptx::reg_fence16(o);
#pragma unroll
        for (int c = 0; c < 16; ++c)
          o[c] = inv == 0.f ? 0u : __float_as_uint(__uint_as_float(o[c]) * inv);
      };
      auto o_done = [&]() {
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&cb->o_free[t]));
        __syncwarp();
      };
      constexpr int kUnits = D / 16;  // of 16 bytes, in each term's place
      if (!whole) {
        // fp32, a quarter of the dims in each place: by two turns, a copy of the
        // warp's rows for each quarter, as they lie (the merge knows how).
        float* part = a.part_o + (size_t)slot * kWideRows * D + (t * 128 + (warp & 3) * 32) * (D / 4);
        const bool some = rows > t * 128 + (warp & 3) * 32;
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
#pragma unroll 1
          for (int c0 = 0; c0 < D / 2; c0 += 16) {
            uint32_t o[16];
            o_of(turn * (D / 2) + c0, o);
            const int unit = c0 / 4;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(unit_at(r, unit / kUnits, unit % kUnits + c)) =
                  make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
          ptx::fence_proxy_async_smem();
          if (turn == 0) __syncwarp();
          else o_done();
          if (lane == 0 && some) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              ptx::bulk_store(part + (size_t)(2 * turn + q) * kWideRows * (D / 4),
                              ptx::smem_u32(q_tile + q * C::kTermBytes + (warp & 3) * 32 * D), 32 * D);
            ptx::bulk_commit();
            ptx::bulk_wait_read_all();
          }
          __syncwarp();
        }
      } else {
        const uint64_t dst =
            valid ? reinterpret_cast<uint64_t>(a.out + ((size_t)row_q * a.heads + row_h) * a.dim) : 0;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t o[16];
          o_of(c0, o);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            o[c] = ptx::pack_bf16x2(__uint_as_float(o[2 * c]), __uint_as_float(o[2 * c + 1]));
          const int unit = c0 / 8;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<uint4*>(unit_at(r, unit / kUnits, unit % kUnits + c)) =
                make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
        o_done();
#pragma unroll 4
        for (int k = 0; k < 2 * kUnits; ++k) {
          // 32 units at a time, those of a row next to each other.
          const int n = (k * 32 + lane) / (2 * kUnits), u = lane % (2 * kUnits);
          const uint64_t to = __shfl_sync(0xffffffffu, dst, n);
          const uint4 v = *reinterpret_cast<const uint4*>(
              unit_at((warp & 3) * 32 + n, u / kUnits, u % kUnits));
          if (to != 0 && u < a.dim / 8) *reinterpret_cast<uint4*>(to + u * 16) = v;
        }
        __syncwarp();
      }
    }
    ptx::bulk_wait_all();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kWideIssueWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the units that CTA boundaries cut (see paged_merge_kernel):
// block (c, y) takes rows y, y + gridDim.y, ... of the unit that starts in CTA c
// and ends in a later one, a warp a row, the parts in CTA order.
constexpr int kWideMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kWideMergeThreads) paged_wide_merge_kernel(const PagedAttnArgs a) {
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::grid_dependency_wait();
  const int4 m0 = a.meta[2 * c], m1 = a.meta[2 * c + 1];
  const int parts = m0.x;
  if (parts == 0) return;
  const float neg_inf = -__int_as_float(0x7f800000);
  auto slot = [&](int p) { return p == 0 ? m1.y : 2 * (c + p); };
  constexpr int kEach = D / 32;  // dims of a lane, next to each other
  const int g = a.shape.group;
  for (int n = blockIdx.y * (kWideMergeThreads / 32) + warp; n < m1.x;
       n += gridDim.y * (kWideMergeThreads / 32)) {
    auto lse_of = [&](int p) { return a.part_lse[(size_t)slot(p) * kWideRows + n]; };
    // (A quarter of the dims of all rows, then the next one's, 16 bytes in the order
    // of the rows' places in shared memory.)
    constexpr int kUnits = D / 16;
    const int u = lane * kEach / 4, place = u % kUnits;
    const int mine = (u / kUnits * kWideRows + n) * (D / 4) + lane * kEach % 4 +
                     (D == 128 ? (place ^ (n & 7)) : (place ^ ((n >> 1) & 3))) * 4;
    float top = neg_inf;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, lse_of(p));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.f, acc[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) acc[k] = 0.f;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float lp = lse_of(p);
      const float* o = a.part_o + (size_t)slot(p) * kWideRows * D + mine;
      const float w = lp == neg_inf ? 0.f : root_ex2(lp - top);
      sum = fmaf(w, w, sum);
      float v[kEach];
      if constexpr (kEach == 4) {
        const float4 f = *reinterpret_cast<const float4*>(o);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(o);
        v[0] = f.x, v[1] = f.y;
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k) acc[k] = fmaf(w, w * v[k], acc[k]);
    }
    const int row = m0.z + n, tok = row / g, h = m0.w * g + row - tok * g;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (lane * kEach < a.dim) {
      uint16_t* out = a.out + ((size_t)(m0.y + tok) * a.heads + h) * a.dim + lane * kEach;
#pragma unroll
      for (int k = 0; k < kEach; k += 2)
        *reinterpret_cast<uint32_t*>(out + k) = ptx::pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
    }
    if (lane == 0 && a.lse)
      a.lse[(size_t)h * a.total_q + m0.y + tok] =
          sum == 0.f ? neg_inf : (top + log2f(sum)) * 0.69314718055994531f;
  }
}

}  // namespace fa
