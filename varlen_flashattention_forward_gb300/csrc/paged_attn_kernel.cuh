// paged_attn_kernel.cuh -- attention of a few query rows per sequence over the
// paged 8-bit cache, for sm_103a.
//
// Rows: the `group` query heads of one kv head times the sequence's query
// tokens (row = token * group + head), N of them (16, 32 or 64) to a tile.
// The work is every row tile's 128-key tiles; CTA c takes an equal contiguous
// range of them (paged_index.h), whatever the lengths, and walks it as
// segments, one per unit it touches.  A segment that covers its unit writes O
// and the LSE, one that covers a part writes a normalised fp32 partial and
// its LSE, and paged_merge_kernel joins the parts.
//
// The transposed form puts the keys on the tensor core's M side, where 128 of
// them fill an instruction whatever the number of rows:
//
//   St[key, row] = K[key, d] . Q[row, d]t     e4m3 x e4m3, M = 128, N = 2 rows
//   Ot[d, row]  += V[key, d]t . Pt[key, row]  f16 x f16,   M = 128 (64), K = 128
//
// K is multiplied as it lies in the cache.  Q is scaled by a power of two to
// at most 448 and held as the sum of two e4m3 numbers, hi = rn(q) and
// lo = rn(q - hi): a bf16 significand has 8 bits and the two terms hold 4
// each, so hi + lo is q exactly down to 2^-10 of the row's largest value and
// within 2^-18 of it below.  The two terms are N-side neighbours of one MMA
// (K is read once for both) and their scores are added in fp32.
//
// V goes through registers to f16 (exact), because P needs more than two
// e4m3 terms can hold: a long row has many small weights, whose sum counts.
// With f16 P is rounded to 11 bits and kept down to 2^-39 of the largest.
// The key's V scale is folded into P: x' = x + log2(vs), and the running
// maximum m is taken over x', so that P' = 2^(x' - m + 7) stays below 2^15;
// the row sum adds 2^(x - m + 7).
//
//   planner warp        walks the segments, publishes each one with its first
//                       page ids and scales in a ring that the other warps
//                       read, and splits its rows of Q into hi and lo; it
//                       runs ahead, so that short segments do not wait for
//                       its chain of dependent loads;
//   producer warp       TMA-loads the pages of each tile (128-byte swizzle;
//                       64-byte at dim 64) into a K and a V ring, with the
//                       next page ids and scales of long segments under way;
//   S issuer warp       St(i) as soon as K(i) has landed;
//   converter warps     V(i) to f16, rows nobody sees as zeros (they may hold
//                       anything, and 0 * NaN is NaN);
//   softmax             thread = key: masks, the vote on a new maximum (only
//                       when some score passes m by 2^8 is the maximum taken,
//                       O rescaled and the sums adjusted), exp2, Pt;
//   PV issuer           Ot += Vt Pt.
//
// One tile's softmax is a chain of waits (S, the vote, the P buffer) about
// as long as a tile's bytes take to arrive, so two warpgroups run it, on even
// and on odd tiles.  Each has its own running maximum, sums and Ot, and they
// are joined at the end of a segment like the parts of a split unit.
//
// TMEM: St at [0, 4N) (two buffers of 2N columns), Ot at [4N, 8N) (of two
// segments and two warpgroups).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "named_bar.cuh"
#include "paged_index.h"
#include "paged_kv_kernels.cuh"
#include "sm103_ptx.cuh"
#include "varlen_fwd_kernel.cuh"     // bounded waits, status word

namespace fa {

// Warps 0-7 softmax, 8-11 converters, 12 S issuer, 13 PV issuer, 14 producer,
// 15 planner.
constexpr int kPagedThreads = 512;
constexpr int kConvertWarp = 8, kSWarp = 12, kPvWarp = 13, kLoadWarp = 14;
// Register split (launch: 128 x 512 = 65536): softmax 256 x 160, converters
// 128 x 80, control 128 x 96 = 63488.
constexpr uint32_t kPagedSoftmaxRegs = 160;
constexpr uint32_t kPagedConvertRegs = 80;
constexpr uint32_t kPagedControlRegs = 96;
constexpr int kPagedMaxBatch = 1024;  // sequences of one launch
constexpr int kPagedInfo = 8;         // tile descriptors in flight
constexpr int kPagedPlans = 4;        // segment descriptors in flight
constexpr int kPlanReaders = 15;      // warps that read them
constexpr int kPlanTiles = 16;        // tiles whose pages are looked up at once
constexpr float kPagedBias = 7.f;     // P' is held times 2^7

struct PagedAttnArgs {
  const uint16_t* q;
  long long q_row, q_head;
  const float *k_scale, *v_scale;
  const int *cu, *seq_lens, *page_table;
  int batch, total_q, heads, dim, max_pages, num_pages;
  AttnShape shape;
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* part_o;    // [2 grid][N][D]
  float* part_lse;  // [2 grid][N], base 2
  // [grid][2] what the first CTA of a split unit leaves for the merge: (parts,
  // the sequence's first q row, first row of the tile, kv head), parts = 0:
  // nothing, and (rows, slot of the first part, -, -).
  int4* meta;
  unsigned int* status;
  uint64_t wait_limit_ns;
};

// One 128-key tile, for the softmax and the converters.
struct TileInfo {
  float ks[2], vs[2], lv[2];  // K scale, V scale and its log2, of the two pages
  int lo, hi;                 // keys of the tile that some row sees, [lo, hi)
  int held;                   // bit p: page p of the tile is in the cache
};

// One segment, for every warp; count = 0 ends the range.
struct SegPlan {
  int count, tile0;            // key tiles
  int lo, hi;                  // keys that some row sees
  int seq, head;
  int q0, row0, rows;          // the sequence's first q row; rows of the tile
  int tok0, tok1;              // tokens of its first and last row
  long long at0;               // position of tok0
  int whole;                   // covers its unit
  int unit_end;                // where the unit starts in this segment but does
                               // not end: the tile number behind it, else -1
  int id[2 * kPlanTiles];      // pages of the first tiles (-1: none)
  float ks[2 * kPlanTiles], vs[2 * kPlanTiles];
};

template <int D, int N>
struct PagedCfg {
  static constexpr int kRow = D;                       // bytes of a K or V row
  static constexpr uint32_t kSwK = D == 128 ? ptx::kLayoutSw128 : ptx::kLayoutSw64;
  static constexpr int kTileBytes = kTileKeys * kRow;  // K or V slot
  static constexpr int kPageBytes = kPageTokens * kRow;
  static constexpr int kVhBytes = kTileKeys * D * 2;
  static constexpr int kPRow = N * 2;
  static constexpr int kPBytes = kTileKeys * kPRow;
  static constexpr int kQBytes = 2 * N * kRow;
  static constexpr int NK = N == 64 ? 3 : 4;
  static constexpr int NV = N == 64 ? 2 : 3;
  static constexpr int NQ = N == 16 ? 4 : 2;
  static constexpr uint32_t kSwP = N == 64   ? ptx::kLayoutSw128
                                   : N == 32 ? ptx::kLayoutSw64
                                             : ptx::kLayoutSw32;
  static constexpr uint32_t kTmemCols = 8 * N;
  // Offsets from a 1024-byte boundary.
  static constexpr int kK = 0;
  static constexpr int kV = kK + NK * kTileBytes;
  static constexpr int kVh = kV + NV * kTileBytes;
  static constexpr int kP = kVh + 2 * kVhBytes;
  static constexpr int kQ = kP + 2 * kPBytes;
  static constexpr int kCtl = kQ + NQ * kQBytes;
};

struct alignas(16) PagedCtl {
  uint64_t plan_full[kPagedPlans], plan_free[kPagedPlans];  // segment published / read (15)
  uint64_t scale_full[kPagedPlans];                         // its scales too
  uint64_t k_full[4], k_free[4];    // K slot landed (TMA bytes) / read by its S MMA
  uint64_t v_full[4], v_free[4];    // V slot landed / converted (128 arrivals)
  uint64_t info_full[kPagedInfo];
  uint64_t vh_full[2];              // f16 V written (128)
  uint64_t s_full[2], s_free[2];    // St computed / loaded (128)
  uint64_t p_full[2], pv_done[2];   // Pt written (128) / PV complete
  uint64_t q_full[4], q_free[4];    // Q terms written (32) / last S of the segment
  uint64_t qs_full[kPagedPlans];    // row scales written (32)
  uint64_t o_free[2];               // Ot of a segment read out (8 warps)
  uint64_t drain, drain_pv;         // everything an issuer started is complete
  uint32_t tmem_base;
  volatile int abort_flag;
  TileInfo info[kPagedInfo];
  SegPlan plan[kPagedPlans];
  alignas(16) float qs[kPagedPlans][64];      // row scale * softmax scale * log2(e)
  // Per softmax warpgroup: per-warp partial maxima or sums, the running
  // maximum less the bias (0 while no key was seen), rescale factors.
  alignas(16) float red[2][4][64];
  alignas(16) float m_used[2][64];
  alignas(16) float alpha[2][64];
  // By segment (mod 4) and warpgroup: maximum so far (-inf: no key seen) and,
  // at the segment's end, the sum.  (A warpgroup may be up to three segments
  // ahead of the other, which still reads these.)
  float end_m[kPagedPlans][2][64], end_l[kPagedPlans][2][64];
  float weight[2][2][64];            // [reader][warpgroup] factors of its Ot
  long long warp_tiles[kPagedThreads / 32];
  int before[kPagedMaxBatch + 1];
};
// (16-byte loads of these.)
static_assert(offsetof(PagedCtl, qs) % 16 == 0 && offsetof(PagedCtl, m_used) % 16 == 0, "align");

template <int D, int N>
constexpr size_t paged_smem() {
  return 1024 + PagedCfg<D, N>::kCtl + sizeof(PagedCtl);
}
static_assert(sizeof(PagedCtl) < 16384, "control block");
static_assert(paged_smem<128, 64>() <= 232448, "shared memory exceeds the per-CTA limit");
static_assert(paged_smem<128, 32>() <= 232448, "shared memory exceeds the per-CTA limit");

// Maximum (kMax) or sum over the 32 lanes of a warp of each of V values (V a
// multiple of 16 up to 64), by repeated halving.  Lane l ends with value
// l / 2 of each 16 in v[g], g < V / 16 (both lanes of a pair hold it).
template <int V, bool kMax>
__device__ __forceinline__ void warp_transpose_reduce(float* v, int lane) {
#pragma unroll
  for (int g = 0; g < V / 16; ++g) {
    float* x = v + 16 * g;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int o = 16 >> s, half = 8 >> s;
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float send = upper ? x[i] : x[i + half];
        const float keep = upper ? x[i + half] : x[i];
        const float recv = __shfl_xor_sync(0xffffffffu, send, o);
        x[i] = kMax ? fmaxf(keep, recv) : keep + recv;
      }
    }
    const float recv = __shfl_xor_sync(0xffffffffu, x[0], 1);
    v[g] = kMax ? fmaxf(x[0], recv) : x[0] + recv;
  }
}

// Page `lane` of the tiles from `tile` on, `count` of which are left: its id,
// or -1 where it is not needed or not in the cache.
__device__ __forceinline__ int page_for(const PagedAttnArgs& a, const int* table, int tile,
                                        int count, int lane, int key_lo, int key_hi) {
  const int p = tile * 2 + lane;
  if (lane / 2 >= count || (long long)p * kPageTokens >= key_hi ||
      (long long)(p + 1) * kPageTokens <= key_lo)
    return -1;
  return checked_page(__ldg(table + p), a.num_pages);
}

template <int D, int N>
__global__ void __launch_bounds__(kPagedThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map, const PagedAttnArgs a) {
  using C = PagedCfg<D, N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  PagedCtl* cb = reinterpret_cast<PagedCtl*>(smem + C::kCtl);
  volatile int* abort_flag = &cb->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const AttnShape& sh = a.shape;
  auto seq_of = [&](int b, RowRange* q, int* len) {
    *q = row_range(__ldg(a.cu + b), __ldg(a.cu + b + 1), a.total_q);
    *len = __ldg(a.seq_lens + b);
  };

  ptx::grid_launch_dependents();
  if (tid == 0) {
    auto init = [&](uint64_t& b, uint32_t n) { ptx::mbar_init(ptx::smem_u32(&b), n); };
    for (int s = 0; s < 4; ++s) {
      init(cb->plan_full[s], 1);
      init(cb->plan_free[s], kPlanReaders);
      init(cb->scale_full[s], 1);
      init(cb->k_full[s], 1);
      init(cb->k_free[s], 1);
      init(cb->v_full[s], 1);
      init(cb->v_free[s], 128);
      init(cb->q_full[s], 32);
      init(cb->q_free[s], 1);
      init(cb->qs_full[s], 32);
    }
    for (int s = 0; s < kPagedInfo; ++s) init(cb->info_full[s], 1);
    for (int s = 0; s < 2; ++s) {
      init(cb->vh_full[s], 128);
      init(cb->s_full[s], 1);
      init(cb->s_free[s], 128);
      init(cb->p_full[s], 128);
      init(cb->pv_done[s], 1);
      init(cb->o_free[s], 8);
    }
    init(cb->drain, 1);
    init(cb->drain_pv, 1);
    cb->abort_flag = 0;
    ptx::fence_mbar_init();
    a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  if (warp == kSWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&cb->tmem_base), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    ptx::prefetch_tmap(&k_map);
    ptx::prefetch_tmap(&v_map);
  }
  // Tiles of the sequences before each one: a scan over the batch, the same
  // in every CTA.
  {
    long long base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPagedThreads) {
      const int b = b0 + tid;
      int n = 0;
      if (b < a.batch) {
        RowRange q;
        int len;
        seq_of(b, &q, &len);
        n = capped_tiles(sh.heads_k * head_tiles(sh, q.n, len));
      }
      long long sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (lane == 31) cb->warp_tiles[warp] = sum;
      __syncthreads();
      long long all = 0, lo = base;
#pragma unroll
      for (int w = 0; w < kPagedThreads / 32; ++w) {
        if (w < warp) lo += cb->warp_tiles[w];
        all += cb->warp_tiles[w];
      }
      if (b < a.batch) cb->before[b + 1] = capped_tiles(lo + sum);
      base += all;
      __syncthreads();
    }
    if (tid == 0) cb->before[0] = 0;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = cb->tmem_base;
  auto before = [&](int b) { return cb->before[b]; };
  const int total = cb->before[a.batch];
  const int cta = blockIdx.x, ctas = gridDim.x;
  // Slot n of a ring of size R: slot n % R, phase parity (n / R) & 1.
  auto wait = [&](uint64_t& b, int parity) {
    return wait_warp(ptx::smem_u32(&b), (uint32_t)parity, abort_flag, a.status, a.wait_limit_ns);
  };
  // The descriptor of segment number seg; every warp that reads it lets it go
  // with plan_done once it has what it needs.
  auto plan_of = [&](int seg, bool* ok) -> const SegPlan& {
    *ok = wait(cb->plan_full[seg % kPagedPlans], (seg / kPagedPlans) & 1);
    return cb->plan[seg % kPagedPlans];
  };
  auto plan_done = [&](int seg) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->plan_free[seg % kPagedPlans]));
  };

  if (warp >= kConvertWarp && warp < kSWarp) {
    ptx::regs_dec<kPagedConvertRegs>();
    // ------------------------------------------------------------ converters
    // A thread takes 16-byte units (16 codes) of a row.  Eight neighbouring
    // lanes take four units of the rows r and r ^ 5 (r even): under the
    // swizzles their eight 16-byte loads, and their eight stores of either
    // half, then lie in different banks.
    constexpr int kChunks = D / 64;          // 64-dim chunks of an f16 row
    constexpr int kIters = 128 * (D / 16) / 128;
    const int t = tid - 32 * kConvertWarp;
    const int u4 = t & 3, odd = (t >> 2) & 1, group = t >> 3;
    bool ok = true;
    int i = 0;
    for (int seg = 0; ok; ++seg) {
      const SegPlan& plan = plan_of(seg, &ok);
      if (!ok) break;
      const int count = plan.count;
      plan_done(seg);
      if (count == 0) break;
      for (int n = 0; n < count; ++n, ++i) {
        const int slot = i % C::NV, hb = i & 1;
        ok = wait(cb->v_full[slot], (i / C::NV) & 1);
        if (ok) ok = wait(cb->info_full[i % kPagedInfo], (i / kPagedInfo) & 1);
        if (!ok) break;
        const TileInfo& ti = cb->info[i % kPagedInfo];
        const int lo = ti.lo, hi = ti.hi, held = ti.held;
        const bool all = lo == 0 && hi == kTileKeys && held == 3;
        const uint8_t* src = smem + C::kV + slot * C::kTileBytes;
        uint4 c[kIters];
        auto place = [&](int k, int* r, int* chunk) {
          const int id = group + 16 * k;  // of 64 row pairs x chunks
          *chunk = id % kChunks;
          const int even = 2 * (id / kChunks);
          *r = odd ? even ^ 5 : even;
        };
#pragma unroll
        for (int k = 0; k < kIters; ++k) {
          int r, ch;
          place(k, &r, &ch);
          const int u = ch * 4 + u4;
          const int us = D == 128 ? (u ^ (r & 7)) : (u ^ ((r >> 1) & 3));
          c[k] = *reinterpret_cast<const uint4*>(src + r * C::kRow + us * 16);
          if (!all && (r < lo || r >= hi || !((held >> (r >> 6)) & 1)))
            c[k] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (i >= 2) {
          ok = wait(cb->pv_done[hb], ((i >> 1) - 1) & 1);
          if (!ok) break;
        }
        uint8_t* dst = smem + C::kVh + hb * C::kVhBytes;
#pragma unroll
        for (int k = 0; k < kIters; ++k) {
          int r, ch;
          place(k, &r, &ch);
          uint8_t* row = dst + ch * (kTileKeys * 128) + r * 128;
          const int p0 = (2 * u4) ^ (r & 7);
          *reinterpret_cast<uint4*>(row + p0 * 16) =
              make_uint4(unpack_e4m3x2(c[k].x), unpack_e4m3x2(c[k].x >> 16),
                         unpack_e4m3x2(c[k].y), unpack_e4m3x2(c[k].y >> 16));
          *reinterpret_cast<uint4*>(row + (p0 ^ 1) * 16) =
              make_uint4(unpack_e4m3x2(c[k].z), unpack_e4m3x2(c[k].z >> 16),
                         unpack_e4m3x2(c[k].w), unpack_e4m3x2(c[k].w >> 16));
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(ptx::smem_u32(&cb->vh_full[hb]));
        ptx::mbar_arrive(ptx::smem_u32(&cb->v_free[slot]));
      }
    }
  } else if (warp >= kSWarp) {
    ptx::regs_dec<kPagedControlRegs>();
    if (warp == kSWarp) {
      // ---------------------------------------------------------- S issuer
      constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, 2 * N);
      bool ok = true;
      int i = 0;
      for (int seg = 0; ok; ++seg) {
        const SegPlan& plan = plan_of(seg, &ok);
        if (!ok) break;
        const int count = plan.count;
        plan_done(seg);
        if (count == 0) break;
        const int qb = seg % C::NQ;
        ok = wait(cb->q_full[qb], (seg / C::NQ) & 1);
        if (!ok) break;
        const uint64_t qd = ptx::smem_desc(ptx::smem_u32(smem + C::kQ + qb * C::kQBytes), 16,
                                           8 * C::kRow, C::kSwK);
        for (int n = 0; n < count; ++n, ++i) {
          const int slot = i % C::NK;
          ok = wait(cb->k_full[slot], (i / C::NK) & 1);
          if (ok && i >= 2) ok = wait(cb->s_free[i & 1], ((i >> 1) - 1) & 1);
          if (!ok) break;
          // (Q was written through the generic proxy; its writers fenced.)
          ptx::tc_fence_after();
          const uint64_t kd = ptx::smem_desc(
              ptx::smem_u32(smem + C::kK + slot * C::kTileBytes), 16, 8 * C::kRow, C::kSwK);
          ptx::mma_f8_elect<D / 32>(tmem + (i & 1) * 2 * N, kd, qd, idesc);
          ptx::mma_commit_elect(ptx::smem_u32(&cb->s_full[i & 1]));
          ptx::mma_commit_elect(ptx::smem_u32(&cb->k_free[slot]));
        }
        if (!ok) break;
        ptx::mma_commit_elect(ptx::smem_u32(&cb->q_free[qb]));
      }
      ptx::mma_commit_elect(ptx::smem_u32(&cb->drain));
      wait_drain_warp(ptx::smem_u32(&cb->drain), 0, a.status);
    } else if (warp == kPvWarp) {
      // --------------------------------------------------------- PV issuer
      constexpr uint32_t idesc = ptx::idesc_f16_f32(D, N, true, true);
      bool ok = true;
      int i = 0;
      for (int seg = 0; ok; ++seg) {
        const SegPlan& plan = plan_of(seg, &ok);
        if (!ok) break;
        const int count = plan.count;
        plan_done(seg);
        if (count == 0) break;
        if (seg >= 2) ok = wait(cb->o_free[seg & 1], ((seg >> 1) - 1) & 1);
        for (int n = 0; ok && n < count; ++n, ++i) {
          const int hb = i & 1;
          ok = wait(cb->vh_full[hb], (i >> 1) & 1);
          if (ok) ok = wait(cb->p_full[hb], (i >> 1) & 1);
          if (!ok) break;
          ptx::tc_fence_after();
          // A = V[keys, d]t, MN-major in chunks of 64 dims; B = Pt, MN-major.
          const uint64_t ad = ptx::smem_desc(ptx::smem_u32(smem + C::kVh + hb * C::kVhBytes),
                                             kTileKeys * 128, 1024, ptx::kLayoutSw128);
          const uint64_t bd = ptx::smem_desc(ptx::smem_u32(smem + C::kP + hb * C::kPBytes),
                                             8 * C::kPRow, 8 * C::kPRow, C::kSwP);
          const uint32_t d = tmem + 4 * N + (seg & 1) * 2 * N + hb * N;
          ptx::mma_ss4_elect<16 * 128 / 16, 16 * C::kPRow / 16>(d, ad, bd, idesc, n > 1 ? 1u : 0u);
          ptx::mma_ss4_elect<16 * 128 / 16, 16 * C::kPRow / 16>(
              d, ptx::desc_add(ad, 64 * 128), ptx::desc_add(bd, 64 * C::kPRow), idesc, 1u);
          ptx::mma_commit_elect(ptx::smem_u32(&cb->pv_done[hb]));
        }
      }
      ptx::mma_commit_elect(ptx::smem_u32(&cb->drain_pv));
      wait_drain_warp(ptx::smem_u32(&cb->drain_pv), 0, a.status);
    } else if (warp == kLoadWarp) {
      // ---------------------------------------------------------- producer
      test_load_delay(a.wait_limit_ns);
      bool ok = true;
      int i = 0, kn = 0, vn = 0;  // tiles; K and V loads issued
      for (int seg = 0; ok; ++seg) {
        const SegPlan& plan = plan_of(seg, &ok);
        if (!ok) break;
        const int count = plan.count, tile0 = plan.tile0, key_lo = plan.lo, key_hi = plan.hi;
        const int head = plan.head;
        const int* table = a.page_table + (size_t)plan.seq * a.max_pages;
        // Lane l holds page l of kPlanTiles tiles: its id, or -1 where the
        // tile needs no such page, and its scales; next_* those of the tiles
        // after them, the ids asked for at the first tile, the scales halfway.
        int id = plan.id[lane], next_id = -1;
        float ks = 0.f, vs = 0.f, next_ks = 0.f, next_vs = 0.f;
        if (count == 0) {
          plan_done(seg);
          break;
        }
        for (int n = 0; n < count; ++n, ++i) {
          const int in = n % kPlanTiles;
          if (n > 0 && in == 0) {
            id = next_id;
            ks = next_ks;
            vs = next_vs;
          }
          if (in == 0 && n + kPlanTiles < count)
            next_id = page_for(a, table, tile0 + n + kPlanTiles, count - n - kPlanTiles, lane,
                               key_lo, key_hi);
          if (in == kPlanTiles / 2 && n + kPlanTiles / 2 < count) {
            next_ks = next_id >= 0 ? __ldg(a.k_scale + (size_t)next_id * sh.heads_k + head) : 0.f;
            next_vs = next_id >= 0 ? __ldg(a.v_scale + (size_t)next_id * sh.heads_k + head) : 0.f;
          }
          const int id0 = __shfl_sync(0xffffffffu, id, 2 * in);
          const int id1 = __shfl_sync(0xffffffffu, id, 2 * in + 1);
          const int held = (id0 >= 0 ? 1 : 0) | (id1 >= 0 ? 2 : 0);
          const uint32_t bytes = ((held & 1) + (held >> 1)) * C::kPageBytes;
          auto load = [&](const CUtensorMap* map, uint64_t& full, uint8_t* slot) {
            if (lane == 0) {
              const uint32_t bar = ptx::smem_u32(&full), dst = ptx::smem_u32(slot);
              ptx::mbar_arrive_expect_tx(bar, bytes);
              if (id0 >= 0) ptx::tma_load_3d(dst, map, bar, 0, 0, id0 * sh.heads_k + head);
              if (id1 >= 0)
                ptx::tma_load_3d(dst + C::kPageBytes, map, bar, 0, 0, id1 * sh.heads_k + head);
            }
          };
          const int sk = i % C::NK, sv = i % C::NV;
          if (i >= C::NK) ok = wait(cb->k_free[sk], (i / C::NK - 1) & 1);
          if (!ok) break;
          load(&k_map, cb->k_full[sk], smem + C::kK + sk * C::kTileBytes);
          ++kn;
          if (i >= C::NV) ok = wait(cb->v_free[sv], (i / C::NV - 1) & 1);
          if (!ok) break;
          load(&v_map, cb->v_full[sv], smem + C::kV + sv * C::kTileBytes);
          ++vn;
          if (n == 0) {
            ok = wait(cb->scale_full[seg % kPagedPlans], (seg / kPagedPlans) & 1);
            if (!ok) break;
            ks = plan.ks[lane];
            vs = plan.vs[lane];
            plan_done(seg);
          }
          TileInfo* ti = &cb->info[i % kPagedInfo];
          if ((lane >> 1) == in) {
            ti->ks[lane & 1] = ks;
            ti->vs[lane & 1] = vs;
            ti->lv[lane & 1] = fmaxf(log2f(vs), -(float)kScaleExpMax);
          }
          if (lane == 0) {
            const int key0 = (tile0 + n) * kTileKeys;
            ti->lo = imax(key_lo - key0, 0);
            ti->hi = imin(key_hi - key0, kTileKeys);
            ti->held = held;
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->info_full[i % kPagedInfo]));
        }
      }
      // Every copy this CTA started lands before it exits.
      for (int s = 0; s < C::NK && s < kn; ++s)
        wait_drain_warp(ptx::smem_u32(&cb->k_full[s]), ((kn - 1 - s) / C::NK) & 1, a.status);
      for (int s = 0; s < C::NV && s < vn; ++s)
        wait_drain_warp(ptx::smem_u32(&cb->v_full[s]), ((vn - 1 - s) / C::NV) & 1, a.status);
    } else {
      // ----------------------------------------------------------- planner
      constexpr int kLanes = D / 8;           // lanes of a Q row, 8 dims each
      constexpr int kGroups = 32 / kLanes;    // rows at once
      constexpr int kBatch = N == 16 ? N / kGroups : 4;  // loads in flight
      const int sub = lane % kLanes, dim0 = sub * 8;
      SegmentWalk walk;
      walk_begin(&walk, range_start(total, ctas, cta), range_start(total, ctas, cta + 1), a.batch,
                 before);
      Segment g = {};
      auto pages = [&]() {
        return page_for(a, a.page_table + (size_t)g.seq * a.max_pages, g.tile0, g.count, lane,
                        g.keys.lo, g.keys.hi);
      };
      bool more = walk_next(&walk, sh, before, seq_of, &g);
      int id = more ? pages() : -1;
      bool ok = true;
      for (int seg = 0;; ++seg) {
        const int slot = seg % kPagedPlans;
        if (seg >= kPagedPlans) ok = wait(cb->plan_free[slot], (seg / kPagedPlans - 1) & 1);
        if (!ok) break;
        SegPlan& plan = cb->plan[slot];
        if (!more) {
          if (lane == 0) {
            plan.count = 0;
            ptx::mbar_arrive(ptx::smem_u32(&cb->plan_full[slot]));
          }
          break;
        }
        const int head = g.head, group = sh.group, q0 = g.q.lo;
        const int row0 = g.row_tile * N, rows = imin(N, g.q.n * group - row0);
        plan.id[lane] = id;
        if (lane == 0) {
          plan.count = g.count;
          plan.tile0 = g.tile0;
          plan.lo = g.keys.lo;
          plan.hi = g.keys.hi;
          plan.seq = g.seq;
          plan.head = head;
          plan.q0 = q0;
          plan.row0 = row0;
          plan.rows = rows;
          plan.tok0 = row0 / group;
          plan.tok1 = (row0 + rows - 1) / group;
          plan.at0 = (long long)g.len - g.q.n + plan.tok0;
          plan.whole = g.count == g.unit_count;
          plan.unit_end =
              g.part_lo == 0 && g.count < g.unit_count ? walk.at - g.count + g.unit_count : -1;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->plan_full[slot]));
        // Scales and the first rows of Q under way, then the next segment's
        // pages.
        const size_t cell = (size_t)imax(id, 0) * sh.heads_k + head;
        const float ks = id >= 0 ? __ldg(a.k_scale + cell) : 0.f;
        const float vs = id >= 0 ? __ldg(a.v_scale + cell) : 0.f;
        uint4 raw[kBatch];
        auto load_rows = [&](int j0) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int n = j0 + j * kGroups + lane / kLanes;
            raw[j] = make_uint4(0u, 0u, 0u, 0u);
            if (n < rows && dim0 < a.dim) {
              const int tok = (row0 + n) / group, h = (row0 + n) - tok * group;
              raw[j] = __ldg(reinterpret_cast<const uint4*>(
                  a.q + (long long)(q0 + tok) * a.q_row + (long long)(head * group + h) * a.q_head +
                  dim0));
            }
          }
        };
        load_rows(0);
        more = walk_next(&walk, sh, before, seq_of, &g);
        id = more ? pages() : -1;
        plan.ks[lane] = ks;
        plan.vs[lane] = vs;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->scale_full[slot]));
        const int qb = seg % C::NQ;
        if (seg >= C::NQ) ok = wait(cb->q_free[qb], (seg / C::NQ - 1) & 1);
        if (!ok) break;
        uint8_t* q_s = smem + C::kQ + qb * C::kQBytes;  // N rows of hi, N of lo
        for (int j0 = 0; j0 < N; j0 += kGroups * kBatch) {
          if (j0 > 0) load_rows(j0);
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int n = j0 + j * kGroups + lane / kLanes;
            float x[8];
            unpack_bf16x8(raw[j], x);
            float mx = 0.f;
            bool finite = true;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              finite = finite && fabsf(x[k]) <= 3.402823466e38f;
              mx = fmaxf(mx, fabsf(x[k]));
            }
            // A row with an infinity or a NaN gets NaN scores.
            if (!finite) mx = __int_as_float(0x7f800000);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // mx in [2^e, 2^(e+1)) goes to [128, 256).  (Rows below 2^-100 keep
            // a smaller size; their scores are zero in fp32 all the same.)
            const int e = imax((int)(__float_as_uint(mx) >> 23) - 127, -100);
            const float f = __uint_as_float((uint32_t)(7 - e + 127) << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float y0 = x[2 * k] * f, y1 = x[2 * k + 1] * f;
              hi[k] = pack_e4m3x2(y0, y1);
              const float2 b = f16x2_floats(unpack_e4m3x2(hi[k]));
              lo[k] = pack_e4m3x2(y0 - b.x, y1 - b.y);
            }
            auto place = [&](int r) {
              const int unit = dim0 >> 4;
              const int us = D == 128 ? (unit ^ (r & 7)) : (unit ^ ((r >> 1) & 3));
              return r * C::kRow + us * 16 + (dim0 & 8);
            };
            *reinterpret_cast<uint2*>(q_s + place(n)) =
                make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(q_s + place(N + n)) =
                make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            if (sub == 0)
              cb->qs[seg % kPagedPlans][n] =
                  mx < __int_as_float(0x7f800000)
                      ? a.scale_log2 * __uint_as_float((uint32_t)(e - 7 + 127) << 23)
                      : __int_as_float(0x7fffffff);
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(ptx::smem_u32(&cb->qs_full[slot]));
        ptx::mbar_arrive(ptx::smem_u32(&cb->q_full[qb]));
      }
    }
  } else {
    ptx::regs_inc<kPagedSoftmaxRegs>();
    // -------------------------------------------------------------- softmax
    const float neg_inf = -__int_as_float(0x7f800000);
    const int wg = warp >> 2;             // tiles i with i % 2 == wg
    const int key = tid & 127;            // of the tile
    const int page = key >> 6;
    const int bar = 1 + 4 * wg;           // named barriers bar .. bar + 2; 4: both warpgroups
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lane_base + wg * 2 * N;
    float (*red)[64] = cb->red[wg];
    float* m_used = cb->m_used[wg];
    float* alpha = cb->alpha[wg];
    uint8_t* prow = smem + C::kP + wg * C::kPBytes + key * C::kPRow;
    float l[N];
    bool ok = true;
    int i = 0;          // tiles before the segment
    for (int seg = 0; ok; ++seg) {
      const SegPlan& plan = plan_of(seg, &ok);
      const int count = plan.count, tile0 = plan.tile0, q0 = plan.q0, head = plan.head;
      const int row0 = plan.row0, rows = plan.rows, tok0 = plan.tok0, tok1 = plan.tok1;
      const int whole = plan.whole, unit_end = plan.unit_end;
      const long long at0 = plan.at0;
      // (A warpgroup goes through a segment as one.)
      ok = named_bar_and(bar + 1, 128, ok);
      if (!ok) break;
      if (count == 0) break;
      const uint32_t o_tmem = tmem + lane_base + 4 * N + (seg & 1) * 2 * N + wg * N;
      const int first = (i & 1) == wg ? 0 : 1;  // this warpgroup's first tile of the segment
      const int last = i + count - 1;           // of the segment's tiles
      // A segment of one tile is its warpgroup's alone; the other one goes on
      // to the next.
      const bool alone = count == 1;
      if (alone && first != 0) {
        plan_done(seg);
        ++i;
        continue;
      }
#pragma unroll
      for (int n = 0; n < N; ++n) l[n] = 0.f;
      // Rows that have seen no key yet have no maximum; while there are any
      // (`unset`), every tile takes the slow path below.
      bool unset = true;
      const float* c = cb->qs[seg % kPagedPlans];
      float* end_m = cb->end_m[seg % kPagedPlans][wg];
      for (int t = first; t < count; t += 2) {
        const int at = i + t;  // tile of the CTA's range
        const uint32_t phase = (uint32_t)(at >> 1) & 1;
        // (A warp whose wait has given up still joins the vote below, after
        // which the whole warpgroup leaves.)
        if (t == first) ok = wait(cb->qs_full[seg % kPagedPlans], (seg / kPagedPlans) & 1);
        if (ok) ok = wait(cb->info_full[at % kPagedInfo], (at / kPagedInfo) & 1);
        const TileInfo& ti = cb->info[at % kPagedInfo];
        const float ks = ti.ks[page], vs = ti.vs[page], lv = ti.lv[page];
        const bool seen = key >= ti.lo && key < ti.hi && ((ti.held >> page) & 1);
        if (ok) ok = wait(cb->s_full[wg], phase);
        ptx::tc_fence_after();
        float x[N];
#pragma unroll
        for (int n0 = 0; n0 < N; n0 += 16) {
          uint32_t hi[16], lo[16];
          ptx::tmem_ld16(s_tmem + n0, hi);
          ptx::tmem_ld16(s_tmem + N + n0, lo);
          ptx::tmem_wait_ld();
          ptx::reg_fence16(hi);
          ptx::reg_fence16(lo);
#pragma unroll
          for (int n = 0; n < 16; n += 4) {
            const float4 f = *reinterpret_cast<const float4*>(c + n0 + n);
            x[n0 + n] = (__uint_as_float(hi[n]) + __uint_as_float(lo[n])) * (f.x * ks);
            x[n0 + n + 1] = (__uint_as_float(hi[n + 1]) + __uint_as_float(lo[n + 1])) * (f.y * ks);
            x[n0 + n + 2] = (__uint_as_float(hi[n + 2]) + __uint_as_float(lo[n + 2])) * (f.z * ks);
            x[n0 + n + 3] = (__uint_as_float(hi[n + 3]) + __uint_as_float(lo[n + 3])) * (f.w * ks);
          }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&cb->s_free[wg]));
        if (!seen) {
#pragma unroll
          for (int n = 0; n < N; ++n) x[n] = neg_inf;
        }
        // Rows of several tokens see different keys: mask the tiles at the
        // edges row by row.
        if (tok0 != tok1) {
          const long long j0 = (long long)(tile0 + t) * kTileKeys, j = j0 + key;
          const bool edge = (sh.causal && j0 > at0 - (kTileKeys - 1)) ||
                            (sh.window >= 0 && j0 < at0 + (tok1 - tok0) - sh.window);
          if (edge) {
            for (int tok = tok0; tok <= tok1; ++tok) {
              const long long pos = at0 + (tok - tok0);
              const bool out = (sh.causal && j > pos) || (sh.window >= 0 && j < pos - sh.window);
              if (out) {
                const int lo = tok * sh.group - row0;
#pragma unroll
                for (int n = 0; n < N; ++n)
                  if (n >= lo && n < lo + sh.group) x[n] = neg_inf;
              }
            }
          }
        }
        // Pt's buffer was last read by the PV of this warpgroup's last tile.
        if (ok && at >= 2) ok = wait(cb->pv_done[wg], phase ^ 1);
        // A new maximum is due where a score passes the old one by 2^8.
        float over = neg_inf;
        if (!unset) {
#pragma unroll
          for (int n = 0; n < N; n += 4) {
            const float4 m = *reinterpret_cast<const float4*>(m_used + n);
            over = ptx::max3(over, x[n] - m.x, x[n + 1] - m.y);
            over = ptx::max3(over, x[n + 2] - m.z, x[n + 3] - m.w);
          }
        }
        const int need = unset || !ok || over + lv > kRescaleLog2 + kPagedBias;
        if (named_bar_or(bar, 128, need)) {
          ok = named_bar_and(bar + 1, 128, ok);
          if (!ok) break;
          float v[N];
#pragma unroll
          for (int n = 0; n < N; ++n) v[n] = x[n] + lv;
          warp_transpose_reduce<N, true>(v, lane);
          if ((lane & 1) == 0) {
#pragma unroll
            for (int k = 0; k < N / 16; ++k) red[warp & 3][16 * k + (lane >> 1)] = v[k];
          }
          named_bar_sync(bar + 2, 128);
          int none = 0;
          if (key < N) {
            const float mt = fmaxf(fmaxf(red[0][key], red[1][key]),
                                   fmaxf(red[2][key], red[3][key])) - kPagedBias;
            const bool had = t != first && end_m[key] != neg_inf;
            const float mu = had ? m_used[key] : neg_inf;
            float al = 1.f;
            if (mt > mu) {
              al = had ? ptx::ex2(mu - mt) : 0.f;
              m_used[key] = mt;
              end_m[key] = mt;
            } else if (!had) {
              m_used[key] = 0.f;
              end_m[key] = neg_inf;
            }
            none = key < rows && end_m[key] == neg_inf;
            alpha[key] = al;
          }
          unset = named_bar_or(bar, 128, none);
#pragma unroll
          for (int n = 0; n < N; ++n) l[n] *= alpha[n];
          if (t != first) {
            // Ot holds this warpgroup's earlier tiles, whose last PV is done.
            ptx::tc_fence_after();
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += 16) {
              uint32_t o[16];
              ptx::tmem_ld16(o_tmem + n0, o);
              ptx::tmem_wait_ld();
              ptx::reg_fence16(o);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha[n0 + k]);
              ptx::tmem_st16(o_tmem + n0, o);
            }
            ptx::tmem_wait_st();
          }
        }
        // Pt row of this key.
#pragma unroll
        for (int n0 = 0; n0 < N; n0 += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 m = *reinterpret_cast<const float2*>(m_used + n0 + 2 * k);
            const float p0 = ptx::ex2(x[n0 + 2 * k] - m.x);
            const float p1 = ptx::ex2(x[n0 + 2 * k + 1] - m.y);
            l[n0 + 2 * k] += p0;
            l[n0 + 2 * k + 1] += p1;
            w[k] = ptx::pack_f16x2(p0 * vs, p1 * vs);
          }
          const int un = n0 / 8;
          const int us = N == 64 ? (un ^ (key & 7))
                                 : N == 32 ? (un ^ ((key >> 1) & 3)) : (un ^ ((key >> 2) & 1));
          *reinterpret_cast<uint4*>(prow + us * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&cb->p_full[wg]));
      }

      // ------------------------------------------------------ segment output
      // (A warpgroup that has given up joins the first barrier.)
      i += count;
      const int slot = 2 * cta + (seg == 0 ? 0 : 1);
      if (ok) {
        warp_transpose_reduce<N, false>(l, lane);
        if ((lane & 1) == 0) {
#pragma unroll
          for (int k = 0; k < N / 16; ++k) red[warp & 3][16 * k + (lane >> 1)] = l[k];
        }
        for (int k = 0; ok && k < 2 && k < count; ++k)
          ok = wait(cb->pv_done[(last - k) & 1], ((last - k) >> 1) & 1);
        named_bar_sync(bar + 2, 128);
        if (key < N)
          cb->end_l[seg % kPagedPlans][wg][key] =
              (red[0][key] + red[1][key]) + (red[2][key] + red[3][key]);
      }
      ok = alone ? named_bar_and(bar + 1, 128, ok) : named_bar_and(4, 256, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      if (key < N) {
        // Weights of the two warpgroups' Ot: 2^(m - M) / sum; a warpgroup
        // that saw no key has m = -inf (or a NaN sum) and nothing to add.
        const float m0 = alone ? end_m[key] : cb->end_m[seg % kPagedPlans][0][key];
        const float m1 = alone ? neg_inf : cb->end_m[seg % kPagedPlans][1][key];
        const float l0 = alone ? cb->end_l[seg % kPagedPlans][wg][key] : cb->end_l[seg % kPagedPlans][0][key];
        const float l1 = alone ? 0.f : cb->end_l[seg % kPagedPlans][1][key];
        const float top = fmaxf(m0, m1);
        const float base = top == neg_inf ? 0.f : top;
        const float e0 = m0 == neg_inf ? (l0 == 0.f ? 0.f : l0) : ptx::ex2(m0 - base);
        const float e1 = m1 == neg_inf ? (l1 == 0.f ? 0.f : l1) : ptx::ex2(m1 - base);
        const float sum = e0 * l0 + e1 * l1;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (a NaN stays one)
        cb->weight[wg][0][key] = e0 * inv;
        cb->weight[wg][1][key] = e1 * inv;
        const float l2 = sum == 0.f ? neg_inf : base + log2f(sum);
        if ((alone || wg == 0) && key < rows) {
          if (!whole) {
            a.part_lse[(size_t)slot * N + key] = l2;
          } else if (a.lse) {
            const int tok = (row0 + key) / sh.group, h = (row0 + key) - tok * sh.group;
            a.lse[(size_t)(head * sh.group + h) * a.total_q + q0 + tok] =
                l2 * 0.69314718055994531f;
          }
        }
      }
      if (unit_end >= 0 && key == 0 && (alone || wg == 0)) {
        // The unit starts here: tell the merge how many CTAs share it.
        int parts = 1;
        while (cta + parts < ctas && range_start(total, ctas, cta + parts) < unit_end) ++parts;
        a.meta[2 * cta + 1] = make_int4(rows, slot, 0, 0);
        a.meta[2 * cta] = make_int4(parts, q0, row0, head);
      }
      named_bar_sync(bar + 2, 128);
      // Dim of this thread's lane: row of a 128-row accumulator, or of a
      // 64-row one, which uses the first 16 lanes of each warp's 32.
      const int d = D == 128 ? key : (warp & 3) * 16 + lane;
      const bool live = d < a.dim && (D == 128 || lane < 16);
      const uint32_t o0 = tmem + lane_base + 4 * N + (seg & 1) * 2 * N;
      // Rows: eight at a time by each warpgroup in turn, or all by the one
      // that is alone, whose Ot is then the only one.
#pragma unroll 1
      for (int n0 = alone ? 0 : 8 * wg; n0 < rows; n0 += alone ? 8 : 16) {
        uint32_t oa[8], ob[8];
        ptx::tmem_ld8(o0 + (alone ? wg * N : 0) + n0, oa);
        ptx::tmem_ld8(o0 + (alone ? wg * N : N) + n0, ob);
        ptx::tmem_wait_ld();
        ptx::reg_fence8(oa);
        ptx::reg_fence8(ob);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int n = n0 + k;
          if (live && n < rows) {
            // (Weight 0: the Ot may hold anything.)
            const float wa = cb->weight[wg][0][n], wb = cb->weight[wg][1][n];
            const float v = (wa == 0.f ? 0.f : wa * __uint_as_float(oa[k])) +
                            (wb == 0.f ? 0.f : wb * __uint_as_float(ob[k]));
            if (whole) {
              const int tok = (row0 + n) / sh.group, h = (row0 + n) - tok * sh.group;
              a.out[((size_t)(q0 + tok) * a.heads + head * sh.group + h) * a.dim + d] =
                  (uint16_t)ptx::pack_bf16x2(v, 0.f);
            } else {
              a.part_o[((size_t)slot * N + n) * D + d] = v;
            }
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        const uint32_t bar_o = ptx::smem_u32(&cb->o_free[seg & 1]);
        ptx::mbar_arrive(bar_o);
        if (alone) ptx::mbar_arrive(bar_o);  // for the other warpgroup
      }
      // Only now: the planner writes over this segment's row scales, and the
      // other warpgroup over its maxima, four segments on at the earliest.
      plan_done(seg);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kSWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the parts of the units that CTA boundaries cut.  Block (c, n): row n
// of the unit that starts in CTA c and ends in a later one.
// O = sum_p w_p O_p, w_p = 2^(lse_p - LSE): the parts are summed in CTA order,
// so the result does not depend on timing.  A unit can have as many parts as
// there are CTAs, so every LSE is loaded at once and eight partials at a time.
constexpr int kPagedMaxGrid = 512;  // CTAs of an attention launch

template <int D, int N>
__global__ void __launch_bounds__(D) paged_merge_kernel(const PagedAttnArgs a) {
  __shared__ float s_w[kPagedMaxGrid];
  __shared__ float s_red[D / 32];
  const int c = blockIdx.x, n = blockIdx.y, tid = threadIdx.x;
  ptx::grid_dependency_wait();
  const int4 m0 = a.meta[2 * c], m1 = a.meta[2 * c + 1];
  const int parts = m0.x;
  if (parts == 0 || n >= m1.x) return;
  auto slot = [&](int p) { return p == 0 ? m1.y : 2 * (c + p); };
  const float neg_inf = -__int_as_float(0x7f800000);
  float top = neg_inf;
  for (int p = tid; p < parts; p += D) {
    const float v = a.part_lse[(size_t)slot(p) * N + n];
    s_w[p] = v;
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) s_red[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < D / 32; ++w) top = fmaxf(top, s_red[w]);
  float sum = 0.f, acc = 0.f;
  for (int p0 = 0; p0 < parts; p0 += 8) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = p0 + k < parts ? a.part_o[((size_t)slot(p0 + k) * N + n) * D + tid] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (p0 + k < parts) {
        const float lp = s_w[p0 + k];
        const float w = lp == neg_inf ? 0.f : ptx::ex2(lp - top);
        sum += w;
        acc = fmaf(w, v[k], acc);
      }
    }
  }
  const int row = m0.z + n, g = a.shape.group;
  const int tok = row / g, h = m0.w * g + row - tok * g;
  if (tid < a.dim)
    a.out[((size_t)(m0.y + tok) * a.heads + h) * a.dim + tid] =
        (uint16_t)ptx::pack_bf16x2(sum == 0.f ? 0.f : acc / sum, 0.f);
  if (tid == 0 && a.lse)
    a.lse[(size_t)h * a.total_q + m0.y + tok] =
        sum == 0.f ? neg_inf : (top + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace fa
