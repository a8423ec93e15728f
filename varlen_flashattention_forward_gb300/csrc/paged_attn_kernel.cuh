// paged_attn_kernel.cuh -- attention of a few query rows per sequence over the
// paged 8-bit cache, for sm_103a.
//
// Rows: the `group` query heads of one kv head times the sequence's query
// tokens (row = token * group + head), N of them (16 or 32) to a tile.
// The work is every row tile's 128-key tiles; CTA c takes an equal contiguous
// range of their costs (paged_index.h), whatever the lengths, and walks it as
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
// K is multiplied as it lies in the cache.  Each row of Q is scaled by a power of
// two, its largest value into [128, 256), and held as the sum of two e4m3
// numbers, hi = rn(q) and lo = rn(q - hi): a bf16 significand has 8 bits and the
// two terms hold 4 each, so hi + lo is q exactly down to 2^-9 of the row's
// largest value and within 2^-17 of that below (e4m3's step ends at 2^-9).  The two terms are N-side neighbours of one MMA
// (K is read once for both) and their scores are added in fp32.
//
// V goes through registers to f16 (exact), because P needs more than two
// e4m3 terms can hold: a long row has many small weights, whose sum counts.
// The key's V scale is folded into P: x' = x + log2(vs), and the running
// maximum m is taken over x', so that P' = 2^(x' - m + 7) stays below 2^15;
// the row sum adds 2^(x - m + 7).  As f16, P' has 11 bits down to 2^-14, that is
// 2^-21 of the maximum, and steps of 2^-24, 2^-31 of it, below.
//
//   planner warp        walks the segments and publishes them in a ring, a
//                       batch of up to 16 tiles at a time with the places and
//                       scales of its pages; splits each segment's rows of Q
//                       into hi and lo.  It runs ahead, so that nobody else
//                       waits for its chains of dependent loads;
//   producer warp       TMA-loads the pages of each tile (128-byte swizzle;
//                       64-byte at dim 64) into a K and a V ring;
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
// TMEM: St in four buffers of 2N columns, Ot behind them (of two segments and
// two warpgroups).
//
// Bound by HBM where sequences are long: 32 of 32768 keys, 32 query and 8 kv
// heads of 128 dims, take 319 us, 6.4 TB/s.  What a unit costs besides its
// bytes (rows of Q, first maximum, output: some 3-4 us of a CTA, part of it
// under the next unit's first tiles) shows in shorter ones: 64 of 100 to 8192
// keys, 32 and 4 heads, 63 us, 4.3 TB/s.  With 32 rows a tile the softmax's own
// latency does: 24 sequences with 2 to 7 rows against windows of 4096 keys, 32
// and 8 heads of 64 dims, 49 us, 1.7 TB/s.  A single sequence of 8192 keys, 32
// and 8 heads of 128 dims, takes 17 us: about 8 until the first tile's score,
// most of them the planner's chain of loads and the first fetch of the kernel's
// instructions, and 4 for the merge.
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
// Register split (launch: 128 x 512 = 65536): softmax 256 x 168, converters
// 128 x 80, control 128 x 96 = 65536.  (Softmax 176 and control 80: 62.4
// instead of 62.9 us at 64 sequences, but 51.0 instead of 48.8 at 32 rows;
// softmax 176 and converters 64: 335 instead of 316 us at 32 x 32768 keys.)
constexpr uint32_t kPagedSoftmaxRegs = 168;
constexpr uint32_t kPagedConvertRegs = 80;
constexpr uint32_t kPagedControlRegs = 96;
// Sequences of one launch (their costs are held in shared memory).
constexpr int kPagedMaxBatch = 1024;
constexpr int kPagedPlans = 4;        // batches in flight
constexpr int kPlanReaders = 15;      // warps that read them
constexpr int kPlanTiles = 16;        // tiles of a batch
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

// A page of a batch: its (page, head) cell of the cache, -1 where there is
// none, and its scales.
struct PagePlan {
  float ks, vs, lv;  // K scale, V scale and its log2
  int held;          // 1: in the cache
};

// Up to kPlanTiles tiles of one segment, for every warp; count = 0 ends the
// range.
template <int N>
struct alignas(16) BatchPlan {
  PagePlan page[2 * kPlanTiles];
  int cell[2 * kPlanTiles];
  int count, tile0;            // key tiles of the batch
  int first, last;             // it begins, ends the segment
  int lo, hi;                  // keys that some row of the segment sees
  int head, q0, row0, rows;    // first q row of the sequence; rows of the tile
  int out[N], lse[N];          // of each row: its place in O (rows) and in the LSE
  int tok0, tok1;              // tokens of its first and last row
  alignas(16) int token[N];    // of each row, from tok0
  long long at0;               // position of tok0
  int tiles;                   // of the segment
  int whole;                   // the segment covers its unit
  int unit_end;                // where the unit starts in this segment but does
                               // not end: the cost up to its end, else -1
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
  // K and V slots: at 128 dims what fits, at 64 dims (8 KB slots) as many as
  // gain anything (24 sequences with 2 to 7 rows, windows of 4096: 4 and 3
  // slots 51.2 us, 6 of each 49.8, 8 the same).
  static constexpr int NK = D == 64 ? 6 : 4;
  static constexpr int NV = D == 64 ? 6 : 3;
  // St buffers, as many as TMEM holds at 32 rows; with two the same case takes
  // 49.0 us, with four 48.6 (by then).
  static constexpr int NS = 4;
  static constexpr int NQ = N == 16 ? 4 : 2;
  static constexpr uint32_t kSwP = N == 32 ? ptx::kLayoutSw64 : ptx::kLayoutSw32;
  static constexpr uint32_t kOt = 2 * N * NS;          // TMEM column of Ot
  static constexpr uint32_t kTmemCols = N == 16 ? 256 : 512;
  static_assert(kOt + 4 * N <= kTmemCols, "tensor memory");
  // Offsets from a 1024-byte boundary.
  static constexpr int kK = 0;
  static constexpr int kV = kK + NK * kTileBytes;
  static constexpr int kVh = kV + NV * kTileBytes;
  static constexpr int kP = kVh + 2 * kVhBytes;
  static constexpr int kQ = kP + 2 * kPBytes;
  static constexpr int kCtl = kQ + NQ * kQBytes;
};

template <int N>
struct alignas(16) PagedCtl {
  uint64_t plan_full[kPagedPlans], plan_free[kPagedPlans];  // batch published / read (15)
  uint64_t scale_full[kPagedPlans];                         // its scales too
  uint64_t k_full[6], k_free[6];    // K slot landed (TMA bytes) / read by its S MMA
  uint64_t v_full[6], v_free[6];    // V slot landed / converted (128 arrivals)
  uint64_t vh_full[2];              // f16 V written (128)
  uint64_t s_full[4], s_free[4];    // St computed / loaded (128)
  uint64_t p_full[2], pv_done[2];   // Pt written (128) / PV complete
  uint64_t q_full[4], q_free[4];    // Q terms written (32) / last S of the segment
  uint64_t qs_full[kPagedPlans];    // row scales written (32)
  uint64_t o_free[2];               // Ot of a segment read out (8 warps)
  uint64_t drain, drain_pv;         // everything an issuer started is complete
  uint32_t tmem_base;
  volatile int abort_flag;
  BatchPlan<N> plan[kPagedPlans];
  alignas(16) float qs[kPagedPlans][N];      // row scale * softmax scale * log2(e)
  // Per softmax warpgroup: of each two rows, the scales and minus the running
  // maxima (less the bias; 0 while no key was seen); per-warp partial maxima
  // or sums; rescale factors.
  alignas(16) float factor[2][N / 2][4];
  alignas(16) float red[2][4][N];
  alignas(16) float alpha[2][2 * N];  // of Ot; of the sums, see root_ex2
  // By segment (mod 4) and warpgroup: maximum so far (-inf: no key seen) and,
  // at the segment's end, the sum.  (A warpgroup may be up to three segments
  // ahead of the other, which still reads these.)
  float end_m[kPagedPlans][2][N], end_l[kPagedPlans][2][N];
  long long warp_tiles[kPagedThreads / 32];
  int before[kPagedMaxBatch + 1];
};
template <int D, int N>
constexpr size_t paged_smem() {
  return 1024 + PagedCfg<D, N>::kCtl + sizeof(PagedCtl<N>);
}
static_assert(paged_smem<128, 32>() <= 232448, "shared memory exceeds the per-CTA limit");

// Bounded wait of a warp (see wait_warp), in as few instructions as will do:
// the clock starts at the 256th probe.  (A launch reads the kernel's
// instructions from L2 or DRAM beside the cache's bytes, and there are many
// waits in it.)
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           unsigned int* status, uint64_t limit_ns) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t spin = 1;
       __builtin_expect(!__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)), 0); ++spin) {
    if ((spin & 255u) != 0 && limit_ns >= kShortWaitNs) continue;
    int give_up = 0;
    if ((threadIdx.x & 31) == 0) {
      const uint64_t now = ptx::globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) {
        atomicOr(status, kStatusTimeout);
        *abort_flag = 1;
      }
      give_up = *abort_flag;
    }
    if (__shfl_sync(0xffffffffu, give_up, 0)) return false;
  }
  return true;
}

// Maximum (kMax) or sum over the 32 lanes of a warp of each of 16 values, by
// repeated halving: lanes 2k and 2k + 1 return that of value k.
template <bool kMax>
__device__ __forceinline__ float warp_transpose_reduce16(float* x, int lane) {
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
  return kMax ? fmaxf(x[0], recv) : x[0] + recv;
}

// The square root of 2^d (d <= 0), to be multiplied by twice: 2^d itself is
// flushed to zero below 2^-126, and a row sum needs more.  The maximum is one of
// score + log2(V scale), so under V scales 2^128 apart a sum is up to 2^96 (2^79
// for each key) where another one that it joins is down to 2^-57.
__device__ __forceinline__ float root_ex2(float d) { return ptx::ex2(0.5f * d); }

template <int D, int N>
__global__ void __launch_bounds__(kPagedThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map, const PagedAttnArgs a) {
  using C = PagedCfg<D, N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  PagedCtl<N>* cb = reinterpret_cast<PagedCtl<N>*>(smem + C::kCtl);
  volatile int* abort_flag = &cb->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const AttnShape& sh = a.shape;
  auto seq_of = [&](int b, RowRange* q, int* len) {
    *q = row_range(__ldg(a.cu + b), __ldg(a.cu + b + 1), a.total_q);
    *len = __ldg(a.seq_lens + b);
  };

  ptx::grid_launch_dependents();
  if (warp == kLoadWarp && lane == 0) {
    auto init = [&](uint64_t& b, uint32_t n) { ptx::mbar_init(ptx::smem_u32(&b), n); };
#pragma unroll 1
    for (int s = 0; s < 4; ++s) {
      init(cb->plan_full[s], 1);
      init(cb->plan_free[s], kPlanReaders);
      init(cb->scale_full[s], 1);
      init(cb->s_full[s], 1);
      init(cb->s_free[s], 128);
      init(cb->q_full[s], 32);
      init(cb->q_free[s], 1);
      init(cb->qs_full[s], 32);
    }
#pragma unroll 1
    for (int s = 0; s < 6; ++s) {
      init(cb->k_full[s], 1);
      init(cb->k_free[s], 1);
      init(cb->v_full[s], 1);
      init(cb->v_free[s], 128);
    }
    for (int s = 0; s < 2; ++s) {
      init(cb->vh_full[s], 128);
      init(cb->p_full[s], 128);
      init(cb->pv_done[s], 1);
      init(cb->o_free[s], 8);
    }
    init(cb->drain, 1);
    init(cb->drain_pv, 1);
    cb->abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&k_map);
    ptx::prefetch_tmap(&v_map);
  }
  if (warp == kSWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&cb->tmem_base), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  // Cost of the sequences before each one: a scan over the batch by the
  // softmax warps, the same in every CTA.
  if (warp < 8) {
    if (tid == 0) {
      cb->before[0] = 0;
      a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    long long base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.batch; b0 += 256) {
      const int b = b0 + tid;
      int n = 0;
      if (b < a.batch) {
        RowRange q;
        int len;
        seq_of(b, &q, &len);
        n = capped_cost(sh.heads_k * head_cost(sh, q.n, len));
      }
      long long sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (lane == 31) cb->warp_tiles[warp] = sum;
      named_bar_sync(1, 256);
      long long all = 0, lo = base;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w < warp) lo += cb->warp_tiles[w];
        all += cb->warp_tiles[w];
      }
      if (b < a.batch) cb->before[b + 1] = capped_cost(lo + sum);
      base += all;
      named_bar_sync(1, 256);
    }
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
    return paged_wait(ptx::smem_u32(&b), (uint32_t)parity, abort_flag, a.status, a.wait_limit_ns);
  };
  // Batch number b of the range; every warp that reads it lets it go with
  // plan_done once it has what it needs.
  auto plan_of = [&](int b, bool* ok) -> const BatchPlan<N>& {
    *ok = wait(cb->plan_full[b % kPagedPlans], (b / kPagedPlans) & 1);
    return cb->plan[b % kPagedPlans];
  };
  auto plan_done = [&](int b) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->plan_free[b % kPagedPlans]));
  };

  if (warp >= kConvertWarp && warp < kSWarp) {
    ptx::regs_dec<kPagedConvertRegs>();
    // ------------------------------------------------------------ converters
    // A thread takes 16-byte units (16 codes) of a row.  Eight neighbouring
    // lanes take four units of the rows r and r ^ 5 (r even): under the
    // swizzles their eight 16-byte loads, and their eight stores of either
    // half, then lie in different banks.  Its rows are a multiple of 8 apart,
    // so that the swizzle is the same for all of them.
    constexpr int kChunks = D / 64;          // 64-dim chunks of an f16 row
    constexpr int kIters = D / 16;           // units of a thread
    constexpr int kStep = 32 / kChunks;      // its rows' distance
    const int t = tid - 32 * kConvertWarp;
    const int u4 = t & 3, pair = t >> 3, chunk = pair % kChunks;
    const int even = 2 * (pair / kChunks), r0 = (t & 4) ? even ^ 5 : even;
    const int u = chunk * 4 + u4;
    const int us = D == 128 ? (u ^ (r0 & 7)) : (u ^ ((r0 >> 1) & 3));
    const uint8_t* src0 = smem + C::kV + r0 * C::kRow + us * 16;
    const int p0 = (2 * u4) ^ (r0 & 7);
    uint8_t* dst0 = smem + C::kVh + chunk * (kTileKeys * 128) + r0 * 128 + p0 * 16;
    uint8_t* dst1 = smem + C::kVh + chunk * (kTileKeys * 128) + r0 * 128 + (p0 ^ 1) * 16;
    bool ok = true;
    int i = 0, slot = 0;
    uint32_t v_phase = 0;
    for (int b = 0; ok; ++b) {
      const BatchPlan<N>& plan = plan_of(b, &ok);
      if (!ok) break;
      const int count = plan.count, tile0 = plan.tile0, key_lo = plan.lo, key_hi = plan.hi;
      if (count == 0) break;
      // (held is written with the scales)
      ok = wait(cb->scale_full[b % kPagedPlans], (b / kPagedPlans) & 1);
      if (!ok) break;
      const unsigned held = __ballot_sync(0xffffffffu, plan.page[lane].held != 0);
      plan_done(b);
#pragma unroll 1
      for (int n = 0; n < count; ++n, ++i) {
        const int hb = i & 1;
        ok = wait(cb->v_full[slot], v_phase);
        if (!ok) break;
        const uint8_t* src = src0 + slot * C::kTileBytes;
        uint4 c[kIters];
#pragma unroll
        for (int k = 0; k < kIters; ++k)
          c[k] = *reinterpret_cast<const uint4*>(src + k * kStep * C::kRow);
        const int key0 = (tile0 + n) * kTileKeys;
        const int lo = key_lo - key0, hi = key_hi - key0;
        const unsigned pages = (held >> (2 * n)) & 3;
        if (__builtin_expect(lo > 0 || hi < kTileKeys || pages != 3, 0)) {
#pragma unroll
          for (int k = 0; k < kIters; ++k) {
            const int r = r0 + k * kStep;
            if (r < lo || r >= hi || !((pages >> (r >> 6)) & 1)) c[k] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        if (i >= 2) {
          ok = wait(cb->pv_done[hb], ((i >> 1) - 1) & 1);
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
        if (++slot == C::NV) {
          slot = 0;
          v_phase ^= 1;
        }
      }
    }
  } else if (warp >= kSWarp) {
    ptx::regs_dec<kPagedControlRegs>();
    if (warp == kSWarp) {
      // ---------------------------------------------------------- S issuer
      constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, 2 * N);
      bool ok = true;
      int i = 0, seg = 0, slot = 0;
      uint32_t k_phase = 0;
      uint64_t qd = 0;
      for (int b = 0; ok; ++b) {
        const BatchPlan<N>& plan = plan_of(b, &ok);
        if (!ok) break;
        const int count = plan.count, first = plan.first, last = plan.last;
        plan_done(b);
        if (count == 0) break;
        const int qb = seg % C::NQ;
        if (first) {
          ok = wait(cb->q_full[qb], (seg / C::NQ) & 1);
          if (!ok) break;
          qd = ptx::smem_desc(ptx::smem_u32(smem + C::kQ + qb * C::kQBytes), 16, 8 * C::kRow,
                              C::kSwK);
        }
#pragma unroll 1
        for (int n = 0; n < count; ++n, ++i) {
          ok = wait(cb->k_full[slot], k_phase);
          const int sb = i % C::NS;
          if (ok && i >= C::NS) ok = wait(cb->s_free[sb], (i / C::NS - 1) & 1);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t kd = ptx::smem_desc(
              ptx::smem_u32(smem + C::kK + slot * C::kTileBytes), 16, 8 * C::kRow, C::kSwK);
          ptx::mma_f8_elect<D / 32>(tmem + sb * 2 * N, kd, qd, idesc);
          ptx::mma_commit_elect(ptx::smem_u32(&cb->s_full[sb]));
          ptx::mma_commit_elect(ptx::smem_u32(&cb->k_free[slot]));
          if (++slot == C::NK) {
            slot = 0;
            k_phase ^= 1;
          }
        }
        if (!ok) break;
        if (last) {
          ptx::mma_commit_elect(ptx::smem_u32(&cb->q_free[qb]));
          ++seg;
        }
      }
      ptx::mma_commit_elect(ptx::smem_u32(&cb->drain));
      wait_drain_warp(ptx::smem_u32(&cb->drain), 0, a.status);
    } else if (warp == kPvWarp) {
      // --------------------------------------------------------- PV issuer
      constexpr uint32_t idesc = ptx::idesc_f16_f32(D, N, true, true);
      bool ok = true;
      int i = 0, seg = 0, in_seg = 0;
      for (int b = 0; ok; ++b) {
        const BatchPlan<N>& plan = plan_of(b, &ok);
        if (!ok) break;
        const int count = plan.count, last = plan.last;
        plan_done(b);
        if (count == 0) break;
        if (in_seg == 0 && seg >= 2) ok = wait(cb->o_free[seg & 1], ((seg >> 1) - 1) & 1);
#pragma unroll 1
        for (int n = 0; ok && n < count; ++n, ++i, ++in_seg) {
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
          const uint32_t d = tmem + C::kOt + (seg & 1) * 2 * N + hb * N;
          ptx::mma_ss4_elect<16 * 128 / 16, 16 * C::kPRow / 16>(d, ad, bd, idesc,
                                                                in_seg > 1 ? 1u : 0u);
          ptx::mma_ss4_elect<16 * 128 / 16, 16 * C::kPRow / 16>(
              d, ptx::desc_add(ad, 64 * 128), ptx::desc_add(bd, 64 * C::kPRow), idesc, 1u);
          ptx::mma_commit_elect(ptx::smem_u32(&cb->pv_done[hb]));
        }
        if (last) {
          ++seg;
          in_seg = 0;
        }
      }
      ptx::mma_commit_elect(ptx::smem_u32(&cb->drain_pv));
      wait_drain_warp(ptx::smem_u32(&cb->drain_pv), 0, a.status);
    } else if (warp == kLoadWarp) {
      // ---------------------------------------------------------- producer
      // Lanes 0 and 1 issue the two pages of a tile with one instruction.
      test_load_delay(a.wait_limit_ns);
      bool ok = true;
      int kn = 0, vn = 0, sk = 0, sv = 0;  // loads issued and slots of K and V
      uint32_t k_phase = 1, v_phase = 1;   // (the first turn finds its slots free)
      for (int b = 0; ok; ++b) {
        const BatchPlan<N>& plan = plan_of(b, &ok);
        if (!ok) break;
        const int count = plan.count;
        const int cell = plan.cell[lane];
        plan_done(b);
        if (count == 0) break;
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
          ok = wait(cb->k_free[sk], k_phase);
          if (!ok) break;
          load(&k_map, cb->k_full[sk], smem + C::kK + sk * C::kTileBytes);
          ++kn;
          if (++sk == C::NK) {
            sk = 0;
            k_phase ^= 1;
          }
          ok = wait(cb->v_free[sv], v_phase);
          if (!ok) break;
          load(&v_map, cb->v_full[sv], smem + C::kV + sv * C::kTileBytes);
          ++vn;
          if (++sv == C::NV) {
            sv = 0;
            v_phase ^= 1;
          }
        }
      }
      // Every copy this CTA started lands before it exits.
#pragma unroll 1
      for (int s = 0; s < C::NK && s < kn; ++s)
        wait_drain_warp(ptx::smem_u32(&cb->k_full[s]), ((kn - 1 - s) / C::NK) & 1, a.status);
#pragma unroll 1
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
      int n0;  // tiles of the segment in earlier batches
      // Lane l: page l of the batch's tiles, as its cell of the cache, or -1
      // where it is not needed or not there.
      auto cells = [&]() {
        const int p = (g.tile0 + n0) * 2 + lane;
        if (n0 + lane / 2 >= g.count || (long long)p * kPageTokens >= g.keys.hi ||
            (long long)(p + 1) * kPageTokens <= g.keys.lo)
          return -1;
        const int id = checked_page(
            __ldg(a.page_table + (size_t)g.seq * a.max_pages + p), a.num_pages);
        return id < 0 ? -1 : id * sh.heads_k + g.head;
      };
      bool more = true, last = true;
      int cell = -1, seg = 0;
      bool ok = true;
      n0 = -kPlanTiles;
      for (int b = -1;; ++b) {
        const int slot = b & (kPagedPlans - 1);
        BatchPlan<N>& plan = cb->plan[slot];
        const bool first = n0 == 0, ends = last;
        uint4 raw[kBatch];
        int rows = 0, row_q = 0, row_h = 0;  // rows; lane's row: token and head
        auto load_rows = [&](int j0) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int n = j0 + j * kGroups + lane / kLanes;
            const int tok = __shfl_sync(0xffffffffu, row_q, n & 31);
            const int h = __shfl_sync(0xffffffffu, row_h, n & 31);
            raw[j] = make_uint4(0u, 0u, 0u, 0u);
            if (n < rows && dim0 < a.dim)
              raw[j] = __ldg(reinterpret_cast<const uint4*>(
                  a.q + (long long)tok * a.q_row + (long long)h * a.q_head + dim0));
          }
        };
        float ks = 0.f, vs = 0.f;
        auto publish = [&]() {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->plan_full[slot]));
        };
        if (b >= 0) {
          if (b >= kPagedPlans) ok = wait(cb->plan_free[slot], (b / kPagedPlans - 1) & 1);
          if (!ok) break;
          if (!more) {
            if (lane == 0) {
              plan.count = 0;
              ptx::mbar_arrive(ptx::smem_u32(&cb->plan_full[slot]));
            }
            break;
          }
          rows = imin(N, g.q.n * sh.group - g.row_tile * N);
          {
            const int row = g.row_tile * N + lane, tok = token_of(sh, row);
            row_q = g.q.lo + tok;
            row_h = g.head * sh.group + row - tok * sh.group;
            if (lane < N) {
              plan.out[lane] = row_q * a.heads + row_h;
              plan.lse[lane] = row_h * a.total_q + row_q;
              plan.token[lane] = tok - token_of(sh, g.row_tile * N);
            }
          }
          if (first) load_rows(0);  // (ahead of the pages' loads in the memory system)
          plan.cell[lane] = cell;
          if (lane == 0) {
            const int row0 = g.row_tile * N;
            plan.count = imin(g.count - n0, kPlanTiles);
            plan.tile0 = g.tile0 + n0;
            plan.first = first;
            plan.last = ends;
            plan.lo = g.keys.lo;
            plan.hi = g.keys.hi;
            plan.head = g.head;
            plan.q0 = g.q.lo;
            plan.row0 = row0;
            plan.rows = rows;
            plan.tok0 = token_of(sh, row0);
            plan.tok1 = token_of(sh, row0 + rows - 1);
            plan.at0 = (long long)g.len - g.q.n + plan.tok0;
            plan.tiles = g.count;
            plan.whole = g.count == g.unit_count;
            plan.unit_end =
                g.part_lo == 0 && g.count < g.unit_count ? g.unit_end : -1;
          }
          // The scales under way.
          if (cell >= 0) {
            ks = __ldg(a.k_scale + cell);
            vs = __ldg(a.v_scale + cell);
          }
          if (b > 0) publish();
        }
        const int held = cell >= 0;
        // On to the next batch.
        n0 += kPlanTiles;
        if (ends) {
          n0 = 0;
          more = walk_next(&walk, sh, before, seq_of, &g);
        }
        last = g.count - n0 <= kPlanTiles;
        cell = more ? cells() : -1;
        if (b >= 0) {
          // The first batch is not published before its scales and rows of Q
          // are here, and the next one's pages asked for: behind the first K
          // and V tiles of all SMs (17 MB) they would take some 3 us.
          if (b == 0) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
              asm volatile("" ::"r"(raw[j].x), "f"(ks), "f"(vs) : "memory");
            publish();
          }
          // Its scales and Q.
          plan.page[lane] = PagePlan{ks, vs, fmaxf(log2f(vs), -(float)kScaleExpMax), held};
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&cb->scale_full[slot]));
          if (first) {
            const int qb = seg % C::NQ;
            if (seg >= C::NQ) ok = wait(cb->q_free[qb], (seg / C::NQ - 1) & 1);
            if (!ok) break;
            uint8_t* q_s = smem + C::kQ + qb * C::kQBytes;  // N rows of hi, N of lo
#pragma unroll 1
            for (int j0 = 0; j0 < N; j0 += kGroups * kBatch) {
              if (j0 > 0) load_rows(j0);
#pragma unroll 1
              for (int j = 0; j < kBatch; ++j) {
                const int n = j0 + j * kGroups + lane / kLanes;
                if (j0 + j * kGroups >= rows) {
                  // Rows past the last: zeros.
                  const int us = D == 128 ? ((dim0 >> 4) ^ (n & 7)) : ((dim0 >> 4) ^ ((n >> 1) & 3));
                  uint8_t* at = q_s + n * C::kRow + us * 16 + (dim0 & 8);
                  *reinterpret_cast<uint2*>(at) = make_uint2(0u, 0u);
                  *reinterpret_cast<uint2*>(at + N * C::kRow) = make_uint2(0u, 0u);
                  if (sub == 0) cb->qs[seg % kPagedPlans][n] = a.scale_log2;
                  continue;
                }
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
                // mx in [2^e, 2^(e+1)) goes to [128, 256).  (Rows below 2^-100
                // keep a smaller size; their scores are zero in fp32 all the
                // same.)
                const int e = imax((int)(__float_as_uint(mx) >> 23) - 127, -100);
                const float f = __uint_as_float((uint32_t)(7 - e + 127) << 23);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float y0 = x[2 * k] * f, y1 = x[2 * k + 1] * f;
                  hi[k] = pack_e4m3x2(y0, y1);
                  const float2 h2 = f16x2_floats(unpack_e4m3x2(hi[k]));
                  lo[k] = pack_e4m3x2(y0 - h2.x, y1 - h2.y);
                }
                // (Rows n and N + n have the same place in the swizzle.)
                const int unit = dim0 >> 4;
                const int us = D == 128 ? (unit ^ (n & 7)) : (unit ^ ((n >> 1) & 3));
                uint8_t* at = q_s + n * C::kRow + us * 16 + (dim0 & 8);
                *reinterpret_cast<uint2*>(at) =
                    make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                *reinterpret_cast<uint2*>(at + N * C::kRow) =
                    make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                if (sub == 0)
                  cb->qs[seg % kPagedPlans][n] =
                      mx < __int_as_float(0x7f800000)
                          ? a.scale_log2 * __uint_as_float((uint32_t)(e - 7 + 127) << 23)
                          : __int_as_float(0x7fffffff);
              }
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(ptx::smem_u32(&cb->qs_full[seg % kPagedPlans]));
            ptx::mbar_arrive(ptx::smem_u32(&cb->q_full[qb]));
          }
          if (ends) ++seg;
        }
      }
    }
  } else {
    ptx::regs_inc<kPagedSoftmaxRegs>();
    // -------------------------------------------------------------- softmax
    const float neg_inf = -__int_as_float(0x7f800000);
    const unsigned full = 0xffffffffu;
    const int wg = warp >> 2;             // tiles i with i % 2 == wg
    const int key = tid & 127;            // of the tile
    const int page = key >> 6;
    const int bar = 1 + 4 * wg;           // named barriers bar .. bar + 2; 4: both warpgroups
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    float (*red)[N] = cb->red[wg];
    float* alpha = cb->alpha[wg];
    uint8_t* prow = smem + C::kP + wg * C::kPBytes + key * C::kPRow;
    // Scales and maxima of the rows, in pairs: at 16 rows they stay in
    // registers, for more they are read from shared memory, both of a pair at
    // once.
    constexpr int kHeld = N == 16 ? N / 2 : 1;
    ulonglong2 f_held[kHeld] = {};
    ulonglong2* factor = reinterpret_cast<ulonglong2*>(cb->factor[wg]);
    auto factor_of = [&](int n) { return N == 16 ? f_held[n % kHeld] : factor[n]; };
    auto pair = [](const float* p, int n) { return *reinterpret_cast<const uint64_t*>(p + n); };
    bool ok = true;
    int i = 0;  // tiles before the batch

    // The output of a segment is written once the next one's first tile is
    // under way (`due`), by when its last P V has long been done.
    struct {
      int seg, batch, last;
      bool alone, due;
    } done;
    done.due = false;
    // The warpgroups meet at barrier 4, once for each segment they share and
    // once more at the end, unless one has learnt there that the other gave
    // up (`parted`): so neither waits there for one that has left.
    bool parted = false;
    // Each warpgroup knows the PV of its own last tile of the segment to be
    // done before they meet: from the wait for Pt's buffer in a tile after it
    // (`later`), or by waiting here.  (Not both: with that tile's PV complete
    // the barrier's phase may have come round again.)
    auto finish = [&](bool later) -> bool {
      done.due = false;
      const bool alone = done.alone;
      const BatchPlan<N>& plan = cb->plan[done.batch % kPagedPlans];  // the segment's last
      const int rows = plan.rows;
      const int ring = done.seg % kPagedPlans;
      const int slot = 2 * cta + (done.seg == 0 ? 0 : 1);
      const int mine = (done.last & 1) == wg ? done.last : done.last - 1;
      bool good = later || wait(cb->pv_done[wg], (mine >> 1) & 1);
      ptx::tc_fence_before();
      good = alone ? named_bar_and(bar + 1, 128, good) : named_bar_and(4, 256, good);
      if (!good) {
        parted = !alone;
        return false;
      }
      ptx::tc_fence_after();
      // Lane n: weights of row n's two Ot, 2^(m - M) / sum; a warpgroup that saw
      // no key has m = -inf (or a NaN sum) and nothing to add.
      float wa = 0.f, wb = 0.f;
      if (lane < N) {
        const int n = lane, w0 = alone ? wg : 0;
        const float m0 = cb->end_m[ring][w0][n], l0 = cb->end_l[ring][w0][n];
        const float m1 = alone ? neg_inf : cb->end_m[ring][1][n];
        const float l1 = alone ? 0.f : cb->end_l[ring][1][n];
        const float top = fmaxf(m0, m1);
        const float base = top == neg_inf ? 0.f : top;
        const float e0 = m0 == neg_inf ? (l0 == 0.f ? 0.f : l0) : root_ex2(m0 - base);
        const float e1 = m1 == neg_inf ? (l1 == 0.f ? 0.f : l1) : root_ex2(m1 - base);
        const float sum = e0 * l0 * e0 + e1 * l1 * e1;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (a NaN stays one)
        // (These may be flushed: Ot goes by the maximum, like P'.)
        wa = e0 * e0 * inv;
        wb = e1 * e1 * inv;
        if (n < rows && (warp & 3) == 0 && (alone || wg == 0)) {
          const float l2 = sum == 0.f ? neg_inf : base + log2f(sum);
          if (!plan.whole)
            a.part_lse[(size_t)slot * N + n] = l2;
          else if (a.lse)
            a.lse[plan.lse[n]] = l2 * 0.69314718055994531f;
        }
      }
      if (plan.unit_end >= 0 && key == 0 && (alone || wg == 0)) {
        // The unit starts here: tell the merge how many CTAs share it.
        int parts = 1;
#pragma unroll 1
        while (cta + parts < ctas && range_start(total, ctas, cta + parts) < plan.unit_end) ++parts;
        a.meta[2 * cta + 1] = make_int4(rows, slot, 0, 0);
        a.meta[2 * cta] = make_int4(parts, plan.q0, plan.row0, plan.head);
      }
      // Dim of this thread's lane: row of a 128-row accumulator, or of a
      // 64-row one, which uses the first 16 lanes of each warp's 32.
      const int d = D == 128 ? key : (warp & 3) * 16 + lane;
      const bool live = d < a.dim && (D == 128 || lane < 16);
      const uint32_t o0 = tmem + lane_base + C::kOt + (done.seg & 1) * 2 * N;
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
          const float fa = __shfl_sync(full, wa, n);
          const float fb = __shfl_sync(full, wb, n);
          if (live && n < rows) {
            // (Weight 0: the Ot may hold anything.)
            const float v = (fa == 0.f ? 0.f : fa * __uint_as_float(oa[k])) +
                            (fb == 0.f ? 0.f : fb * __uint_as_float(ob[k]));
            if (plan.whole)
              a.out[(size_t)plan.out[n] * a.dim + d] = (uint16_t)ptx::pack_bf16x2(v, 0.f);
            else
              a.part_o[((size_t)slot * N + n) * D + d] = v;
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        const uint32_t bar_o = ptx::smem_u32(&cb->o_free[done.seg & 1]);
        ptx::mbar_arrive(bar_o);
        if (alone) ptx::mbar_arrive(bar_o);  // for the other warpgroup
      }
      // Only now: the planner writes over the segment's row scales, and the
      // other warpgroup over its maxima, four batches on at the earliest.
      plan_done(done.batch);
      return true;
    };

    int seg = 0, seg0 = 0;  // segment, its first tile
    uint64_t l[N / 2];
    bool unset = true;
    for (int b = 0; ok; ++b) {
      const BatchPlan<N>& plan = plan_of(b, &ok);
      if (ok && plan.count > 0) ok = wait(cb->scale_full[b % kPagedPlans], (b / kPagedPlans) & 1);
      const int count = plan.count, tile0 = plan.tile0, rows = plan.rows;
      const int tok0 = plan.tok0, tok1 = plan.tok1;
      const long long at0 = plan.at0;
      if (plan.first) seg0 = i;
      // This warpgroup's first tile of the batch and of the segment.
      const int first = (i & 1) == wg ? 0 : 1;
      const int start = seg0 + ((seg0 & 1) == wg ? 0 : 1);
      // (A warpgroup goes through a batch as one.)
      ok = named_bar_and(bar + 1, 128, ok);
      if (!ok) break;
      // A segment of one tile is its warpgroup's alone; the other one goes on
      // to the next.
      const bool alone = plan.tiles == 1;
      const bool skip = count == 0 || (alone && first != 0);
      const uint32_t o_tmem = tmem + lane_base + C::kOt + (seg & 1) * 2 * N + wg * N;
      const float* c = cb->qs[seg % kPagedPlans];
      float* end_m = cb->end_m[seg % kPagedPlans][wg];
      if (plan.first && !skip) {
#pragma unroll
        for (int n = 0; n < N / 2; ++n) l[n] = 0;
        // Rows that have seen no key yet have no maximum (0 stands in for
        // it); while there are any (`unset`), every tile takes the slow path
        // below.
        unset = true;
        ok = wait(cb->qs_full[seg % kPagedPlans], (seg / kPagedPlans) & 1);
        if (key < N) {
          cb->factor[wg][key / 2][key & 1] = c[key];
          cb->factor[wg][key / 2][2 + (key & 1)] = 0.f;
        }
        ok = named_bar_and(bar + 1, 128, ok);
        if (!ok) break;
        if constexpr (N == 16) {
#pragma unroll
          for (int n = 0; n < N / 2; ++n) f_held[n] = factor[n];
        }
      }
      // The tiles in a loop of their own, so that its instructions lie
      // together; it is left for a new maximum (`slow`), which comes back to
      // the same tile, and after a segment's first tile for the output that
      // is due.  A batch that is skipped comes by for that alone.
      bool settled = false;  // the tile's maximum is known to do
      for (int t = first;;) {
        const int stop = done.due ? imin(start - i + 1, count) : count;
        bool slow = false;
        uint64_t x[N / 2];  // score less the maximum, log2
        float lv = 0.f;
#pragma unroll 1
        for (; t < stop && !skip; t += 2) {
          const int at = i + t;  // tile of the CTA's range
          const uint32_t phase = (uint32_t)(at >> 1) & 1;
          const PagePlan pp = plan.page[2 * t + page];
          lv = pp.lv;
          const int j0 = (tile0 + t) * kTileKeys;
          const bool seen = j0 + key >= plan.lo && (unsigned)(j0 + key) < (unsigned)plan.hi && pp.held;
          // Rows of several tokens see different keys: the tiles at the edges
          // are masked row by row.
          const bool edge =
              tok0 != tok1 &&
              ((sh.causal && (long long)j0 + kTileKeys - 1 > at0) ||
               (sh.window >= 0 && (long long)j0 < at0 + (tok1 - tok0) - sh.window));
          // (A warp whose wait has given up still joins the votes below,
          // after which the whole warpgroup leaves.)
          const int sb = at % C::NS;
          const uint32_t s_tmem = tmem + lane_base + sb * 2 * N;
          if (ok) ok = wait(cb->s_full[sb], (at / C::NS) & 1);
          // Pt's buffer was last read by the PV of this warpgroup's last tile.
          if (ok && at >= 2) ok = wait(cb->pv_done[wg], phase ^ 1);
          ptx::tc_fence_after();
          const uint64_t ks2 = ptx::f2_pack(pp.ks, pp.ks);
          uint32_t qh[N], ql[N];
#pragma unroll
          for (int n = 0; n < N; n += 16) {
            ptx::tmem_ld16(s_tmem + n, qh + n);
            ptx::tmem_ld16(s_tmem + N + n, ql + n);
          }
          ptx::tmem_wait_ld();
#pragma unroll
          for (int n = 0; n < N; n += 16) {
            ptx::reg_fence16(qh + n);
            ptx::reg_fence16(ql + n);
          }
#pragma unroll
          for (int n = 0; n < N; n += 2) {
            const ulonglong2 f = factor_of(n / 2);
            const uint64_t h2 = ptx::f2_pack(__uint_as_float(qh[n]), __uint_as_float(qh[n + 1]));
            const uint64_t l2 = ptx::f2_pack(__uint_as_float(ql[n]), __uint_as_float(ql[n + 1]));
            x[n / 2] = ptx::fma2(ptx::add2(h2, l2), ptx::mul2(f.x, ks2), f.y);
          }
          if (edge) {
            // Row n stands at at0 + token[n].
            const long long r = (long long)j0 + key - at0;
            const long long w = r + sh.window;
            const int lo = sh.causal ? (int)(r < kMaxCost ? (r > -1 ? r : -1) : kMaxCost) : -1;
            const int hi = sh.window < 0 ? kMaxCost : (int)(w < kMaxCost ? (w > -1 ? w : -1) : kMaxCost);
#pragma unroll
            for (int n = 0; n < N; n += 4) {
              const int4 o = *reinterpret_cast<const int4*>(plan.token + n);
              float u, v;
              ptx::f2_unpack(x[n / 2], u, v);
              x[n / 2] = ptx::f2_pack(o.x >= lo && o.x <= hi ? u : neg_inf,
                                      o.y >= lo && o.y <= hi ? v : neg_inf);
              ptx::f2_unpack(x[n / 2 + 1], u, v);
              x[n / 2 + 1] = ptx::f2_pack(o.z >= lo && o.z <= hi ? u : neg_inf,
                                          o.w >= lo && o.w <= hi ? v : neg_inf);
            }
          }
          if (!seen) {
#pragma unroll
            for (int n = 0; n < N / 2; ++n) x[n] = ptx::f2_pack(neg_inf, neg_inf);
          }
          if (!settled) {
            // A new maximum is due where a score passes the old one by 2^8.
            float over = neg_inf;
#pragma unroll
            for (int n = 0; n < N / 2; ++n) {
              float u, v;
              ptx::f2_unpack(x[n], u, v);
              over = ptx::max3(over, u, v);
            }
            const int need = unset || !ok || over + lv > kRescaleLog2 + kPagedBias;
            if (named_bar_or(bar, 128, need)) {
              slow = true;
              break;
            }
          }
          settled = false;
          ptx::tc_fence_before();
          ptx::mbar_arrive(ptx::smem_u32(&cb->s_free[sb]));
          // Pt row of this key.
          const uint64_t vs2 = ptx::f2_pack(pp.vs, pp.vs);
#pragma unroll
          for (int n0 = 0; n0 < N; n0 += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float u, v;
              ptx::f2_unpack(x[n0 / 2 + k], u, v);
              const uint64_t p2 = ptx::f2_pack(ptx::ex2(u), ptx::ex2(v));
              l[n0 / 2 + k] = ptx::add2(l[n0 / 2 + k], p2);
              ptx::f2_unpack(ptx::mul2(p2, vs2), u, v);
              w[k] = ptx::pack_f16x2(u, v);
            }
            const int un = n0 / 8;
            const int us = N == 32 ? (un ^ ((key >> 1) & 3)) : (un ^ ((key >> 2) & 1));
            *reinterpret_cast<uint4*>(prow + us * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(ptx::smem_u32(&cb->p_full[wg]));
        }
        if (slow) {
          ok = named_bar_and(bar + 1, 128, ok);
          if (!ok) break;
          const int at = i + t;
#pragma unroll
          for (int n0 = 0; n0 < N; n0 += 16) {
            float v[16];
#pragma unroll
            for (int n = 0; n < 16; n += 2) {
              float u0, u1, m0, m1;
              ptx::f2_unpack(x[(n0 + n) / 2], u0, u1);
              ptx::f2_unpack(factor_of((n0 + n) / 2).y, m0, m1);
              v[n] = u0 - m0 + lv;
              v[n + 1] = u1 - m1 + lv;
            }
            const float top = warp_transpose_reduce16<true>(v, lane);
            if ((lane & 1) == 0) red[warp & 3][n0 + (lane >> 1)] = top;
          }
          named_bar_sync(bar + 2, 128);
          int none = 0;
          if (key < N) {
            const float mt = fmaxf(fmaxf(red[0][key], red[1][key]),
                                   fmaxf(red[2][key], red[3][key])) - kPagedBias;
            const float mu = at == start ? neg_inf : end_m[key];
            float al = 1.f;
            if (mt > mu) {
              al = mu == neg_inf ? 0.f : root_ex2(mu - mt);
              cb->factor[wg][key / 2][2 + (key & 1)] = -mt;
              end_m[key] = mt;
            } else if (at == start) {
              end_m[key] = neg_inf;
            }
            none = key < rows && end_m[key] == neg_inf;
            alpha[key] = al * al;
            alpha[N + key] = al;
          }
          unset = named_bar_or(bar, 128, none);
          if constexpr (N == 16) {
#pragma unroll
            for (int n = 0; n < N / 2; ++n) f_held[n] = factor[n];
          }
          if (at != start) {
#pragma unroll
            for (int n = 0; n < N; n += 2) {
              const uint64_t root = pair(alpha, N + n);
              l[n / 2] = ptx::mul2(ptx::mul2(l[n / 2], root), root);
            }
            // Ot holds this warpgroup's earlier tiles, whose last PV is done.
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
          settled = true;
          continue;
        }
        if (done.due && (skip || t > start - i)) {
          ok = finish(!skip);
          if (!ok) break;
        }
        if (skip || t >= count) break;
      }
      if (!ok || count == 0) break;
      if (skip) {
        plan_done(b);
        ++i;
        ++seg;
        continue;
      }
      i += count;
      if (!plan.last) {
        plan_done(b);
        continue;
      }
      // The segment's sums; its output comes later.
#pragma unroll
      for (int n0 = 0; n0 < N; n0 += 16) {
        float v[16];
#pragma unroll
        for (int n = 0; n < 16; n += 2) ptx::f2_unpack(l[(n0 + n) / 2], v[n], v[n + 1]);
        const float sum = warp_transpose_reduce16<false>(v, lane);
        if ((lane & 1) == 0) red[warp & 3][n0 + (lane >> 1)] = sum;
      }
      named_bar_sync(bar + 2, 128);
      if (key < N)
        cb->end_l[seg % kPagedPlans][wg][key] =
            (red[0][key] + red[1][key]) + (red[2][key] + red[3][key]);
      done.seg = seg;
      done.batch = b;
      done.last = i - 1;
      done.alone = alone;
      done.due = true;
      ++seg;
    }
    if (!parted) named_bar_and(4, 256, ok);
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
// so the result does not depend on timing.  (A small weight can meet the larger
// values, of pages with a larger scale, hence its root.)  A unit can have as many
// parts as there are CTAs, so every LSE is loaded at once and 16 partials at a
// time.
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
  constexpr int kAtOnce = 16;
  float v[kAtOnce];
  auto load = [&](int p0) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      v[k] = p0 + k < parts ? a.part_o[((size_t)slot(p0 + k) * N + n) * D + tid] : 0.f;
  };
  load(0);
  const float neg_inf = -__int_as_float(0x7f800000);
  float top = neg_inf;
  for (int p = tid; p < parts; p += D) {
    const float lp = a.part_lse[(size_t)slot(p) * N + n];
    s_w[p] = lp;
    top = fmaxf(top, lp);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) s_red[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < D / 32; ++w) top = fmaxf(top, s_red[w]);
  float sum = 0.f, acc = 0.f;
#pragma unroll 1
  for (int p0 = 0; p0 < parts; p0 += kAtOnce) {
    if (p0 > 0) load(p0);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (p0 + k < parts) {
        const float lp = s_w[p0 + k];
        const float w = lp == neg_inf ? 0.f : root_ex2(lp - top);
        sum = fmaf(w, w, sum);
        acc = fmaf(w, w * v[k], acc);
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
