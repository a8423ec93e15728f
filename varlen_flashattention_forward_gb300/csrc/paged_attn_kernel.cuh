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
//   producer warp 10    walks the segments, loads page ids and scales ahead,
//                       and TMA-loads the pages of each tile (128-byte
//                       swizzle; 64-byte at dim 64) into a K and a V ring;
//   Q warp 11           splits each segment's rows into hi and lo;
//   S issuer warp 8     St(i) as soon as K(i) has landed;
//   converter warps 4-7 V(i) to f16, rows nobody sees as zeros (they may hold
//                       anything, and 0 * NaN is NaN);
//   softmax warps 0-3   thread = key: masks, the vote on a new maximum (only
//                       when some score passes m by 2^8 is the maximum taken,
//                       O rescaled and the sums adjusted), exp2, Pt;
//   PV issuer warp 9    Ot += Vt Pt.
//
// TMEM: St at [0, 4N) (two buffers of 2N columns), Ot at [4N, 6N) (two).
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

constexpr int kPagedThreads = 384;
// Register split (launch: 168 x 384 = 64512): softmax 128 x 232, converters
// 128 x 88, control 128 x 96 = 53248.
constexpr uint32_t kPagedSoftmaxRegs = 232;
constexpr uint32_t kPagedConvertRegs = 88;
constexpr uint32_t kPagedControlRegs = 96;
constexpr int kPagedMaxBatch = 1024;  // sequences of one launch
constexpr int kPagedInfo = 8;         // tile descriptors in flight
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
  static constexpr int NV = N == 64 ? 2 : N == 32 ? 3 : 4;
  static constexpr uint32_t kSwP = N == 64   ? ptx::kLayoutSw128
                                   : N == 32 ? ptx::kLayoutSw64
                                             : ptx::kLayoutSw32;
  static constexpr uint32_t kTmemCols = N == 16 ? 128 : N == 32 ? 256 : 512;
  // Offsets from a 1024-byte boundary.
  static constexpr int kK = 0;
  static constexpr int kV = kK + NK * kTileBytes;
  static constexpr int kVh = kV + NV * kTileBytes;
  static constexpr int kP = kVh + 2 * kVhBytes;
  static constexpr int kQ = kP + 2 * kPBytes;
  static constexpr int kCtl = kQ + 2 * kQBytes;
};

struct alignas(16) PagedCtl {
  uint64_t k_full[4], k_free[4];    // K slot landed (TMA bytes) / read by its S MMA
  uint64_t v_full[4], v_free[4];    // V slot landed / converted (128 arrivals)
  uint64_t info_full[kPagedInfo];
  uint64_t vh_full[2];              // f16 V written (128)
  uint64_t s_full[2], s_free[2];    // St computed / loaded (128)
  uint64_t p_full[2], pv_done[2];   // Pt written (128) / PV complete
  uint64_t q_full[2], q_free[2];    // Q terms written (32) / last S of the segment
  uint64_t qs_full[4];              // row scales written (32)
  uint64_t o_free[2];               // Ot read out (128)
  uint64_t drain, drain_pv;         // everything an issuer started is complete
  uint32_t tmem_base;
  volatile int abort_flag;
  TileInfo info[kPagedInfo];
  alignas(16) float qs[4][64];      // row scale * softmax scale * log2(e)
  alignas(16) float red[4][64];     // per-warp partial maxima / sums
  alignas(16) float m_used[64];     // running maximum - bias
  alignas(16) float alpha[64];      // rescale factors; at the end reciprocal sums
  long long warp_sum[kPagedThreads / 32];
  long long before[kPagedMaxBatch + 1];
};

// (16-byte loads of these.)
static_assert(offsetof(PagedCtl, qs) % 16 == 0 && offsetof(PagedCtl, m_used) % 16 == 0, "align");

template <int D, int N>
constexpr size_t paged_smem() {
  return 1024 + PagedCfg<D, N>::kCtl + sizeof(PagedCtl);
}
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
      init(cb->k_full[s], 1);
      init(cb->k_free[s], 1);
      init(cb->v_full[s], 1);
      init(cb->v_free[s], 128);
      init(cb->qs_full[s], 32);
    }
    for (int s = 0; s < kPagedInfo; ++s) init(cb->info_full[s], 1);
    for (int s = 0; s < 2; ++s) {
      init(cb->vh_full[s], 128);
      init(cb->s_full[s], 1);
      init(cb->s_free[s], 128);
      init(cb->p_full[s], 128);
      init(cb->pv_done[s], 1);
      init(cb->q_full[s], 32);
      init(cb->q_free[s], 1);
      init(cb->o_free[s], 128);
    }
    init(cb->drain, 1);
    init(cb->drain_pv, 1);
    cb->abort_flag = 0;
    ptx::fence_mbar_init();
    a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  if (warp == 8) {
    ptx::tmem_alloc(ptx::smem_u32(&cb->tmem_base), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (warp == 10 && lane == 0) {
    ptx::prefetch_tmap(&k_map);
    ptx::prefetch_tmap(&v_map);
  }
  // Tiles of the sequences before each one: a scan over the batch, the same
  // in every CTA.
  {
    long long base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPagedThreads) {
      const int b = b0 + tid;
      long long n = 0;
      if (b < a.batch) {
        RowRange q;
        int len;
        seq_of(b, &q, &len);
        n = sh.heads_k * head_tiles(sh, q.n, len);
      }
      long long sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (lane == 31) cb->warp_sum[warp] = sum;
      __syncthreads();
      long long all = 0, lo = base;
#pragma unroll
      for (int w = 0; w < kPagedThreads / 32; ++w) {
        if (w < warp) lo += cb->warp_sum[w];
        all += cb->warp_sum[w];
      }
      if (b < a.batch) cb->before[b + 1] = lo + sum;
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
  const long long total = cb->before[a.batch];
  const int cta = blockIdx.x, ctas = gridDim.x;
  SegmentWalk walk;
  walk_begin(&walk, range_start(total, ctas, cta), range_start(total, ctas, cta + 1), a.batch,
             before);
  Segment g;
  // Slot n of a ring of size R: slot n % R, phase parity (n / R) & 1.
  auto wait = [&](uint64_t& b, int parity) {
    return wait_warp(ptx::smem_u32(&b), (uint32_t)parity, abort_flag, a.status, a.wait_limit_ns);
  };

  if (warp >= 4 && warp < 8) {
    ptx::regs_dec<kPagedConvertRegs>();
    // ------------------------------------------------------------ converters
    // Thread t: 16-byte unit u = t % (D / 16) of rows t / (D / 16) + k * 128 / (D / 16).
    constexpr int kUnits = D / 16;          // 8 or 4 units of a row
    constexpr int kRows = 128 / kUnits;     // rows at once
    const int t = tid - 128;
    const int u = t % kUnits, r0 = t / kUnits;
    bool ok = true;
    int i = 0;
    while (ok && walk_next(&walk, sh, before, seq_of, &g)) {
      for (int n = 0; n < g.count; ++n, ++i) {
        const int slot = i % C::NV, hb = i & 1;
        ok = wait(cb->v_full[slot], (i / C::NV) & 1);
        if (!ok) break;
        const TileInfo& ti = cb->info[i % kPagedInfo];
        const int lo = ti.lo, hi = ti.hi, held = ti.held;
        if (i >= 2) {
          ok = wait(cb->pv_done[hb], ((i >> 1) - 1) & 1);
          if (!ok) break;
        }
        const uint8_t* src = smem + C::kV + slot * C::kTileBytes;
        uint8_t* dst = smem + C::kVh + hb * C::kVhBytes;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
          const int r = r0 + k * kRows;
          const int us = D == 128 ? (u ^ (r & 7)) : (u ^ ((r >> 1) & 3));
          uint4 c = *reinterpret_cast<const uint4*>(src + r * C::kRow + us * 16);
          if (r < lo || r >= hi || !((held >> (r >> 6)) & 1)) c = make_uint4(0u, 0u, 0u, 0u);
          uint4 h0, h1;
          h0.x = unpack_e4m3x2(c.x);
          h0.y = unpack_e4m3x2(c.x >> 16);
          h0.z = unpack_e4m3x2(c.y);
          h0.w = unpack_e4m3x2(c.y >> 16);
          h1.x = unpack_e4m3x2(c.z);
          h1.y = unpack_e4m3x2(c.z >> 16);
          h1.z = unpack_e4m3x2(c.w);
          h1.w = unpack_e4m3x2(c.w >> 16);
          // f16 rows of 128 bytes in chunks of 64 dims, 128-byte swizzle;
          // lanes of the upper chunk store their second half first, so that
          // the eight lanes of a row hit eight different 16-byte banks.
          uint8_t* row = dst + (u >> 2) * (kTileKeys * 128) + r * 128;
          const int p0 = ((u & 3) * 2) ^ (r & 7), p1 = p0 ^ 1;
          const bool swap = u >= 4;
          *reinterpret_cast<uint4*>(row + (swap ? p1 : p0) * 16) = swap ? h1 : h0;
          *reinterpret_cast<uint4*>(row + (swap ? p0 : p1) * 16) = swap ? h0 : h1;
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(ptx::smem_u32(&cb->vh_full[hb]));
        ptx::mbar_arrive(ptx::smem_u32(&cb->v_free[slot]));
      }
    }
  } else if (warp >= 8) {
    ptx::regs_dec<kPagedControlRegs>();
    if (warp == 8) {
      // ---------------------------------------------------------- S issuer
      constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, 2 * N);
      bool ok = true;
      int i = 0;
      for (int seg = 0; ok && walk_next(&walk, sh, before, seq_of, &g); ++seg) {
        ok = wait(cb->q_full[seg & 1], (seg >> 1) & 1);
        if (!ok) break;
        const uint64_t qd = ptx::smem_desc(ptx::smem_u32(smem + C::kQ + (seg & 1) * C::kQBytes), 16,
                                           8 * C::kRow, C::kSwK);
        for (int n = 0; n < g.count; ++n, ++i) {
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
        ptx::mma_commit_elect(ptx::smem_u32(&cb->q_free[seg & 1]));
      }
      ptx::mma_commit_elect(ptx::smem_u32(&cb->drain));
      wait_drain_warp(ptx::smem_u32(&cb->drain), 0, a.status);
    } else if (warp == 9) {
      // --------------------------------------------------------- PV issuer
      constexpr uint32_t idesc = ptx::idesc_f16_f32(D, N, true, true);
      bool ok = true;
      int i = 0;
      for (int seg = 0; ok && walk_next(&walk, sh, before, seq_of, &g); ++seg) {
        if (seg >= 2) ok = wait(cb->o_free[seg & 1], ((seg >> 1) - 1) & 1);
        for (int n = 0; ok && n < g.count; ++n, ++i) {
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
          const uint32_t d = tmem + 4 * N + (seg & 1) * N;
          ptx::mma_ss4_elect<16 * 128 / 16, 16 * C::kPRow / 16>(d, ad, bd, idesc, n > 0 ? 1u : 0u);
          ptx::mma_ss4_elect<16 * 128 / 16, 16 * C::kPRow / 16>(
              d, ptx::desc_add(ad, 64 * 128), ptx::desc_add(bd, 64 * C::kPRow), idesc, 1u);
          ptx::mma_commit_elect(ptx::smem_u32(&cb->pv_done[hb]));
        }
      }
      ptx::mma_commit_elect(ptx::smem_u32(&cb->drain_pv));
      wait_drain_warp(ptx::smem_u32(&cb->drain_pv), 0, a.status);
    } else if (warp == 10) {
      // ---------------------------------------------------------- producer
      test_load_delay(a.wait_limit_ns);
      bool ok = true;
      int i = 0, kn = 0, vn = 0;  // tiles; K and V loads issued
      while (ok && walk_next(&walk, sh, before, seq_of, &g)) {
        const int* table = a.page_table + (size_t)g.seq * a.max_pages;
        // Lane l holds page l of a batch of 16 tiles: its id, or -1 where the
        // tile needs no such page, and its scales.
        int id = -1;
        float ks = 0.f, vs = 0.f, lv = 0.f;
        for (int n = 0; n < g.count; ++n, ++i) {
          if (n % 16 == 0) {
            const int p = (g.tile0 + n) * 2 + lane;
            id = -1;
            ks = vs = 0.f;
            lv = -kScaleExpMax;
            if (n + lane / 2 < g.count && p * (long long)kPageTokens < g.keys.hi &&
                (p + 1) * (long long)kPageTokens > g.keys.lo)
              id = checked_page(__ldg(table + p), a.num_pages);
            if (id >= 0) {
              const size_t cell = (size_t)id * sh.heads_k + g.head;
              ks = __ldg(a.k_scale + cell);
              vs = __ldg(a.v_scale + cell);
              lv = fmaxf(log2f(vs), -(float)kScaleExpMax);
            }
          }
          const int l0 = (n % 16) * 2;
          const int id0 = __shfl_sync(0xffffffffu, id, l0), id1 = __shfl_sync(0xffffffffu, id, l0 + 1);
          const int ks_slot = i % C::NK, vs_slot = i % C::NV;
          if (i >= C::NK) ok = wait(cb->k_free[ks_slot], (i / C::NK - 1) & 1);
          if (!ok) break;
          TileInfo* ti = &cb->info[i % kPagedInfo];
          if ((lane & ~1) == l0) {
            ti->ks[lane & 1] = ks;
            ti->vs[lane & 1] = vs;
            ti->lv[lane & 1] = lv;
          }
          const int held = (id0 >= 0 ? 1 : 0) | (id1 >= 0 ? 2 : 0);
          const uint32_t bytes = ((held & 1) + (held >> 1)) * C::kPageBytes;
          if (lane == 0) {
            const long long key0 = (long long)(g.tile0 + n) * kTileKeys;
            ti->lo = (int)(g.keys.lo > key0 ? g.keys.lo - key0 : 0);
            ti->hi = (int)(g.keys.hi < key0 + kTileKeys ? g.keys.hi - key0 : kTileKeys);
            ti->held = held;
          }
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(ptx::smem_u32(&cb->info_full[i % kPagedInfo]));
            const uint32_t bar = ptx::smem_u32(&cb->k_full[ks_slot]);
            const uint32_t dst = ptx::smem_u32(smem + C::kK + ks_slot * C::kTileBytes);
            ptx::mbar_arrive_expect_tx(bar, bytes);
            if (id0 >= 0) ptx::tma_load_3d(dst, &k_map, bar, 0, 0, id0 * sh.heads_k + g.head);
            if (id1 >= 0)
              ptx::tma_load_3d(dst + C::kPageBytes, &k_map, bar, 0, 0, id1 * sh.heads_k + g.head);
          }
          ++kn;
          if (i >= C::NV) ok = wait(cb->v_free[vs_slot], (i / C::NV - 1) & 1);
          if (!ok) break;
          if (lane == 0) {
            const uint32_t bar = ptx::smem_u32(&cb->v_full[vs_slot]);
            const uint32_t dst = ptx::smem_u32(smem + C::kV + vs_slot * C::kTileBytes);
            ptx::mbar_arrive_expect_tx(bar, bytes);
            if (id0 >= 0) ptx::tma_load_3d(dst, &v_map, bar, 0, 0, id0 * sh.heads_k + g.head);
            if (id1 >= 0)
              ptx::tma_load_3d(dst + C::kPageBytes, &v_map, bar, 0, 0, id1 * sh.heads_k + g.head);
          }
          ++vn;
        }
      }
      // Every copy this CTA started lands before it exits.
      for (int s = 0; s < C::NK && s < kn; ++s)
        wait_drain_warp(ptx::smem_u32(&cb->k_full[s]), ((kn - 1 - s) / C::NK) & 1, a.status);
      for (int s = 0; s < C::NV && s < vn; ++s)
        wait_drain_warp(ptx::smem_u32(&cb->v_full[s]), ((vn - 1 - s) / C::NV) & 1, a.status);
    } else {
      // ------------------------------------------------------------ Q warp
      constexpr int kLanes = D / 8;           // lanes of a row, 8 dims each
      constexpr int kGroups = 32 / kLanes;
      const int sub = lane % kLanes, dim0 = sub * 8;
      bool ok = true;
      for (int seg = 0; ok && walk_next(&walk, sh, before, seq_of, &g); ++seg) {
        if (seg >= 2) ok = wait(cb->q_free[seg & 1], ((seg >> 1) - 1) & 1);
        if (!ok) break;
        const int row0 = g.row_tile * N;
        const int rows = imin(N, g.q.n * sh.group - row0);
        uint8_t* q_s = smem + C::kQ + (seg & 1) * C::kQBytes;  // N rows of hi, N of lo
        constexpr int kBatch = 4;
        for (int j0 = 0; j0 < N; j0 += kGroups * kBatch) {
          uint4 raw[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int n = j0 + j * kGroups + lane / kLanes;
            raw[j] = make_uint4(0u, 0u, 0u, 0u);
            if (n < rows && dim0 < a.dim) {
              const int tok = (row0 + n) / sh.group, h = (row0 + n) - tok * sh.group;
              raw[j] = __ldg(reinterpret_cast<const uint4*>(
                  a.q + (long long)(g.q.lo + tok) * a.q_row +
                  (long long)(g.head * sh.group + h) * a.q_head + dim0));
            }
          }
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
            int e;
            frexpf(mx * (1.f / 256.f), &e);  // mx * 2^-e in [128, 256)
            if (!(mx > 0.f)) e = 0;
            // Two factors: 2^-e itself may be past fp32 for tiny rows.
            const float f0 = ldexpf(1.f, -(e / 2)), f1 = ldexpf(1.f, -(e - e / 2));
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float y0 = x[2 * k] * f0 * f1, y1 = x[2 * k + 1] * f0 * f1;
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
              cb->qs[seg & 3][n] = mx < __int_as_float(0x7f800000)
                                       ? ldexpf(a.scale_log2, e)
                                       : __int_as_float(0x7fffffff);
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(ptx::smem_u32(&cb->qs_full[seg & 3]));
        ptx::mbar_arrive(ptx::smem_u32(&cb->q_full[seg & 1]));
      }
    }
  } else {
    ptx::regs_inc<kPagedSoftmaxRegs>();
    // -------------------------------------------------------------- softmax
    const float neg_inf = -__int_as_float(0x7f800000);
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const int key = tid;           // of the tile
    const int page = key >> 6;
    float l[N];
    bool ok = true;
    int i = 0;
    for (int seg = 0; ok && walk_next(&walk, sh, before, seq_of, &g); ++seg) {
      const int row0 = g.row_tile * N;
      const int rows = imin(N, g.q.n * sh.group - row0);
      const int tok0 = row0 / sh.group, tok1 = (row0 + rows - 1) / sh.group;
      const long long at0 = (long long)g.len - g.q.n + tok0;  // position of the first row
#pragma unroll
      for (int n = 0; n < N; ++n) l[n] = 0.f;
      if (tid < N) cb->m_used[tid] = neg_inf;
      ok = wait(cb->qs_full[seg & 3], (seg >> 2) & 1);
      ok = named_bar_and(3, 128, ok);
      if (!ok) break;
      float c[N];
#pragma unroll
      for (int n = 0; n < N; n += 4) {
        const float4 v = *reinterpret_cast<const float4*>(&cb->qs[seg & 3][n]);
        c[n] = v.x; c[n + 1] = v.y; c[n + 2] = v.z; c[n + 3] = v.w;
      }
      for (int t = 0; t < g.count; ++t, ++i) {
        const int sb = i & 1;
        ok = wait(cb->info_full[i % kPagedInfo], (i / kPagedInfo) & 1);
        if (ok) ok = wait(cb->s_full[sb], (i >> 1) & 1);
        // (Every wait is followed by a warpgroup-wide agreement, so that no
        // warp is left alone at a later named barrier.)
        ok = named_bar_and(3, 128, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const TileInfo& ti = cb->info[i % kPagedInfo];
        const float ks = ti.ks[page], vs = ti.vs[page], lv = ti.lv[page];
        const bool seen = key >= ti.lo && key < ti.hi && ((ti.held >> page) & 1);
        float x[N];
#pragma unroll
        for (int n0 = 0; n0 < N; n0 += 16) {
          uint32_t hi[16], lo[16];
          ptx::tmem_ld16(tmem + lane_base + sb * 2 * N + n0, hi);
          ptx::tmem_ld16(tmem + lane_base + sb * 2 * N + N + n0, lo);
          ptx::tmem_wait_ld();
          ptx::reg_fence16(hi);
          ptx::reg_fence16(lo);
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const float s = __uint_as_float(hi[n]) + __uint_as_float(lo[n]);
            x[n0 + n] = seen ? s * (c[n0 + n] * ks) : neg_inf;
          }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&cb->s_free[sb]));
        // Rows of several tokens see different keys: mask the tiles at the
        // edges row by row.
        if (tok0 != tok1) {
          const long long j = (long long)(g.tile0 + t) * kTileKeys + key;
          const long long j0 = j - key;
          const bool edge = (sh.causal && j0 + kTileKeys - 1 > at0) ||
                            (sh.window >= 0 && j0 < at0 + (tok1 - tok0) - sh.window);
          if (edge) {
            for (int tok = tok0; tok <= tok1; ++tok) {
              const long long at = at0 + (tok - tok0);
              const bool out = (sh.causal && j > at) || (sh.window >= 0 && j < at - sh.window);
              if (out) {
                const int first = tok * sh.group - row0;
#pragma unroll
                for (int n = 0; n < N; ++n)
                  if (n >= first && n < first + sh.group) x[n] = neg_inf;
              }
            }
          }
        }
        // A new maximum is due where a score passes the old one by 2^8.
        int need = 0;
#pragma unroll
        for (int n0 = 0; n0 < N; n0 += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&cb->m_used[n0]);
          need |= x[n0] + lv > m.x + kRescaleLog2 + kPagedBias;
          need |= x[n0 + 1] + lv > m.y + kRescaleLog2 + kPagedBias;
          need |= x[n0 + 2] + lv > m.z + kRescaleLog2 + kPagedBias;
          need |= x[n0 + 3] + lv > m.w + kRescaleLog2 + kPagedBias;
        }
        if (named_bar_or(2, 128, need)) {
          float v[N];
#pragma unroll
          for (int n = 0; n < N; ++n) v[n] = x[n] + lv;
          warp_transpose_reduce<N, true>(v, lane);
          if ((lane & 1) == 0) {
#pragma unroll
            for (int k = 0; k < N / 16; ++k) cb->red[warp][16 * k + (lane >> 1)] = v[k];
          }
          named_bar_sync(1, 128);
          if (tid < N) {
            const float mt = fmaxf(fmaxf(cb->red[0][tid], cb->red[1][tid]),
                                   fmaxf(cb->red[2][tid], cb->red[3][tid])) - kPagedBias;
            const float mu = cb->m_used[tid];
            float al = 1.f;
            if (mt > mu) {
              al = mu == neg_inf ? 0.f : ptx::ex2(mu - mt);
              cb->m_used[tid] = mt;
            }
            cb->alpha[tid] = al;
          }
          named_bar_sync(1, 128);
#pragma unroll
          for (int n = 0; n < N; ++n) l[n] *= cb->alpha[n];
          if (t > 0) {
            // Ot holds the segment's earlier tiles: wait for their last PV.
            ok = wait(cb->pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1);
            ok = named_bar_and(3, 128, ok);
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += 16) {
              uint32_t o[16];
              const uint32_t addr = tmem + lane_base + 4 * N + (seg & 1) * N + n0;
              ptx::tmem_ld16(addr, o);
              ptx::tmem_wait_ld();
              ptx::reg_fence16(o);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                o[k] = __float_as_uint(__uint_as_float(o[k]) * cb->alpha[n0 + k]);
              ptx::tmem_st16(addr, o);
            }
            ptx::tmem_wait_st();
          }
        }
        // Pt row of this key.  The buffer's last reader was PV(i - 2).
        if (i >= 2) {
          ok = wait(cb->pv_done[sb], ((i >> 1) - 1) & 1);
          ok = named_bar_and(3, 128, ok);
          if (!ok) break;
        }
        uint8_t* prow = smem + C::kP + sb * C::kPBytes + key * C::kPRow;
#pragma unroll
        for (int n0 = 0; n0 < N; n0 += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 m = *reinterpret_cast<const float2*>(&cb->m_used[n0 + 2 * k]);
            // (A row that has seen no key yet: its scores are -inf, and so
            // must not meet the maximum -inf.)
            const float p0 = ptx::ex2(x[n0 + 2 * k] - (m.x == neg_inf ? 0.f : m.x));
            const float p1 = ptx::ex2(x[n0 + 2 * k + 1] - (m.y == neg_inf ? 0.f : m.y));
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
        ptx::mbar_arrive(ptx::smem_u32(&cb->p_full[sb]));
      }
      if (!ok) break;

      // ------------------------------------------------------ segment output
      const bool whole = g.count == g.unit_count;
      const int slot = 2 * cta + (seg == 0 ? 0 : 1);
      if (!whole && g.part_lo == 0 && tid == 0) {
        // The unit starts here: tell the merge how many CTAs share it.
        const long long unit_end = walk.at - g.count + g.unit_count;
        int parts = 1;
        while (cta + parts < ctas && range_start(total, ctas, cta + parts) < unit_end) ++parts;
        a.meta[2 * cta] = make_int4(parts, g.q.lo, row0, g.head);
        a.meta[2 * cta + 1] = make_int4(rows, slot, 0, 0);
      }
      warp_transpose_reduce<N, false>(l, lane);
      if ((lane & 1) == 0) {
#pragma unroll
        for (int k = 0; k < N / 16; ++k) cb->red[warp][16 * k + (lane >> 1)] = l[k];
      }
      named_bar_sync(1, 128);
      if (tid < N) {
        const float sum = (cb->red[0][tid] + cb->red[1][tid]) + (cb->red[2][tid] + cb->red[3][tid]);
        // (0: no key seen; a NaN stays one.)
        cb->alpha[tid] = sum == 0.f ? 0.f : 1.f / sum;
        const float l2 = sum == 0.f ? neg_inf : cb->m_used[tid] + log2f(sum);
        if (tid < rows) {
          if (!whole) {
            a.part_lse[(size_t)slot * N + tid] = l2;
          } else if (a.lse) {
            const int tok = (row0 + tid) / sh.group, h = (row0 + tid) - tok * sh.group;
            a.lse[(size_t)(g.head * sh.group + h) * a.total_q + g.q.lo + tok] =
                l2 * 0.69314718055994531f;
          }
        }
      }
      named_bar_sync(1, 128);
      ok = wait(cb->pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1);
      ok = named_bar_and(3, 128, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      // Dim of this thread's lane: row of a 128-row accumulator, or of a
      // 64-row one, which uses the first 16 lanes of each warp's 32.
      const int d = D == 128 ? tid : warp * 16 + lane;
      const bool live = d < a.dim && (D == 128 || lane < 16);
#pragma unroll 1
      for (int n0 = 0; n0 < rows; n0 += 16) {
        uint32_t o[16];
        ptx::tmem_ld16(tmem + lane_base + 4 * N + (seg & 1) * N + n0, o);
        ptx::tmem_wait_ld();
        ptx::reg_fence16(o);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int n = n0 + k;
          if (live && n < rows) {
            const float v = __uint_as_float(o[k]) * cb->alpha[n];
            if (whole) {
              const int tok = (row0 + n) / sh.group, h = (row0 + n) - tok * sh.group;
              a.out[((size_t)(g.q.lo + tok) * a.heads + g.head * sh.group + h) * a.dim + d] =
                  (uint16_t)ptx::pack_bf16x2(v, 0.f);
            } else {
              a.part_o[((size_t)slot * N + n) * D + d] = v;
            }
          }
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_u32(&cb->o_free[seg & 1]));
      named_bar_sync(1, 128);  // alpha is read before the next segment writes it
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the parts of the units that CTA boundaries cut.  Block (c, y): the
// unit that starts in CTA c and ends in a later one, rows y of it.
// O = sum_p w_p O_p, w_p = 2^(lse_p - LSE): the parts are summed in CTA order,
// so the result does not depend on timing.
template <int D, int N>
__global__ void __launch_bounds__(D) paged_merge_kernel(const PagedAttnArgs a) {
  const int c = blockIdx.x, tid = threadIdx.x;
  ptx::grid_dependency_wait();
  const int4 m0 = a.meta[2 * c];
  if (m0.x == 0) return;
  const int4 m1 = a.meta[2 * c + 1];
  const int n = blockIdx.y;
  if (n >= m1.x) return;
  auto slot = [&](int p) { return p == 0 ? m1.y : 2 * (c + p); };
  const float neg_inf = -__int_as_float(0x7f800000);
  float top = neg_inf;
  for (int p = 0; p < m0.x; ++p) top = fmaxf(top, a.part_lse[(size_t)slot(p) * N + n]);
  float sum = 0.f, acc = 0.f;
  for (int p = 0; p < m0.x; ++p) {
    const float lp = a.part_lse[(size_t)slot(p) * N + n];
    const float w = lp == neg_inf ? 0.f : ptx::ex2(lp - top);
    sum += w;
    acc = fmaf(w, a.part_o[((size_t)slot(p) * N + n) * D + tid], acc);
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
