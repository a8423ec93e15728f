// paged_kv_kernels.cuh -- writing the paged 8-bit key/value cache, and reading
// it back as packed bf16.
//
// Cache: e4m3 [pages, kv heads, 64 tokens, dim] with one fp32 scale for each
// (page, kv head); a value is code * scale.  The scale is the smallest power
// of two that keeps the largest value of the page within 448, the largest
// e4m3 number, so that moving codes to a larger scale only drops bits at the
// subnormal end.  A page that is filled over several calls only ever raises
// its scale, and ends with the one that writing it at once would have given
// (unless rows were written over, as after rejected drafts: theirs counts too).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "find_unit.cuh"
#include "named_bar.cuh"
#include "paged_index.h"
#include "rope_row.cuh"
#include "sm103_ptx.cuh"

namespace fa {

// ------------------------------------------------------------------ append
struct KvAppendArgs {
  const uint16_t *k, *v;
  long long k_row, k_head, v_row, v_head;
  const int *cu, *seq_lens, *page_table;
  int batch, total, heads, dim, max_pages, num_pages;
  int limit;  // positions that exist
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  const float* k_weight;  // or null
  float inv_dim, eps;
  RopeParams rope;
  int per_block, key_blocks;  // heads of a block, blocks for keys (prompt kernel)
};

struct AppendChunk {
  int page, slot, count;  // the page, its first new slot and their number
  int row0, pos0;         // row and position of the first
};

// One item: the new tokens of one page and head, keys (KEYS) or values, taken
// by a team of TEAM warps (TEAM = 1 or the block).  Rows go ROWS at a time to
// each LANES-lane group; an item of at most TEAM * ROWS * (32 / LANES) rows is
// held in registers between the maximum and the rounding, a longer one is
// loaded again for the second pass.
template <int LANES, int ROWS, int TEAM, bool KEYS>
struct AppendItem {
  static constexpr int kGroups = 32 / LANES;           // rows of a warp at once
  static constexpr int kPass = TEAM * ROWS * kGroups;  // rows of the team's pass
  static constexpr bool kOnePass = kPass >= kPageTokens;
  const KvAppendArgs& a;
  const AppendChunk ch;
  const float* table;  // row of the chunk's first position
  int team_warp, lane, sub;
  RowPieces p;
  uint64_t w[4];
  // The current item.
  const uint16_t* src;
  uint8_t* codes;
  float* scale;
  float old;
  RowBits raw[ROWS];
  uint64_t x[ROWS][4];
  int turn_no = 0;

  __device__ __forceinline__ AppendItem(const KvAppendArgs& a_, const AppendChunk& c, int tw,
                                        const float* table_)
      : a(a_), ch(c), table(table_), team_warp(tw) {
    lane = threadIdx.x & 31;
    sub = lane % LANES;
    if constexpr (KEYS) {
      p = row_pieces(a.rope, sub, a.dim);
      if (a.k_weight && p.a >= 0) load_weights(a.k_weight, p, w);
    } else {
      p.a = sub * 8 < a.dim ? sub * 8 : -1;
      p.b = sub * 8 + 4;
    }
  }
  __device__ __forceinline__ bool whole() const { return !KEYS || whole_pieces(a.rope); }
  __device__ __forceinline__ int row_of(int pass, int i) const {
    return pass * kPass + (i * TEAM + team_warp) * kGroups + lane / LANES;
  }
  __device__ __forceinline__ void load(int pass) {
    const long long stride = KEYS ? a.k_row : a.v_row;
    const uint16_t* row = src + (long long)(ch.row0 + row_of(pass, 0)) * stride;
    const long long step = (long long)(TEAM * kGroups) * stride;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      raw[i].a = raw[i].b = make_uint2(0u, 0u);
      if (row_of(pass, i) < ch.count && p.a >= 0) raw[i] = load_row(row, p, whole());
      row += step;
    }
  }
  // (Keys and values of one block can be two teams of it.)
  __device__ __forceinline__ void team_sync() const { named_bar_sync(KEYS ? 1 : 2, TEAM * 32); }
  // Head `head` of the chunk: its first loads under way.
  __device__ __forceinline__ void begin(int head) {
    src = KEYS ? a.k + head * a.k_head : a.v + head * a.v_head;
    const size_t cell = (size_t)ch.page * a.heads + head;
    codes = (KEYS ? a.k_cache : a.v_cache) + cell * kPageTokens * a.dim;
    scale = (KEYS ? a.k_scale : a.v_scale) + cell;
    old = ch.slot > 0 ? *scale : 0.f;
    load(0);
  }
  __device__ __forceinline__ void values(int pass) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      unpack_row(raw[i], x[i]);
      if constexpr (KEYS) {
        if (a.k_weight) norm_row<LANES>(x[i], w, a.inv_dim, a.eps);
        const int r = row_of(pass, i);
        if (p.turns && r < ch.count)
          rotate_row(x[i], a.rope, load_rope(a.rope, table + r * a.rope.rot_dim, sub));
      }
    }
  }
  // The item that begin() has under way; `next` (a head, or -1) is under way
  // when it returns.
  __device__ __forceinline__ void finish(int next, float* s_amax) {
    float amax = 0.f;
    const int passes = kOnePass ? 1 : (ch.count + kPass - 1) / kPass;
#pragma unroll 1
    for (int ps = 0; ps < passes; ++ps) {
      if (ps > 0) load(ps);
      values(ps);
      // Infinite and NaN values take no part in the scale: an infinity
      // saturates and a NaN stays one, and the rest of the page keeps its
      // precision.  (Rows and lanes past the end hold zeros; the maximum
      // passes over NaN by itself.)
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float u, v;
          ptx::f2_unpack(x[i][j], u, v);
          top = ptx::max3(top, fabsf(u), fabsf(v));
        }
      }
      if (__builtin_expect(!(top <= 3.402823466e38f), 0)) {
        top = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float u, v;
            ptx::f2_unpack(x[i][j], u, v);
            if (fabsf(u) <= 3.402823466e38f) top = fmaxf(top, fabsf(u));
            if (fabsf(v) <= 3.402823466e38f) top = fmaxf(top, fabsf(v));
          }
        }
      }
      amax = fmaxf(amax, top);
    }
    uint8_t* const codes_ = codes;
    float* const scale_ = scale;
    const float old_ = old;
    if (passes == 1 && next >= 0) begin(next);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if constexpr (TEAM > 1) {
      // (Two rows in turn: those of the last item may still be being read.)
      float* row = s_amax + turn_no * TEAM;
      turn_no ^= 1;
      if (lane == 0) row[team_warp] = amax;
      team_sync();  // (and every warp has read the old scale)
#pragma unroll
      for (int i = 0; i < TEAM; ++i) amax = fmaxf(amax, row[i]);
    }
    const float s = fmaxf(scale_for(amax), old_);
    const float inv = 1.f / s;
    const uint64_t inv2 = ptx::f2_pack(inv, inv);
    __syncwarp();
    if (lane == 0 && team_warp == 0) *scale_ = s;
#pragma unroll 1
    for (int ps = 0; ps < passes; ++ps) {
      if (passes > 1) {
        load(ps);
        values(ps);
      }
      uint8_t* at = codes_ + (ch.slot + row_of(ps, 0)) * a.dim;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        uint8_t* row = at + i * (TEAM * kGroups) * a.dim;
        if (row_of(ps, i) < ch.count && p.a >= 0) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            ptx::f2_unpack(ptx::mul2(x[i][j], inv2), f[2 * j], f[2 * j + 1]);
          const uint32_t lo = pack_e4m3x2(f[0], f[1]) | pack_e4m3x2(f[2], f[3]) << 16;
          const uint32_t hi = pack_e4m3x2(f[4], f[5]) | pack_e4m3x2(f[6], f[7]) << 16;
          if (whole()) {
            *reinterpret_cast<uint2*>(row + p.a) = make_uint2(lo, hi);
          } else {
            *reinterpret_cast<uint32_t*>(row + p.a) = lo;
            *reinterpret_cast<uint32_t*>(row + p.b) = hi;
          }
        }
      }
    }
    // Earlier tokens of the page follow a scale that has grown.
    if (ch.slot > 0 && s > old_) {
      const float f = old_ * inv;
      const int words = ch.slot * a.dim / 4;
      uint32_t* c = reinterpret_cast<uint32_t*>(codes_);
#pragma unroll 1
      for (int i = team_warp * 32 + lane; i < words; i += TEAM * 32) {
        const uint32_t u = c[i];
        const float2 lo = f16x2_floats(unpack_e4m3x2(u)), hi = f16x2_floats(unpack_e4m3x2(u >> 16));
        c[i] = pack_e4m3x2(lo.x * f, lo.y * f) | pack_e4m3x2(hi.x * f, hi.y * f) << 16;
      }
    }
    if (passes > 1 && next >= 0) begin(next);
  }
  // Heads first, first + step, ... below `end`.
  __device__ __forceinline__ void run(int first, int end, int step, float* s_amax) {
#pragma unroll 1
    for (int h = first; h < end; h += step) finish(h + step < end ? h + step : -1, s_amax);
  }
};

// The page of the cache and the rows that chunk x (page by page of each
// sequence's new tokens) fills; false if there is nothing to write.
__device__ __forceinline__ bool append_chunk(const KvAppendArgs& a, int x, AppendChunk* c) {
  auto span = [&](int b, int* lo) {
    const RowRange r = row_range(__ldg(a.cu + b), __ldg(a.cu + b + 1), a.total);
    *lo = r.lo;
    return append_span(r.n, __ldg(a.seq_lens + b), a.limit);
  };
  const FoundUnit u = find_unit(x, a.batch, [&](int b) {
    int lo;
    const AppendSpan s = span(b, &lo);
    return pages_touched(s.first, s.n);
  });
  if (u.seq < 0) return false;
  int lo;
  const AppendSpan s = span(u.seq, &lo);
  const int p = s.first / kPageTokens + u.at;
  const PageSpan sp = page_span(s.first, s.n, p);
  c->slot = sp.slot;
  c->count = sp.count;
  c->row0 = lo + sp.row;
  c->pos0 = s.first + sp.row;
  c->page = checked_page(__ldg(a.page_table + (size_t)u.seq * a.max_pages + p), a.num_pages);
  return c->page >= 0;
}

// Few tokens of each sequence: a block takes a chunk, its even warps the heads
// of K and its odd warps those of V, one warp an item.  A chunk of more than
// kStepAlone tokens among them has the whole block as a team, head by head (255
// sequences with one token and one with 2048, 8 heads of 128 dims: 23.0 us, one
// warp an item 45.2; 64 sequences of 15 tokens: team 17.6, one warp 12.3).
// What bounds it is latency, 4.9 us for 256 tokens: launch, search for the block's
// sequence, its page, rows, maximum, codes, each waiting for the one before.
constexpr int kStepThreads = 512;
constexpr int kStepAlone = 16;
template <int LANES>
__global__ void __launch_bounds__(kStepThreads, 2) kv_append_step_kernel(const KvAppendArgs a) {
  constexpr int kTeam = kStepThreads / 32;
  AppendChunk ch;
  if (!append_chunk(a, blockIdx.x, &ch)) return;
  const int warp = threadIdx.x >> 5;
  const float* table = a.rope.table + (long long)ch.pos0 * a.rope.rot_dim;
  if (ch.count > kStepAlone) {
    __shared__ float s_amax[2][2 * kTeam];
    {
      AppendItem<LANES, 2, kTeam, true> it(a, ch, warp, table);
      it.begin(0);
      it.run(0, a.heads, 1, s_amax[0]);
    }
    AppendItem<LANES, 2, kTeam, false> it(a, ch, warp, nullptr);
    it.begin(0);
    it.run(0, a.heads, 1, s_amax[1]);
    return;
  }
  const int head = warp >> 1, step = kTeam / 2;
  if (head >= a.heads) return;
  if (warp & 1) {
    AppendItem<LANES, 1, 1, false> it(a, ch, 0, nullptr);
    it.begin(head);
    it.run(head, a.heads, step, nullptr);
  } else {
    AppendItem<LANES, 1, 1, true> it(a, ch, 0, table);
    it.begin(head);
    it.run(head, a.heads, step, nullptr);
  }
}

// Many tokens: a block of LANES / 2 warps (4 rows of each lane group fill a
// page) takes `a.per_block` heads of a chunk in turn, keys (the first
// a.key_blocks in y) or values, with the next head's rows under way.  The
// positions' table rows (32 KB of 64 positions of 128 dims) come into shared
// memory for all its heads.
// 4 x 2048 tokens x 8 heads of 128 dims take 16.7 us, 3.1 TB/s: one wave of
// blocks, of which the launch, the search and the first loads are about half
// and the issue of the norm's, rotation's and packing's instructions the rest.
// (One wave of blocks with keys and values in turn and no loads ahead: 19.4.)
template <int LANES>
__global__ void __launch_bounds__(16 * LANES, 48 / LANES)
    kv_append_prompt_kernel(const KvAppendArgs a) {
  constexpr int kTeam = LANES / 2;
  extern __shared__ __align__(16) float s_table[];
  __shared__ float s_amax[2 * kTeam];
  AppendChunk ch;
  if (!append_chunk(a, blockIdx.x, &ch)) return;
  const bool keys = blockIdx.y < (unsigned)a.key_blocks;
  const int first = (keys ? blockIdx.y : blockIdx.y - a.key_blocks) * a.per_block;
  const int end = imin(first + a.per_block, a.heads);
  if (keys) {
    const float4* rows =
        reinterpret_cast<const float4*>(a.rope.table + (long long)ch.pos0 * a.rope.rot_dim);
#pragma unroll 1
    for (int k = threadIdx.x; k < ch.count * a.rope.rot_dim / 4; k += blockDim.x)
      ptx::cp_async_16(ptx::smem_u32(s_table) + k * 16, rows + k);
    AppendItem<LANES, 4, kTeam, true> it(a, ch, threadIdx.x >> 5, s_table);
    it.begin(first);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    it.run(first, end, 1, s_amax);
  } else {
    AppendItem<LANES, 4, kTeam, false> it(a, ch, threadIdx.x >> 5, nullptr);
    it.begin(first);
    it.run(first, end, 1, s_amax);
  }
}

// ------------------------------------------------------------------ gather
struct KvGatherArgs {
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int *cu, *page_table;
  int batch, total, heads, dim, max_pages, num_pages;
  uint16_t *k, *v;
  int wide_stores;  // both outputs are 32-byte aligned
};

// A block takes one page of one sequence, K or V; each thread 16 codes at a
// time, which leave with one 32-byte store where the outputs are aligned to
// that (two of 16 bytes: 2 x 32768 tokens 71.5 us, one: 66.5 us).  One load of
// a thread in flight is best: with two, four or eight the reads and writes of
// the same DRAM pages drift apart (71, 74, 77 us).
// Positions whose page is not in the cache (or not in the table) read as zero.
__global__ void __launch_bounds__(256) kv_gather_kernel(const KvGatherArgs a) {
  const FoundUnit u = find_unit(blockIdx.x, a.batch, [&](int b) {
    const RowRange r = row_range(__ldg(a.cu + b), __ldg(a.cu + b + 1), a.total);
    return pages_touched(0, r.n);
  });
  if (u.seq < 0) return;
  const RowRange r = row_range(__ldg(a.cu + u.seq), __ldg(a.cu + u.seq + 1), a.total);
  const PageSpan sp = page_span(0, r.n, u.at);
  const int page =
      u.at < a.max_pages
          ? checked_page(__ldg(a.page_table + (size_t)u.seq * a.max_pages + u.at), a.num_pages)
          : -1;
  const int per_row = a.dim / 16;
  const int per_token = a.heads * per_row;
  const uint8_t* cache = blockIdx.y ? a.v_cache : a.k_cache;
  const float* scales = blockIdx.y ? a.v_scale : a.k_scale;
  uint16_t* out = blockIdx.y ? a.v : a.k;
  for (int i = threadIdx.x; i < sp.count * per_token; i += blockDim.x) {
    const int t = i / per_token, j = i - t * per_token;
    const int h = j / per_row, c = j - h * per_row;
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (page >= 0) {
      const size_t cell = (size_t)page * a.heads + h;
      const uint4 code = __ldg(reinterpret_cast<const uint4*>(
          cache + (cell * kPageTokens + sp.slot + t) * a.dim + c * 16));
      const float s = __ldg(scales + cell);
      const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 lo = f16x2_floats(unpack_e4m3x2(cw[k]));
        const float2 hi = f16x2_floats(unpack_e4m3x2(cw[k] >> 16));
        w[2 * k] = ptx::pack_bf16x2(lo.x * s, lo.y * s);
        w[2 * k + 1] = ptx::pack_bf16x2(hi.x * s, hi.y * s);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(out + ((size_t)(r.lo + sp.row + t) * a.heads + h) * a.dim +
                                          c * 16);
    if (a.wide_stores) {
      ptx::st_global_v8(dst, w);
    } else {
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

}  // namespace fa
