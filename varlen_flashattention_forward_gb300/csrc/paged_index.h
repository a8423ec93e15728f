// paged_index.h -- index arithmetic of the paged-cache kernels, for host and
// device.  Plain C++ without CUDA types, so that it also runs (and is tested)
// on the CPU.
//
// Every number that reaches a kernel from device memory (cu_seqlens,
// seq_lens, page ids) goes through one of these functions before it becomes
// an address: a malformed array then gives empty or shortened work, never an
// access outside the tensors.
#pragma once

#if defined(__CUDACC__)
#define FA_HD __host__ __device__ __forceinline__
#define FA_ROLLED _Pragma("unroll 1")  // short code over speed
#else
#define FA_HD inline
#define FA_ROLLED
#endif

namespace fa {

constexpr int kPageTokens = 64;  // tokens of a cache page

FA_HD int imin(int a, int b) { return a < b ? a : b; }
FA_HD int imax(int a, int b) { return a > b ? a : b; }

// Rows of sequence b in a packed tensor of `total` rows: the cu_seqlens
// entries clamped to [0, total], the end to at least the start.
struct RowRange {
  int lo, n;
};
FA_HD RowRange row_range(int cu0, int cu1, int total) {
  RowRange r;
  r.lo = imin(imax(cu0, 0), total);
  r.n = imin(imax(cu1, r.lo), total) - r.lo;
  return r;
}

// New tokens of a sequence as positions [first, first + n) of its cache: n
// rows are the last n of `len` positions; a sequence whose length is below
// its number of rows is malformed and gets none.  `limit` positions exist
// (pages of the table, rows of the rotation table); the rows past it are cut.
struct AppendSpan {
  int first, n;
};
FA_HD AppendSpan append_span(int n, int len, int limit) {
  AppendSpan s;
  s.first = len - n;
  s.n = n;
  if (n <= 0 || len < n) {
    s.first = 0;
    s.n = 0;
  } else if (len > limit) {
    s.n = imax(0, limit - s.first);
  }
  return s;
}

// Pages that the positions [first, first + n) touch.
FA_HD int pages_touched(int first, int n) {
  return n > 0 ? (first + n - 1) / kPageTokens - first / kPageTokens + 1 : 0;
}

// Slots of page number `p` (counted within the sequence) that the positions
// [first, first + n) fill: [slot, slot + count), row of the first one.
struct PageSpan {
  int slot, count, row;
};
FA_HD PageSpan page_span(int first, int n, int p) {
  PageSpan s;
  const int lo = imax(first, p * kPageTokens);
  const int hi = imin(first + n, (p + 1) * kPageTokens);
  s.slot = lo - p * kPageTokens;
  s.count = imax(0, hi - lo);
  s.row = lo - first;
  return s;
}

// Page id of the table, or -1 where it names no page of the cache.
FA_HD int checked_page(int id, int num_pages) { return id >= 0 && id < num_pages ? id : -1; }

// Keys [lo, hi) that any of the query rows i0 .. i1 (inclusive) of a sequence
// with n rows and `len` keys sees, of which `held` at most are in the table.
// Row i stands at position len - n + i; causal rows see no later key,
// window >= 0 bounds the keys before it.
struct KeyRange {
  int lo, hi;
};
FA_HD KeyRange key_range(int i0, int i1, int n, int len, int held, bool causal, int window) {
  KeyRange r;
  const int keys = imin(imax(len, 0), held);
  const long long at = (long long)len - n;
  long long hi = keys, lo = 0;
  if (causal && at + i1 + 1 < hi) hi = at + i1 + 1;
  if (window >= 0 && at + i0 - window > 0) lo = at + i0 - window;
  if (hi < 0) hi = 0;
  if (lo > hi) lo = hi;
  r.lo = (int)lo;
  r.hi = (int)hi;
  return r;
}

// ---------------------------------------------------- attention work split
// A work unit is one row tile (`rows` of the n * group rows of a sequence and
// kv head, row = token * group + head of the group) against its key tiles of
// kTileKeys keys.  Units come by sequence, then head, then row tile.  A unit
// costs its key tiles and kUnitCost more, for what a CTA does once for each
// (its rows of Q, the first maximum, its output); the costs, in that order,
// are cut into equal contiguous ranges, one for each CTA.  A unit's first
// kUnitCost places hold no tile, so a cut among them leaves it whole.
constexpr int kTileKeys = 128;
// In tiles.  Measured with 5, 6, 7, 8, 9: 64 sequences of 100 to 8192 keys, 4 kv
// heads of 128 dims 65.0, 62.7, 62.6, 62.4, 63.3 us; 24 sequences with 2 to 7
// rows, windows of 4096, 8 kv heads of 64 dims 49.7, 48.9, 48.6, 49.1, 50.3.
constexpr int kUnitCost = 7;

struct AttnShape {
  int heads_k, group, rows;  // kv heads, query heads of one, rows of a tile
  int causal, window, held;  // held: positions of the page table
};
FA_HD int token_of(const AttnShape& s, unsigned row) { return (int)(row / (unsigned)s.group); }

// n * group is at most the number of query rows of the call, below 2^31.
FA_HD int row_tiles(const AttnShape& s, int n) {
  return (int)(((unsigned)n * (unsigned)s.group + s.rows - 1) / (unsigned)s.rows);
}
// Keys of row tile t of a sequence with n query rows and len keys.
FA_HD KeyRange tile_keys(const AttnShape& s, int t, int n, int len) {
  const unsigned r0 = (unsigned)t * s.rows, all = (unsigned)n * s.group;
  unsigned r1 = r0 + s.rows;
  if (r1 > all) r1 = all;
  return key_range(token_of(s, r0), token_of(s, r1 - 1), n, len, s.held, s.causal != 0, s.window);
}
// First key tile and number of key tiles; a unit without keys keeps one (all
// masked), which writes its empty rows.
struct TileRange {
  int first, count;
};
FA_HD TileRange key_tiles(const KeyRange& k) {
  TileRange t;
  t.first = k.lo / kTileKeys;
  t.count = k.hi > k.lo ? (int)(((unsigned)k.hi + kTileKeys - 1) / kTileKeys) - t.first : 1;
  return t;
}
// Cost of all row tiles of one (sequence, head).
FA_HD long long head_cost(const AttnShape& s, int n, int len) {
  long long sum = 0;
  const int m = n > 0 ? row_tiles(s, n) : 0;
  FA_ROLLED
  for (int t = 0; t < m; ++t) sum += kUnitCost + key_tiles(tile_keys(s, t, n, len)).count;
  return sum;
}

// Costs are 32-bit.  The host splits a batch so that those of a launch stay
// below 2^31 where cu_seqlens is well formed; a sum past that (from
// overlapping sequences) stops at the limit, and what lies behind it is not
// done.
constexpr int kMaxCost = 0x7fffffff;
FA_HD int capped_cost(long long n) { return n < kMaxCost ? (int)n : kMaxCost; }

// Start of CTA c's range of `total` among `ctas`: the first total % ctas
// ranges are one longer.
FA_HD int range_start(int total, int ctas, int c) {
  const int q = (int)((unsigned)total / (unsigned)ctas), r = total - q * ctas;
  return c * q + (c < r ? c : r);
}

// Walks the segments of a range: the part of each unit's tiles inside it.
// before(b) is the cost of the sequences before b (b up to the batch).
struct Segment {
  int seq, head, row_tile;
  RowRange q;        // the sequence's query rows
  int len;           // its keys
  KeyRange keys;     // of the row tile
  int tile0;         // first key tile of the segment (tile t: keys 128 t ..)
  int count;         // its key tiles
  int part_lo, unit_count;  // place of tile0 among the unit's tiles, and their number
  int unit_end;      // cost up to the end of the unit
};
struct SegmentWalk {
  int at, end;  // cost done, end of the range
  int seq, head, row_tile;
  int in_unit;  // cost of the current unit that is done
};

template <typename Before>
FA_HD void walk_begin(SegmentWalk* w, int lo, int hi, int batch, const Before& before) {
  w->at = lo;
  w->end = hi;
  int a = 0, b = batch;  // before(a) <= lo < before(b)
  FA_ROLLED
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (before(m) <= lo) a = m; else b = m;
  }
  w->seq = a;
  w->head = -1;  // place within the sequence still to be found
  w->row_tile = 0;
  w->in_unit = 0;
}

// The next segment, or false at the end of the range.  seq_of(b, &q, &len)
// gives a sequence's query rows and keys.
template <typename Before, typename SeqOf>
FA_HD bool walk_next(SegmentWalk* w, const AttnShape& s, const Before& before, const SeqOf& seq_of,
                     Segment* g) {
  FA_ROLLED
  while (w->at < w->end) {
    if (w->head < 0) {
      FA_ROLLED
      while (before(w->seq + 1) <= w->at) ++w->seq;  // sequences without query rows
      seq_of(w->seq, &g->q, &g->len);
      const int in_seq = w->at - before(w->seq);
      // (The sequence's cost without the cap, so that no head is past the last.)
      const int per_head = capped_cost(head_cost(s, g->q.n, g->len));
      w->head = (int)((unsigned)in_seq / (unsigned)per_head);
      int left = in_seq - w->head * per_head;
      w->row_tile = 0;
      FA_ROLLED
      for (;;) {
        const int c = kUnitCost + key_tiles(tile_keys(s, w->row_tile, g->q.n, g->len)).count;
        if (left < c) break;
        left -= c;
        ++w->row_tile;
      }
      w->in_unit = left;
    } else {
      seq_of(w->seq, &g->q, &g->len);
    }
    g->seq = w->seq;
    g->head = w->head;
    g->row_tile = w->row_tile;
    g->keys = tile_keys(s, w->row_tile, g->q.n, g->len);
    const TileRange t = key_tiles(g->keys);
    const int cost = kUnitCost + t.count;
    int n = cost - w->in_unit;
    if (n > w->end - w->at) n = w->end - w->at;
    const int lo = w->in_unit > kUnitCost ? w->in_unit - kUnitCost : 0;
    const int hi = w->in_unit + n > kUnitCost ? w->in_unit + n - kUnitCost : 0;
    g->tile0 = t.first + lo;
    g->count = hi - lo;
    g->part_lo = lo;
    g->unit_count = t.count;
    w->at += n;
    w->in_unit += n;
    // (Past the limit of 32 bits the unit ends with the range.)
    g->unit_end = cost - w->in_unit < kMaxCost - w->at ? w->at + (cost - w->in_unit) : kMaxCost;
    if (w->in_unit == cost) {
      w->in_unit = 0;
      if (++w->row_tile == row_tiles(s, g->q.n)) {
        w->row_tile = 0;
        if (++w->head == s.heads_k) {
          w->head = -1;
          ++w->seq;
        }
      }
    }
    if (g->count > 0) return true;
  }
  return false;
}

}  // namespace fa
