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
#else
#define FA_HD inline
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

}  // namespace fa
