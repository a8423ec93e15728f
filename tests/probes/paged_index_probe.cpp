// Host build of the paged kernels' index arithmetic, for a CPU test.
#include "../../varlen_flashattention_forward_gb300/csrc/paged_index.h"

extern "C" {
void probe_row_range(int c0, int c1, int total, int* out) {
  const fa::RowRange r = fa::row_range(c0, c1, total);
  out[0] = r.lo;
  out[1] = r.n;
}
void probe_append_span(int n, int len, int limit, int* out) {
  const fa::AppendSpan s = fa::append_span(n, len, limit);
  out[0] = s.first;
  out[1] = s.n;
}
int probe_pages_touched(int first, int n) { return fa::pages_touched(first, n); }
void probe_page_span(int first, int n, int p, int* out) {
  const fa::PageSpan s = fa::page_span(first, n, p);
  out[0] = s.slot;
  out[1] = s.count;
  out[2] = s.row;
}
int probe_checked_page(int id, int num) { return fa::checked_page(id, num); }
void probe_key_range(int i0, int i1, int n, int len, int held, int causal, int window, int* out) {
  const fa::KeyRange r = fa::key_range(i0, i1, n, len, held, causal != 0, window);
  out[0] = r.lo;
  out[1] = r.hi;
}
}
