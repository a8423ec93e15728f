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

// Walks every CTA's range; writes (cta, seq, head, row_tile, tile0, count,
// part_lo, unit_count) of each segment and returns how many there are (at
// most `most`), -1 past that.
extern "C" int probe_walk(const int* cu, const int* lens, int batch, int total_q, int heads_k,
                          int group, int rows, int causal, int window, int held, int ctas, int most,
                          int* out) {
  fa::AttnShape s = {heads_k, group, rows, causal, window, held};
  auto seq_of = [&](int b, fa::RowRange* q, int* len) {
    *q = fa::row_range(cu[b], cu[b + 1], total_q);
    *len = lens[b];
  };
  int pre[4097];
  long long sum = 0;
  pre[0] = 0;
  for (int b = 0; b < batch; ++b) {
    fa::RowRange q;
    int len;
    seq_of(b, &q, &len);
    sum += heads_k * fa::head_cost(s, q.n, len);
    pre[b + 1] = fa::capped_cost(sum);
  }
  auto before = [&](int b) { return pre[b]; };
  int found = 0;
  for (int c = 0; c < ctas; ++c) {
    fa::SegmentWalk w;
    fa::Segment g;
    fa::walk_begin(&w, fa::range_start(pre[batch], ctas, c), fa::range_start(pre[batch], ctas, c + 1),
                   batch, before);
    while (fa::walk_next(&w, s, before, seq_of, &g)) {
      if (found == most) return -1;
      // A part that is not the unit's last ends where the CTA's range does.
      if (g.part_lo + g.count < g.unit_count && w.at != w.end) return -2;
      // The parts a merge would look for: CTAs whose range starts in the unit.
      int parts = 1;
      while (c + parts < ctas && fa::range_start(pre[batch], ctas, c + parts) < g.unit_end) ++parts;
      const int v[8] = {c,      g.seq,   g.head,    g.row_tile,
                        g.tile0, g.count, g.part_lo, g.part_lo == 0 ? g.unit_count + 65536 * parts
                                                                     : g.unit_count};
      for (int k = 0; k < 8; ++k) out[8 * found + k] = v[k];
      ++found;
    }
  }
  return found;
}
