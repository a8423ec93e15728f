// Host build of the masked attention's work split, for a CPU test.
#include "../../varlen_flashattention_forward_gb300/csrc/paged_index.h"

// Walks every CTA's range; writes (cta, seq, head, row_tile, part_lo, count,
// unit_count, tile0) of each segment and returns how many there are (at most
// `most`), -1 past that, -2 where tile0 is not the tile of part_lo.
extern "C" int probe_masked_walk(const int* cu, const int* lens, int batch, int total_q,
                                 int heads_k, int group, int rows, int causal, int window, int held,
                                 int sinks, int tree, int ctas, int most, int* out) {
  const fa::AttnShape s = {heads_k, group, rows, causal, window, held, sinks, tree};
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
    sum += heads_k * fa::head_cost<true>(s, q.n, len);
    pre[b + 1] = fa::capped_cost(sum);
  }
  auto before = [&](int b) { return pre[b]; };
  int found = 0;
  for (int c = 0; c < ctas; ++c) {
    fa::SegmentWalk w;
    fa::Segment g;
    fa::walk_begin(&w, fa::range_start(pre[batch], ctas, c),
                   fa::range_start(pre[batch], ctas, c + 1), batch, before);
    while (fa::walk_next<true>(&w, s, before, seq_of, &g)) {
      if (found == most) return -1;
      if (g.tile0 != fa::tile_of(g.tiles, g.part_lo)) return -2;
      const int v[8] = {c, g.seq, g.head, g.row_tile, g.part_lo, g.count, g.unit_count, g.tile0};
      for (int k = 0; k < 8; ++k) out[8 * found + k] = v[k];
      ++found;
    }
  }
  return found;
}

extern "C" int probe_range_start(int total, int ctas, int c) { return fa::range_start(total, ctas, c); }
extern "C" int probe_range_of(int total, int ctas, int p) { return fa::range_of(total, ctas, p); }

// Key tile of the u-th tile of row tile t of a sequence.
extern "C" int probe_tile_of(int n, int len, int t, int heads_k, int group, int rows, int causal,
                             int window, int held, int sinks, int tree, int u) {
  const fa::AttnShape s = {heads_k, group, rows, causal, window, held, sinks, tree};
  return fa::tile_of(fa::key_tiles<true>(fa::tile_keys<true>(s, t, n, len)), u);
}
