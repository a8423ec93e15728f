// varlen_shape.h -- how many key tiles an item of the packed forward walks.
// Plain C++, so that it also runs (and is tested) on the CPU.
#pragma once

namespace fa {

// Key tiles (of `tile` keys) of a work item of at most `rows` query rows, estimated
// from the call's sizes and hints; it steers the split over a cluster and nothing
// else.  max_seqlen_k: 0 for unknown.  tree_nodes: rows that a sequence is expected to
// have where they are the nodes of a tree (causal is not used then), else 0.  sinks:
// first keys that stay visible behind the window; the tiles between are left out.
inline long long item_key_tiles(long long total_k, int max_seqlen_k, int causal, int window_left,
                                int window_right, int sinks, long long tree_nodes, int rows,
                                int tile) {
  auto tiles = [&](long long keys) { return (keys + tile - 1) / tile; };
  const long long keys = max_seqlen_k > 0 && max_seqlen_k < total_k ? max_seqlen_k : total_k;
  const bool tree = tree_nodes > 0;
  if (window_left < 0 || !(tree || causal || window_right >= 0)) return tiles(keys);
  const long long span =
      (long long)window_left + (tree ? tree_nodes : (long long)(causal ? 0 : window_right) + rows);
  if (span >= keys) return tiles(keys);
  const long long first = sinks < keys - span ? sinks : keys - span;
  const long long sum = tiles(span) + tiles(first);
  return sum < tiles(keys) ? sum : tiles(keys);
}

}  // namespace fa
