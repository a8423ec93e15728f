// Host build of the packed forward's estimate of an item's key tiles, for a CPU test.
#include "../../varlen_flashattention_forward_gb300/csrc/varlen_shape.h"

extern "C" long long probe_item_key_tiles(long long total_k, int max_seqlen_k, int causal,
                                          int window_left, int window_right, int sinks,
                                          long long tree_nodes) {
  return fa::item_key_tiles(total_k, max_seqlen_k, causal, window_left, window_right, sinks,
                            tree_nodes, 256, 128);
}
