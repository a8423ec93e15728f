// draft_tree_kernel.cuh -- ancestor masks and positions of drafted trees.
//
//   mask(i) = { i } + mask(parent(i)),   position(i) = seq_len - n + depth(i)
//
// and under a window w, for an attention with the same one, of these only the nodes
// that i sees when its path is decoded one after another: itself and its ancestors up
// to w nodes back, and those whose position is below `sinks`.  (The attention takes a
// node's depth from the bits of its mask.  Where some are left out there are w + 1 of
// them or more, and that window ends behind the context as the node's own does.)
//
// A thread takes a node and walks up to the root.  Parents are smaller
// numbers, so the walk passes the words of its mask from the last to the
// first and writes each once; it takes at most as many steps as there are
// nodes.  Latency alone bounds it, a launch and the chain of loads, which after
// the first come from L1: one tree of 16 nodes 3.2 us, 24 of 33 to 64 nodes 3.8.
#pragma once

#include <cuda_runtime.h>

#include "paged_index.h"

namespace fa {

struct DraftTreeArgs {
  const int *parents, *cu, *seq_lens;
  int total, words;
  int window, sinks;  // window: 0x7fffffff for none
  int *mask, *positions;
};

constexpr int kTreeThreads = 64;
constexpr int kTreeBlocks = 1024;  // of a sequence, at most

// Block (x, b): nodes of sequence b from kTreeThreads * x on, in steps of the
// grid.
__global__ void __launch_bounds__(kTreeThreads) draft_tree_kernel(const DraftTreeArgs a) {
  const int b = blockIdx.y;
  const RowRange r = row_range(__ldg(a.cu + b), __ldg(a.cu + b + 1), a.total);
  const long long context = (long long)__ldg(a.seq_lens + b) - r.n;
  for (int i = blockIdx.x * kTreeThreads + threadIdx.x; i < r.n; i += gridDim.x * kTreeThreads) {
    int* row = a.mask + (size_t)(r.lo + i) * a.words;
    auto parent = [&](int node) {
      const int up = __ldg(a.parents + r.lo + node);
      return up < node ? up : -1;
    };
    // Ancestors more than `late` nodes back are sinks.  (Only where the sinks reach
    // past the context.)
    int late = 0x7fffffff;
    if (a.window != 0x7fffffff && a.sinks > context) {
      long long d = 0;
      for (int node = parent(i); node >= 0; node = parent(node)) ++d;
      d += context - a.sinks;
      late = (int)(d > -1 ? d : -1);
    }
    int node = i, depth = -1, word = a.words - 1;
    unsigned bits = 0;
    while (node >= 0) {
      ++depth;
      const int w = node >> 5;
      // (Nodes past the mask's words leave no bit.)
      if (w <= word) {
        for (; word > w; --word) {
          row[word] = (int)bits;
          bits = 0;
        }
        if (depth <= a.window || depth > late) bits |= 1u << (node & 31);
      }
      node = parent(node);
    }
    for (; word >= 0; --word) {
      row[word] = (int)bits;
      bits = 0;
    }
    if (a.positions) {
      const long long p = context + depth;
      a.positions[r.lo + i] = (int)(p > -0x80000000ll ? p : -0x80000000ll);
    }
  }
}

}  // namespace fa
