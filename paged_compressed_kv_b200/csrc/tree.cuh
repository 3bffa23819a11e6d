// The tree description shared by the drafted-token kernels.
#pragma once

#include "common.cuh"

namespace v4kv {

// rows [first, first + n) of the per-node arrays belong to sequence b; n is
// clamped to the host's bounds (and flagged), so every row index stays inside
// the arrays whatever cu_nodes holds
struct TreeSeq {
  int first, n;
};

__device__ __forceinline__ TreeSeq tree_seq(const int32_t* cu_nodes, int b, int total, int max_nodes,
                                            int32_t* st) {
  const int lo = cu_nodes[b], hi = cu_nodes[b + 1];
  TreeSeq s;
  s.first = min(max(lo, 0), total);
  const int last = min(max(hi, s.first), total);
  s.n = min(last - s.first, max_nodes);
  if (s.n != hi - lo || s.first != lo) flag(st, V4KV_DEV_OVERFLOW);
  return s;
}

// a node's parent, -1 for a root and for a parent that does not come before it
__device__ __forceinline__ int tree_parent(const int32_t* parents, int first, int i, int32_t* st) {
  const int p = parents[first + i];
  if (p < -1 || p >= i) {
    flag(st, V4KV_DEV_BAD_INDEX);
    return -1;
  }
  return p;
}

}  // namespace v4kv
