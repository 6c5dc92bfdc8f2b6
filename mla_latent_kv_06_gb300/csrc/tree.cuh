// tree.cuh -- one node of a drafted token tree.
//
// The S new tokens of a sequence form a tree given by parent indices: -1 for a
// child of the last cached token, s' < s for a child of node s', -2 for an
// absent node.  Node s sees itself and its ancestors, and its rotary position
// is the prefix length plus its depth (its number of ancestors).
#pragma once

#include <float.h>
#include <stdint.h>

#include "../../include/mla.h"

namespace mla {

enum TreeState { kNodePresent = 0, kNodeAbsent = 1, kNodeBad = 2 };

// Where the running maximum of a node's scores starts.  Not at -inf: a tile may
// show it no key, and its weights are then exp(-inf - maximum) = 0.
constexpr float kMaxFloor = -FLT_MAX;

struct TreeNode {
  unsigned long long mask;  // bit j: node j is visible (0 for an absent or bad node)
  int depth;
  int state;
};

// Node s of the tree whose S parents start at `par`.  The walk up visits
// strictly decreasing indices, so it ends after at most S <= 64 steps; a
// parent at or above its child, below -2, or absent makes the node bad.
__device__ __forceinline__ TreeNode tree_node(const int32_t* par, int s) {
  TreeNode n{1ull << s, 0, kNodePresent};
  int cur = s, up = __ldg(par + s);
  if (up == -2) return TreeNode{0ull, 0, kNodeAbsent};
  while (up >= 0 && up < cur) {
    cur = up;
    n.mask |= 1ull << cur;
    ++n.depth;
    up = __ldg(par + cur);
  }
  if (up != -1) return TreeNode{0ull, 0, kNodeBad};
  return n;
}

}  // namespace mla
