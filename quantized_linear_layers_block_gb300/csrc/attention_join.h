// Who joins whose partials in paged attention: a segment's keys are cut over n neighbouring blocks, from block c0
// on, each of which leaves a partial. The blocks of a group count themselves in, and the last of them to arrive joins the
// group's partials into the first of them; where that leaves several, every fan-th one, they are grouped in the same way.
//
// A counter must have one user at a time. Of the blocks of a segment only the first and the last may hold a part of
// another cut segment; this one's c0 is no other's, for no second cut segment can begin in a block. The second level's only
// group is counted at c0. A group of the first level is counted at its first block, which lies before the segment's
// last unless that is a group for itself. The next segment may begin there, and count its own first group there: so a
// group of one has no counter, and needs none, being complete when it arrives.
//
// Plain C++: compiled for the GPU with the kernel, and by itself for the test.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define TL_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TL_HOST_DEVICE inline
#endif

namespace tl {

constexpr int kAttnMaxGrid = 4096;     // the workspace begins with a counter for each block and level
constexpr int kAttnLevels = 2;

namespace attn {

constexpr int kJoinBytes = 320 * 1024;

struct JoinGroup {
  int first, size;          // its first partial, counted from c0, and how many
  int counter;              // among the workspace's counters; -1 for a group of one
};

// Partials to a group. One join of all up to kJoinBytes, which cost about what a second level does (3 us); else two
// levels: the least fan with fan^2 >= n.
TL_HOST_DEVICE int join_fan(int n, int partial_bytes) {
  return static_cast<long long>(n) * partial_bytes <= kJoinBytes ? n : static_cast<int>(ceilf(sqrtf(static_cast<float>(n))));
}

// The group to which `block`'s partial belongs on a level on which every `step`-th one is left.
TL_HOST_DEVICE JoinGroup join_group(int block, int c0, int n, int fan, int step, int level) {
  JoinGroup g;
  g.first = (block - c0) / (step * fan) * (step * fan);
  g.size = (n - g.first + step - 1) / step;
  if (g.size > fan) g.size = fan;
  g.counter = g.size == 1 ? -1 : level * kAttnMaxGrid + c0 + g.first;
  return g;
}

}  // namespace attn
}  // namespace tl
