// Ancestor masks, positions and cache slots of drafted trees, from the nodes' parents.
//
// A warp takes a request, a lane its nodes i and i + 32. Ancestors by doubling: with m_i the nodes that i reaches in up to
// 2^k steps and p_i the one 2^k steps up,
//   m_i |= m_{p_i},  p_i = p_{p_i}
// six times, all by shuffles, instead of a chain of up to 63 dependent steps. A few bytes for each
// node: bound by the launch and one chain of loads (starts, parents and length, page). GB300: one request of 26 nodes 2.9 us, 500
// requests of up to 64 3.0.
#include "tl_internal.cuh"

#include "tree.cuh"

namespace tl {
namespace {

constexpr int kWarps = 4;

__global__ void __launch_bounds__(kWarps * 32) tree_plan_kernel(const __grid_constant__ TreePlanParams p) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x * kWarps + (threadIdx.x >> 5);
  pdl_wait_prior();
  pdl_launch_dependents();
  if (b > p.B) return;
  auto pad = [&](int64_t t) { p.masks[t] = 0, p.positions[t] = 0, p.slots[t] = -1; };
  // Rows of no request, where starts are not what they have to be: append stores nothing of them.
  auto pad_others = [&](int64_t from, int64_t to) {
    for (int64_t t = max(from, int64_t{0}) + lane; t < min(to, static_cast<int64_t>(p.T)); t += 32) {
      bool taken = false;
      for (int i = 0; i < p.B && !taken; ++i) {
        int first, nodes;
        taken = tree_rows(p.starts, i, p.T, first, nodes) && t >= first && t - first < nodes;
      }
      if (!taken) pad(t);
    }
  };
  if (b == p.B) {            // one warp more, for the rows before all requests and behind the last
    const int first = __ldg(p.starts), last = __ldg(p.starts + p.B);
    if (first > 0) {
      int least = min(first, p.T);
      for (int i = lane; i <= p.B; i += 32) least = min(least, __ldg(p.starts + i));
      least = __reduce_min_sync(0xffffffffu, least);
      for (int t = lane; t < least; t += 32) pad(t);
    }
    if (last < 0 || last > p.T) {
      if (lane == 0) set_status(p.status, TL_EDATA);
      if (last < 0) pad_others(0, p.T);
      return;
    }
    for (int64_t t = static_cast<int64_t>(last) + lane; t < p.T; t += 32) pad(t);
    return;
  }
  const int len = __ldg(p.lens + b);
  int begin, n;
  if (!tree_rows(p.starts, b, p.T, begin, n)) {
    if (lane == 0) set_status(p.status, TL_EDATA);
    pad_others(begin, __ldg(p.starts + b + 1));
    return;
  }
  const bool fits = len >= 0 && len <= p.capacity - n;
  unsigned long long mask[2];
  int up[2];
  bool bad = !fits;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    mask[h] = 1ull << i;
    up[h] = i < n ? __ldg(p.parents + begin + i) : -1;
    if (up[h] < -1 || up[h] >= i) bad = true, up[h] = -1;
  }
#pragma unroll
  for (int step = 0; step < 6; ++step) {
    unsigned long long seen[2];
    int next[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int from = up[h] & 31;
      const unsigned long long m0 = __shfl_sync(0xffffffffu, mask[0], from), m1 = __shfl_sync(0xffffffffu, mask[1], from);
      const int u0 = __shfl_sync(0xffffffffu, up[0], from), u1 = __shfl_sync(0xffffffffu, up[1], from);
      seen[h] = up[h] < 0 ? 0 : up[h] < 32 ? m0 : m1;
      next[h] = up[h] < 0 ? -1 : up[h] < 32 ? u0 : u1;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) mask[h] |= seen[h], up[h] = next[h];
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    if (i >= n) continue;
    const int64_t t = static_cast<int64_t>(begin) + i;
    p.masks[t] = static_cast<int64_t>(mask[h]);
    p.positions[t] = fits ? len + __popcll(mask[h]) - 1 : 0;
    int64_t slot = -1;
    if (fits) {
      const int key = len + i, at = key / p.page_size;
      const int page = __ldg(p.pages + b * p.ldp + at);
      if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages))
        slot = static_cast<int64_t>(page) * p.page_size + (key - at * p.page_size);
      else
        bad = true;
    }
    p.slots[t] = slot;
  }
  if (bad) set_status(p.status, TL_EDATA);
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.B / kWarps + 1);
  return launch_pdl(tree_plan_kernel, dim3(grid), dim3(kWarps * 32), 0, st, p);
}

}  // namespace tl
