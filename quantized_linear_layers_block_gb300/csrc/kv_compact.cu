// Moves the rows of accepted nodes together in a paged cache.
//
// A row's destination may be an earlier row's source, so a block takes all moves of a request for some 16-byte columns of
// the cache's rows: every thread loads what it moves, the block meets, every thread stores. A few rows of each
// request: bound by the launch and one chain of loads (starts, path, pages, rows). GB300: 24 requests, 4 heads of 256 channels 2.9 us;
// 160 requests in 8 bits, 8 heads of 128, 3.4.
#include "tl_internal.cuh"

#include "tree.cuh"

namespace tl {
namespace {

constexpr int kThreads = 256;
constexpr int kColumns = 32;                                             // 16-byte columns of a block
constexpr int kMoves = TL_TREE_NODES - 1;                                // node 0 stays
constexpr int kItems = (kMoves * kColumns + kThreads - 1) / kThreads;

__global__ void __launch_bounds__(kThreads) kv_compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int64_t s_from[TL_TREE_NODES], s_to[TL_TREE_NODES];
  __shared__ int s_moves;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  pdl_wait_prior();
  pdl_launch_dependents();
  if (tid < 32) {            // one warp looks the moves up, two places to a lane
    const int len = __ldg(p.lens + b), count = __ldg(p.counts + b);
    int begin, n, moves = 0;
    bool bad = !tree_rows(p.starts, b, p.T, begin, n) || count < 0 || count > n || len < 0 || len > p.capacity - n;
    int node[2] = {-1, -1}, before[2];
    if (!bad) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < count) node[h] = __ldg(p.path + begin + lane + 32 * h);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) before[h] = __shfl_up_sync(0xffffffffu, node[h], 1);
    const int last = __shfl_sync(0xffffffffu, node[0], 31);
    if (lane == 0) before[0] = -1, before[1] = last;
    int64_t from[2], to[2];
    bool moved[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 32 * h;
      const bool there = !bad && j < count;
      if (there && (node[h] <= before[h] || node[h] >= n)) bad = true;
      moved[h] = there && !bad && node[h] != j;      // (increasing from -1 on: node[h] >= j)
      from[h] = to[h] = 0;
      if (moved[h]) {
        const int a = len + node[h], z = len + j, pa = a / p.page_size, pz = z / p.page_size;
        const int page_a = __ldg(p.pages + b * p.ldp + pa), page_z = __ldg(p.pages + b * p.ldp + pz);
        if (static_cast<unsigned>(page_a) >= static_cast<unsigned>(p.num_pages) ||
            static_cast<unsigned>(page_z) >= static_cast<unsigned>(p.num_pages))
          bad = true;
        from[h] = page_a * p.page_stride + (a - pa * p.page_size) * p.token_stride;
        to[h] = page_z * p.page_stride + (z - pz * p.page_size) * p.token_stride;
      }
    }
    if (__any_sync(0xffffffffu, bad)) {
      if (lane == 0 && blockIdx.y == 0) set_status(p.status, TL_EDATA);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned who = __ballot_sync(0xffffffffu, moved[h]);
        const int at = moves + __popc(who & ((1u << lane) - 1));
        if (moved[h]) s_from[at] = from[h], s_to[at] = to[h];
        moves += __popc(who);
      }
    }
    if (lane == 0) s_moves = moves;
  }
  __syncthreads();
  const int moves = s_moves;
  if (moves == 0) return;
  // columns: K's heads, then V's
  const int64_t column = static_cast<int64_t>(blockIdx.y) * kColumns + tid % kColumns, half = static_cast<int64_t>(p.kv_heads) * p.row;
  const bool live = column < 2 * half;
  const int64_t c = column < half ? column : column - half;
  uint8_t* const at = (column < half ? p.k : p.v) + c / p.row * p.head_stride + c % p.row * 16;
  uint4 x[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int move = i * (kThreads / kColumns) + tid / kColumns;
    if (live && move < moves) x[i] = *reinterpret_cast<const uint4*>(at + s_from[move]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int move = i * (kThreads / kColumns) + tid / kColumns;
    if (live && move < moves) *reinterpret_cast<uint4*>(at + s_to[move]) = x[i];
  }
}

}  // namespace

cudaError_t launch_kv_compact(const CompactParams& p, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(p.B), static_cast<unsigned>((2ll * p.kv_heads * p.row + kColumns - 1) / kColumns));
  return launch_pdl(kv_compact_kernel, grid, dim3(kThreads), 0, st, p);
}

}  // namespace tl
