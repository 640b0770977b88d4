// Which drafted tokens hold against the target's probabilities, and the token after them.
//
// The walk is a handful of comparisons of single probabilities; what costs are the rows: where a child is refused the
// rest max(R - S q, 0) is needed as a sum (for the next child) or as a distribution to draw from (at the end), and
// where the walk ends after an accepted node, that node's row. A cluster of blocks takes a request, each block
// a part of the vocabulary. All blocks read the nodes' few probabilities, walk alike, and meet only
// in a pass over a row. Most of these are not needed: R(x) = 0 refuses and u q S' < R(x), S' an
// upper bound of S, accepts without S; chosen tokens take their own probability from S and no more. R is not kept: it is worked out again, element by element, from p, q and the sums so
// far, so a pass after the first comes from L2 and any vocabulary fits.
//
// A token drawn at random has to be the one of the definition, wherever the number falls: sums in 32 bits would move the borders of
// a hundred thousand tokens, GB300's FP64 units do 2 operations a clock and SM, and 64-bit integers cost 60 instructions a
// probability (64 requests, 100001 tokens: 211 us). So a thread sums its share as a pair of floats, the sum and what its
// roundings lost (about 48 bits, a dozen fp32 operations an element), and the threads' sums meet as 64-bit integers in units of 2^-60.
//
// GB300: those 64 requests 50 to 57 us by their numbers (rows once from HBM: 8; the request with most refusals makes several passes, one
// after the other, of some 8 us, of L2's throughput 8 %), chosen tokens 28; a chain of 8 with 131072 tokens 8.5, chosen 7.8.
#include "tl_internal.cuh"

#include "tree.cuh"

namespace tl {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBits = 60;
using u64 = unsigned long long;
constexpr u64 kOne = 1ull << kBits;

// A probability in units of 2^-60, rounded down; NaN and below 0 as 0, above 1 as 1.
__device__ __forceinline__ u64 fixed(float x) { return __float2ull_rz(__saturatef(x) * 0x1p60f); }

// s q in units of 2^-60, rounded down
__device__ __forceinline__ u64 times(u64 s, u64 q) { return __umul64hi(s << 2, q << 2); }

__device__ __forceinline__ float unit(float u) { return !(u > 0.f) ? 0.f : fminf(u, 1.f - 0x1p-24f); }

__device__ __forceinline__ float2 less(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }

// Two sums of floats and what their roundings lost.
struct Pair {
  float2 s = {0.f, 0.f}, c = {0.f, 0.f};
  __device__ __forceinline__ void add(float2 x, float2 low) {
    const float2 t = __fadd2_rn(s, x), b = less(t, s);
    c = __fadd2_rn(c, __fadd2_rn(low, __fadd2_rn(less(s, less(t, b)), less(x, b))));
    s = t;
  }
  // in units of 2^-60, at least 0
  __device__ __forceinline__ u64 units() const {
    const long long x = __float2ll_rz(s.x * 0x1p60f) + __float2ll_rz(c.x * 0x1p60f) + __float2ll_rz(s.y * 0x1p60f) + __float2ll_rz(c.y * 0x1p60f);
    return x > 0 ? x : 0;
  }
};

// What the walk has to know of a node, worked out by a thread for each: its probabilities, u q, and whether it is taken as a first child.
struct Node {
  int parent, token;
  u64 p, q, need;
  bool first;
};

// A row of target sums to no more than this: what a refusal leaves, too.
constexpr u64 kMost = kOne + (kOne >> 8);

// a b < c for numbers in [0, 1], exactly: the product's rounding error decides where the rounded product is c. All by powers of two as
// large, by which no product that comes near c > 0, nor its error, is subnormal.
__device__ __forceinline__ bool product_below(float a, float b, float c) {
  a *= 0x1p60f, b *= 0x1p60f, c *= 0x1p120f;
  const float h = __fmul_rn(a, b);
  return h < c || (h == c && __fmaf_rn(a, b, -h) < 0.f);
}

struct Shared {
  Node node[TL_TREE_NODES];
  u64 sum[TL_TREE_NODES + 1];            // S of each refusal at the node where the walk stands
  float2 pair[TL_TREE_NODES + 1];        // the same as two floats
  int token[TL_TREE_NODES];              // the tokens refused there; -1: one outside the vocabulary
  u64 warp_sum[kWarps], step_sum[kWarps];
  int step_last[kWarps];
  u64 block_sum[2][kMaxCluster];         // of every block of the cluster, for two passes in turn
};

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t rank, u64 v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote), "l"(v) : "memory");
}

// What is left of a row after `refused` refusals, for four neighbouring tokens.
struct Rest {
  const float* p;
  const float* q;                        // NULL: chosen tokens
  int refused, vocab;
  bool wide;                             // both rows 16-byte aligned from their element -shift on
  int shift;                             // elements of an aligned vector that lie before the row

  __device__ __forceinline__ void load(const float* row, int x, float (&f)[4]) const {
    if (wide && x >= 0 && x + 4 <= vocab) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(row + x));
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = x + i >= 0 && x + i < vocab ? __ldg(row + x + i) : 0.f;
    }
  }

  // r + low becomes at least 0.
  static __device__ __forceinline__ void floor0(float2& r, float2& low) {
    low.x = r.x > 0.f ? low.x : 0.f;
    low.y = r.y > 0.f ? low.y : 0.f;
    r.x = fmaxf(r.x, 0.f);
    r.y = fmaxf(r.y, 0.f);
  }
  // r + low less f b, f being S_k as two floats.
  static __device__ __forceinline__ void further(float2 f, float2 b, float2& r, float2& low) {
    const float2 f1 = make_float2(f.x, f.x), f2 = make_float2(f.y, f.y);
    const float2 h = __fmul2_rn(f1, b), l = __ffma2_rn(f2, b, __ffma2_rn(f1, b, make_float2(-h.x, -h.y)));
    const float2 t = less(r, h), v = less(t, r);
    low = __fadd2_rn(less(low, l), less(less(r, less(t, v)), __fadd2_rn(h, v)));
    r = __fadd2_rn(t, low);
    low = less(low, less(r, t));
    floor0(r, low);
  }

  // The sum of what is left of this lane's tokens: four of each 128 from `first` on.
  template <int KIND>      // 0: nothing was refused; 1: drawn tokens were; 2: chosen ones
  __device__ __forceinline__ u64 sum(const Shared& s, int first, int steps, int lane) const {
    constexpr int U = KIND == 1 ? 2 : 4;
    Pair part;
#pragma unroll 1
    for (int i0 = 0; i0 < steps; i0 += U) {
      float pf[U][4], qf[U][4];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int x = first + (i0 + i) * 128 + 4 * lane;
        const bool here = i0 + i < steps && x < vocab;
#pragma unroll
        for (int e = 0; e < 4; ++e) pf[i][e] = qf[i][e] = 0.f;
        if (here) load(p, x, pf[i]);
        if (KIND == 1 && here) load(q, x, qf[i]);
      }
      float2 r[2 * U], low[2 * U];                      // (NaN saturates to 0)
#pragma unroll
      for (int i = 0; i < 2 * U; ++i) {
        r[i] = make_float2(__saturatef(pf[i / 2][i % 2 * 2]), __saturatef(pf[i / 2][i % 2 * 2 + 1]));
        low[i] = make_float2(0.f, 0.f);
      }
      if constexpr (KIND == 1) {
        float2 b[2 * U];
#pragma unroll
        for (int i = 0; i < 2 * U; ++i) {
          const float2 a = r[i];
          b[i] = make_float2(__saturatef(qf[i / 2][i % 2 * 2]), __saturatef(qf[i / 2][i % 2 * 2 + 1]));
          r[i] = less(a, b[i]);
          low[i] = less(less(a, r[i]), b[i]);           // a - b = r + low where a > b
          floor0(r[i], low[i]);
        }
        // all tokens of a lane side by side: one after the other these chains took three times as long
#pragma unroll 1
        for (int k = 1; k < refused; ++k) {
          const float2 f = s.pair[k];
#pragma unroll
          for (int i = 0; i < 2 * U; ++i) further(f, b[i], r[i], low[i]);
        }
      }
      if constexpr (KIND == 2) {
#pragma unroll 1
        for (int k = 0; k < refused; ++k) {
          const int x = s.token[k] - (first + i0 * 128 + 4 * lane);
#pragma unroll
          for (int i = 0; i < 2 * U; ++i) {
            r[i].x = x == i / 2 * 128 + i % 2 * 2 ? 0.f : r[i].x;
            r[i].y = x == i / 2 * 128 + i % 2 * 2 + 1 ? 0.f : r[i].y;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * U; ++i) part.add(r[i], low[i]);
    }
    return part.units();
  }

  // In units of 2^-60: of tokens x .. x + 3, x = 4 j - shift
  __device__ __forceinline__ void take(const Shared& s, int x, const float (&pf)[4], const float (&qf)[4], u64 (&r)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = fixed(pf[i]);
      if (refused == 0) continue;
      if (q != nullptr) {
        const u64 f = fixed(qf[i]);
        r[i] = r[i] > f ? r[i] - f : 0;
        for (int k = 1; k < refused; ++k) {
          const u64 less = times(s.sum[k], f);
          r[i] = r[i] > less ? r[i] - less : 0;
        }
      } else {
        for (int k = 0; k < refused; ++k)
          if (s.token[k] == x + i) r[i] = 0;
      }
    }
  }
};

// One lane's share of a pass, out of line: a kernel with several copies of it waits for its instructions.
__device__ __noinline__ u64 part_of(const Rest rest, const Shared& s, int first, int steps, int lane) {
  if (rest.refused == 0) return rest.sum<0>(s, first, steps, lane);
  return rest.q != nullptr ? rest.sum<1>(s, first, steps, lane) : rest.sum<2>(s, first, steps, lane);
}

__global__ void __launch_bounds__(kThreads, 4) verify_tree_kernel(const __grid_constant__ VerifyParams p, const int blocks) {
  __shared__ Shared s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / blocks, rank = blockIdx.x - b * blocks;
  pdl_wait_prior();
  pdl_launch_dependents();
  int begin, n;
  const bool ok = tree_rows(p.starts, b, p.T, begin, n);
  if (!ok && tid == 0 && rank == 0) set_status(p.status, TL_EDATA);
  if (b == p.B - 1 && rank == blocks - 1) {          // padding
    const int end = __ldg(p.starts + p.B);
    if (end >= 0)
      for (int64_t t = static_cast<int64_t>(end) + tid; t < p.T; t += kThreads) p.path[t] = -1;
  }
  if (b == 0 && rank == 0 && begin > 0) {            // padding before all requests, in whatever order they are
    int least = min(begin, p.T);
    for (int i = lane; i <= p.B; i += 32) least = min(least, __ldg(p.starts + i));
    least = __reduce_min_sync(0xffffffffu, least);
    for (int t = tid; t < least; t += kThreads) p.path[t] = -1;
  }
  if (n == 0) {                                      // the same for all blocks of the cluster
    if (rank == 0 && tid == 0) p.counts[b] = 0, p.next[b] = -1;
    return;
  }
  if (blocks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (rank == 0 && tid == 0) p.next[b] = p.vocab - 1;                   // what a row gives whose sum is beyond all bounds
  if (tid < n) {
    Node x;
    x.parent = __ldg(p.parents + begin + tid);
    x.token = tid > 0 ? __ldg(p.tokens + begin + tid) : 0;
    const float u = unit(__ldg(p.uniform + begin + tid));
    float a = 0.f, b = 0.f;
    const bool bad = x.parent < -1 || x.parent >= tid, there = static_cast<unsigned>(x.token) < static_cast<unsigned>(p.vocab);
    if ((bad || !there) && rank == 0) set_status(p.status, TL_EDATA);
    if (bad) x.parent = -1;                          // never reached
    if (!there) x.token = -1;                        // refused: neither distribution gives it any probability
    if (x.parent >= 0 && there) {
      a = __ldg(p.target + static_cast<int64_t>(begin + x.parent) * p.ldt + x.token);
      b = p.draft == nullptr ? 1.f : __ldg(p.draft + static_cast<int64_t>(begin + x.parent) * p.ldd + x.token);
    }
    a = __saturatef(a), b = __saturatef(b);          // below 0 and NaN count as 0, above 1 as 1: here as in the sums
    x.p = fixed(a), x.q = fixed(b), x.first = product_below(u, b, a);
    x.need = tid == 0 ? fixed(u) : times(fixed(u), x.q);
    s.node[tid] = x;
  }
  __syncthreads();
  if (blocks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");      // all blocks run: their memory may be written

  int at = 0, refused = 0, known = 0, count = 1, turn = 0;      // known: S_1 .. S_known of the refusals here are in s.sum
  u64 total = 0, before = 0;                         // of the last pass: the whole sum, and that of the blocks before this one
  if (rank == 0 && tid == 0) p.path[begin] = 0;
  // a pass over what is left of the row at `at`: this warp's part of the vocabulary, neighbours in order
  Rest rest;
  int first, steps;
  auto aim = [&]() {
    rest.p = p.target + static_cast<int64_t>(begin + at) * p.ldt;
    rest.q = p.draft == nullptr ? nullptr : p.draft + static_cast<int64_t>(begin + at) * p.ldd;
    rest.refused = refused, rest.vocab = p.vocab;
    rest.shift = static_cast<int>(reinterpret_cast<uintptr_t>(rest.p) >> 2) & 3;
    rest.wide = rest.q == nullptr || (static_cast<int>(reinterpret_cast<uintptr_t>(rest.q) >> 2) & 3) == rest.shift;
    const int vectors = (p.vocab + rest.shift + 3) / 4, parts = blocks * kWarps;
    steps = ((vectors + parts - 1) / parts + 31) / 32;
    first = (rank * kWarps + warp) * steps * 128 - rest.shift;
  };
  auto pass = [&]() {
    aim();
    u64 sum = part_of(rest, s, first, steps, lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s.warp_sum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      u64 mine = lane < kWarps ? s.warp_sum[lane] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
      if (blocks == 1) {
        if (lane == 0) s.block_sum[turn][0] = mine;
      } else if (lane < blocks) {
        st_cluster(smem_u32(&s.block_sum[turn][rank]), lane, mine);
      }
    }
    if (blocks > 1)
      cluster_sync();
    else
      __syncthreads();
    total = before = 0;
    for (int i = 0; i < blocks; ++i) {
      const u64 x = s.block_sum[turn][i];
      if (i < rank) before += x;
      total += x;
    }
    turn ^= 1;
  };

  // S_1 .. S_k of the node where the walk stands
  auto know = [&](int k) {
    while (known < k) {
      u64 next;
      if (p.draft == nullptr && known > 0) {         // the token that was refused takes its own with it, unless it was refused before
        const int x = s.token[known];
        bool again = false;
        for (int j = 0; j < known; ++j) again |= s.token[j] == x;
        next = s.sum[known] - (again || x < 0 ? 0 : fixed(__ldg(p.target + static_cast<int64_t>(begin + at) * p.ldt + x)));
      } else {
        const int all = refused;
        refused = known + 1;
        pass();
        refused = all;
        next = total;
      }
      ++known;
      if (tid == 0) {
        const float h = __ull2float_rz(next);
        s.sum[known] = next;
        s.pair[known] = make_float2(h * 0x1p-60f, __ull2float_rz(next - static_cast<u64>(h)) * 0x1p-60f);
      }
      __syncthreads();
    }
  };
  for (int i = 1; i < n; ++i) {
    const Node& c = s.node[i];
    if (c.parent != at) continue;
    bool taken = c.first;
    if (refused > 0) {
      u64 r = c.p;
      if (p.draft == nullptr) {
        for (int k = 0; k < refused; ++k)
          if (s.token[k] == c.token) r = 0;
      } else {
        r = r > c.q ? r - c.q : 0;
        if (r > 0) know(refused - 1);
        for (int k = 1; k < refused && r > 0; ++k) {
          const u64 less = times(s.sum[k], c.q);
          r = r > less ? r - less : 0;
        }
      }
      taken = r > 0 && times(known > 0 ? s.sum[known] : kMost, c.need) < r;
      if (r > 0 && !taken) {
        know(refused);
        taken = times(s.sum[refused], c.need) < r;
      }
    }
    if (taken) {
      at = i, refused = 0, known = 0;
      if (rank == 0 && tid == 0) p.path[begin + count] = i;
      ++count;
    } else {
      __syncthreads();
      if (tid == 0) s.token[refused] = c.token;
      ++refused;
      __syncthreads();
    }
  }
  if (p.draft != nullptr) know(refused - 1);
  for (;;) {
    pass();
    if (total != 0 || refused == 0) break;
    refused = 0;                                     // the draft left nothing: the target's own
  }
  if (rank == 0) {
    if (tid == 0) p.counts[b] = count;
    for (int j = count + tid; j < n; j += kThreads) p.path[begin + j] = -1;
  }
  // the smallest x with sum_{y <= x} R(y) > u sum R: floor(u sum R) in units of 2^-60
  const u64 goal = times(total, s.node[0].need);
  const u64 inside = goal - before;                  // of this block's part, if it lies there
  if (total > 0 && goal >= before && inside < s.block_sum[turn ^ 1][rank]) {      // one block of the cluster
    u64 run = 0;
    int w = 0;
    while (w < kWarps - 1 && inside >= run + s.warp_sum[w]) run += s.warp_sum[w++];
    // that warp's part once more, 128 tokens to a warp: first their sums, then within them
    const int start = first + (w - warp) * steps * 128;
    int found = -1, last = -1;                       // (the sums of a pass and these may differ in their last bits)
    u64 need = inside - run;
    for (int i0 = 0; i0 < steps && found < 0; i0 += kWarps) {
      const int x = start + (i0 + warp) * 128 + 4 * lane;
      float pf[4] = {0.f, 0.f, 0.f, 0.f}, qf[4] = {0.f, 0.f, 0.f, 0.f};
      if (i0 + warp < steps && x < p.vocab) {
        rest.load(rest.p, x, pf);
        if (rest.refused > 0 && rest.q != nullptr) rest.load(rest.q, x, qf);
      }
      u64 r[4];
      rest.take(s, x, pf, qf, r);
      const u64 mine = (r[0] + r[1]) + (r[2] + r[3]);
      u64 incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      int top = -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) top = r[k] > 0 ? x + k : top;
      top = __reduce_max_sync(0xffffffffu, top);
      __syncthreads();                               // (what the turn before left has been read)
      if (lane == 31) s.step_sum[warp] = incl;
      if (lane == 0) s.step_last[warp] = top;
      __syncthreads();
      for (int v = 0; v < kWarps && found < 0; ++v) {
        last = max(last, s.step_last[v]);
        if (need < s.step_sum[v]) found = v;
        else need -= s.step_sum[v];
      }
      if (found == warp) {
        const unsigned who = __ballot_sync(0xffffffffu, incl > need);
        if (lane == __ffs(who) - 1) {
          u64 sum = incl - mine;
          int k = 0;
#pragma unroll
          for (; k < 3; ++k) {
            sum += r[k];
            if (sum > need) break;
          }
          p.next[b] = x + k;
        }
      }
    }
    if (found < 0 && last >= 0 && tid == 0) p.next[b] = last;
  }
  if (blocks > 1) cluster_sync();                    // no block leaves while another writes its sum here
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyParams& p, int sms, cudaStream_t st) {
  // As many blocks to a request as run at once, four to an SM, while each warp has 128 tokens at least.
  int blocks = kMaxCluster;
  while (blocks > 1 && (static_cast<long long>(p.B) * blocks > 4ll * sms || p.vocab < blocks * kWarps * 128)) blocks >>= 1;
  static int ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE) == 0) {
    e = cudaFuncSetAttribute(verify_tree_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
  }
  return launch_pdl_cluster(verify_tree_kernel, dim3(static_cast<unsigned>(p.B) * blocks), dim3(kThreads), 0, st, blocks, p, blocks);
}

}  // namespace tl
