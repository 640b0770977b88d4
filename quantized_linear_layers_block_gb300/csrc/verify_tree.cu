// Which drafted tokens hold against the target's probabilities, and the token after them.
//
// The walk is a handful of comparisons of single probabilities; what costs are the rows: where a child is refused the
// rest max(R - S q, 0) is needed as a sum (for the next child) or as a distribution to draw from (at the end), and
// where the walk ends after an accepted node, that node's row. A cluster of blocks takes a request, each block
// a part of the vocabulary. All blocks read the nodes' few probabilities, walk alike, and meet only
// in a pass over a row. R is not kept: it is worked out again, element by element, from p, q and the sums so
// far, so a pass after the first comes from L2 and any vocabulary fits.
//
// A token drawn at random has to be the one of the definition, wherever the number falls: sums in 32 bits would move the borders of
// a hundred thousand tokens. Probabilities are taken as multiples of 2^-60 in 64-bit integers, which holds what fp32 holds
// above 2^-37 exactly; sums and differences of them are exact, whatever their order, and 64-bit adds
// cost two instructions where GB300's FP64 units would bound the pass (2 a clock and SM).
#include "tl_internal.cuh"

#include "tree.cuh"

namespace tl {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBits = 60;
using u64 = unsigned long long;
constexpr u64 kOne = 1ull << kBits;

// A probability in units of 2^-60, rounded down; NaN and below 0 as 0, above 1 as 1.
__device__ __forceinline__ u64 fixed(float x) {
  if (!(x > 0.f)) return 0;
  const unsigned bits = __float_as_uint(fminf(x, 1.f));
  const int e = static_cast<int>(bits >> 23) - (127 + 23 - kBits);      // x = m 2^(e - 60)
  const u64 m = (bits & 0x7FFFFFu) | 0x800000u;
  return e >= 0 ? m << e : e > -24 ? m >> -e : 0;                       // (a subnormal is far below)
}

// s q in units of 2^-60, rounded down
__device__ __forceinline__ u64 times(u64 s, u64 q) { return __umul64hi(s << 2, q << 2); }

__device__ __forceinline__ float unit(float u) { return !(u > 0.f) ? 0.f : fminf(u, 1.f - 0x1p-24f); }

struct Node {
  int parent, token;
  float u, p, q;
};

struct Shared {
  Node node[TL_TREE_NODES];
  u64 sum[TL_TREE_NODES + 1];            // S of each refusal at the node where the walk stands
  int token[TL_TREE_NODES];              // the tokens refused there
  u64 warp_sum[kWarps];
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

  // of tokens x .. x + 3, x = 4 j - shift
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

__global__ void __launch_bounds__(kThreads, 2) verify_tree_kernel(const __grid_constant__ VerifyParams p, const int blocks) {
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
    x.u = unit(__ldg(p.uniform + begin + tid));
    x.p = x.q = 0.f;
    if (x.parent < -1 || x.parent >= tid || static_cast<unsigned>(x.token) >= static_cast<unsigned>(p.vocab)) {
      if (rank == 0) set_status(p.status, TL_EDATA);
      x.parent = -1;                                 // never reached
    }
    if (x.parent >= 0) {
      x.p = __ldg(p.target + static_cast<int64_t>(begin + x.parent) * p.ldt + x.token);
      x.q = p.draft == nullptr ? 1.f : __ldg(p.draft + static_cast<int64_t>(begin + x.parent) * p.ldd + x.token);
    }
    s.node[tid] = x;
  }
  __syncthreads();
  if (blocks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");      // all blocks run: their memory may be written

  int at = 0, refused = 0, known = 1, count = 1, turn = 0;
  u64 total = 0, before = 0;                         // of the last pass: the whole sum, and that of the blocks before this one
  if (tid == 0) {
    s.sum[0] = kOne;
    if (rank == 0) p.path[begin] = 0;
  }
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
    u64 sum = 0;
    constexpr int U = 4;
    for (int i0 = 0; i0 < steps; i0 += U) {
      float pf[U][4], qf[U][4];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int x = first + (i0 + i) * 128 + 4 * lane;
        if (i0 + i < steps && x < p.vocab) {
          rest.load(rest.p, x, pf[i]);
          if (rest.refused > 0 && rest.q != nullptr) rest.load(rest.q, x, qf[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int x = first + (i0 + i) * 128 + 4 * lane;
        if (i0 + i < steps && x < p.vocab) {
          u64 r[4];
          rest.take(s, x, pf[i], qf[i], r);
          sum += (r[0] + r[1]) + (r[2] + r[3]);
        }
      }
    }
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

  for (int i = 1; i < n; ++i) {
    const Node c = s.node[i];
    if (c.parent != at) continue;
    while (known <= refused) {                       // a sibling was refused: what it left, as a sum
      const int all = refused;
      refused = known;
      pass();
      refused = all;
      if (tid == 0) s.sum[known] = total;
      __syncthreads();
      ++known;
    }
    u64 r = fixed(c.p);
    const u64 q = fixed(c.q);
    for (int k = 0; k < refused; ++k) {
      const u64 less = p.draft == nullptr ? (s.token[k] == c.token ? r : 0) : k == 0 ? q : times(s.sum[k], q);
      r = r > less ? r - less : 0;
    }
    // u q S < R; for the first child both sides as they were given, exactly
    const bool taken = refused == 0 ? static_cast<double>(c.u) * static_cast<double>(c.q) < static_cast<double>(c.p)
                                    : static_cast<double>(c.u) * static_cast<double>(c.q) * static_cast<double>(s.sum[refused]) < static_cast<double>(r);
    __syncthreads();
    if (taken) {
      at = i, refused = 0, known = 1;
      if (rank == 0 && tid == 0) p.path[begin + count] = i;
      ++count;
    } else {
      if (tid == 0) s.token[refused] = c.token;
      ++refused;
      __syncthreads();
    }
  }
  while (known < refused) {
    const int all = refused;
    refused = known;
    pass();
    refused = all;
    if (tid == 0) s.sum[known] = total;
    __syncthreads();
    ++known;
  }
  pass();
  if (total == 0 && refused > 0) {                   // the draft left nothing: the target's own
    refused = 0;
    pass();
  }
  if (rank == 0) {
    if (tid == 0) p.counts[b] = count;
    for (int j = count + tid; j < n; j += kThreads) p.path[begin + j] = -1;
  }
  // the smallest x with sum_{y <= x} R(y) > u sum R: floor(u sum R) in units of 2^-60
  const u64 goal = __umul64hi(total << 1, static_cast<u64>(static_cast<double>(s.node[0].u) * 0x1p63));
  const u64 inside = goal - before;                  // of this block's part, if it lies there
  if (total > 0 && goal >= before) {
    u64 run = 0;
    int w = 0;
    for (; w < kWarps; ++w) {
      const u64 x = s.warp_sum[w];
      if (inside < run + x) break;
      run += x;
    }
    if (w == warp) {                                 // one warp of the cluster
      u64 need = inside - run;
      for (int i = 0; i < steps; ++i) {
        const int x = first + i * 128 + 4 * lane;
        u64 r[4] = {0, 0, 0, 0};
        if (x < p.vocab) {
          float pf[4], qf[4] = {0.f, 0.f, 0.f, 0.f};
          rest.load(rest.p, x, pf);
          if (rest.refused > 0 && rest.q != nullptr) rest.load(rest.q, x, qf);
          rest.take(s, x, pf, qf, r);
        }
        const u64 mine = (r[0] + r[1]) + (r[2] + r[3]);
        u64 incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const unsigned who = __ballot_sync(0xffffffffu, incl > need);
        if (who != 0) {
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
          break;
        }
        need -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  }
  if (blocks > 1) cluster_sync();                    // no block leaves while another writes its sum here
}

}  // namespace

cudaError_t launch_verify_tree(const VerifyParams& p, int sms, cudaStream_t st) {
  // As many blocks to a request as run at once, two to an SM, while each warp has 128 tokens at least.
  int blocks = 8;
  while (blocks > 1 && (static_cast<long long>(p.B) * blocks > 2ll * sms || p.vocab < blocks * kWarps * 128)) blocks >>= 1;
  return launch_pdl_cluster(verify_tree_kernel, dim3(static_cast<unsigned>(p.B) * blocks), dim3(kThreads), 0, st, blocks, p, blocks);
}

}  // namespace tl
