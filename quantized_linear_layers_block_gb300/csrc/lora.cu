// Low-rank adapters of many requests beside a projection:
//   y[m] = base[m] + scale[a] B[a] (A[a] x[m]),  a = ids[m].
//
// A plan kernel sorts the tokens by adapter once per step; an item is up to 16 or 32
// tokens of one adapter, so an adapter's matrices are read once per item,
// by however many tokens use it. One kernel does both products: a cluster of blocks takes an item.
//
// First h = A x: the rank is small and K long, so K is cut over all warps of the cluster, whose sums meet through
// distributed shared memory in a fixed order; h never goes to memory. The adapter's rows are the 16
// rows of the MMA, 8 of the item's tokens its columns. Nothing is used twice but through registers, so
// the operands come straight from global memory: with the K axis permuted alike on both sides
// (thread t of a quad takes the 8 consecutive elements 8t .. 8t + 7 of 32) every load is 16 bytes.
//
// Then y = base + scale B h: every block has h and takes its part of the columns. Tokens are the rows of the MMA, the
// columns of B are permuted so that a thread ends with 8 of a token, in 16-byte pieces side by side with its
// quad's: loads of base and stores of y, whose bytes bound the kernel for many tokens. h is scaled by a
// power of two of its own per token (the f16 range) and split in 16-bit parts, so that it keeps 16 bits or more.
//
// A few items leave most SMs idle, and the expansion long: then several clusters take
// an item's columns, and each forms h for itself (its A is in L2 by then).
//
// Measured on GB300: 4096 tokens, rank 16, K = 5120, N = 34816, bf16: 102 us, 6.05 TB/s, 0.89 of the copy rate (two kernels
// with h in memory: 169 us). 515 tokens, rank 64, K = 17408, N = 5120, fp32 out: 19.7 us, of which the first
// product takes 6 (96 MB of x and A per item into the SMs, 83 B/ns each), the second 3 and the chain
// around them (plan, sums, meetings of the cluster, parts) the rest. 48 tokens of 32 adapters, rank 32, K = N = 5120:
// 7.6 us; one token, rank 16, N = 17408: 5.2 us, all of it that chain. 4096 tokens, rank 128, K = 5120, N = 17408: 148 us,
// where the bytes take 52 and the MMAs of both parts 69. The plan, once per step: 2.8 us for one token, 3.1 for 48, 5.5 for
// 515, 24 for 4096 (one block, whose warps take turns: 6 us per 1024 tokens).
#include "lora.cuh"
#include "tl_internal.cuh"

#include <algorithm>

#include <cuda_bf16.h>

namespace tl {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kLoraWarps = 8;
constexpr int kLoraMaxCluster = 16;

// ----------------------------------------------------------------- plan
// Shared memory: for each adapter, and for the tokens without one, a counter and its first item.
__global__ void __launch_bounds__(kPlanThreads)
lora_plan_kernel(const int32_t* __restrict__ ids, int M, int n, int tile, LoraPlanHeader* head, LoraItem* items, int* status) {
  extern __shared__ int next[];
  int* const first = next + n + 1;
  __shared__ int s_items[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait_prior();
  for (int i = tid; i <= n; i += kPlanThreads) next[i] = 0;
  __syncthreads();
  auto bin = [&](int id) { return id >= 0 && id < n ? id : n; };
  for (int i = tid; i < M; i += kPlanThreads) {
    const int id = __ldg(ids + i);
    if (id >= n) set_status(status, TL_EDATA);
    atomicAdd(next + bin(id), 1);
  }
  __syncthreads();
  // exclusive sum of the items over the bins; a thread owns consecutive bins
  const int per = (n + kPlanThreads) / kPlanThreads;
  int tiles = 0;
  for (int i = tid * per; i < min(n + 1, (tid + 1) * per); ++i) tiles += (next[i] + tile - 1) / tile;
  int incl = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_items[warp] = incl;
  __syncthreads();
  int item = incl - tiles, all = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) item += s_items[w];
    all += s_items[w];
  }
  for (int i = tid * per; i < min(n + 1, (tid + 1) * per); ++i) {
    const int c = next[i];
    next[i] = 0;
    first[i] = item;
    for (int k = 0; k < c; k += tile, ++item) {
      items[item].adapter = i < n ? i : -1;
      items[item].count = min(tile, c - k);
    }
  }
  if (tid == 0) *head = LoraPlanHeader{M, n, all, 0};
  __syncthreads();
  // places, in the order of the tokens: the warps of each round take their turns
  for (int base = 0; base < M; base += kPlanThreads) {
    const int i = base + tid;
    const int b = i < M ? bin(__ldg(ids + i)) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, b);
    const int leader = __ffs(same) - 1, rank = __popc(same & ((1u << lane) - 1));
    for (int w = 0; w < kPlanThreads / 32 && base + 32 * w < M; ++w) {
      if (w == warp) {
        int at = 0;
        if (lane == leader && b >= 0) {
          at = next[b];
          next[b] = at + __popc(same);
        }
        at = __shfl_sync(0xffffffffu, at, leader) + rank;
        if (b >= 0) items[first[b] + at / tile].token[at % tile] = i;
      }
      __syncthreads();
    }
  }
}

// ----------------------------------------------------------------- common
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t rank, uint32_t v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, uint32_t rank, uint32_t a, uint32_t b) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(remote), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// base + up d of two 16-bit values; `up` is a power of two, so the fused product is exact
template <int YD>
__device__ __forceinline__ uint32_t add2(uint32_t base, float lo, float hi, float up) {
  uint32_t r;
  if constexpr (YD == TL_BF16) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
        : "=r"(r)
        : "f"(__fmaf_rn(hi, up, __uint_as_float(base & 0xFFFF0000u))), "f"(__fmaf_rn(lo, up, __uint_as_float(base << 16))));
  } else {
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&base));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__fmaf_rn(hi, up, b.y)), "f"(__fmaf_rn(lo, up, b.x)));
  }
  return r;
}

// ----------------------------------------------------------------- the operator
// Both products stream their operands through rings of cp.async slots in shared memory, each written and
// read by one thread only, so that no barrier is needed; registers could not hold enough bytes in flight
// (4096 tokens: 134 us with operands a step ahead in registers). A stage of the first ring is a whole K step: finer
// stages keep more bytes on their way and took longer, by their own instructions.
// Shared memory: the first product's ring [RS][slots][threads], then in its place
// the warps' sums, then the second product's ring [YS][slots][threads]. Behind the larger of these two h's sums
// [TILE][RP] in fp32, RP the rank rounded up to 16 (RT = 1) or a multiple of 32, and the parts of h [PARTS][TILE][RP + 8].
// A rank above 64 is cut over the two halves of the warps, which share K among four then.
template <bool BF16, int YD, int RT, int TILE>
struct Lora {
  // A third part where the bits of two, 16 of bf16, would be the largest error of an fp32 y. Two of fp16 give 22, and fp32 sums over
  // K and the rank err by about as much (515 tokens, rank 64: 3.9e-7 of y, 3.6e-7 in plain fp32); a third one would
  // cost 5 % there (19.7 to 20.7 us) and 20 % at 4096 tokens and rank 128 (168 to 201 us).
  static constexpr int PARTS = YD == TL_F32 && BF16 ? 3 : 2;
  static constexpr int V = YD == TL_F32 ? 2 : 1;                // 16-byte vectors of 8 columns
  static constexpr int ROWS = 16 * RT, RPITCH = ROWS + 4;
  static constexpr int THREADS = kLoraWarps * 32, VEC = THREADS * 16;
  static constexpr int SLOTS = 2 * RT + TILE / 8, RS = RT == 4 ? 2 : RT == 2 && TILE == 32 ? 3 : 4, RING = RS * SLOTS * VEC;
  // The second product's ring. Up to rank 16, a thread's part of B is 8 bytes a row and goes to registers, one group
  // ahead (8-byte slots in the ring: 4096 tokens 112 us instead of 103); above, B has stages of its own.
  static constexpr bool REG_B = RT == 1;
  static constexpr int BASES = V == 1 ? TILE / 8 : 4;          // vectors of base in a stage
  static constexpr int YSLOTS = REG_B ? BASES : 4;
  static constexpr int YS = REG_B ? 16 / YSLOTS : RT == 2 ? 6 : 4, YSTAGE = YSLOTS * VEC, YRING = YS * YSTAGE;
  static constexpr int RED = kLoraWarps * TILE * RPITCH * 4;
  static constexpr int AREA = RED > YRING ? RED : YRING;
  static_assert(YRING <= RING, "layout");
  // the K of the second product: one MMA for ranks up to 16, else pairs of them
  static constexpr int KSTEP = RT == 1 ? 16 : 32;
  __host__ __device__ static int padded(int rank) { return (rank + KSTEP - 1) / KSTEP * KSTEP; }
  static constexpr bool SHARED = RT == 4;        // each block sums some tokens for all
  __host__ __device__ static int hs_at(int rank) { return AREA + TILE * padded(rank) * 4; }
  static int smem(int rank) {
    const int hs = hs_at(rank) + PARTS * TILE * (padded(rank) + 8) * 2;
    return hs > RING ? hs : RING;
  }
};

// blockIdx.x = (item * NS + part of the columns) * CS + rank of the block in its cluster
template <bool BF16, int YD, int RT, int TILE>
__global__ void __launch_bounds__(kLoraWarps * 32, 2) lora_kernel(const __grid_constant__ LoraParams p, int CS, int NS) {
  using L = Lora<BF16, YD, RT, TILE>;
  constexpr int NT = TILE / 8, V = L::V, ROWS = L::ROWS;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float s_up[TILE];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int me = blockIdx.x % CS, part = blockIdx.x / CS % NS, idx = blockIdx.x / CS / NS;
  const int RP = L::padded(p.rank);
  const int PITCH = RP + 8;
  float* const sum = reinterpret_cast<float*>(smem + L::AREA);
  float* const red = reinterpret_cast<float*>(smem);
  uint16_t* const hs = reinterpret_cast<uint16_t*>(smem + L::hs_at(p.rank));
  const uint32_t slot0 = smem_u32(smem) + tid * 16;
  // No early start for the next kernel: its clusters would be placed where the first SMs fall free, two blocks
  // on some and none on others (515 tokens of rank 64, calls back to back: 29 us with it, 22 without).
  pdl_wait_prior();
  const LoraPlanHeader head = *p.plan;
  const LoraItem* const item = p.items + idx;
  int adapter, count, tok[NT];
  auto read_item = [&]() {
    adapter = item->adapter;
    count = item->count;
#pragma unroll
    for (int n = 0; n < NT; ++n) tok[n] = item->token[8 * n + g];
  };
  // Every plan has a first item, which is read beside the header; another one's place may lie past the end of a plan of
  // fewer tokens or adapters, so the header is asked first.
  if (idx == 0) read_item();
  if (head.M != p.M || head.n_adapters != p.n_adapters) {
    if (tid == 0) set_status(p.status, TL_EDATA);
    return;
  }
  if (idx >= head.items) return;                                          // whole clusters leave
  if (idx > 0) read_item();
  if (adapter < 0 && !p.copy_bare) return;
#pragma unroll
  for (int n = 0; n < NT; ++n)
    if (8 * n + g >= count) tok[n] = -1;

  const int steps = adapter < 0 ? 0 : RP / L::KSTEP;
  if (steps > 0) {
    // ---- h = A x
    const bool two = RT == 4 && p.rank > ROWS;                                    // the upper warps take ranks 64 and up
    const int per_block = two ? kLoraWarps / 2 : kLoraWarps, r0 = two ? warp / (kLoraWarps / 2) * ROWS : 0;
    const int chunks = (p.K + 31) / 32, workers = CS * per_block, worker = me * per_block + (warp & (per_block - 1));
    const int c0 = static_cast<int>(static_cast<long long>(chunks) * worker / workers);
    const int c1 = static_cast<int>(static_cast<long long>(chunks) * (worker + 1) / workers);
    const uint16_t* xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xr[n] = p.x + (tok[n] >= 0 ? tok[n] * p.ldx : 0) + 8 * t;
    const int nts = (count + 7) / 8;
    const uint16_t* const ar = p.A + (static_cast<int64_t>(adapter) * p.rank + r0 + g) * p.K + 8 * t;
    float acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
    auto ask = [&](int c) {
      if (c < c1) {
        const int k = 32 * c;
        const bool in = k + 8 * t < p.K;
        const uint32_t dst = slot0 + (c - c0) % L::RS * (L::SLOTS * L::VEC);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool row = in && r0 + 16 * i + 8 * e + g < p.rank;
            cp_async16(dst + (2 * i + e) * L::VEC, row ? ar + static_cast<int64_t>(16 * i + 8 * e) * p.K + k : p.A, row ? 16 : 0);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const bool row = in && tok[n] >= 0;
          if (n < nts) cp_async16(dst + (2 * RT + n) * L::VEC, row ? xr[n] + k : p.x, row ? 16 : 0);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int c = 0; c < L::RS - 1; ++c) ask(c0 + c);
    for (int c = c0; c < c1; ++c) {
      cp_async_wait<L::RS - 2>();
      ask(c + L::RS - 1);                      // the slots that the last turn read
      const uint32_t src = slot0 + (c - c0) % L::RS * (L::SLOTS * L::VEC);
      uint4 a[RT][2];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) a[i][e] = ld_shared16(src + (2 * i + e) * L::VEC);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n < nts) {
          const uint4 b = ld_shared16(src + (2 * RT + n) * L::VEC);
#pragma unroll
          for (int i = 0; i < RT; ++i) mma16816<BF16>(acc[i][n], a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y, b.x, b.y);
#pragma unroll
          for (int i = 0; i < RT; ++i) mma16816<BF16>(acc[i][n], a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w, b.z, b.w);
        }
      }
    }
    // the warps' sums
    __syncthreads();                             // the rings have been read
    float* const mine = red + warp * TILE * L::RPITCH + g;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n < nts) {
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[(8 * n + 2 * t + (e & 1)) * L::RPITCH + 16 * i + 8 * (e >> 1)] = acc[i][n][e];
        }
    __syncthreads();
    constexpr int W = ROWS / 4;
    for (int x = tid; x < count * (two ? 2 * W : W); x += kLoraWarps * 32) {
      const int m = two ? x / (2 * W) : x / W, r = 4 * (two ? x % (2 * W) : x % W);
      const float* const from = red + ((r / ROWS) * (kLoraWarps / 2) * TILE + m) * L::RPITCH + r % ROWS;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kLoraWarps; ++w) {
        if (w < per_block) {
          const float4 q = *reinterpret_cast<const float4*>(from + w * TILE * L::RPITCH);
          v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
        }
      }
      if (r < RP) *reinterpret_cast<float4*>(sum + m * RP + r) = v;
    }
    if (CS > 1) cluster_arrive();
    __syncthreads();                             // the sums have been taken: their place is the ring's
  }

  // ---- this warp's columns: groups of 32, col, col + 8, ... below g1. Each passes through the ring as `steps`
  // stages with B's rows for one K step (none up to rank 16), then one or two with base; the pointers run
  // ahead of the products.
  const int groups = (p.N + 31) / 32, share = part * CS + me, shares = NS * CS;
  const int g1 = static_cast<int>(static_cast<long long>(groups) * (share + 1) / shares);
  int col = static_cast<int>(static_cast<long long>(groups) * share / shares) + warp;
  // A thread has 8 columns of a group of 32: 8t .. 8t + 7 of 16-bit rows, 4t .. 4t + 3 of each half of fp32 rows, so that
  // every 16-byte access of a quad covers 64 bytes (8 consecutive columns in fp32 touch each sector twice: 1743 tokens,
  // rank 8, N = 33688: 153 us).
  constexpr int YB = V == 2 ? 4 : 2, SIDE = 8 / V, STEP = kLoraWarps * 32;
  const int n_end = min(32 * g1, p.N);
  int n = 32 * col + SIDE * t;                   // this thread's first column of the group asked for
  const char* bp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) bp[i] = static_cast<const char*>(p.base) + (tok[i] * p.ldb + n) * YB;
  // rows of B: columns permuted so that tile j's column c is column SIDE (c / 2) + tile_col(j) + c % 2 of the group
  auto tile_col = [](int j) { return V == 2 ? 2 * (j & 1) + 16 * (j >> 1) : 2 * j; };
  constexpr int KV = RT == 1 ? 4 : 8;            // elements of a row that a thread takes
  int nb = 32 * col + SIDE * (g >> 1) + (g & 1);    // its row in tile 0 of the group that wp points to
  const uint16_t* wp = p.B + (static_cast<int64_t>(adapter) * p.N + nb) * p.rank + KV * t;
  const int mts = TILE > 16 && count > 16 ? 2 : 1, halves = V == 2 && mts == 2 ? 2 : 1;      // stages with base
  const int b_stages = L::REG_B ? 0 : steps;
  int kind = 0, ask_at = 0, take_at = 0;         // which of a group's stages is asked for next; places in the ring
  auto ask_next = [&]() {
    const uint32_t dst = slot0 + ask_at * L::YSTAGE;
    if (n - SIDE * t < n_end) {
      if (kind < b_stages) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool in = nb + tile_col(j) < n_end && 32 * kind + KV * t < p.rank;
          cp_async16(dst + j * L::VEC, in ? wp + tile_col(j) * p.rank + 32 * kind : p.B, in ? 16 : 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < L::BASES; ++i) {
          // V = 1: token 8i + g; V = 2: the two vectors of tokens 8 (i / 2) + g, and 16 more in the second stage
          const int half = kind - b_stages, r = V == 1 ? i : (i >> 1) + 2 * half;
          const char* const src = V == 1 ? bp[i] : (half == 0 ? bp[i >> 1] : bp[(NT - 2) + (i >> 1)]) + 64 * (i & 1);
          if (n + (V == 1 ? 0 : 16 * (i & 1)) < n_end && 8 * r + g < count) cp_async16(dst + i * L::VEC, src, 16);
        }
      }
    }
    cp_async_commit();
    if (++kind == b_stages + halves) {
      kind = 0;
      n += STEP;
      if constexpr (!L::REG_B) {
        nb += STEP;
        wp += static_cast<int64_t>(STEP) * p.rank;
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) bp[i] += STEP * YB;
    }
    ask_at = ask_at + 1 == L::YS ? 0 : ask_at + 1;
  };
  // REG_B: B's rows of the groups in turn; two sets by name, for a set that is moved waits for its loads
  uint2 b_even[4] = {}, b_odd[4] = {};
  auto load_b = [&](uint2 (&w)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = nb + tile_col(j) < n_end && KV * t < p.rank ? __ldg(reinterpret_cast<const uint2*>(wp + tile_col(j) * p.rank)) : make_uint2(0, 0);
    nb += STEP;
    wp += static_cast<int64_t>(STEP) * p.rank;
  };
  auto take_next = [&]() {
    cp_async_wait<L::YS - 2>();
    ask_next();                                  // into the slots that the last turn read
    const uint32_t src = slot0 + take_at * L::YSTAGE;
    take_at = take_at + 1 == L::YS ? 0 : take_at + 1;
    return src;
  };
  // the first columns' operands arrive while the blocks meet
#pragma unroll 1
  for (int s = 0; s < L::YS - 1; ++s) ask_next();
  if constexpr (L::REG_B) {
    if (steps > 0) load_b(b_even);
  }
  float up[NT] = {};
  if (steps > 0) {
    if (CS > 1) cluster_wait();
    // ---- some lanes take a token: sum over the blocks, power of two, then the parts in the K order of the MMAs below.
    // A lane has four elements of the rank; 32 / wide tokens to a warp. Up to rank 32 every block does this for all tokens.
    // Above, what they read from one another would take longest (rank 128, 8 blocks: 64 KB each at 27 B/ns, 2.5 us): a
    // block sums the tokens me, me + CS, ... and stores their parts to every block, which costs a second meeting.
    constexpr bool SHARED = L::SHARED;
    const float sc = __ldg(p.scale + adapter);
    const uint32_t sums = smem_u32(sum);
    int wide = 4;
    while (4 * wide < RP) wide *= 2;
    const int sub = lane & (wide - 1), per_warp = 32 / wide;
    const int m_first = SHARED ? me : 0, m_step = SHARED ? CS : 1;
    for (int j0 = warp * per_warp; m_first + j0 * m_step < count; j0 += kLoraWarps * per_warp) {     // rows past the last token may hold anything: they reach no other row
      const int m = m_first + (j0 + lane / wide) * m_step;
      float v[4] = {};
      if (m < count && 4 * sub < p.rank) {
        for (int q0 = 0; q0 < (SHARED ? CS : 1); q0 += 8) {       // (eight blocks at most if not SHARED)
          float4 f[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) f[q] = q0 + q < CS ? ld_cluster4(sums + (m * RP + 4 * sub) * 4, q0 + q) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[0] += f[q].x, v[1] += f[q].y, v[2] += f[q].z, v[3] += f[q].w;
        }
      }
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] *= sc;
        top = fmaxf(top, fabsf(v[e]));
      }
      for (int o = wide / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e2 = min(max(static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127, -126), 126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
      const uint32_t back = static_cast<uint32_t>(127 + e2) << 23;
      // element 8q + j of 32 (thread q of the quad loads it): MMA j / 4, column 2q + (j & 1) + 8 ((j & 2) / 2);
      // of 16, for one MMA, element 4q + j
      const int at = RT == 1 ? 2 * sub : 32 * (sub >> 3) + 16 * (sub & 1) + 2 * (sub >> 1 & 3);
      const bool live = m < count && 4 * sub < RP;
      if (live && sub == 0) {
        if (SHARED && CS > 1) {
          for (int q = 0; q < CS; ++q) st_cluster(smem_u32(&s_up[m]), q, back);
        } else {
          s_up[m] = __uint_as_float(back);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= down;
#pragma unroll
      for (int h = 0; h < L::PARTS; ++h) {
        uint32_t w[2];                           // j & 2 = 0: columns 2q, 2q + 1; j & 2 = 2: columns 8 + 2q, 9 + 2q
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float lo, hi;
          if constexpr (BF16) {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(v[2 * e + 1]), "f"(v[2 * e]));
            lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xFFFF0000u);
          } else {
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(v[2 * e + 1]), "f"(v[2 * e]));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
            lo = f.x, hi = f.y;
          }
          // an infinity is in the first part alone
          v[2 * e] = isinf(v[2 * e]) ? 0.f : v[2 * e] - lo;
          v[2 * e + 1] = isinf(v[2 * e + 1]) ? 0.f : v[2 * e + 1] - hi;
        }
        uint16_t* const row = hs + (h * TILE + m) * PITCH;
        if (SHARED && CS > 1) {
          // with the lane of the next q: one takes the lower columns of both, the other the upper
          const bool upper = sub & 2;
          const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? w[0] : w[1], 2);
          const uint32_t to = smem_u32(row + at + (upper ? 6 : 0));
          if (live)
            for (int q = 0; q < CS; ++q) st_cluster2(to, q, upper ? other : w[0], upper ? w[1] : other);
        } else if (live) {
          *reinterpret_cast<uint32_t*>(row + at) = w[0];
          *reinterpret_cast<uint32_t*>(row + at + 8) = w[1];
        }
      }
    }
    if (CS > 1) cluster_arrive();                // this block has read the others' sums, and written to them
    if (SHARED && CS > 1)
      cluster_wait();
    else
      __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i) up[i] = s_up[8 * i + g];
  }

  // ---- y = base + B h
  char* yp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) yp[i] = static_cast<char*>(p.y) + (tok[i] * p.ldy + 32 * col + SIDE * t) * YB;
  const uint32_t hbase = smem_u32(hs) + ((lane & 15) * PITCH + (lane >> 4) * 8) * 2;
  auto group = [&](const uint2 (&mine)[4], uint2 (&next)[4]) {
    const int left = n_end - 32 * col - SIDE * t;              // columns from this thread's first to the end
    float acc[NT / 2][4][4];
#pragma unroll
    for (int m = 0; m < NT / 2; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.f;
    for (int s = 0; s < steps; ++s) {
      uint4 b[4];
      if constexpr (L::REG_B) {
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = make_uint4(mine[j].x, mine[j].y, 0, 0);
        load_b(next);
      } else {
        const uint32_t at = take_next();
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = ld_shared16(at + j * L::VEC);
      }
#pragma unroll
      for (int m = 0; m < NT / 2; ++m) {
        if (m < mts) {
#pragma unroll
          for (int h = 0; h < L::PARTS; ++h) {
#pragma unroll
            for (int half = 0; half < L::KSTEP / 16; ++half) {
              uint32_t a[4];
              asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                           : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                           : "r"(hbase + ((h * TILE + 16 * m) * PITCH + 32 * s + 16 * half) * 2)
                           : "memory");
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma16816<BF16>(acc[m][j], a[0], a[1], a[2], a[3], half ? b[j].z : b[j].x, half ? b[j].w : b[j].y);
            }
          }
        }
      }
    }
    uint32_t src = take_next();
    // token 8i + g: columns SIDE t + tile_col(j) + {0, 1} of the group are elements 2 (i & 1) + {0, 1} of acc[i / 2][j]
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (V == 2 && i == 2 && mts == 2) src = take_next();
      if (left > 0 && tok[i] >= 0) {
        uint4 r[V];
#pragma unroll
        for (int e = 0; e < V; ++e) r[e] = ld_shared16(src + (V == 1 ? i : 2 * (i & 1) + e) * L::VEC);
        if (steps > 0) {
          uint32_t w[4 * V];
#pragma unroll
          for (int e = 0; e < V; ++e) w[4 * e] = r[e].x, w[4 * e + 1] = r[e].y, w[4 * e + 2] = r[e].z, w[4 * e + 3] = r[e].w;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = acc[i >> 1][j][2 * (i & 1)], hi = acc[i >> 1][j][2 * (i & 1) + 1];
            if constexpr (V == 2) {
              w[2 * j] = __float_as_uint(__fmaf_rn(lo, up[i], __uint_as_float(w[2 * j])));
              w[2 * j + 1] = __float_as_uint(__fmaf_rn(hi, up[i], __uint_as_float(w[2 * j + 1])));
            } else {
              w[j] = add2<YD>(w[j], lo, hi, up[i]);
            }
          }
#pragma unroll
          for (int e = 0; e < V; ++e) r[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (16 * e < left) reinterpret_cast<uint4*>(yp[i])[4 * e] = r[e];
      }
      yp[i] += STEP * YB;
    }
    col += kLoraWarps;
  };
  while (col < g1) {
    group(b_even, b_odd);
    if constexpr (L::REG_B) {
      if (col < g1) group(b_odd, b_even);
    }
  }
  cp_async_wait<0>();
  if (!L::SHARED && steps > 0 && CS > 1) cluster_wait();        // no block leaves while another reads its sums
}

template <bool BF16, int YD, int RT, int TILE>
cudaError_t apply(const LoraParams& p, int sms, cudaStream_t st) {
  using L = Lora<BF16, YD, RT, TILE>;
  static int ready[64];                            // the shared memory limit is set, by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (__atomic_load_n(&ready[dev], __ATOMIC_RELAXED) == 0) {
    e = cudaFuncSetAttribute(lora_kernel<BF16, YD, RT, TILE>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::smem(kLoraMaxRank));
    if (e != cudaSuccess) return e;
    if (L::SHARED) {
      e = cudaFuncSetAttribute(lora_kernel<BF16, YD, RT, TILE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    __atomic_store_n(&ready[dev], 1, __ATOMIC_RELAXED);
  }
  // Blocks of a cluster (cs) share an item's K and clusters of an item (ns) repeat that; both share its columns.
  // All blocks run at once, two to an SM at most, and the SM with most of them sets the time: taken is the pair with the
  // fewest bytes into it, of those that leave every warp a piece of K and columns. A block alone takes in 1 / 0.75 of
  // what each of two does (0.5 to 0.85 tried). Bound to powers of two, 3000 tokens, rank 64, K = 4096,
  // N = 14336: 75 us, so 54; with the largest cs and then the largest ns, 256 tokens, rank 128, K = 5120, N = 17408:
  // 32 us, so 25. Sixteen blocks, above rank 32, find room on four fifths of the GPU or less (2 tokens of 2 adapters, rank 128,
  // K = 8488, N = 33832: at most eight 18.1 us, so 13.3; ten and twelve as well: 200 tokens, rank 64, 17.0 us, so 11.4).
  const long long items = lora_max_items(p.M, p.n_adapters);
  const int per_block = p.rank > L::ROWS ? kLoraWarps / 2 : kLoraWarps;           // warps that share K
  const int chunks = (p.K + 31) / 32, groups = (p.N + 31) / 32;
  int cs = 1, ns = 1;
  float best = 0.f;
  for (int c = 1; c <= (L::SHARED ? kLoraMaxCluster : 8); c = c < 8 ? c + 1 : 2 * c) {
    const int room = c > 8 ? sms * 4 / 5 : sms;
    if (c > 1 && (chunks < c * per_block || items * c > 2LL * room)) break;
    for (int full = 1; full <= 2; ++full) {
      const int fit = static_cast<int>(full * static_cast<long long>(room) / (items * c)), most = groups / (c * kLoraWarps);
      const int n = std::max(1, std::min(fit, most));
      const float a = 2.f * p.K * (p.rank + TILE), b = 2.f * p.N * (p.rank + 2 * L::V * TILE);   // x and A; B, base and y
      const float bytes = (a + b / n) / c * (items * c * n <= sms ? 0.75f : 1.f);
      if (c + full == 2 || bytes <= best) best = bytes, cs = c, ns = n;
    }
  }
  return launch_pdl_cluster(lora_kernel<BF16, YD, RT, TILE>, dim3(static_cast<unsigned>(items * ns * cs)), dim3(kLoraWarps * 32),
                            L::smem(p.rank), st, cs, p, cs, ns);
}

template <bool BF16, int YD, int TILE>
cudaError_t apply_rank(const LoraParams& p, int sms, cudaStream_t st) {
  return p.rank <= 16   ? apply<BF16, YD, 1, TILE>(p, sms, st)
         : p.rank <= 32 ? apply<BF16, YD, 2, TILE>(p, sms, st)
                        : apply<BF16, YD, 4, TILE>(p, sms, st);
}

template <bool BF16, int YD>
cudaError_t apply_tile(const LoraParams& p, int sms, cudaStream_t st) {
  return lora_tile(p.M) == 16 ? apply_rank<BF16, YD, 16>(p, sms, st) : apply_rank<BF16, YD, 32>(p, sms, st);
}

template <bool BF16>
cudaError_t apply_type(const LoraParams& p, int sms, cudaStream_t st) {
  switch (p.y_dtype) {
    case TL_BF16: return apply_tile<BF16, TL_BF16>(p, sms, st);
    case TL_F16: return apply_tile<BF16, TL_F16>(p, sms, st);
    default: return apply_tile<BF16, TL_F32>(p, sms, st);
  }
}

}  // namespace

cudaError_t launch_lora_plan(const int32_t* ids, int M, int n_adapters, void* plan, int* status, cudaStream_t st) {
  auto* head = static_cast<LoraPlanHeader*>(plan);
  return launch_pdl(lora_plan_kernel, dim3(1), dim3(kPlanThreads), 2 * sizeof(int) * (n_adapters + 1), st, ids, M, n_adapters, lora_tile(M), head,
                    reinterpret_cast<LoraItem*>(head + 1), status);
}

cudaError_t launch_lora_apply(const LoraParams& p, bool bf16, int sms, cudaStream_t st) {
  return bf16 ? apply_type<true>(p, sms, st) : apply_type<false>(p, sms, st);
}

}  // namespace tl
