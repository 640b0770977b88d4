// Low-rank adapters of many requests beside a projection:
//   y[m] = base[m] + scale[a] B[a] (A[a] x[m]),  a = ids[m].
//
// A plan kernel sorts the tokens by adapter once per step; its items are up
// to 32 tokens of one adapter, so an adapter's matrices are read once per item,
// by however many tokens use it. Two kernels per projection:
//
// shrink  h = A x for an item. The rank is small and K long, so the K axis is
//   cut over the warps of a cluster of blocks, whose sums meet through distributed
//   shared memory in a fixed order. The adapter's rows are the 16 rows of the MMA and the
//   item's tokens its 8 columns. Nothing is used twice but through registers, so the
//   operands come straight from global memory: with the K axis permuted alike on
//   both sides (thread t of a quad takes the 8 consecutive elements 8t .. 8t + 7 of 32) every
//   load is 16 bytes.
// expand  y = base + scale B h for an item and a range of columns: tokens are the rows
//   of the MMA, the columns of B are permuted so that a thread ends with 8
//   consecutive ones of a token: 16-byte loads of base and stores of y. The
//   bytes of base and y bound it. h is scaled by a power of two of its own per
//   token (the f16 range) and split in 16-bit parts, so that it keeps 16 bits or more.
#include "lora.cuh"
#include "tl_internal.cuh"

#include <cuda_bf16.h>

namespace tl {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kLoraWarps = 4;

// ----------------------------------------------------------------- plan
// Shared memory: one counter per adapter, and one for the tokens without.
__global__ void __launch_bounds__(kPlanThreads)
lora_plan_kernel(const int32_t* __restrict__ ids, int M, int n, LoraPlanHeader* head, LoraItem* items, int* order, int* status) {
  extern __shared__ int next[];
  __shared__ int s_tokens[kPlanThreads / 32], s_items[kPlanThreads / 32];
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
  // exclusive sums of tokens and items over the bins; a thread owns consecutive bins
  const int per = (n + kPlanThreads) / kPlanThreads;
  int tokens = 0, tiles = 0;
  for (int i = tid * per; i < min(n + 1, (tid + 1) * per); ++i) {
    tokens += next[i];
    tiles += (next[i] + kLoraTile - 1) / kLoraTile;
  }
  int it = tokens, ii = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, it, o), b = __shfl_up_sync(0xffffffffu, ii, o);
    if (lane >= o) it += a, ii += b;
  }
  if (lane == 31) s_tokens[warp] = it, s_items[warp] = ii;
  __syncthreads();
  int start = it - tokens, item = ii - tiles, all = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) start += s_tokens[w], item += s_items[w];
    all += s_items[w];
  }
  for (int i = tid * per; i < min(n + 1, (tid + 1) * per); ++i) {
    const int c = next[i];
    next[i] = start;
    for (int k = 0; k < c; k += kLoraTile) items[item++] = LoraItem{i < n ? i : -1, start + k, min(kLoraTile, c - k), 0};
    start += c;
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
        at = __shfl_sync(0xffffffffu, at, leader);
        if (b >= 0) order[at + rank] = i;
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

__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

// ----------------------------------------------------------------- shrink
// blockIdx.x = item * CS + rank of the block in its cluster; blockIdx.y: 16 RT rows of A
template <bool BF16, int RT>
__global__ void __launch_bounds__(kLoraWarps * 32) lora_shrink_kernel(const __grid_constant__ LoraParams p, int CS) {
  constexpr int NT = kLoraTile / 8, ROWS = 16 * RT;
  __shared__ float red[kLoraWarps][ROWS][kLoraTile + 1];
  __shared__ float sum[ROWS * kLoraTile];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int idx = blockIdx.x / CS, rank = blockIdx.x - idx * CS, r0 = blockIdx.y * ROWS;
  pdl_wait_prior();
  pdl_launch_dependents();
  if (p.plan->M != p.M || p.plan->n_adapters != p.n_adapters) return;      // expand reports it
  if (idx >= p.plan->items) return;                                         // the whole cluster leaves
  const LoraItem item = p.items[idx];
  if (item.adapter < 0) return;

  const int chunks = (p.K + 31) / 32, workers = CS * kLoraWarps, me = rank * kLoraWarps + warp;
  const int c0 = static_cast<int>(static_cast<long long>(chunks) * me / workers);
  const int c1 = static_cast<int>(static_cast<long long>(chunks) * (me + 1) / workers);
  const uint16_t* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    xr[n] = 8 * n + g < item.count ? p.x + p.order[item.start + 8 * n + g] * p.ldx + 8 * t : nullptr;
  const uint16_t* const ar = p.A + (static_cast<int64_t>(item.adapter) * p.rank + r0 + g) * p.K + 8 * t;
  const int nts = (item.count + 7) / 8;

  float acc[RT][NT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
  for (int c = c0; c < c1; ++c) {
    const int k = 32 * c;
    const bool in = k + 8 * t < p.K;
    uint4 a[RT][2], b[NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        a[i][e] = in && r0 + 16 * i + 8 * e + g < p.rank
                      ? __ldg(reinterpret_cast<const uint4*>(ar + static_cast<int64_t>(16 * i + 8 * e) * p.K + k))
                      : zero;
#pragma unroll
    for (int n = 0; n < NT; ++n) b[n] = in && xr[n] != nullptr ? __ldg(reinterpret_cast<const uint4*>(xr[n] + k)) : zero;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n < nts) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          mma16816<BF16>(acc[i][n], a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y, b[n].x, b[n].y);
          mma16816<BF16>(acc[i][n], a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w, b[n].z, b[n].w);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[warp][16 * i + g + 8 * (e >> 1)][8 * n + 2 * t + (e & 1)] = acc[i][n][e];
  __syncthreads();
  for (int x = tid; x < ROWS * kLoraTile; x += kLoraWarps * 32) {
    const int r = x % ROWS, m = x / ROWS;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) v += red[w][r][m];
    sum[x] = v;
  }
  if (CS > 1) cluster_sync(); else __syncthreads();
  const uint32_t base = smem_u32(sum);
  for (int x = rank * kLoraWarps * 32 + tid; x < ROWS * item.count; x += CS * kLoraWarps * 32) {
    const int r = x % ROWS, m = x / ROWS;
    float v = 0.f;
    if (CS > 1)
      for (int q = 0; q < CS; ++q) v += ld_cluster(base + 4 * x, q);
    else
      v = sum[x];
    if (r0 + r < p.rank) p.h[static_cast<int64_t>(item.start + m) * p.rank + r0 + r] = v;
  }
  if (CS > 1) cluster_sync();           // no block leaves while another reads its sums
}

// ----------------------------------------------------------------- expand
template <int YD>
struct YType;
template <>
struct YType<TL_BF16> { static constexpr int V = 1; };
template <>
struct YType<TL_F16> { static constexpr int V = 1; };
template <>
struct YType<TL_F32> { static constexpr int V = 2; };     // 16-byte vectors per 8 columns

template <int YD>
__device__ __forceinline__ uint32_t add2(uint32_t base, float lo, float hi) {
  uint32_t r;
  if constexpr (YD == TL_BF16) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(base & 0xFFFF0000u) + hi), "f"(__uint_as_float(base << 16) + lo));
  } else {
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&base));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b.y + hi), "f"(b.x + lo));
  }
  return r;
}

// blockIdx.x: item; blockIdx.y: 32 IT columns for each warp
template <bool BF16, int YD>
__global__ void __launch_bounds__(kLoraWarps * 32) lora_expand_kernel(const __grid_constant__ LoraParams p, int IT) {
  constexpr int PARTS = YD == TL_F32 && BF16 ? 3 : 2, V = YType<YD>::V, PITCH = kLoraMaxRank + 8;
  __shared__ __align__(16) uint16_t hs[PARTS][kLoraTile][PITCH];
  __shared__ float s_up[kLoraTile];
  __shared__ int s_tok[kLoraTile];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_wait_prior();
  pdl_launch_dependents();
  if (p.plan->M != p.M || p.plan->n_adapters != p.n_adapters) {
    if (tid == 0) set_status(p.status, TL_EDATA);
    return;
  }
  if (static_cast<int>(blockIdx.x) >= p.plan->items) return;
  const LoraItem item = p.items[blockIdx.x];
  if (item.adapter < 0 && !p.copy_bare) return;
  const int steps = item.adapter < 0 ? 0 : (p.rank + 31) / 32, rp = 32 * steps;
  if (tid < kLoraTile) s_tok[tid] = tid < item.count ? p.order[item.start + tid] : -1;
  if (steps > 0) {
    // a warp takes a token: power of two, then the parts, in the K order of the MMAs below
    const float sc = __ldg(p.scale + item.adapter);
    for (int m = warp; m < kLoraTile; m += kLoraWarps) {
      float v[kLoraMaxRank / 32], top = 0.f;
#pragma unroll
      for (int i = 0; i < kLoraMaxRank / 32; ++i) {
        const int r = 32 * i + lane;
        v[i] = r < p.rank && m < item.count ? sc * p.h[static_cast<int64_t>(item.start + m) * p.rank + r] : 0.f;
        top = fmaxf(top, fabsf(v[i]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = min(max(static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127, -126), 126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (lane == 0) s_up[m] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      // element r = 8 q + j of 32 (thread q of the quad loads it): MMA j / 4, column 2 q + (j & 1) + 8 (j & 2) / 2
      const int q = lane >> 3, j = lane & 7;
      const int col = 16 * (j >> 2) + 2 * q + (j & 1) + 4 * (j & 2);
#pragma unroll
      for (int i = 0; i < kLoraMaxRank / 32; ++i) {
        if (i < steps) {
          float rest = v[i] * down;
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
            uint16_t bits;
            if constexpr (BF16) {
              const __nv_bfloat16 b = __float2bfloat16_rn(rest);
              bits = __bfloat16_as_ushort(b);
              rest = isinf(rest) ? 0.f : rest - __bfloat162float(b);       // an infinity is in the first part alone
            } else {
              const __half b = __float2half_rn(rest);
              bits = __half_as_ushort(b);
              rest = isinf(rest) ? 0.f : rest - __half2float(b);
            }
            hs[part][m][32 * i + col] = bits;
          }
        }
      }
    }
  }
  __syncthreads();
  int tok[4];
  float up[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tok[i] = s_tok[8 * i + g];
    up[i] = steps > 0 ? s_up[8 * i + g] : 0.f;
  }
  const int mts = item.count > 16 ? 2 : 1;
  const uint32_t hbase = smem_u32(&hs[0][0][0]) + ((lane & 15) * PITCH + (lane >> 4) * 8) * 2;
  for (int it = 0; it < IT; ++it) {
    const int n0 = ((blockIdx.y * IT + it) * kLoraWarps + warp) * 32;
    if (n0 >= p.N) break;
    const bool live = n0 + 8 * t < p.N;
    uint4 base[4][V];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (live && tok[i] >= 0) {
        const char* src = static_cast<const char*>(p.base) + (tok[i] * p.ldb + n0 + 8 * t) * (V == 2 ? 4 : 2);
#pragma unroll
        for (int e = 0; e < V; ++e) base[i][e] = reinterpret_cast<const uint4*>(src)[e];
      }
    }
    float acc[2][4][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.f;
    for (int s = 0; s < steps; ++s) {
      uint4 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
        b[j] = n < p.N && 32 * s + 8 * t < p.rank
                   ? __ldg(reinterpret_cast<const uint4*>(p.B + (static_cast<int64_t>(item.adapter) * p.N + n) * p.rank + 32 * s + 8 * t))
                   : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (m < mts) {
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t a[4];
              asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                           : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                           : "r"(hbase + ((part * kLoraTile + 16 * m) * PITCH + 32 * s + 16 * half) * 2)
                           : "memory");
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma16816<BF16>(acc[m][j], a[0], a[1], a[2], a[3], half ? b[j].z : b[j].x, half ? b[j].w : b[j].y);
            }
          }
        }
      }
    }
    // token 8 i + g: columns n0 + 8 t + 2 j + {0, 1} are elements 2 (i & 1) + {0, 1} of acc[i / 2][j]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (live && tok[i] >= 0) {
        float d[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[2 * j] = acc[i >> 1][j][2 * (i & 1)] * up[i];
          d[2 * j + 1] = acc[i >> 1][j][2 * (i & 1) + 1] * up[i];
        }
        char* dst = static_cast<char*>(p.y) + (tok[i] * p.ldy + n0 + 8 * t) * (V == 2 ? 4 : 2);
        uint32_t w[4 * V] = {};
#pragma unroll
        for (int e = 0; e < V; ++e) {
          w[4 * e] = base[i][e].x, w[4 * e + 1] = base[i][e].y, w[4 * e + 2] = base[i][e].z, w[4 * e + 3] = base[i][e].w;
        }
        if (steps > 0) {
          if constexpr (V == 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) + d[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = add2<YD>(w[e], d[2 * e], d[2 * e + 1]);
          }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) reinterpret_cast<uint4*>(dst)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
      }
    }
  }
}

template <bool BF16, int RT>
cudaError_t shrink(const LoraParams& p, int items, int sms, cudaStream_t st) {
  const int ry = (p.rank + 16 * RT - 1) / (16 * RT);
  // the fewest blocks per cluster that fill the GPU three times over
  int cs = 1;
  while (cs < 8 && static_cast<long long>(items) * ry * cs < 3LL * sms) cs *= 2;
  return launch_pdl_cluster(lora_shrink_kernel<BF16, RT>, dim3(items * cs, ry), dim3(kLoraWarps * 32), 0, st, cs, p, cs);
}

template <bool BF16, int YD>
cudaError_t expand(const LoraParams& p, int items, int sms, cudaStream_t st) {
  const int cols = (p.N + 32 * kLoraWarps - 1) / (32 * kLoraWarps);
  // more columns per block (h is split once per block) as long as the GPU stays full
  int it = 1;
  while (it < 8 && static_cast<long long>(items) * cols > 16LL * sms * it) it *= 2;
  return launch_pdl(lora_expand_kernel<BF16, YD>, dim3(items, (cols + it - 1) / it), dim3(kLoraWarps * 32), 0, st, p, it);
}

template <bool BF16>
cudaError_t apply(const LoraParams& p, int sms, cudaStream_t st) {
  const int items = lora_max_items(p.M, p.n_adapters);
  cudaError_t e = p.rank <= 16   ? shrink<BF16, 1>(p, items, sms, st)
                  : p.rank <= 32 ? shrink<BF16, 2>(p, items, sms, st)
                                 : shrink<BF16, 4>(p, items, sms, st);
  if (e != cudaSuccess) return e;
  switch (p.y_dtype) {
    case TL_BF16: return expand<BF16, TL_BF16>(p, items, sms, st);
    case TL_F16: return expand<BF16, TL_F16>(p, items, sms, st);
    default: return expand<BF16, TL_F32>(p, items, sms, st);
  }
}

}  // namespace

cudaError_t launch_lora_plan(const int32_t* ids, int M, int n_adapters, void* plan, int* status, cudaStream_t st) {
  auto* head = static_cast<LoraPlanHeader*>(plan);
  auto* items = reinterpret_cast<LoraItem*>(head + 1);
  auto* order = reinterpret_cast<int*>(items + lora_max_items(M, n_adapters));
  return launch_pdl(lora_plan_kernel, dim3(1), dim3(kPlanThreads), sizeof(int) * (n_adapters + 1), st, ids, M, n_adapters, head, items,
                    order, status);
}

cudaError_t launch_lora_apply(const LoraParams& p, bool bf16, int sms, cudaStream_t st) {
  return bf16 ? apply<true>(p, sms, st) : apply<false>(p, sms, st);
}

}  // namespace tl
