// Attention of one new token per request over a paged key-value cache.
//
//   out[h] = sum_j p_j V_j / sum_j p_j,   p_j = exp(scale q[h] . K_j)
//
// Every cached byte is used by the G = q_heads / kv_heads queries that share a
// key-value head and by nothing else: 2 G flops a 16-bit element, so the cache's bytes bound the kernel
// and the tensor cores' legacy path (mma.sync, which needs no tensor memory and
// takes tiles of 8 queries) has room to spare. One pass: the running maximum m,
// the sum l and the output o of a softmax over the keys seen so far,
//   m' = max(m, s),  l' = l 2^(m - m') + sum 2^(s - m'),  o' likewise,
// with s in units of log2(e).
//
// Work. A (request, group of query heads) is a segment; its keys are cut into
// tiles of 4 KT keys and the tiles of all segments form one list, cut into
// equal shares for the blocks of one resident wave. So a batch of ragged lengths
// needs no plan from the host, which never learns the lengths, and no block waits
// for the longest request. A segment inside one block's share is finished there;
// one that is cut leaves a partial (m, l, o) per block in the workspace, and the
// block that arrives last joins them in block order (the order of arrival does not
// reach the result). At most two of a block's segments are cut, the first and
// the last, so the workspace depends on the grid alone.
//
// Tiles. A tile's keys go through four rings of STAGES buffers (cp.async), KT keys each. A ring has a warp for
// up to 8 or 16 query heads of the segment, or two warps, which fill it together and read it each for its
// heads; there is no block barrier in the loop. Each warp keeps its own (m, l, o);
// the rings meet once per segment. The scores are computed transposed, S^T = K q^T: the
// keys are the rows of the MMA and 8 query heads its columns, so 8 heads need
// half the MMAs that 16 padded rows would, and S^T and O^T = V^T P^T have their heads on the same
// lanes, which keeps the rescaling in registers. P^T becomes an operand by an 8x8 transpose (movmatrix).
// Probabilities are split in two 16-bit numbers, high and low part, so that they count with 16 (bf16)
// or 22 (f16) bits instead of 8 or 11; the MMAs for it are not what bounds the kernel. Both parts are positive, and never zero,
// so that an infinite value makes its channel infinite: a low part of either sign, or a zero, would make it NaN.
//
// An 8-bit cache is widened to f16 in registers (exact); q is then scaled by a
// power of two of its own per head so that a bf16 query fits f16's range.
//
// Few segments of up to some thousand keys take the same way with one to sixteen blocks each, a cluster, which join
// through their shared memory; many segments of few keys with a ring each: no list, no workspace, no atomics.
//
// Measured on GB300 (copy rate 6.79 TB/s): the loop streams at 7.4-7.7 TB/s. 160 requests of 512-16384 tokens, 8 heads of 128
// channels, 8 bits: 226 us, 6.7 TB/s of 1.51 GB. 24 requests of 40-9000 tokens, 4 heads of 256, bf16: 37 us, 4.7 TB/s;
// 23 us of it stream, 3.4 us pass before the first loads are out (lengths, place in the list, page
// table) and 8 us in meetings and joins. One request of 80001: 62 us, 5.3 TB/s. 577 tokens of
// one request: 5.8 us. 1024 requests of 1-400 tokens, 8 heads of 128: 155 us, 5.6 TB/s. The 16-bit loop takes 1.3 us for a tile of
// 64 KB per SM whatever is left out of its arithmetic; above 16 query heads to a key-value head it is the arithmetic that
// bounds (32 heads of 128 channels: 106 us where the bytes take 50).
#pragma once

#include "attention_join.h"
#include "tl_internal.cuh"

#include <type_traits>

#include <cuda_bf16.h>

namespace tl {

enum AttnCache { kCacheBf16 = 0, kCacheF16 = 1, kCacheF8 = 2 };

// n / d for 0 <= n < 2^31 by a multiplication: m = floor(2^(31 + s) / d) + 1 with
// s = ceil(log2 d) exceeds 2^(31 + s) / d by at most 1, so n m / 2^(31 + s)
// exceeds n / d by less than 2^-s <= 1 / d.
struct FastDiv {
  uint32_t d, m, s;
  static FastDiv make(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.s) < d) ++f.s;
    f.m = static_cast<uint32_t>(((1ull << (31 + f.s)) / d) + 1);
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return d == 1 ? n : __umulhi(n, m) >> (s - 1);
  }
};

struct AttnParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride, head_stride, token_stride;   // bytes
  int num_pages;
  FastDiv page;
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq, ldo;
  const int32_t* pages;
  int64_t ldp;
  int max_len;              // max_pages * page_size, at most 2^31 - 1
  const int32_t* lens;
  float* lse;
  float scale_log2;
  int B, q_heads, kv_heads, group, groups_per_kv, window, q_bf16;
  int runs16;               // page_size is a multiple of 16: 16 keys from a multiple of 16 lie at equal distances
  int cluster_log;          // kCluster: 2^cluster_log blocks share a segment
  int* counters;            // [kAttnLevels][kAttnMaxGrid] (attention_join.h), zero between calls
  float* partials;          // two per block
  int* status;
};

constexpr int kAttnRings = 4;          // rings of key tiles in a block, each with HW warps
constexpr int kAttnMaxBlocksPerSm = 2;
constexpr int kAttnClusterLog = 4;     // of the most blocks that share a segment of a small call
constexpr int kJoinFew = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// floats of one partial: m and l of each head, then o
__host__ __device__ constexpr size_t attn_partial_floats(int heads, int dim) {
  return static_cast<size_t>(heads) * (dim + 2);
}

cudaError_t launch_attn_bf16(const AttnParams& p, int dim, int columns, int sms, cudaStream_t st);
cudaError_t launch_attn_f16(const AttnParams& p, int dim, int columns, int sms, cudaStream_t st);
cudaError_t launch_attn_f8(const AttnParams& p, int dim, int columns, int sms, cudaStream_t st);

namespace attn {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// d += a b, 16 x 8 x 16
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Towards zero, and then at least the least positive number (f16) or normal number (bf16): the parts of a probability.
template <bool BF16>
__device__ __forceinline__ uint32_t above_zero(uint32_t v) {
  uint32_t r;
  if constexpr (BF16)
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x00800080));
  else
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x00010001));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2_down(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return above_zero<BF16>(r);
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
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
// two e4m3 values (low, high byte) as f16, exact
__device__ __forceinline__ uint32_t widen_lo(uint32_t v) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t v) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^x, by which sums of earlier keys or of another share are scaled down; no infinity among them may meet a zero.
__device__ __forceinline__ float faded(float x) { return fmaxf(exp2_approx(x), 0x1p-126f); }

// HW warps to a ring, 8 NT query heads to a warp
template <int CACHE, int D, int HW, int NT>
struct Traits {
  static constexpr bool F8 = CACHE == kCacheF8;
  static constexpr bool BF16 = CACHE == kCacheBf16;      // the MMA's operand type (f16 otherwise)
  static constexpr int THREADS = kAttnRings * HW * 32;
  static constexpr int ROW = D * (F8 ? 1 : 2);           // bytes of a key
  static constexpr int KT = 4096 / ROW > 16 ? 4096 / ROW : 16;   // keys of a ring's buffer: 4 KB of K (8 for 512-byte rows)
  static constexpr int TILE = kAttnRings * KT;
  static constexpr int BUF = 2 * KT * ROW;
  static constexpr int HEADS = 8 * HW * NT;
  static constexpr int OPITCH = D + 4;                   // floats; the warps' o meet here, conflict-free
  static constexpr int MEET = (HEADS * OPITCH + 2 * HEADS) * 4;
  // buffers of a ring: up to three where two blocks share an SM (whose 228 KB hold a KB more for each
  // block), else as many as fit
  static constexpr int stages() {
    for (int s = 3; s >= 2 && HW * NT < 4; --s)        // 256 threads of 255 registers are alone on their SM
      if (kAttnRings * (s * BUF + MEET) <= 115500) return s;
    int s = 6;
    while (kAttnRings * (s * BUF + MEET) > 231000) --s;
    return s;
  }
  static constexpr int STAGES = stages();
  static constexpr int SMEM = kAttnRings * (STAGES * BUF + MEET);
  // partials that the rings hold, at most a warp's lanes
  static constexpr int HOLD = kAttnRings * STAGES * BUF / (HEADS * (D + 2) * 4), FIT = HOLD < 32 ? HOLD : 32;
  static constexpr int BLOCKS = HW * NT == 4 || SMEM > 115500 ? 1 : kAttnMaxBlocksPerSm;     // per SM
  // 2^15 in the probabilities keeps an f16 low part of the small ones out of the subnormals, and makes the least f16 number,
  // which every key with a value at least counts with, 2^-39 of the largest probability
  static constexpr float POFF = BF16 ? 0.f : 15.f;
};

// byte offset of 16-byte chunk c of row r, swizzled so that 8 rows' equal chunks lie in different banks
template <int ROW>
__device__ __forceinline__ uint32_t at(int r, int c) {
  if constexpr (ROW >= 128)
    return r * ROW + ((c ^ (r & 7)) << 4);
  else
    return r * ROW + ((c ^ ((r >> 1) & 3)) << 4);
}

struct Segment {            // where in the list of tiles
  int b, h, tile, tiles;    // request, group of query heads, tile, tiles of this segment
  int begin, first, end;    // where its tiles begin, its first key, one past the last
};

// 64-bit quotient of non-negative numbers, by the 32-bit division where both fit
__device__ __forceinline__ long long divide(long long n, long long d) {
  if (((n | d) >> 32) == 0) return static_cast<unsigned>(n) / static_cast<unsigned>(d);
  return n / d;
}

__device__ __forceinline__ void seg_keys(const AttnParams& p, int len, int tile_keys, Segment& s) {
  const int n = min(max(len, 0), p.max_len);
  s.end = n;
  s.first = p.window > 0 ? max(0, n - p.window) : 0;
  s.begin = p.runs16 ? s.first & ~15 : s.first;       // a window's tiles begin with its first key's run
  s.tiles = max(1, (s.end - s.begin + tile_keys - 1) / tile_keys);
}

// A segment that n blocks share, from block c0 on: c0 began it (its second partial), the others found it
// begun (their first). The partials are joined by the last block to arrive; where they are many, `fan` neighbours
// by the last of them, and their results in the same way, so that the joins run on many SMs.
struct Shared {
  int c0, n, fan, b, h0, heads;
  float v_scale;
};

// Four channels of head h of request b, from the joined (m, l, o).
template <class T>
__device__ __forceinline__ void write_out(const AttnParams& p, int b, int h, int d, int dim, const float4& o, float m, float l, float vs) {
  const float inv = l == 0.f ? 0.f : vs / l;
  uint2 r;
  r.x = p.q_bf16 ? pack2<true>(o.x * inv, o.y * inv) : pack2<false>(o.x * inv, o.y * inv);
  r.y = p.q_bf16 ? pack2<true>(o.z * inv, o.w * inv) : pack2<false>(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.out + b * p.ldo + static_cast<int64_t>(h) * dim + d) = r;
  if (d == 0 && p.lse != nullptr)
    p.lse[static_cast<int64_t>(b) * p.q_heads + h] = l == 0.f ? -INFINITY : (m - T::POFF) * kLn2 + logf(l);
}

// Called by one thread, after a barrier behind which all of the block's writes lie: counts this block in and
// says whether it is the last of its group. The counter is zero again then, and what the others wrote is visible.
__device__ __forceinline__ int count_in(const AttnParams& p, const JoinGroup& g) {
  if (g.counter < 0) return 1;
  int* const counter = p.counters + g.counter;
  int before;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
  if (before != g.size - 1) return 0;
  *counter = 0;
  return 1;
}

// Joins the n partials of blocks first, first + step, ... counted from the segment's first: with LAST, into the
// segment's result; otherwise into the first of them. One block works alone here, with few warps, so what
// counts is the number of latencies and of instructions: bulk copies bring the partials to the
// ring, which is free by now, as many at a time as fit; the warps turn maxima and sums into one weight per
// partial and head, and each thread adds up its channels.
template <class T, int D>
__device__ __forceinline__ void join(const AttnParams& p, const Shared& s, int first, int step, int n, bool last, uint8_t* ring,
                                     float* meet, uint32_t bar, uint32_t& phase) {
  constexpr size_t PF = attn_partial_floats(T::HEADS, D);
  constexpr int THREADS = T::THREADS, COLS = T::HEADS * D / 4 / THREADS;
  static_assert(T::FIT >= 2 && T::FIT <= 32 && T::HEADS * D / 4 % THREADS == 0 && (T::FIT + 3) * T::HEADS * 4 <= kAttnRings * T::MEET, "join");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto part = [&](int i) {
    const int at = first + i * step;
    return p.partials + static_cast<size_t>(2 * (s.c0 + at) + (at == 0)) * PF;
  };
  const float* const in = reinterpret_cast<const float*>(ring);
  // [k + 1][HEADS]: of this round's partials, and of the rounds before; then the maximum and sum per head so far
  float* const weight = meet;
  float* const all = meet + (T::FIT + 1) * T::HEADS;
  float4 a[COLS];
#pragma unroll
  for (int c = 0; c < COLS; ++c) a[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += T::FIT) {
    const int k = min(T::FIT, n - i0);
    if (warp == 0) {
      const uint32_t bytes = (2 * T::HEADS + s.heads * D) * 4;
      // other blocks' ordinary writes, which count_in made visible, before the copies that read them
      asm volatile("fence.proxy.async;" ::: "memory");
      if (lane == 0) mbar_arrive_expect_tx(bar, k * bytes);
      __syncwarp();
      if (lane < k)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem_u32(ring) + lane * static_cast<uint32_t>(PF * 4)),
                     "l"(part(i0 + lane)), "r"(bytes), "r"(bar)
                     : "memory");
    }
    if (!mbar_wait(bar, phase, nullptr)) set_status(p.status, TL_ETIMEOUT);
    phase ^= 1;
    for (int h = warp; h < s.heads; h += THREADS / 32) {
      const float m = lane < k ? in[lane * PF + h] : -INFINITY, l = lane < k ? in[lane * PF + T::HEADS + h] : 0.f;
      const float m0 = i0 > 0 ? all[h] : -INFINITY, l0 = i0 > 0 ? all[T::HEADS + h] : 0.f;
      float top = fmaxf(m, m0);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float base = top == -INFINITY ? 0.f : top, w = faded(m - base), w0 = faded(m0 - base);
      float sum = w * l;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane < k) weight[lane * T::HEADS + h] = w;
      if (lane == 0) {
        weight[T::FIT * T::HEADS + h] = w0;
        all[h] = top;
        all[T::HEADS + h] = sum + w0 * l0;
      }
    }
    __syncthreads();
    const float4* v = reinterpret_cast<const float4*>(in + 2 * T::HEADS) + tid;
    const float* w = weight;
    if (i0 > 0) {
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        const float f = weight[T::FIT * T::HEADS + (tid + c * THREADS) / (D / 4)];
        a[c].x *= f, a[c].y *= f, a[c].z *= f, a[c].w *= f;
      }
    }
    // (heads past s.heads add up whatever lies there, which is not written out: no branches)
#pragma unroll 4
    for (int i = 0; i < k; ++i, v += PF / 4, w += T::HEADS) {
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        const float f = w[(tid + c * THREADS) / (D / 4)];
        const float4 x = v[c * THREADS];
        a[c].x += f * x.x;
        a[c].y += f * x.y;
        a[c].z += f * x.z;
        a[c].w += f * x.w;
      }
    }
    if (i0 + T::FIT < n) {
      fence_proxy_async_smem();
      __syncthreads();
    }
  }
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    const int x = tid + c * THREADS, h = x / (D / 4), d = 4 * (x % (D / 4));
    if (h < s.heads) {
      if (last) {
        write_out<T>(p, s.b, s.h0 + h, d, D, a[c], all[h], all[T::HEADS + h], s.v_scale);
      } else {
        float* const dst = part(0);
        reinterpret_cast<float4*>(dst + 2 * T::HEADS)[x] = a[c];
        if (d == 0) {
          dst[h] = all[h];
          dst[T::HEADS + h] = all[T::HEADS + h];
        }
      }
    }
  }
  fence_proxy_async_smem();
  __syncthreads();            // `meet` and the ring are free again
}

// The same of up to kJoinFew partials, all of a segment's: every thread reads what it needs at once, one latency.
template <class T, int D>
__device__ __forceinline__ void join_few(const AttnParams& p, const Shared& s) {
  constexpr size_t PF = attn_partial_floats(T::HEADS, D);
  for (int x = threadIdx.x; x < s.heads * (D / 4); x += T::THREADS) {
    const int h = x / (D / 4);
    float m[kJoinFew], l[kJoinFew], top = -INFINITY;
    float4 v[kJoinFew];
#pragma unroll
    for (int i = 0; i < kJoinFew; ++i) {
      m[i] = -INFINITY, l[i] = 0.f, v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < s.n) {
        const float* const q = p.partials + static_cast<size_t>(2 * (s.c0 + i) + (i == 0)) * PF;
        m[i] = __ldcg(q + h);
        l[i] = __ldcg(q + T::HEADS + h);
        v[i] = __ldcg(reinterpret_cast<const float4*>(q + 2 * T::HEADS) + x);
      }
      top = fmaxf(top, m[i]);
    }
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kJoinFew; ++i) {
      const float f = faded(m[i] - base);
      sum += f * l[i];
      a.x += f * v[i].x;
      a.y += f * v[i].y;
      a.z += f * v[i].z;
      a.w += f * v[i].w;
    }
    write_out<T>(p, s.b, s.h0 + h, 4 * (x % (D / 4)), D, a, top, sum, s.v_scale);
  }
}

// What a block does that arrived as the last of its group of partials; ring, meet, flag and barrier in shared memory.
template <class T, int D>
__device__ __forceinline__ void finish(const AttnParams& p, const Shared& s, uint8_t* ring, float* meet, int* flag, uint32_t bar,
                                       uint32_t& phase) {
  if (s.n <= kJoinFew) {
    join_few<T, D>(p, s);
    return;
  }
  for (int step = 1, level = 0;; ++level) {
    const JoinGroup g = join_group(static_cast<int>(blockIdx.x), s.c0, s.n, s.fan, step, level);
    const bool last = g.first == 0 && step * s.fan >= s.n;
    join<T, D>(p, s, g.first, step, g.size, last, ring, meet, bar, phase);
    if (last) return;
    step *= s.fan;
    if (threadIdx.x == 0) *flag = count_in(p, join_group(static_cast<int>(blockIdx.x), s.c0, s.n, s.fan, step, level + 1));
    __syncthreads();
    if (*flag == 0) return;
  }
}

enum AttnMode {
  kList,      // the list of tiles, in equal shares
  kCluster,   // a cluster of blocks takes a segment, and joins it through its shared memory
  kSolo       // each ring takes whole segments for itself, of KT keys a tile: no meetings, no joins
};

template <int CACHE, int D, int HW, int NT, AttnMode MODE>
__global__ void __launch_bounds__(kAttnRings * HW * 32, Traits<CACHE, D, HW, NT>::BLOCKS)
paged_attention_kernel(const __grid_constant__ AttnParams p) {
  using T = Traits<CACHE, D, HW, NT>;
  constexpr bool CL = MODE == kCluster, SOLO = MODE == kSolo;
  constexpr int TILE = SOLO ? T::KT : T::TILE;        // keys of a tile, of the whole block or of one ring
  constexpr int KT = T::KT, ROW = T::ROW, MT = KT / 16, DT = D / 16, S = T::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_bar;
  __shared__ int s_last[2];
  __shared__ Shared s_pend[2];                        // segments shared with other blocks: the first, the last
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int w = warp / HW, hw = warp % HW;            // the warp's ring, and its 8 NT heads
  const int HG = p.kv_heads * p.groups_per_kv;

  pdl_wait_prior();

  long long share = 0, t0 = 0;
  int count;                                          // places of this block's share
  int skip;                                           // places of the first segment that lie before t0
  Segment cur;
  if constexpr (CL) {
    // ---- an equal part of a segment's tiles
    const int seg = blockIdx.x >> p.cluster_log, rank = blockIdx.x & ((1 << p.cluster_log) - 1);
    cur.b = seg / HG;
    cur.h = seg - cur.b * HG;
    const int len = __ldg(p.lens + cur.b);
    if ((len < 0 || len > p.max_len) && tid == 0) set_status(p.status, TL_EDATA);
    seg_keys(p, len, TILE, cur);
    cur.tile = static_cast<int>(static_cast<long long>(cur.tiles) * rank >> p.cluster_log);
    count = static_cast<int>(static_cast<long long>(cur.tiles) * (rank + 1) >> p.cluster_log) - cur.tile;
    skip = 1;
  } else if constexpr (SOLO) {
    // ---- the block's segments, shared out to its rings; `count` of them, whole
    const long long segments = static_cast<long long>(p.B) * HG;
    const long long s0 = segments * blockIdx.x / gridDim.x;
    const int n = static_cast<int>(segments * (blockIdx.x + 1) / gridDim.x - s0);
    const long long mine = s0 + static_cast<long long>(n) * w / kAttnRings;
    count = static_cast<int>(s0 + static_cast<long long>(n) * (w + 1) / kAttnRings - mine);
    if (count == 0) return;
    cur.b = static_cast<int>(divide(mine, HG));
    cur.h = static_cast<int>(mine - static_cast<long long>(cur.b) * HG);
    const int len = __ldg(p.lens + cur.b);
    if ((len < 0 || len > p.max_len) && lane == 0) set_status(p.status, TL_EDATA);
    seg_keys(p, len, TILE, cur);
    cur.tile = 0;
    skip = 1;
  } else {
    // ---- the share of this block: `count` places from t0 of the list, in which a segment has one place for
    // what it costs besides its tiles, then its tiles. Every warp finds it for itself.
    long long total = 0;
    int len = 0;
    bool bad = false;
    for (int base = 0; base < p.B; base += 32) {
      len = base + lane < p.B ? __ldg(p.lens + base + lane) : 0;
      bad |= len < 0 || len > p.max_len;
      seg_keys(p, len, TILE, cur);
      if (base + lane < p.B) total += cur.tiles + 1;
    }
    if (bad && blockIdx.x == 0) set_status(p.status, TL_EDATA);
    // a lane's sum is below 2^50 (2^27 tiles a request, 2^23 requests a lane)
    total = static_cast<long long>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(total & 0x1FFFFFF))) +
            (static_cast<long long>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(total >> 25))) << 25);
    total *= HG;
    share = divide(total + gridDim.x - 1, gridDim.x);
    t0 = share * blockIdx.x;
    if (t0 >= total) return;
    count = static_cast<int>(min(share, total - t0));
    long long run = 0;                                // places of the requests before this round's, of one head group
    for (int base = 0;; base += 32) {
      if (p.B > 32) len = base + lane < p.B ? __ldg(p.lens + base + lane) : 0;
      seg_keys(p, len, TILE, cur);
      const unsigned places = base + lane < p.B ? cur.tiles + 1 : 0;
      unsigned incl = places;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned at = __ballot_sync(0xffffffffu, t0 < HG * (run + incl));
      if (at != 0) {
        const int who = __ffs(at) - 1;
        cur.b = base + who;
        seg_keys(p, __shfl_sync(0xffffffffu, len, who), TILE, cur);
        const long long left = t0 - HG * (run + __shfl_sync(0xffffffffu, incl - places, who));
        cur.h = static_cast<int>(divide(left, cur.tiles + 1));
        skip = static_cast<int>(left - cur.h * (cur.tiles + 1ll));
        cur.tile = max(skip - 1, 0);
        break;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
  }

  // ---- the ring, filled by its HW warps together
  const uint32_t ring = smem_u32(smem) + w * S * T::BUF;
  float* const meet = reinterpret_cast<float*>(smem + kAttnRings * S * T::BUF);
  auto ring_sync = [&]() {
    if constexpr (HW == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + w), "n"(HW * 32) : "memory");
  };

  const int at0 = SOLO ? 0 : w * KT;                  // the ring's first key of a tile
  constexpr int CPR = ROW / 16;                       // 16-byte chunks of a row
  constexpr int RPI = 32 / CPR;                       // rows that one instruction of a warp copies
  constexpr int KPL = (KT + 31) / 32;                 // keys whose address a lane computes
  static_assert(16 / RPI * MT % HW == 0, "rows are shared out evenly");
  Segment ld = cur;
  int next_len = 0;                                   // length of the request after ld's
  int pid[KPL];
  const int chunk = (lane % CPR) * 16, row0 = lane / CPR;
  auto fetch_len = [&]() {
    if constexpr (!CL) next_len = ld.b + 1 < p.B ? __ldg(p.lens + ld.b + 1) : 0;
  };
  auto fetch_pages = [&]() {
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const int key = ld.begin + ld.tile * TILE + at0 + i * 32 + lane;
      pid[i] = key >= ld.first && key < ld.end && i * 32 + lane < KT ? __ldg(p.pages + ld.b * p.ldp + p.page.div(key)) : -1;
    }
  };
  int left = count - (skip == 0);                     // places of the tiles (kSolo: segments) not yet asked for
  fetch_len();
  if (left > 0) fetch_pages();
  auto load_tile = [&](int stage) {
    if (left > 0) {
      const int k0 = ld.begin + ld.tile * TILE + at0;
      if (k0 < ld.end) {
        const int kvh = ld.h / p.groups_per_kv;
        int64_t off[KPL];                             // bytes from the cache's first row to key i * 32 + lane; -1: no such row
        bool bad = false;
#pragma unroll
        for (int i = 0; i < KPL; ++i) {
          const int key = k0 + i * 32 + lane;
          off[i] = -1;
          if (key >= ld.first && key < ld.end && i * 32 + lane < KT) {
            if (static_cast<unsigned>(pid[i]) < static_cast<unsigned>(p.num_pages))
              off[i] = pid[i] * p.page_stride + kvh * p.head_stride +
                       static_cast<int64_t>(key - p.page.div(key) * p.page.d) * p.token_stride;
            else
              bad = true;
          }
        }
        const uint32_t kb = ring + stage * T::BUF;
        // a tile of whole pages, or parts of pages, of 16 rows each: one address for 16 rows
        if (p.runs16 && k0 >= ld.first && k0 + KT <= ld.end && !__any_sync(0xffffffffu, bad)) {
#pragma unroll
          for (int x = 0; x < 16 / RPI * MT / HW; ++x) {
            const int step = x * HW + hw, j = step / (16 / RPI), i = step % (16 / RPI);
            const int64_t o = __shfl_sync(0xffffffffu, off[KPL == 1 ? 0 : j / 2], (16 * j) & 31) +
                              static_cast<int64_t>(i * RPI + row0) * p.token_stride + chunk;
            const uint32_t dst = kb + at<ROW>(step * RPI + row0, chunk >> 4);
            cp_async16(dst, p.k + o);
            cp_async16(dst + KT * ROW, p.v + o);
          }
        } else {
          if (bad) set_status(p.status, TL_EDATA);
#pragma unroll
          for (int x = 0; x < KT / RPI / HW; ++x) {
            const int r = (x * HW + hw) * RPI + row0;
            const int64_t o = __shfl_sync(0xffffffffu, off[KPL == 1 ? 0 : (x * HW + hw) * RPI / 32], r & 31);
            const uint32_t bytes = o < 0 ? 0u : 16u;
            const int64_t src = (o < 0 ? 0 : o) + chunk;
            const uint32_t dst = kb + at<ROW>(r, chunk >> 4);
            cp_async16(dst, p.k + src, bytes);
            cp_async16(dst + KT * ROW, p.v + src, bytes);
          }
        }
      }
      if constexpr (!SOLO) --left;
      if (++ld.tile == ld.tiles) {
        ld.tile = 0;
        --left;
        if (++ld.h == HG) {
          ld.h = 0;
          ++ld.b;
          if (SOLO && (next_len < 0 || next_len > p.max_len) && left > 0 && lane == 0) set_status(p.status, TL_EDATA);
          seg_keys(p, next_len, TILE, ld);
          fetch_len();
        }
      }
      if (left > 0) fetch_pages();
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) load_tile(i);

  // ---- the segments
  int stage = 0, done = skip == 0;
  bool starts_before = cur.tile > 0;
  // queries as B operands: k = 16 channels, n = 8 heads. For an 8-bit cache thread t takes channels
  // 4t .. 4t + 3, as its ldmatrix of K gives them. Asked for while the segment before is being finished.
  uint32_t qf[DT][NT][2];
  int h0, heads;
  float kscale = 1.f, vscale = 1.f;
  auto fetch_q = [&]() {
    const int kvh = cur.h / p.groups_per_kv;
    h0 = kvh * p.group + (cur.h - kvh * p.groups_per_kv) * T::HEADS;
    heads = min(T::HEADS, kvh * p.group + p.group - h0);
    if constexpr (T::F8) {
      kscale = __ldg(p.k_scale + kvh);
      vscale = __ldg(p.v_scale + kvh);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = 8 * (hw * NT + n) + g;
      const uint16_t* qr = p.q + cur.b * p.ldq + static_cast<int64_t>(h0 + h) * D;
      const bool live = h < heads;
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        if constexpr (T::F8) {
          const uint2 x = live ? __ldg(reinterpret_cast<const uint2*>(qr + 16 * i + 4 * t)) : make_uint2(0, 0);
          qf[i][n][0] = x.x;
          qf[i][n][1] = x.y;
        } else {
          qf[i][n][0] = live ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * i + 2 * t)) : 0u;
          qf[i][n][1] = live ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * i + 8 + 2 * t)) : 0u;
        }
      }
    }
  };
  fetch_q();
  if (MODE == kList && tid == 0) {
    s_pend[0].n = s_pend[1].n = 0;
    mbar_init(smem_u32(&s_bar), 1);
    fence_barrier_init();
  }
  while (CL || done < count) {
    // tiles of this segment in this block's share (none for some blocks of a cluster)
    const int here = SOLO ? cur.tiles : min(cur.tiles - cur.tile, count - done);

    float sc[NT][2];                                  // log2(e) scale of heads 2t and 2t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      sc[n][0] = sc[n][1] = p.scale_log2;
      if constexpr (T::F8) {
        float up = 1.f;
        if (p.q_bf16) {
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < DT; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 f = unpack2<true>(qf[i][n][e]);
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // 2^e <= top < 2^(e + 1); e is kept where both 2^e and 2^-e are normal (an infinite or NaN q stays one)
          const int e = min(max(static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127, -126), 126);
          up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
          const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
          for (int i = 0; i < DT; ++i) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float2 f = unpack2<true>(qf[i][n][x]);
              qf[i][n][x] = pack2<false>(f.x * down, f.y * down);
            }
          }
        }
        sc[n][0] *= kscale * __shfl_sync(0xffffffffu, up, 8 * t);    // head 2t is lane group g = 2t
        sc[n][1] *= kscale * __shfl_sync(0xffffffffu, up, 8 * t + 4);
      }
    }

    float m[NT][2], l[NT][2], o[DT][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }
    for (int it = 0; it < here; ++it) {
      cp_async_wait<S - 2>();
      ring_sync();
      load_tile(stage == 0 ? S - 1 : stage - 1);      // the buffer that the last turn read
      const int k0 = cur.begin + (cur.tile + it) * TILE + at0;
      const uint32_t kb = ring + stage * T::BUF, vb = kb + KT * ROW;
      if (k0 < cur.end) {
        float s[MT][NT][4], s2[MT][NT][4];            // two chains of dependent MMAs
#pragma unroll
        for (int j = 0; j < MT; ++j) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][n][e] = s2[j][n][e] = 0.f;
          const int r = 16 * j + (lane & 15);
          if constexpr (T::F8) {
#pragma unroll
            for (int i = 0; i < DT; i += 2) {
              uint32_t x[4];
              ldsm4(kb + at<ROW>(r, i + (lane >> 4)), x);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t a[4] = {widen_lo(x[2 * e]), widen_lo(x[2 * e + 1]), widen_hi(x[2 * e]), widen_hi(x[2 * e + 1])};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma<false>(e ? s2[j][n] : s[j][n], a, qf[i + e][n][0], qf[i + e][n][1]);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < DT; ++i) {
              uint32_t a[4];
              ldsm4(kb + at<ROW>(r, 2 * i + (lane >> 4)), a);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma<T::BF16>(i & 1 ? s2[j][n] : s[j][n], a, qf[i][n][0], qf[i][n][1]);
            }
          }
        }
        // rows 16 j + g (elements 0, 1) and + 8 (2, 3); columns: heads 2t, 2t + 1
        const int live = cur.end - k0, early = cur.first - k0;
        bool moved = false;
        float al[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            const int r = 16 * j + g;
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][n][e] = (s[j][n][e] + s2[j][n][e]) * sc[n][e & 1];
            if (live < KT) {
              if (r >= live) s[j][n][0] = s[j][n][1] = -INFINITY;
              if (r + 8 >= live) s[j][n][2] = s[j][n][3] = -INFINITY;
            }
            if (early > 0) {
              if (r < early) s[j][n][0] = s[j][n][1] = -INFINITY;
              if (r + 8 < early) s[j][n][2] = s[j][n][3] = -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = m[n][e];
#pragma unroll
            for (int j = 0; j < MT; ++j) top = fmaxf(top, fmaxf(s[j][n][e], s[j][n][e + 2]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            moved |= top != m[n][e];
            // no key seen so far scored above -inf: any finite base will do
            const float base = top == -INFINITY ? 0.f : top;
            al[n][e] = faded(m[n][e] - base);
            m[n][e] = top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              s[j][n][e] = exp2_approx(s[j][n][e] - (base - T::POFF));
              s[j][n][e + 2] = exp2_approx(s[j][n][e + 2] - (base - T::POFF));
              sum += s[j][n][e] + s[j][n][e + 2];
            }
            l[n][e] = l[n][e] * al[n][e] + sum;
          }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int i = 0; i < DT; ++i) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              o[i][n][0] *= al[n][0];
              o[i][n][1] *= al[n][1];
              o[i][n][2] *= al[n][0];
              o[i][n][3] *= al[n][1];
            }
          }
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = s[j][n][2 * e], y = s[j][n][2 * e + 1];
              // e4m3 has no infinities: there the high part is the nearest, its low part has either sign
              const uint32_t hi = T::F8 ? pack2<T::BF16>(x, y) : pack2_down<T::BF16>(x, y);
              const float2 back = unpack2<T::BF16>(hi);
              const uint32_t lo = pack2<T::BF16>(x - back.x, y - back.y);
              ph[n][e] = transpose8x8(hi);
              pl[n][e] = transpose8x8(T::F8 ? lo : above_zero<T::BF16>(lo));
            }
          }
          if constexpr (T::F8) {
            const int r = 16 * j + (lane & 15);
#pragma unroll
            for (int i = 0; i < DT; i += 2) {
              uint32_t x[4];
              ldsm4t(vb + at<ROW>(r, i + (lane >> 4)), x);
              uint32_t a[2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // bytes (key 2t: d, d + 1; key 2t + 1: d, d + 1) -> (d of both keys, d + 1 of both keys)
                const uint32_t y = __byte_perm(x[2 * e], 0, 0x3120), z = __byte_perm(x[2 * e + 1], 0, 0x3120);
                a[e][0] = widen_lo(y), a[e][1] = widen_hi(y), a[e][2] = widen_lo(z), a[e][3] = widen_hi(z);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) mma<false>(o[i + e][n], a[e], ph[n][0], ph[n][1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) mma<false>(o[i + e][n], a[e], pl[n][0], pl[n][1]);
              }
            }
          } else {
            const int r = 16 * j + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int i = 0; i < DT; i += 4) {         // four independent MMAs before the first dependent one
              uint32_t a[4][4];
#pragma unroll
              for (int e = 0; e < 4; ++e) ldsm4t(vb + at<ROW>(r, 2 * (i + e) + ((lane >> 3) & 1)), a[e]);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) mma<T::BF16>(o[i + e][n], a[e], ph[n][0], ph[n][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mma<T::BF16>(o[i + e][n], a[e], pl[n][0], pl[n][1]);
              }
            }
          }
        }
      }
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    done += SOLO ? 1 : here;

    // ---- the warps meet: each leaves (m, l, o) in shared memory
    float* const mo = meet + w * (T::MEET / 4);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
        const int h = 8 * (hw * NT + n) + 2 * t + e;
        if (g == 0) {
          mo[h] = m[n][e];
          mo[T::HEADS + h] = l[n][e];
        }
        float* row = mo + 2 * T::HEADS + h * T::OPITCH;
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          if constexpr (T::F8) {
            *reinterpret_cast<float2*>(row + 16 * i + 2 * g) = make_float2(o[i][n][e], o[i][n][e + 2]);
          } else {
            row[16 * i + g] = o[i][n][e];
            row[16 * i + g + 8] = o[i][n][e + 2];
          }
        }
      }
    }
    const Segment seg = cur;
    const int sh0 = h0, sheads = heads;
    const float vs = vscale;
    if constexpr (SOLO) {
      // a warp alone: its heads pass through its part of the ring's place of meeting to whole rows
      cur.tile = 0;
      if (++cur.h == HG) {
        cur.h = 0;
        ++cur.b;
        if (done < count) seg_keys(p, __ldg(p.lens + cur.b), TILE, cur);
      }
      if (done < count) fetch_q();
      __syncwarp();
      const int first_head = 8 * NT * hw, live = min(8 * NT, sheads - first_head);
      for (int x = lane; x < live * (D / 4); x += 32) {
        const int h = first_head + x / (D / 4), d = 4 * (x % (D / 4));
        const float4 v = *reinterpret_cast<const float4*>(mo + 2 * T::HEADS + h * T::OPITCH + d);
        write_out<T>(p, seg.b, sh0 + h, d, D, v, mo[h], mo[T::HEADS + h], vs);
      }
      __syncwarp();
      continue;
    }
    const bool whole = CL ? p.cluster_log == 0 : !starts_before && seg.tile + here == seg.tiles, second = !starts_before;
    const long long first = t0 + (done - here) - seg.tile;      // the place of its first tile
    if constexpr (CL) {
      pdl_launch_dependents();
      cp_async_wait<0>();                             // the ring is where the block's result goes
    } else {
      ++done;                                         // the next segment's first place
      starts_before = false;
      cur.tile = 0;
      if (++cur.h == HG) {
        cur.h = 0;
        ++cur.b;
        if (done < count) seg_keys(p, __ldg(p.lens + cur.b), TILE, cur);
      }
      if (done < count) fetch_q();
    }
    __syncthreads();
    float* const part = CL ? reinterpret_cast<float*>(smem)
                           : p.partials + (static_cast<size_t>(blockIdx.x) * 2 + second) * attn_partial_floats(T::HEADS, D);
    for (int x = tid; x < sheads * (D / 4); x += T::THREADS) {
      const int h = x / (D / 4), d = 4 * (x % (D / 4));
      float mw[kAttnRings], top = -INFINITY;
#pragma unroll
      for (int r = 0; r < kAttnRings; ++r) {
        mw[r] = meet[r * (T::MEET / 4) + h];
        top = fmaxf(top, mw[r]);
      }
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < kAttnRings; ++r) {
        const float* q = meet + r * (T::MEET / 4) + T::HEADS;
        const float f = faded(mw[r] - base);
        const float4 v = *reinterpret_cast<const float4*>(q + T::HEADS + h * T::OPITCH + d);
        sum += f * q[h];
        a.x += f * v.x;
        a.y += f * v.y;
        a.z += f * v.z;
        a.w += f * v.w;
      }
      if (whole) {
        write_out<T>(p, seg.b, sh0 + h, d, D, a, top, sum, vs);
      } else {
        if (d == 0) {
          part[h] = top;
          part[T::HEADS + h] = sum;
        }
        *reinterpret_cast<float4*>(part + 2 * T::HEADS + h * D + d) = a;
      }
    }
    if constexpr (CL) {
      if (whole) return;
      // ---- the cluster's blocks join: each takes an equal part of the channels
      cluster_sync();
      const int size = 1 << p.cluster_log, rank = blockIdx.x & (size - 1);
      const uint32_t mine = smem_u32(smem);
      for (int x = rank * T::THREADS + tid; x < sheads * (D / 4); x += size * T::THREADS) {
        const int h = x / (D / 4), d = 4 * (x % (D / 4));
        float top = -INFINITY, sum = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        // N blocks' results with one latency
        auto take = [&](auto count, int r0) {
          constexpr int N = decltype(count)::value;
          float mr[N], lr[N], most = top;
          float4 v[N];
#pragma unroll
          for (int r = 0; r < N; ++r) {
            mr[r] = ld_cluster(mine + 4 * h, r0 + r);
            lr[r] = ld_cluster(mine + 4 * (T::HEADS + h), r0 + r);
            v[r] = ld_cluster4(mine + 4 * (2 * T::HEADS + h * D + d), r0 + r);
            most = fmaxf(most, mr[r]);
          }
          const float base = most == -INFINITY ? 0.f : most, f0 = faded(top - base);
          top = most;
          sum *= f0, a.x *= f0, a.y *= f0, a.z *= f0, a.w *= f0;
#pragma unroll
          for (int r = 0; r < N; ++r) {
            const float f = faded(mr[r] - base);
            sum += f * lr[r];
            a.x += f * v[r].x;
            a.y += f * v[r].y;
            a.z += f * v[r].z;
            a.w += f * v[r].w;
          }
        };
        if (size >= 8)
          for (int r0 = 0; r0 < size; r0 += 8) take(std::integral_constant<int, 8>{}, r0);
        else if (size == 4)
          take(std::integral_constant<int, 4>{}, 0);
        else
          take(std::integral_constant<int, 2>{}, 0);
        write_out<T>(p, seg.b, sh0 + h, d, D, a, top, sum, vs);
      }
      cluster_sync();                                 // no block leaves while another reads its result
      return;
    }
    __syncthreads();          // the partial is written, and `meet` is free again
    if (!whole && tid == 0) {
      // Blocks c0 .. c0 + n - 1 share this segment. Thread 0 says that this block's partial is there; who
      // joins them is looked up when the block has nothing else to do.
      const int c0 = static_cast<int>(divide(first, share));
      const int n = static_cast<int>(divide(first + seg.tiles - 1, share)) - c0 + 1;
      const int fan = join_fan(n, sheads * D * 4);
      s_pend[second] = Shared{c0, n, fan, seg.b, sh0, sheads, vs};
      s_last[second] = count_in(p, join_group(static_cast<int>(blockIdx.x), c0, n, fan, 1, 0));
    }
  }
  if constexpr (SOLO) return;
  pdl_launch_dependents();             // the stream is over: the next kernel may begin its own beside the joins
  cp_async_wait<0>();
  fence_proxy_async_smem();            // joins copy to the ring by the async proxy
  __syncthreads();
  uint32_t phase = 0;
#pragma unroll 1
  for (int e = 0; e < 2; ++e)
    if (s_pend[e].n > 0 && s_last[e]) finish<T, D>(p, s_pend[e], smem, meet, s_last + e, smem_u32(&s_bar), phase);
}

template <int CACHE, int D, int HW, int NT>
cudaError_t launch(const AttnParams& p, int sms, cudaStream_t st) {
  using T = Traits<CACHE, D, HW, NT>;
  // by device: blocks per SM, and how many clusters of 2^i blocks run at once
  static int per_sm[64], at_once[64][kAttnClusterLog + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = __atomic_load_n(&per_sm[dev], __ATOMIC_ACQUIRE);
  if (n == 0) {
    for (auto* kernel : {paged_attention_kernel<CACHE, D, HW, NT, kList>, paged_attention_kernel<CACHE, D, HW, NT, kCluster>,
                         paged_attention_kernel<CACHE, D, HW, NT, kSolo>}) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM);
      if (e != cudaSuccess) return e;
    }
    auto* const kernel = paged_attention_kernel<CACHE, D, HW, NT, kCluster>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, paged_attention_kernel<CACHE, D, HW, NT, kList>, T::THREADS, T::SMEM);
    if (e != cudaSuccess) return e;
    n = n < 1 ? 1 : n > kAttnMaxBlocksPerSm ? kAttnMaxBlocksPerSm : n;
    __atomic_store_n(&at_once[dev][0], sms * n, __ATOMIC_RELAXED);
    for (int log = 1; log <= kAttnClusterLog; ++log) {
      cudaLaunchAttribute size;
      size.id = cudaLaunchAttributeClusterDimension;
      size.val.clusterDim.x = 1 << log, size.val.clusterDim.y = size.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1 << log), cfg.blockDim = dim3(T::THREADS), cfg.dynamicSmemBytes = T::SMEM;
      cfg.attrs = &size, cfg.numAttrs = 1;
      int clusters = 0;
      e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
      if (e != cudaSuccess) return e;
      __atomic_store_n(&at_once[dev][log], clusters, __ATOMIC_RELAXED);
    }
    __atomic_store_n(&per_sm[dev], n, __ATOMIC_RELEASE);
  }
  const long long keys = p.window > 0 && p.window < p.max_len ? p.window : p.max_len;
  const long long segments = static_cast<long long>(p.B) * p.kv_heads * p.groups_per_kv;
  long long grid = static_cast<long long>(sms) * n;
  if (grid > kAttnMaxGrid) grid = kAttnMaxGrid;
  // Few segments: a cluster each, of 16 to 1 blocks, the most of which all run at once (sixteens on SMs of their own), while a
  // block has eight tiles at most. A cluster of 16 is for more than 8 tiles, of 8 for more than 4, of 4 for more than 2, as blocks
  // without a tile only lengthen the join; a pair for more than 4, as up to there a single block is as fast (the last figures
  // here). The last list figure is a loss that the rule accepts. bf16, 128 channels, list against clusters:
  // 4 segments of 4000 keys 14.5, 10.1 (7.5 with sixteens), 5 of 8000 14.5, 11.1; 36 of 2000 12.1, 9.0; 56 of 600 9.9, 7.5; 152 of
  // 600 14.2, 10.2; 300 of 200 8.6, 6.9, of 50 to 400 12.8, 8.7, of 100 to 800 16.8, 15.3, of 187 to 1500 24.7, 27.4. Pairs
  // against single blocks: 152 of 200 6.7, 5.9, of 400 8.3, 9.0. Clusters that do not all run at once lose (256
  // channels, 16 eights: list 10.5, eights 11.5).
  const long long tiles = (keys + T::TILE - 1) / T::TILE;
  for (int log = kAttnClusterLog; log >= 0; --log) {
    const int c = 1 << log;
    if (segments > __atomic_load_n(&at_once[dev][log], __ATOMIC_RELAXED) / (c == 16 ? n : 1)) continue;
    if (tiles <= (c == 16 ? 8 : c == 8 || c == 2 ? 4 : c == 4 ? 2 : 0)) continue;
    if (tiles > 8 * c) break;
    AttnParams shared = p;
    shared.cluster_log = log;
    return launch_pdl_cluster(paged_attention_kernel<CACHE, D, HW, NT, kCluster>, dim3(static_cast<unsigned>(segments * c)),
                              dim3(T::THREADS), T::SMEM, st, c, shared);
  }
  // Many short ones: a ring for each, while that is one step or two, or eight where the blocks would have one and a half
  // segments each or more (bf16, 128 channels, 456 segments of 60 keys, 4 steps: 7.4 -> 6.4 us, of 120 9.8 -> 9.5; 912 of 120 13.1 ->
  // 10.0; the one loss known is 256 channels in 16 bits, where a block has an SM: 304 of 120 keys 10.9 -> 12.0).
  if (keys <= (2 * segments < 3 * grid ? 2 : 8) * T::KT)
    return launch_pdl(paged_attention_kernel<CACHE, D, HW, NT, kSolo>, dim3(static_cast<unsigned>(segments < grid ? segments : grid)),
                      dim3(T::THREADS), T::SMEM, st, p);
  // most places that the list can have; a window's tiles may begin up to 15 keys before it
  const long long most = segments * ((keys + 15 + T::TILE - 1) / T::TILE + 1);
  if (grid > most) grid = most;
  return launch_pdl(paged_attention_kernel<CACHE, D, HW, NT, kList>, dim3(static_cast<unsigned>(grid)), dim3(T::THREADS), T::SMEM, st, p);
}

// `columns`: 1, 2 or 4 times 8 query heads to a segment. A warp that takes 16 heads reads K and V half as often as two
// that take 8 each, and has the registers for it up to 128 channels.
template <int CACHE>
cudaError_t launch_dim(const AttnParams& p, int dim, int columns, int sms, cudaStream_t st) {
  switch (dim) {
    case 64:
      return columns == 1 ? launch<CACHE, 64, 1, 1>(p, sms, st)
             : columns == 2 ? launch<CACHE, 64, 1, 2>(p, sms, st)
                            : launch<CACHE, 64, 2, 2>(p, sms, st);
    case 128:
      return columns == 1 ? launch<CACHE, 128, 1, 1>(p, sms, st)
             : columns == 2 ? launch<CACHE, 128, 1, 2>(p, sms, st)
                            : launch<CACHE, 128, 2, 2>(p, sms, st);
    case 256: return columns == 1 ? launch<CACHE, 256, 1, 1>(p, sms, st) : launch<CACHE, 256, 2, 1>(p, sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
}  // namespace tl
