// Appending keys and values to a paged cache, with the rotary position applied
// to keys and queries on the way.
//
//   (a, b) -> (a c - b s, b c + a s)   for each pair of rotated channels
//
// in fp32, every product and sum rounded on its own, so that the result is
// the plain fp32 formula's bit for bit, and rounded once to the type that is stored. Each byte is
// read and written once: bound by HBM for prompts, by the launch and one chain of loads (slot
// and position, angles, data) for the few tokens of a decode step. One block takes one token: a thread owns
// 16 channels (two 16-byte vectors, which hold both halves of their 8 pairs in either pairing) at a
// fixed place of the head and walks over the heads, so it reads its angles once for all of them. Measured on
// GB300: 16000 tokens of 40 + 16 heads of 128, fp16: 72 us, 6.5 TB/s, 0.96 of the copy rate; 24 tokens of 24 + 8 heads of 256:
// 2.3 us, about what an empty kernel between others takes.
//
// With NORM every head of queries and keys is first divided by the root of its mean square and weighted: a head's lanes add their
// squares up by shuffles, in fp32, and nothing is rounded to the stored type in between. Instructions then weigh as much as bytes (issue slots 70 %
// busy, L1 59 %, 16000 tokens into 8 bits): squares, weights and products go two to an instruction. Weights lie in shared memory, by thread:
// from L1, 64 bytes apart, they were four lines to a read, and L1 was 84 % busy (92 us). Measured: those 16000 tokens, 40 + 16
// heads of 128, into 8 bits 79.5 us, into bf16 79.5 (floors 65 and 69); 4000 tokens of 24 + 8 heads of 256 25.5; 192 tokens of those 3.8.
#include "tl_internal.cuh"

#include <cuda_bf16.h>

#include "kv_append.cuh"

namespace tl {
namespace {

// 16 channels as 8 pairs: first and second elements. Pairs are neighbours, or lie across the two vectors.
template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& v0, const uint4& v1, bool neighbours, float2 (&x)[4], float2 (&y)[4]) {
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  float2 f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = BF16 ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)) : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = neighbours ? make_float2(f[2 * i].x, f[2 * i + 1].x) : f[i];
    y[i] = neighbours ? make_float2(f[2 * i].y, f[2 * i + 1].y) : f[4 + i];
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  uint32_t w;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

template <bool BF16>
__device__ __forceinline__ void narrow8(const float2 (&x)[4], const float2 (&y)[4], bool neighbours, uint4& v0, uint4& v1) {
  if (neighbours) {
    v0 = make_uint4(narrow2<BF16>(x[0].x, y[0].x), narrow2<BF16>(x[0].y, y[0].y), narrow2<BF16>(x[1].x, y[1].x), narrow2<BF16>(x[1].y, y[1].y));
    v1 = make_uint4(narrow2<BF16>(x[2].x, y[2].x), narrow2<BF16>(x[2].y, y[2].y), narrow2<BF16>(x[3].x, y[3].x), narrow2<BF16>(x[3].y, y[3].y));
  } else {
    v0 = make_uint4(narrow2<BF16>(x[0].x, x[0].y), narrow2<BF16>(x[1].x, x[1].y), narrow2<BF16>(x[2].x, x[2].y), narrow2<BF16>(x[3].x, x[3].y));
    v1 = make_uint4(narrow2<BF16>(y[0].x, y[0].y), narrow2<BF16>(y[1].x, y[1].y), narrow2<BF16>(y[2].x, y[2].y), narrow2<BF16>(y[3].x, y[3].y));
  }
}

__device__ __forceinline__ uint32_t narrow4_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return lo | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ void narrow8_e4m3(float2 (&x)[4], float2 (&y)[4], bool neighbours, float inv, uint2& v0, uint2& v1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __fmul2_rn(x[i], make_float2(inv, inv)), y[i] = __fmul2_rn(y[i], make_float2(inv, inv));
  if (neighbours) {
    v0 = make_uint2(narrow4_e4m3(x[0].x, y[0].x, x[0].y, y[0].y), narrow4_e4m3(x[1].x, y[1].x, x[1].y, y[1].y));
    v1 = make_uint2(narrow4_e4m3(x[2].x, y[2].x, x[2].y, y[2].y), narrow4_e4m3(x[3].x, y[3].x, x[3].y, y[3].y));
  } else {
    v0 = make_uint2(narrow4_e4m3(x[0].x, x[0].y, x[1].x, x[1].y), narrow4_e4m3(x[2].x, x[2].y, x[3].x, x[3].y));
    v1 = make_uint2(narrow4_e4m3(y[0].x, y[0].y, y[1].x, y[1].y), narrow4_e4m3(y[2].x, y[2].y, y[3].x, y[3].y));
  }
}

template <bool PACKED>
__device__ __forceinline__ float2 products(float2 a, float2 b) {
  if constexpr (PACKED) return __fmul2_rn(a, b);
  return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y));       // (the 48 registers of small blocks have no pairs to spare)
}

// the least power of two that is at least n <= 32
__host__ __device__ constexpr int power_of_two(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// lanes = head_dim / 16 threads cover a head; `rows` heads are taken at a time. With NORM they are a power of two of neighbouring
// lanes of one warp, the last of them idle for other sizes, and add up the squares of their head by shuffles.
template <bool BF16, bool F8, int THREADS, bool NORM>
__global__ void __launch_bounds__(THREADS, THREADS == 64 ? (NORM ? 14 : 20) : THREADS == 256 ? (NORM ? 2 : 4) : 1) kv_append_kernel(const __grid_constant__ AppendParams p) {
  const int lanes = NORM ? power_of_two(p.dim >> 4) : p.dim >> 4;
  const int row = threadIdx.x / lanes, j = threadIdx.x - row * lanes;
  const int rows = blockDim.x / lanes;
  const int tok = blockIdx.x;
  pdl_wait_prior();
  // (no early start for the next kernel, whose blocks would take this one's room: 1500 tokens, calls back to back, 12 us with it,
  // 6.5 without; 512 tokens 4.1 and 3.7)
  const int64_t slot = __ldg(p.slots + tok);
  const bool turn = 16 * j < p.rot;
  // the thread's two vectors of 8 channels: pairs (a[i], b[i]), or pairs of neighbours in a, then in b
  const int c0 = turn && !p.interleaved ? 8 * j : 16 * j;
  const int c1 = turn && !p.interleaved ? 8 * j + (p.rot >> 1) : 16 * j + 8;
  const bool idle = NORM && 16 * j >= p.dim;
  // q may be q_out: not the read-only path
  auto load = [&](int h, uint4& v0, uint4& v1) {
    if (idle) {
      v0 = v1 = make_uint4(0, 0, 0, 0);
      return;
    }
    const bool is_v = h >= p.q_heads + p.kv_heads;
    const uint16_t* src = h < p.q_heads ? p.q + tok * p.ldq + h * p.dim
                          : is_v        ? p.v + tok * p.ldv + (h - p.q_heads - p.kv_heads) * p.dim
                                        : p.k + tok * p.ldk + (h - p.q_heads) * p.dim;
    v0 = *reinterpret_cast<const uint4*>(src + c0);
    v1 = *reinterpret_cast<const uint4*>(src + c1);
  };
  // the first head's data wait for neither slot nor angles
  uint4 first0 = make_uint4(0, 0, 0, 0), first1 = first0;
  if (row < p.q_heads + 2 * p.kv_heads) load(row, first0, first1);
  // Norm weights, by thread of a head: float4 i of thread j at [i][j], where all heads' threads j read it with one wavefront.
  __shared__ float4 s_w[NORM ? 2 : 1][4][NORM ? 32 : 1];
  if constexpr (NORM) {
    for (int i = threadIdx.x; i < 8 * lanes; i += blockDim.x) {
      const int at = i % lanes, part = i / lanes % 4;
      const float* const w = i < 4 * lanes ? p.q_norm : p.k_norm;
      const int c = 16 * at < p.rot ? 8 * at + part % 2 * 4 + (part < 2 ? 0 : p.rot >> 1) : 16 * at + 4 * part;
      if (w == nullptr || 16 * at >= p.dim) continue;
      if (p.interleaved) {              // every other channel from 16 at + 8 (part % 2) on
        const float* const z = w + 16 * at + part % 2 * 8 + part / 2;
        s_w[i / (4 * lanes)][part][at] = make_float4(__ldg(z), __ldg(z + 2), __ldg(z + 4), __ldg(z + 6));
      } else {
        s_w[i / (4 * lanes)][part][at] = __ldg(reinterpret_cast<const float4*>(w + c));
      }
    }
  }
  bool ok = true;
  float cs[8], sn[8];
  if (p.rot > 0) {
    const int pos = __ldg(p.positions + tok);
    ok = static_cast<unsigned>(pos) < static_cast<unsigned>(p.max_pos);
    if (ok && turn) {
      const float* a = p.cos_sin + static_cast<int64_t>(pos) * p.rot + 8 * j;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(a) + h);
        const float4 s = __ldg(reinterpret_cast<const float4*>(a + (p.rot >> 1)) + h);
        cs[4 * h] = c.x, cs[4 * h + 1] = c.y, cs[4 * h + 2] = c.z, cs[4 * h + 3] = c.w;
        sn[4 * h] = s.x, sn[4 * h + 1] = s.y, sn[4 * h + 2] = s.z, sn[4 * h + 3] = s.w;
      }
    }
  }
  if (!ok || slot >= p.num_slots) {
    if (threadIdx.x == 0) set_status(p.status, TL_EDATA);
    if (!ok) return;
  }
  const bool keep = slot >= 0 && slot < p.num_slots;
  int64_t cell = 0;                     // element offset of the token's row in the cache
  if (keep) {
    const int64_t page = slot / p.page_size;
    cell = page * p.page_stride + (slot - page * p.page_size) * p.token_stride;
  }
  const int heads = p.q_heads + (keep ? 2 * p.kv_heads : 0);
  const unsigned head_lanes = NORM ? (lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1) << ((threadIdx.x & 31) / lanes * lanes)) : 0u;
  const float per_channel = 1.f / static_cast<float>(p.dim);
  auto store = [&](int h, const uint4& v0, const uint4& v1) {
    const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + p.kv_heads;
    const int kh = h - p.q_heads - (is_v ? p.kv_heads : 0);
    uint4 r0 = v0, r1 = v1;
    float2 x[4], y[4];                  // first and second elements of the 8 pairs
    const bool turned = turn && !is_v;
    const bool normed = NORM && !is_v && (is_q ? p.q_norm : p.k_norm) != nullptr;
    if (turned || normed || (F8 && !is_q)) {
      widen8<BF16>(v0, v1, p.interleaved, x, y);
    }
    if (normed) {
      float2 sums = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) sums = __ffma2_rn(y[i], y[i], __ffma2_rn(x[i], x[i], sums));
      float sum = sums.x + sums.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) sum += __shfl_xor_sync(head_lanes, sum, o);
      const float inv = __frsqrt_rn(sum * per_channel + p.eps);
      const float4(&weight)[4][NORM ? 32 : 1] = s_w[NORM && !is_q];
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float4 w = weight[i / 2][NORM ? j : 0], z = weight[2 + i / 2][NORM ? j : 0];
        const float2 by = make_float2(inv, inv);
        x[i] = __fmul2_rn(x[i], __fmul2_rn(by, make_float2(w.x, w.y)));
        x[i + 1] = __fmul2_rn(x[i + 1], __fmul2_rn(by, make_float2(w.z, w.w)));
        y[i] = __fmul2_rn(y[i], __fmul2_rn(by, make_float2(z.x, z.y)));
        y[i + 1] = __fmul2_rn(y[i + 1], __fmul2_rn(by, make_float2(z.z, z.w)));
      }
    }
    if (idle) return;
    if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = make_float2(cs[2 * i], cs[2 * i + 1]), s = make_float2(sn[2 * i], sn[2 * i + 1]), a = x[i], b = y[i];
        // (sums of pairs would be joined with the products to multiply-adds, rounded once)
        const float2 ac = products<NORM>(a, c), bs = products<NORM>(b, s), bc = products<NORM>(b, c), as = products<NORM>(a, s);
        x[i] = make_float2(__fsub_rn(ac.x, bs.x), __fsub_rn(ac.y, bs.y));
        y[i] = make_float2(__fadd_rn(bc.x, as.x), __fadd_rn(bc.y, as.y));
      }
    }
    if ((turned || normed) && (!F8 || is_q)) narrow8<BF16>(x, y, p.interleaved, r0, r1);
    if (is_q) {
      uint16_t* dst = p.q_out + tok * p.ldqo + h * p.dim;
      *reinterpret_cast<uint4*>(dst + c0) = r0;
      *reinterpret_cast<uint4*>(dst + c1) = r1;
    } else {
      const int64_t at = cell + kh * p.head_stride;
      if constexpr (F8) {
        const float inv = __frcp_rn(__ldg((is_v ? p.v_scale : p.k_scale) + kh));
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.cv : p.ck) + at;
        uint2 lo, hi;
        narrow8_e4m3(x, y, p.interleaved, inv, lo, hi);
        *reinterpret_cast<uint2*>(dst + c0) = lo;
        *reinterpret_cast<uint2*>(dst + c1) = hi;
      } else {
        uint16_t* dst = static_cast<uint16_t*>(is_v ? p.cv : p.ck) + at;
        *reinterpret_cast<uint4*>(dst + c0) = r0;
        *reinterpret_cast<uint4*>(dst + c1) = r1;
      }
    }
  };
  if constexpr (NORM) __syncthreads();
  if constexpr (NORM) {                 // the next head's data are on their way while this one's squares are summed (8 bits: 101 -> 92 us)
#pragma unroll 1
    for (int h = row; h < heads; h += rows) {
      uint4 v0, v1;
      load(h + rows < heads ? h + rows : h, v0, v1);
      store(h, first0, first1);
      first0 = v0, first1 = v1;
    }
    return;
  }
  if (row < heads) store(row, first0, first1);
#pragma unroll 2
  for (int h = row + rows; h < heads; h += rows) {
    uint4 v0, v1;
    load(h, v0, v1);
    store(h, v0, v1);
  }
}

template <int THREADS, bool NORM>
cudaError_t launch(const AppendParams& p, int T, bool bf16, bool f8, cudaStream_t st) {
  const int lanes = NORM ? power_of_two(p.dim / 16) : p.dim / 16;
  const dim3 grid(static_cast<unsigned>(T)), block(static_cast<unsigned>(THREADS / lanes * lanes));
  if (bf16)
    return f8 ? launch_pdl(kv_append_kernel<true, true, THREADS, NORM>, grid, block, 0, st, p)
              : launch_pdl(kv_append_kernel<true, false, THREADS, NORM>, grid, block, 0, st, p);
  return f8 ? launch_pdl(kv_append_kernel<false, true, THREADS, NORM>, grid, block, 0, st, p)
            : launch_pdl(kv_append_kernel<false, false, THREADS, NORM>, grid, block, 0, st, p);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, int T, bool bf16, bool f8, int sms, cudaStream_t st) {
  // One block for each token. Few tokens: all their heads at once, as the latency of one pass is the time (24 tokens of 32
  // heads of 256: 2.4 us with 512 threads, 2.6 with 256, 3.1 with 128, 4.4 with 64). Many: small blocks, which start and end
  // out of step and so keep the memory busy (40 + 16 heads of 128, us with 256, 128 and 64 threads: bf16, 512 tokens 4.1, 4.1, 5.0;
  // 1000: 6.9, 6.5, 7.9; 4000: 27.2, 22.1, 22.1; 16000: 97.8, 77.9, 72.0, 0.96 of the copy rate. Into 8 bits, where 64 threads have
  // 48 registers and spill some: 512: 4.0, 4.3, 6.1; 1000: 6.4, 5.5, 7.6; 4000: 27.8, 24.4, 25.5; 16000: 99.8, 86.3, 77.1, 0.82 of it).
  // Around 1000 tokens, and for 8 bits up to some thousand, the rule gives away up to a quarter of the time.
  // With norms 64 threads have 72 registers, 14 blocks an SM (12 or 16 of them: 87 us where 14 take 83.5; 18: 137).
  if (p.q_norm != nullptr || p.k_norm != nullptr)
    return T <= sms ? launch<512, true>(p, T, bf16, f8, st) : T < 4 * sms ? launch<256, true>(p, T, bf16, f8, st) : launch<64, true>(p, T, bf16, f8, st);
  return T <= sms ? launch<512, false>(p, T, bf16, f8, st) : T < 4 * sms ? launch<256, false>(p, T, bf16, f8, st) : launch<64, false>(p, T, bf16, f8, st);
}

}  // namespace tl
