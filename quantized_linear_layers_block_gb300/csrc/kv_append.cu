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
#include "tl_internal.cuh"

#include <cuda_bf16.h>

#include "kv_append.cuh"

namespace tl {
namespace {

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    else
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 narrow8_e4m3(const float (&f)[8], float inv) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(h[i])
        : "f"(__fmul_rn(f[2 * i + 1], inv)), "f"(__fmul_rn(f[2 * i], inv)));
  return make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16));
}

// lanes = head_dim / 16 threads cover a head; `rows` heads are taken at a time
template <bool BF16, bool F8, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 64 ? 20 : THREADS == 256 ? 4 : 1) kv_append_kernel(const __grid_constant__ AppendParams p) {
  const int lanes = p.dim >> 4;
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
  // q may be q_out: not the read-only path
  auto load = [&](int h, uint4& v0, uint4& v1) {
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
  auto store = [&](int h, const uint4& v0, const uint4& v1) {
    const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + p.kv_heads;
    const int kh = h - p.q_heads - (is_v ? p.kv_heads : 0);
    uint4 r0 = v0, r1 = v1;
    float a[8], b[8];
    const bool turned = turn && !is_v;
    if (turned || (F8 && !is_q)) {
      widen8<BF16>(v0, a);
      widen8<BF16>(v1, b);
    }
    if (turned) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = a[2 * i], y = a[2 * i + 1];
          a[2 * i] = __fsub_rn(__fmul_rn(x, cs[i]), __fmul_rn(y, sn[i]));
          a[2 * i + 1] = __fadd_rn(__fmul_rn(y, cs[i]), __fmul_rn(x, sn[i]));
          x = b[2 * i], y = b[2 * i + 1];
          b[2 * i] = __fsub_rn(__fmul_rn(x, cs[4 + i]), __fmul_rn(y, sn[4 + i]));
          b[2 * i + 1] = __fadd_rn(__fmul_rn(y, cs[4 + i]), __fmul_rn(x, sn[4 + i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = a[i], y = b[i];
          a[i] = __fsub_rn(__fmul_rn(x, cs[i]), __fmul_rn(y, sn[i]));
          b[i] = __fadd_rn(__fmul_rn(y, cs[i]), __fmul_rn(x, sn[i]));
        }
      }
      if (!F8 || is_q) {
        r0 = narrow8<BF16>(a);
        r1 = narrow8<BF16>(b);
      }
    }
    if (is_q) {
      uint16_t* dst = p.q_out + tok * p.ldqo + h * p.dim;
      *reinterpret_cast<uint4*>(dst + c0) = r0;
      *reinterpret_cast<uint4*>(dst + c1) = r1;
    } else {
      const int64_t at = cell + kh * p.head_stride;
      if constexpr (F8) {
        const float inv = __frcp_rn(__ldg((is_v ? p.v_scale : p.k_scale) + kh));
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.cv : p.ck) + at;
        const uint2 x = narrow8_e4m3(a, inv), y = narrow8_e4m3(b, inv);
        *reinterpret_cast<uint2*>(dst + c0) = x;
        *reinterpret_cast<uint2*>(dst + c1) = y;
      } else {
        uint16_t* dst = static_cast<uint16_t*>(is_v ? p.cv : p.ck) + at;
        *reinterpret_cast<uint4*>(dst + c0) = r0;
        *reinterpret_cast<uint4*>(dst + c1) = r1;
      }
    }
  };
  if (row < heads) store(row, first0, first1);
#pragma unroll 2
  for (int h = row + rows; h < heads; h += rows) {
    uint4 v0, v1;
    load(h, v0, v1);
    store(h, v0, v1);
  }
}

template <int THREADS>
cudaError_t launch(const AppendParams& p, int T, bool bf16, bool f8, cudaStream_t st) {
  const int lanes = p.dim / 16;
  const dim3 grid(static_cast<unsigned>(T)), block(static_cast<unsigned>(THREADS / lanes * lanes));
  if (bf16)
    return f8 ? launch_pdl(kv_append_kernel<true, true, THREADS>, grid, block, 0, st, p)
              : launch_pdl(kv_append_kernel<true, false, THREADS>, grid, block, 0, st, p);
  return f8 ? launch_pdl(kv_append_kernel<false, true, THREADS>, grid, block, 0, st, p)
            : launch_pdl(kv_append_kernel<false, false, THREADS>, grid, block, 0, st, p);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, int T, bool bf16, bool f8, int sms, cudaStream_t st) {
  // One block for each token. Few tokens: all their heads at once, as the latency of one pass is the time (24 tokens of 32
  // heads of 256: 2.4 us with 512 threads, 2.6 with 256, 3.1 with 128, 4.4 with 64). Many: small blocks, which start and end
  // out of step and so keep the memory busy (40 + 16 heads of 128, us with 256, 128 and 64 threads: bf16, 512 tokens 4.1, 4.1, 5.0;
  // 1000: 6.9, 6.5, 7.9; 4000: 27.2, 22.1, 22.1; 16000: 97.8, 77.9, 72.0, 0.96 of the copy rate. Into 8 bits, where 64 threads have
  // 48 registers and spill some: 512: 4.0, 4.3, 6.1; 1000: 6.4, 5.5, 7.6; 4000: 27.8, 24.4, 25.5; 16000: 99.8, 86.3, 77.1, 0.82 of it).
  // Around 1000 tokens, and for 8 bits up to some thousand, the rule gives away up to a quarter of the time.
  return T <= sms ? launch<512>(p, T, bf16, f8, st) : T < 4 * sms ? launch<256>(p, T, bf16, f8, st) : launch<64>(p, T, bf16, f8, st);
}

}  // namespace tl
