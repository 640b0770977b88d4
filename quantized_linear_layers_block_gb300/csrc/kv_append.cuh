// What tl_kv_append hands to its kernel.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace tl {

struct AppendParams {
  void* ck;
  void* cv;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride, head_stride, token_stride, num_slots;   // elements; pages * page_size
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  int64_t ldq, ldk, ldv, ldqo;
  const float* cos_sin;
  const int32_t* positions;
  const int64_t* slots;
  int* status;
  int q_heads, kv_heads, dim, page_size, rot, max_pos, interleaved;
};

cudaError_t launch_kv_append(const AppendParams& p, int T, bool bf16, bool f8, int sms, cudaStream_t st);

}  // namespace tl
