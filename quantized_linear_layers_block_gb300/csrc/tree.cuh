// What the entry points for trees of drafted tokens hand to their kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/tl.h"

namespace tl {

struct TreePlanParams {
  const int32_t* parents;
  const int32_t* starts;
  const int32_t* lens;
  const int32_t* pages;
  int64_t ldp;
  int64_t* masks;
  int32_t* positions;
  int64_t* slots;
  int* status;
  int B, T, page_size, num_pages;
  int capacity;              // max_pages * page_size, at most 2^31 - 2^16
};

struct VerifyParams {
  const float* target;
  const float* draft;
  int64_t ldt, ldd;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* starts;
  const float* uniform;
  int32_t* path;
  int32_t* counts;
  int32_t* next;
  int* status;
  int vocab, B, T;
};

struct CompactParams {
  uint8_t* k;
  uint8_t* v;
  int64_t page_stride, head_stride, token_stride;     // bytes
  const int32_t* path;
  const int32_t* counts;
  const int32_t* starts;
  const int32_t* lens;
  const int32_t* pages;
  int64_t ldp;
  int* status;
  int B, T, page_size, num_pages, capacity;
  int kv_heads, row;                                  // 16-byte chunks of a head's row
};

cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t st);
cudaError_t launch_verify_tree(const VerifyParams& p, int sms, cudaStream_t st);
cudaError_t launch_kv_compact(const CompactParams& p, cudaStream_t st);

// Rows of request b; false where its starts are not what they have to be.
__device__ __forceinline__ bool tree_rows(const int32_t* starts, int b, int T, int& begin, int& n) {
  begin = __ldg(starts + b);
  const int end = __ldg(starts + b + 1);
  const bool ok = begin >= 0 && begin <= end && end <= T && end - begin <= TL_TREE_NODES;
  n = ok ? end - begin : 0;
  return ok;
}

}  // namespace tl
