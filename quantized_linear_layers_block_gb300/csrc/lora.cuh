// What the adapter entry points hand to their kernels, and the layout of a plan.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace tl {

constexpr int kLoraTile = 32;           // most tokens that an item can have
constexpr int kLoraMaxM = 1 << 20;
constexpr int kLoraMaxAdapters = 4096;
constexpr int kLoraMaxRank = 128;

// A plan: a header and the items, each up to lora_tile(M) tokens of one adapter (or of none), adapter by
// adapter, the tokens of one in their own order.
struct LoraItem {
  int adapter, count, unused[2];        // adapter -1: none
  int token[kLoraTile];
};
struct LoraPlanHeader {
  int M, n_adapters, items, unused;
};

// Tokens of an item. 32 read an adapter's matrices half as often as 16 and fill the matrix instructions' rows as
// well; 16 leave twice as many items, which blocks share the SMs more evenly with, and a shorter chain. The plan
// serves adapters of any rank and width, and both sides meet at about the same M for all of them (K = 5120, N = 17408,
// 4 adapters, 16 against 32 tokens, us: rank 8: 512 tokens 12.8, 16.6; 1024: 24.4, 19.9; 2048: 43, 33;
// rank 128: 512 tokens 35, 52; 1024: 54, 53; 2048: 96, 83).
inline int lora_tile(int M) { return M >= 1024 ? 32 : 16; }

// most items that M tokens of n_adapters adapters (and none) can need
inline int lora_max_items(int M, int n_adapters) {
  const int bins = n_adapters + 1 < M ? n_adapters + 1 : M;
  return (M - bins) / lora_tile(M) + bins;
}
inline size_t lora_plan_bytes(int M, int n_adapters) {
  return sizeof(LoraPlanHeader) + sizeof(LoraItem) * static_cast<size_t>(lora_max_items(M, n_adapters));
}

struct LoraParams {
  const uint16_t* x;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const LoraPlanHeader* plan;
  const LoraItem* items;
  const void* base;
  void* y;
  int64_t ldx, ldb, ldy;
  int M, N, K, rank, n_adapters, y_dtype;
  int copy_bare;            // base and y differ: tokens without an adapter are copied
  int* status;
};

cudaError_t launch_lora_plan(const int32_t* ids, int M, int n_adapters, void* plan, int* status, cudaStream_t st);
cudaError_t launch_lora_apply(const LoraParams& p, bool bf16, int sms, cudaStream_t st);

}  // namespace tl
