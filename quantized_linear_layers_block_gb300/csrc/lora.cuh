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
// serves adapters of any rank and width, and both sides meet at about the same M for all of them (bf16, K = 5120, N = 17408,
// 4 adapters, 16 against 32 tokens, us: rank 8: 256 tokens 8.8, 9.8; 512: 14.9, 14.8; 1024: 22.5, 19.9; 2048: 38.6, 32.7;
// rank 32: 512 tokens 16.0, 17.4; 1024: 23.9, 23.2; rank 64: 21.0, 23.0; 32.9, 30.0; rank 128: 30.8, 34.1; 53.0, 46.0; 2048:
// 96.5, 79.0; 515 tokens of 5 adapters, rank 64, K = 17408, N = 5120, fp16 to fp32: 19.8, 28.8).
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
