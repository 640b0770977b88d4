// Paged attention over a bf16 cache: the instantiations of paged_attention.cuh.
#include "paged_attention.cuh"

namespace tl {

cudaError_t launch_attn_bf16(const AttnParams& p, int dim, int columns, int sms, cudaStream_t st) {
  return attn::launch_dim<kCacheBf16>(p, dim, columns, sms, st);
}

}  // namespace tl
