// Tree attention over a bf16 cache: the instantiations of tree_attention.cuh.
#include "tree_attention.cuh"

namespace tl {

cudaError_t launch_tree_attn_bf16(TreeAttnParams p, int dim, int sms, cudaStream_t st) {
  return tree::launch_dim<kCacheBf16>(p, dim, sms, st);
}

}  // namespace tl
