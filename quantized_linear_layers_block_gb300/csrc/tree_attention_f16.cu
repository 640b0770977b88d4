// Tree attention over a f16 cache: the instantiations of tree_attention.cuh.
#include "tree_attention.cuh"

namespace tl {

cudaError_t launch_tree_attn_f16(TreeAttnParams p, int dim, int sms, cudaStream_t st) {
  return tree::launch_dim<kCacheF16>(p, dim, sms, st);
}

}  // namespace tl
