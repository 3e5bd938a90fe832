// Tree attention, head dimension 64 (see tree_attn.cuh).
#include "tree_attn.cuh"

namespace llmq {
cudaError_t launch_tree_attn_64(TreeAttnParams p, bool f32, bool q8, int n_sm, cudaStream_t st) {
  return launch_tree_attn_hd<64>(p, f32, q8, n_sm, st);
}
}  // namespace llmq
