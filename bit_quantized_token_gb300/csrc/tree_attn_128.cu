// Tree attention, head dimension 128 (see tree_attn.cuh, tree_attn_q8.cuh).
#include "tree_attn_q8.cuh"

namespace llmq {
cudaError_t launch_tree_attn_128(const TreeAttnParams& p, bool f32, bool q8, int n_sm, cudaStream_t st) {
  return q8 ? launch_tree_q8<128>(p, f32, n_sm, st) : launch_tree_tc<128>(p, f32, n_sm, st);
}
}  // namespace llmq
