// Tree attention, head dimension 64 (see tree_attn.cuh, tree_attn_tc.cuh, tree_attn_q8.cuh).
#include "tree_attn_q8.cuh"

namespace llmq {
cudaError_t launch_tree_attn_64(TreeAttnParams p, bool f32, bool q8, int n_sm, cudaStream_t st) {
  cudaError_t e;
  if (q8 ? launch_tree_q8<64>(p, f32, n_sm, st, &e) : launch_tree_tc<64>(p, f32, n_sm, st, &e)) return e;
  return launch_tree_attn_hd<64>(p, f32, q8, n_sm, st);
}
}  // namespace llmq
