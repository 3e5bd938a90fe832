// Attention of sequences that share prefixes: two launches, of which the second
// overlaps the first (see serve.cuh, tree_attn.cuh).
#include "op_call.cuh"
#include "serve.cuh"

namespace llmq {

cudaError_t launch_prefix_attn(const TreeAttnParams& first, const TreeAttnParams& second, int hd, bool f32, bool q8,
                               int n_sm, cudaStream_t st) {
  const cudaError_t e = launch_tree_attn(first, hd, f32, q8, n_sm, st);
  return e == cudaSuccess ? launch_tree_attn(second, hd, f32, q8, n_sm, st) : e;
}

}  // namespace llmq

// ---- C entries -------------------------------------------------------------------
using namespace llmq;

namespace {

// [rows][head_dim] results, then [rows] (reference, sum), of rows = sequences x nodes x heads
int64_t part_bytes(int64_t n_seq, int64_t n_nodes, int64_t n_heads, int64_t head_dim) {
  return n_seq * n_nodes * n_heads * (head_dim * 4 + 8);
}

}  // namespace

extern "C" {

int64_t llm_prefix_workspace(int32_t n_seq, int32_t n_nodes, int32_t n_heads, int32_t head_dim) {
  Call c;
  if (!c.need(n_seq > 0 && n_seq <= 65535 && n_nodes > 0 && n_nodes <= kTreeMaxNodes && n_heads > 0 && n_heads <= 65535 &&
                  (head_dim == 64 || head_dim == 128),
              LLM_ERR_INVALID_ARG, "a size is out of range"))
    return c.rc;
  return part_bytes(n_seq, n_nodes, n_heads, head_dim);
}

int llm_prefix_attention(const llm_prefix_attention_args* a, void* cuda_stream) {
  Call c;
  TreeAttnParams p{};
  if (!c.need(a != nullptr, LLM_ERR_INVALID_ARG, "the arguments are null")) return c.rc;
  const llm_tree_attention_args& t = a->attention;
  if (!attention_params(c, &t, p) || !check_view(c, a->prefix, "prefix")) return c.rc;
  const llm_kv_view &v = *t.cache, &f = *a->prefix;
  const int64_t nodes = (int64_t)t.n_seq * t.n_nodes, gq = t.n_heads / v.n_heads;
  if (!c.need(a->n_groups >= 1 && a->n_groups <= f.n_seq, LLM_ERR_INVALID_ARG,
              "n_groups is not positive or over the prefix view's sequences") ||
      !c.need(f.dtype == v.dtype && f.head_dim == v.head_dim && f.n_heads == v.n_heads && f.n_layers == 1,
              LLM_ERR_INVALID_ARG, "the prefix's rows do not match the cache") ||
      !c.need(v.n_heads * (nodes * gq / 16 + 1) <= 65535 && (nodes + 128) * gq * gq < (1ll << 32) &&
                  nodes * t.n_nodes < (1ll << 32),
              LLM_ERR_UNSUPPORTED, "too many sequences and heads") ||
      !view_memory(c, a->prefix, "prefix") || !c.device("starts", a->starts, 4) ||
      !c.device("prefix_lens", a->prefix_lens, 4) || !c.device("workspace", a->workspace, 16) ||
      !c.need(a->workspace_bytes >= part_bytes(t.n_seq, t.n_nodes, t.n_heads, v.head_dim), LLM_ERR_INVALID_ARG,
              "the workspace is smaller than llm_prefix_workspace says"))
    return c.rc;
  const bool f32 = t.dtype == LLM_F32, q8 = v.dtype == LLM_Q8G32;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (f.rows == 0) return finish(launch_tree_attn(p, v.head_dim, f32, q8, c.n_sm, st), "attention launch");
  p.starts = a->starts;
  p.G = a->n_groups;
  p.all = t.n_seq;
  p.by_n = FastDiv(t.n_nodes);
  p.part_o = static_cast<float*>(a->workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + nodes * t.n_heads * v.head_dim);
  TreeAttnParams first = p;
  p.part = TreeAttnParams::kSecond;
  first.part = TreeAttnParams::kFirst;
  first.cache = rows_of(f);
  first.tree = KvRows();
  first.lens = a->prefix_lens;
  first.counts = nullptr;
  first.B = a->n_groups;
  first.nodes = (int)nodes;
  return finish(launch_prefix_attn(first, p, v.head_dim, f32, q8, c.n_sm, st), "prefix attention launch");
}

}  // extern "C"
