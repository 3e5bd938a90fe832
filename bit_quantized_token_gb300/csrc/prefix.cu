// Attention of sequences that share prefixes: two launches, of which the second
// overlaps the first (see serve.cuh, tree_attn.cuh).
#include "op_call.cuh"
#include "own_attn.cuh"
#include "prefix_attn.cuh"
#include "serve.cuh"

namespace llmq {

cudaError_t launch_prefix_attn(const TreeAttnParams& first, const TreeAttnParams& second, int hd, bool f32, bool q8,
                               int n_sm, cudaStream_t st) {
  // By the rows of a kv head that a group can have. The tree attention's kernel splits the keys further, the wide one
  // reads them once for 256 rows. Measured, wide / narrow, us a call: 64 dims, 4 kv heads, 128 rows behind 2048 /
  // 8192 prefix rows 12.6 / 12.9, 20.7 / 18.0; 256 rows 15.3 / 14.2, 26.0 / 20.5; 512 rows 15.5 / 17.7, 26.2 / 27.8;
  // 128 dims, 8 kv heads, 128 rows 18.5 / 19.1, 27.7 / 29.1; 256 rows 28.9 / 29.2, 42.4 / 48.3.
  const int wide_from = hd == 64 ? 257 : 128;
  const int64_t rows = (int64_t)first.nodes * first.gq;
  const bool wide = !f32 && !q8 && rows >= wide_from && first.B <= kWideGroups &&
                    (rows / kWideRows + first.B) * first.Hkv * (first.cache.rows / 128 + 1) < (1ll << 31) &&
                    rows * first.Hkv < (1ll << 30);
  const cudaError_t e = !wide ? launch_tree_attn(first, hd, f32, q8, n_sm, st)
                        : hd == 64 ? launch_wide<64>(first, n_sm, st) : launch_wide<128>(first, n_sm, st);
  if (e != cudaSuccess) return e;
  if (!own_fits(second, hd, q8)) return launch_tree_attn(second, hd, f32, q8, n_sm, st);
  const auto launch = hd == 64 ? (f32 ? (q8 ? launch_own<64, true, true> : launch_own<64, true, false>)
                                      : (q8 ? launch_own<64, false, true> : launch_own<64, false, false>))
                               : (f32 ? (q8 ? launch_own<128, true, true> : launch_own<128, true, false>)
                                      : (q8 ? launch_own<128, false, true> : launch_own<128, false, false>));
  return launch(second, n_sm, st);
}

}  // namespace llmq

// ---- C entries -------------------------------------------------------------------
using namespace llmq;

namespace {

// [parts][rows][head_dim] results, [parts][rows] (reference, sum), [rows] numbers of parts, of rows = sequences x
// nodes x heads
int64_t part_bytes(int64_t rows, int64_t head_dim) { return rows * (wide_parts(rows) * (head_dim * 4 + 8) + 4); }

}  // namespace

extern "C" {

int64_t llm_prefix_workspace(int32_t n_seq, int32_t n_nodes, int32_t n_heads, int32_t head_dim) {
  Call c;
  if (!c.need(n_seq > 0 && n_seq <= 65535 && n_nodes > 0 && n_nodes <= kTreeMaxNodes && n_heads > 0 && n_heads <= 65535 &&
                  (head_dim == 64 || head_dim == 128),
              LLM_ERR_INVALID_ARG, "a size is out of range"))
    return c.rc;
  return part_bytes((int64_t)n_seq * n_nodes * n_heads, head_dim);
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
      !c.need(v.n_heads * (nodes * gq / 16 + 1) <= 65535 && (nodes + 256) * gq * gq < (1ll << 32) &&
                  nodes * t.n_nodes < (1ll << 32),
              LLM_ERR_UNSUPPORTED, "too many sequences and heads") ||
      !view_memory(c, a->prefix, "prefix") || !c.device("starts", a->starts, 4) ||
      !c.device("prefix_lens", a->prefix_lens, 4) || !c.device("workspace", a->workspace, 32) ||
      !c.need(a->workspace_bytes >= part_bytes(nodes * t.n_heads, v.head_dim), LLM_ERR_INVALID_ARG,
              "the workspace is smaller than llm_prefix_workspace says"))
    return c.rc;
  const bool f32 = t.dtype == LLM_F32, q8 = v.dtype == LLM_Q8G32;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (f.rows == 0) return finish(launch_tree_attn(p, v.head_dim, f32, q8, c.n_sm, st), "attention launch");
  p.starts = a->starts;
  p.G = a->n_groups;
  p.all = t.n_seq;
  p.by_n = FastDiv(t.n_nodes);
  p.part_rows = nodes * t.n_heads;
  p.max_parts = wide_parts(p.part_rows);
  p.part_o = static_cast<float*>(a->workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + p.max_parts * p.part_rows * v.head_dim);
  p.part_n = reinterpret_cast<int*>(p.part_ml + p.max_parts * p.part_rows);
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
