// Serving operators: parameters and launchers of what stands around the
// attention of a served batch on the caller's own tensors: new tokens' q, k and v
// into the cache and cached rows back out (kv_rows.cu), attention behind shared
// prefixes (prefix.cu, over tree_attn.cuh and prefix_attn.cuh) and the next tokens
// from logits (sample_rows.cu).
#pragma once
#include "tree.cuh"

namespace llmq {

struct AppendParams {
  const void *q, *k, *v;     // [token][head][dim], bf16 or fp32; q null: no queries
  void* q_out;               // bf16 or fp32
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head;  // strides in elements
  KvRows cache;              // one layer
  const int *seqs, *rows;    // [T] where a token's row goes
  const int* positions;      // [T] or null: rows
  const float *q_norm, *k_norm;  // [head_dim] or null
  float eps;
  int T, Hq, Hkv, n_seq;
  bool rotate, neox, f32, out_f32;
  int passes;                // set by the launch: rows that a group of lanes takes one after the other
  bool pdl = true;
  // turn of pair i a position, in 2^-64 turns: a product with a position, modulo 2^64, is the angle
  uint64_t freq[64];
};
cudaError_t launch_append_kv(AppendParams& p, int hd, bool q8, int n_sm, cudaStream_t st);

struct ReadParams {
  KvRows cache;              // strides of one layer
  int64_t layer, slayer;     // strides of the layers
  const int *seqs, *rows;    // [T]
  void *k, *v;               // [layer][token][head][dim], bf16 or fp32
  int64_t o_layer, o_tok, o_head;
  int T, L, H, n_seq;
  FastDiv by_heads;
  bool f32;
  bool pdl = true;
};
cudaError_t launch_read_kv(const ReadParams& p, int hd, bool q8, cudaStream_t st);

// Attention in two parts: every group's queries over the rows that its sequences
// share (first), then every sequence's over its own, joined (second; see TreeAttnParams::Part).
cudaError_t launch_prefix_attn(const TreeAttnParams& first, const TreeAttnParams& second, int hd, bool f32, bool q8,
                               int n_sm, cudaStream_t st);

constexpr int kSampleList = 4096;  // tokens around the borders that one CTA sorts

struct SampleRowsParams {
  const float* logits;
  int64_t stride;            // of the rows, in elements
  const float *u, *temperature, *top_p, *min_p;  // [R]; all but u may be null
  const int* top_k;          // [R] or null
  int* tokens;               // [R]
  float* probs;              // [R] or null
  int R, V;
  int slice;                 // set by the launch: logits of a CTA
  bool pdl = true;
};
cudaError_t launch_sample_rows(SampleRowsParams& p, int n_sm, cudaStream_t st);

}  // namespace llmq
