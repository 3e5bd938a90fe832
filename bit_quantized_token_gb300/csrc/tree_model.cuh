// A drafted tree through the batched pipeline: what stands around the tree
// attention in a layer of the model.
#pragma once
#include "batch.cuh"
#include "tree.cuh"

namespace llmq {

struct TreeRowsParams {
  const float* qkv;          // [n][q_dim + 2 kv_dim]
  int qkv_cols, q_dim, kv_dim, n_heads, n_kv;
  const int* pos;            // [n] position of each node
  const float2* rope;        // [cap][hd / 2]
  int rope_neox, cap;
  const float *q_norm, *k_norm;  // per-head RMSNorm weights, or null
  float eps;
  float* q;                  // [n][n_heads][hd] out
  uint16_t *k, *v;           // the tree's rows of this layer [n_kv][rows][hd]: bf16
  int8_t *k8, *v8;           // or int8 codes and fp16 scales
  uint16_t *ks, *vs;
  int rows;
  int* status;
};

// The nodes' queries and own K/V rows from the layer's q|k|v: RMSNorm of q and
// k heads, RoPE at the node's position, K and V in the cache's format (the
// roundings of the cache's own append). A warp per (node, head); lane holds
// dims lane + 32 e, so a group of 32 values is one per lane.
template <int HD>
__global__ void __launch_bounds__(128) tree_rows_kernel(const TreeRowsParams p) {
  constexpr int E = HD / 32;
  __shared__ float buf[4][HD];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, node = blockIdx.y;
  const int h = blockIdx.x * 4 + warp;  // q heads, k heads, v heads
  if (h >= p.n_heads + 2 * p.n_kv) return;
  const bool is_q = h < p.n_heads, is_v = h >= p.n_heads + p.n_kv;
  const int pos = p.pos[node];
  if (pos < 0 || pos >= p.cap) {
    if (lane == 0) atomicOr(p.status, ST_CTX_FULL);
    return;
  }
  const float* src = p.qkv + (size_t)node * p.qkv_cols + (size_t)h * HD;  // q, k and v heads lie in this order
  float x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = __ldcg(src + lane + 32 * e);
  if (!is_v) {
    const float* w = is_q ? p.q_norm : p.k_norm;
    if (w) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) ss += x[e] * x[e];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = 1.0f / sqrtf(ss / (float)HD + p.eps);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = x[e] * inv * __ldg(w + lane + 32 * e);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) buf[warp][lane + 32 * e] = x[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane + 32 * e;
      const int i = p.rope_neox ? d % (HD / 2) : d / 2;               // the pair
      const bool second = p.rope_neox ? d >= HD / 2 : d & 1;
      const float2 cs = __ldg(p.rope + (size_t)pos * (HD / 2) + i);
      const float other = buf[warp][p.rope_neox ? (second ? d - HD / 2 : d + HD / 2) : d ^ 1];
      x[e] = second ? other * cs.y + x[e] * cs.x : x[e] * cs.x - other * cs.y;
    }
  }
  if (is_q) {
    float* dst = p.q + ((size_t)node * p.n_heads + h) * HD;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[lane + 32 * e] = x[e];
    return;
  }
  const size_t row = ((size_t)(h - p.n_heads - (is_v ? p.n_kv : 0)) * p.rows + node) * HD;
  if (p.k8) {
    int8_t* codes = (is_v ? p.v8 : p.k8) + row;
    uint16_t* scales = (is_v ? p.vs : p.ks) + row / 32;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float amax = fabsf(x[e]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const __half dh = __float2half_rn(amax / 127.0f);
      const float dq = __half2float(dh);
      const float cf = dq == 0.0f ? 0.0f : fminf(fmaxf(roundf(x[e] / dq), -127.0f), 127.0f);
      codes[lane + 32 * e] = (int8_t)(int)cf;
      if (lane == 0) scales[e] = __half_as_ushort(dh);
    }
  } else {
    uint16_t* dst = (is_v ? p.v : p.k) + row;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[lane + 32 * e] = __bfloat16_as_ushort(__float2bfloat16_rn(x[e]));
  }
}

// The attention's output staged for the o-projection: XL [64][cols].
struct TreeStageParams {
  const float* o;            // [n][cols]
  uint16_t* xl;
  int cols;
};
__global__ void __launch_bounds__(256) tree_stage_kernel(const TreeStageParams p) {
  pdl_wait();
  pdl_trigger();
  const int node = blockIdx.y, i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < p.cols) store_hl(p.xl, p.cols, node, i, p.o[(size_t)node * p.cols + i]);
}

}  // namespace llmq
