// Token probabilities, draft verification and the commit of accepted rows, and
// the C entries of the tree-decoding operators (see tree.cuh).
#include <cooperative_groups.h>

#include <cmath>
#include <cstdio>
#include <utility>

#include "common.cuh"
#include "llmq.h"
#include "sample_key.cuh"
#include "tree.cuh"

namespace llmq {
namespace cg = cooperative_groups;

cudaError_t launch_tree_attn(const TreeAttnParams& p, int hd, bool f32, bool q8, int n_sm, cudaStream_t st) {
  return hd == 64 ? launch_tree_attn_64(p, f32, q8, n_sm, st) : launch_tree_attn_128(p, f32, q8, n_sm, st);
}

namespace {

template <typename Kern, typename Params>
cudaError_t launch_cluster(Kern kern, dim3 grid, int threads, int cluster, size_t smem, cudaStream_t st,
                           const Params& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// ---- token probabilities -----------------------------------------------------
// p_j = 2^(c (l_j - m)) / sum over the kept tokens, c = log2(e) / T. A cluster
// owns a row: every CTA keeps its slice in shared memory, so the row is read
// once and written once; a CTA's (max, sum) and, with top_k, its sorted top_k
// candidates are all that crosses the cluster. A NaN counts as -inf, +inf as
// the largest finite value; a row without a finite logit is all zeros.
constexpr int kProbThreads = 512;
constexpr int kProbSlice = 51200;  // floats of a row that one CTA keeps

__device__ __forceinline__ float clean_logit(float x) { return x != x ? -INFINITY : fminf(x, 3.402823466e38f); }

// Sum / max over the CTA in a fixed order, to every thread.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* s_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, y) : v + y;
  }
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_warp[threadIdx.x & 31 & (kProbThreads / 32 - 1)];
#pragma unroll
  for (int o = kProbThreads / 64; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, y) : v + y;
  }
  __syncthreads();
  return v;
}

// The slice [a, a + n) of a row to shared memory, aligned as in global memory
// (the returned offset, 0..3 floats), 16 bytes at a time where it is; f(x, i)
// maps the value of element i.
template <typename F>
__device__ __forceinline__ int load_slice(float* sx, const float* src, int n, F f) {
  const int off = (int)((reinterpret_cast<uintptr_t>(src) >> 2) & 3);
  const float* base = src - off;
  const int end = off + n, v0 = (off + 3) / 4, v1 = end / 4;
  for (int i = v0 + threadIdx.x; i < v1; i += kProbThreads) {
    float4 x = __ldcs(reinterpret_cast<const float4*>(base) + i);
    x.x = f(x.x), x.y = f(x.y), x.z = f(x.z), x.w = f(x.w);
    reinterpret_cast<float4*>(sx)[i] = x;
  }
  const int head = min(4 * v0, end), tail = max(4 * v1, head);
  if (threadIdx.x < head - off) sx[off + threadIdx.x] = f(base[off + threadIdx.x]);
  if (threadIdx.x < end - tail) sx[tail + threadIdx.x] = f(base[tail + threadIdx.x]);
  return off;
}

struct ProbRange {  // slice of CTA `rank` of C: starts on a multiple of 4
  int a, n;
  __device__ ProbRange(int V, int rank, int C) {
    const int q = (V + 4 * C - 1) / (4 * C) * 4;
    a = min(V, q * rank);
    n = min(V, a + q) - a;
  }
};

__global__ void __launch_bounds__(kProbThreads) softmax_rows_kernel(const TokenProbsParams p) {
  extern __shared__ __align__(16) float sx[];
  __shared__ float s_warp[32];
  __shared__ float2 s_ms;
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), row = blockIdx.x / C, tid = threadIdx.x;
  const ProbRange r(p.V, rank, C);
  float mx = -INFINITY;
  const int off = load_slice(sx, p.logits + (int64_t)row * p.l_row + r.a, r.n, [&](float x) {
    x = clean_logit(x);
    mx = fmaxf(mx, x);
    return x;
  });
  mx = block_reduce<true>(mx, s_warp);  // its barriers publish sx
  const float m = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
  for (int i = off + tid; i < off + r.n; i += kProbThreads) {
    const float e = exp2f((sx[i] - m) * p.c);
    sx[i] = e;
    sum += e;
  }
  sum = block_reduce<false>(sum, s_warp);
  if (tid == 0) s_ms = make_float2(mx, sum);
  cl.sync();
  float M = -INFINITY, S = 0.f;
  for (int k = 0; k < C; ++k) M = fmaxf(M, cl.map_shared_rank(&s_ms, k)->x);
  for (int k = 0; k < C; ++k) {
    const float2 o = *cl.map_shared_rank(&s_ms, k);
    if (o.x != -INFINITY) S += o.y * exp2f((o.x - M) * p.c);
  }
  const float f = S > 0.f && mx != -INFINITY ? exp2f((mx - M) * p.c) / S : 0.f;
  float* dst = p.probs + (int64_t)row * p.p_row + r.a;
  const int doff = (int)((reinterpret_cast<uintptr_t>(dst) >> 2) & 3);
  if (doff == off) {
    float* base = dst - off;
    const int end = off + r.n, v0 = (off + 3) / 4, v1 = end / 4, head = min(4 * v0, end), tail = max(4 * v1, head);
    for (int i = v0 + tid; i < v1; i += kProbThreads) {
      float4 x = reinterpret_cast<const float4*>(sx)[i];
      x.x *= f, x.y *= f, x.z *= f, x.w *= f;
      __stcs(reinterpret_cast<float4*>(base) + i, x);
    }
    if (tid < head - off) base[off + tid] = sx[off + tid] * f;
    if (tid < end - tail) base[tail + tid] = sx[tail + tid] * f;
  } else {
    for (int i = tid; i < r.n; i += kProbThreads) dst[i] = sx[off + i] * f;
  }
  cl.sync();  // s_ms lives until every rank has read it
}

// With top_k: 64-bit keys (order-preserving value, complement of the token id)
// make every logit's place unique, ties to the lower id. Of G = 128 groups of a
// CTA's threads the k-th largest group maximum is at most the CTA's k-th
// largest key, so the keys from it on, a few more than k, hold the CTA's top k;
// their ranks among themselves sort them, and rank 0 of the cluster merges the
// C sorted lists by binary search, cuts the nucleus and writes the kept tokens
// over the zeros that every CTA has written to its slice.
constexpr int kProbGroups = 128;

struct TopKShared {
  unsigned long long gmax[kProbGroups];
  unsigned long long top[kSampleMaxK];  // this CTA's largest keys, sorted
  int n_top, n_cand;
  unsigned long long thr;
  unsigned long long all[16 * kSampleMaxK];
  unsigned long long sorted[kSampleMaxK];
  int n_all[16];
};

__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u ^ 0x80000000u) : ~u);
}

__global__ void __launch_bounds__(kProbThreads) topk_rows_kernel(const TokenProbsParams p) {
  extern __shared__ __align__(16) float sx[];
  __shared__ TopKShared s;
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), row = blockIdx.x / C, tid = threadIdx.x;
  const ProbRange r(p.V, rank, C);
  const int K = min(p.top_k, p.V);
  int* cand = reinterpret_cast<int*>(sx + p.cap + 4);
  const int off = load_slice(sx, p.logits + (int64_t)row * p.l_row + r.a, r.n,
                             [&](float x) { return clean_logit(x); });
  if (tid == 0) s.n_cand = 0;
  __syncthreads();
  auto key = [&](int i) {  // of slice element i; 0: a logit that can never be kept
    const float x = sx[off + i];
    return x == -INFINITY ? 0ull
                          : ((unsigned long long)sample_key(x) << 32) | (uint32_t)(0x7FFFFFFF - (r.a + i));
  };
  unsigned long long best = 0;
  for (int i = tid; i < r.n; i += kProbThreads) best = max(best, key(i));
  best = max(best, __shfl_xor_sync(0xffffffffu, best, 1));
  best = max(best, __shfl_xor_sync(0xffffffffu, best, 2));
  if ((tid & 3) == 0) s.gmax[tid >> 2] = best;
  __syncthreads();
  if (tid < kProbGroups) {  // the group maximum with K - 1 larger ones (group maxima differ, or are 0)
    const unsigned long long v = s.gmax[tid];
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < kProbGroups; ++j) above += s.gmax[j] > v || (s.gmax[j] == v && j < tid);
    if (above == K - 1) s.thr = v;
  }
  // zeros while the candidates are found
  float* dst = p.probs + (int64_t)row * p.p_row + r.a;
  const unsigned long long* sthr = &s.thr;
  __syncthreads();
  const unsigned long long thr = max(*sthr, 1ull);
  for (int i = tid; i < r.n; i += kProbThreads)
    if (key(i) >= thr) cand[atomicAdd(&s.n_cand, 1)] = i;
  {
    const int doff = (int)((reinterpret_cast<uintptr_t>(dst) >> 2) & 3);
    float* base = dst - doff;
    const int end = doff + r.n, v0 = (doff + 3) / 4, v1 = end / 4, head = min(4 * v0, end), tail = max(4 * v1, head);
    for (int i = v0 + tid; i < v1; i += kProbThreads)
      __stcs(reinterpret_cast<float4*>(base) + i, make_float4(0.f, 0.f, 0.f, 0.f));
    if (tid < head - doff) base[doff + tid] = 0.f;
    if (tid < end - tail) base[tail + tid] = 0.f;
  }
  __syncthreads();
  const int nc = s.n_cand;
  if (tid == 0) s.n_top = min(nc, K);
  for (int i = tid; i < nc; i += kProbThreads) {  // the order of the list does not matter: keys are unique
    const unsigned long long v = key(cand[i]);
    int above = 0;
    for (int j = 0; j < nc; ++j) above += key(cand[j]) > v;
    if (above < K) s.top[above] = v;
  }
  cl.sync();
  if (rank == 0) {
    if (tid < C) s.n_all[tid] = cl.map_shared_rank(&s.n_top, tid)[0];
    __syncthreads();
    for (int i = tid; i < C * kSampleMaxK; i += kProbThreads) {
      const int k = i / kSampleMaxK, j = i % kSampleMaxK;
      if (j < s.n_all[k]) s.all[i] = cl.map_shared_rank(s.top, k)[j];
    }
    __syncthreads();
    int total = 0;
    for (int k = 0; k < C; ++k) total += s.n_all[k];
    const int n = min(total, K);
    for (int i = tid; i < C * kSampleMaxK; i += kProbThreads) {
      const int own = i / kSampleMaxK;
      if (i % kSampleMaxK >= s.n_all[own]) continue;
      const unsigned long long v = s.all[i];
      int above = i % kSampleMaxK;
      for (int k = 0; k < C; ++k) {
        if (k == own) continue;
        int lo = 0, hi = s.n_all[k];  // keys of list k larger than v
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (s.all[k * kSampleMaxK + mid] > v) lo = mid + 1;
          else hi = mid;
        }
        above += lo;
      }
      if (above < n) s.sorted[above] = v;
    }
    __syncthreads();
    if (tid < 32) {  // lane l: tokens l and l + 32 in order; sums in fp64 (a cut-off compares them with top_p)
      const float m = n > 0 ? key_value(s.sorted[0]) : 0.f;
      float e[2];
      double w[2], cum[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = tid + 32 * h;
        e[h] = j < n ? exp2f((key_value(s.sorted[j]) - m) * p.c) : 0.f;
        w[h] = e[h];
        cum[h] = w[h];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, cum[h], o);
          if (tid >= o) cum[h] += y;
        }
      }
      cum[1] += __shfl_sync(0xffffffffu, cum[0], 31);
      const double tot = __shfl_sync(0xffffffffu, cum[1], 31);
      bool in[2];
      double kept = 0.0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        in[h] = tid + 32 * h < n && (tid + 32 * h == 0 || cum[h] - w[h] < (double)p.top_p * tot);
        kept += in[h] ? w[h] : 0.0;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) kept += __shfl_xor_sync(0xffffffffu, kept, o);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = tid + 32 * h;
        if (j < n) s.sorted[j] = (s.sorted[j] & 0xFFFFFFFFull) |
                                 ((unsigned long long)__float_as_uint(in[h] ? (float)(w[h] / kept) : 0.f) << 32);
      }
    }
    if (tid == 0) s.n_top = n;
  }
  cl.sync();  // every slice's zeros are written, the kept tokens are known
  if (rank == 0 && tid < s.n_top) {
    const unsigned long long v = s.sorted[tid];
    const int id = 0x7FFFFFFF - (int)(uint32_t)v;
    p.probs[(int64_t)row * p.p_row + id] = __uint_as_float((uint32_t)(v >> 32));
  }
}

// ---- draft verification ---------------------------------------------------------
// Sums over a vocabulary decide an integer, so they are exact far beyond fp32:
// each thread adds unevaluated pairs of floats (two-sums, ~2^-46 relative), the
// pairs meet in fp64. fp64 arithmetic per element would cost 50 times more here
// (2 results per clock and SM against 128).
struct Two {
  float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ void two_add(Two& acc, Two x) {
  const Two t = two_sum(acc.h, x.h);
  acc.h = t.h;
  acc.l = __fadd_rn(acc.l, __fadd_rn(t.l, x.l));
}
__device__ __forceinline__ double two_double(Two x) { return (double)x.h + (double)x.l; }

constexpr int kVerThreads = 512;

struct VerShared {
  int tok[kTreeMaxNodes], par[kTreeMaxNodes], path[kTreeMaxNodes];
  float u[kTreeMaxNodes], px[kTreeMaxNodes], qx[kTreeMaxNodes];
  double mass[kTreeMaxNodes + 1];  // what rejection k - 1 left, in all
  Two inv[kTreeMaxNodes + 1];      // its reciprocal
  double warp_sum[kVerThreads / 32];
  double sums[2][16];              // every rank's slice sum, in two buffers used in turn
};

// What k rejections leave of p(j), unnormalised after the last one.
__device__ __forceinline__ Two residual(float p, float q, const Two* inv, int k) {
  Two r = {fmaxf(p, 0.f), 0.f};  // a NaN probability counts as 0
  q = fmaxf(q, 0.f);
  for (int i = 0; i < k; ++i) {
    if (i > 0) {
      const Two f = inv[i];
      const float h = __fmul_rn(r.h, f.h);
      r = {h, __fmaf_rn(r.h, f.h, -h) + (r.h * f.l + r.l * f.h)};
    }
    const Two t = two_sum(r.h, -q);
    const Two d = two_sum(t.h, __fadd_rn(t.l, r.l));
    r = d.h > 0.f ? d : Two{0.f, 0.f};
  }
  return r;
}

// One cluster per sequence. Every CTA walks the tree on the same prefetched
// values, so the walk needs no communication; the vocabulary is read only for
// the masses of rejections that a later sibling needs, and once for the final
// draw: each rank sums its slice, the ranks exchange their sums, and the rank,
// the warp, the lane and the token where the running sum passes u tot are
// found level by level.
template <bool SOFT>  // SOFT: draft probabilities are given
__global__ void __launch_bounds__(kVerThreads) verify_kernel(const VerifyParams p) {
  __shared__ VerShared s;
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = kVerThreads / 32;
  const int cnt = p.counts ? min(max(p.counts[b], 0), p.n) : p.n, V = p.V;
  int* path_out = p.path + (int64_t)b * p.n;
  if (cnt == 0) {  // nothing is chosen (the same in every CTA of the cluster)
    if (rank == 0) {
      if (tid < p.n) path_out[tid] = -1;
      if (tid == 0) p.n_path[b] = 0, p.next[b] = -1;
    }
    return;
  }
  const float* pb = p.p + (int64_t)b * p.p_seq;
  const float* qb = SOFT ? p.q + (int64_t)b * p.q_seq : nullptr;
  if (tid < cnt) {  // every node's test values at once
    const int64_t at = (int64_t)b * p.n + tid;
    const int par = tid ? p.parents[at] : -1, tok = p.tokens[at];
    const bool ok = par >= 0 && par < tid && tok >= 0 && tok < V;
    s.tok[tid] = tok;
    s.par[tid] = par < tid ? par : -1;
    s.u[tid] = p.u[at];
    s.px[tid] = ok ? fmaxf(pb[(int64_t)par * p.p_node + tok], 0.f) : 0.f;
    s.qx[tid] = ok && SOFT ? fmaxf(qb[(int64_t)par * p.q_node + tok], 0.f) : 1.f;
  }
  if (tid == 0) s.path[0] = 0, s.mass[0] = 1.0;
  __syncthreads();
  // warp `warp` owns elements w0 .. w1 of the row, a multiple of 32 but for the end
  const int chunk = (V + 32 * C * NW - 1) / (32 * C * NW);  // elements of a lane when lanes own runs
  const int w0 = (int)min((int64_t)V, (int64_t)32 * chunk * (rank * NW + warp)), w1 = min(V, w0 + 32 * chunk);
  int turn = 0, cur = 0, n_path = 1, k = 0;  // k: rejections that count at `cur`
  auto removed = [&](int j) {  // !SOFT: a rejected child's token
    for (int i = cur + 1; i < cnt; ++i)
      if (s.par[i] == cur && s.tok[i] == j) return true;
    return false;
  };
  bool holes = false;  // !SOFT: whether a rejected token falls into this warp's elements
  const float *pr = nullptr, *qr = nullptr;
  auto element = [&](int j) {
    if constexpr (SOFT) {
      return residual(pr[j], k ? qr[j] : 0.f, s.inv, k);
    } else {
      const float x = fmaxf(pr[j], 0.f);
      return Two{holes && removed(j) ? 0.f : x, 0.f};
    }
  };
  auto total = [&]() {  // the sum over the row of `cur` after k rejections; leaves warp_sum and sums
    pr = pb + (int64_t)cur * p.p_node;
    if constexpr (SOFT) qr = qb + (int64_t)cur * p.q_node;
    else
      for (int i = cur + 1; i < cnt; ++i) holes |= s.par[i] == cur && s.tok[i] >= w0 && s.tok[i] < w1;
    Two acc = {0.f, 0.f};
#pragma unroll 8
    for (int i = w0 + lane; i < w1; i += 32) two_add(acc, element(i));
    double d = two_double(acc);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) s.warp_sum[warp] = d;
    __syncthreads();
    if (warp == 0) {
      d = lane < NW ? s.warp_sum[lane] : 0.0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      if (lane < C) cl.map_shared_rank(&s.sums[turn][0], lane)[rank] = d;
    }
    cl.sync();
    double t = 0.0;
    for (int r = 0; r < C; ++r) t += s.sums[turn][r];
    turn ^= 1;  // the other ranks have left the other buffer before this call's barrier
    return t;
  };
  bool known = true;  // s.mass[k], s.inv[k] are set
  double gone = 0.0;  // !SOFT: probability of the rejected children
  for (int i = 1; i < cnt; ++i) {
    if (s.par[i] != cur) continue;
    bool take;
    if constexpr (SOFT) {
      if (!known) {
        const double m = total();
        if (m > 0.0) {
          if (tid == 0) {
            const float h = (float)(1.0 / m);
            s.inv[k] = {h, (float)(1.0 / m - (double)h)};
            s.mass[k] = m;
          }
          __syncthreads();
        } else {  // nothing is left: that rejection does not count
          --k;
        }
        known = true;
      }
      take = (double)s.u[i] * (double)s.qx[i] * s.mass[k] < two_double(residual(s.px[i], s.qx[i], s.inv, k));
    } else {  // an earlier sibling with the same token has taken its probability
      double x = s.px[i];
      for (int j = cur + 1; j < i; ++j)
        if (s.par[j] == cur && s.tok[j] == s.tok[i]) x = 0.0;
      take = (double)s.u[i] * (1.0 - gone) < x;
      gone += x;
    }
    if (take) {
      if (tid == 0) s.path[n_path] = i;
      cur = i;
      ++n_path;
      k = 0;
      gone = 0.0;
      known = true;
    } else if (SOFT) {
      ++k;
      known = false;
    }
  }
  // ---- the next token, from what is left at `cur`
  double tot = total();
  while (SOFT && k > 0 && !(tot > 0.0)) {
    --k;
    tot = total();
  }
  const double* sums = s.sums[turn ^ 1];
  const double target = (double)s.u[0] * tot;
  int owner = -1, last = -1;
  double base = 0.0, cum = 0.0;
  for (int r = 0; r < C && owner < 0; ++r) {
    if (sums[r] > 0.0) last = r, base = cum;
    cum += sums[r];
    if (cum > target) owner = r;
  }
  if (owner < 0) owner = last;  // u beyond the sum's last bit
  if (rank == 0 && tid < p.n) path_out[tid] = tid < n_path ? s.path[tid] : -1;
  if (rank == 0 && tid == 0) {
    p.n_path[b] = n_path;
    if (owner < 0) p.next[b] = V - 1;  // a row without mass
  }
  if (owner == rank) {
    int ow = -1, lw = 0;
    double wbase = base, wcum = base;
    for (int w = 0; w < NW && ow < 0; ++w) {
      if (s.warp_sum[w] > 0.0) lw = w, wbase = wcum;
      wcum += s.warp_sum[w];
      if (wcum > target) ow = w;
    }
    if (ow < 0) ow = lw;
    if (warp == ow) {
      // lane l: the run of `chunk` elements from w0 + l chunk
      const int l0 = min(w1, w0 + lane * chunk), l1 = min(w1, l0 + chunk);
      Two acc = {0.f, 0.f};
#pragma unroll 8
      for (int i = l0; i < l1; ++i) two_add(acc, element(i));
      const double mine = two_double(acc);
      double incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned over = __ballot_sync(0xffffffffu, wbase + incl > target && mine > 0.0);
      const unsigned some = __ballot_sync(0xffffffffu, mine > 0.0);
      const int ol = over ? __ffs(over) - 1 : 31 - __clz(some);
      double run = wbase + __shfl_sync(0xffffffffu, incl - mine, ol);
      const int r0 = __shfl_sync(0xffffffffu, l0, ol), r1 = __shfl_sync(0xffffffffu, l1, ol);
      int pick = -1, fallback = V - 1;
      for (int i0 = r0; i0 < r1 && pick < 0; i0 += 32) {
        const double x = i0 + lane < r1 ? two_double(element(i0 + lane)) : 0.0;
        double in = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, in, o);
          if (lane >= o) in += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, x > 0.0 && run + in > target);
        const unsigned pos = __ballot_sync(0xffffffffu, x > 0.0);
        if (hit) pick = i0 + __ffs(hit) - 1;
        if (pos) fallback = i0 + 31 - __clz(pos);
        run += __shfl_sync(0xffffffffu, in, 31);
      }
      if (lane == 0) p.next[b] = pick >= 0 ? pick : fallback;
    }
  }
}

// Greedy: a child is kept when it is the target's own choice after its parent.
__global__ void __launch_bounds__(kTreeMaxNodes) verify_greedy_kernel(const VerifyParams p) {
  __shared__ int tok[kTreeMaxNodes], par[kTreeMaxNodes], tgt[kTreeMaxNodes], path[kTreeMaxNodes];
  __shared__ int s_n;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int cnt = p.counts ? min(max(p.counts[b], 0), p.n) : p.n;
  if (tid < cnt) {
    const int64_t at = (int64_t)b * p.n + tid;
    tok[tid] = p.tokens[at];
    par[tid] = p.parents[at];
    tgt[tid] = p.targets[at];
  }
  __syncthreads();
  if (tid == 0) {
    int cur = 0, n = 0;
    if (cnt > 0) path[n++] = 0;
    for (int i = 1; i < cnt; ++i)
      if (par[i] == cur && tok[i] == tgt[cur]) path[n++] = cur = i;
    s_n = n;
    p.n_path[b] = n;
    p.next[b] = cnt > 0 ? tgt[cur] : -1;
  }
  __syncthreads();
  if (tid < p.n) p.path[(int64_t)b * p.n + tid] = tid < s_n ? path[tid] : -1;
}

// ---- commit -----------------------------------------------------------------------
// cache row len + k = tree row path[k] for every layer, head, K and V: 16-byte
// copies, a thread per chunk, four rows' loads of a thread in flight.
__global__ void __launch_bounds__(256) commit_kernel(const CommitParams p) {
  __shared__ int s_path[kTreeMaxNodes];
  const int b = blockIdx.y, tid = threadIdx.x;
  const int len = max(p.lens[b], 0);
  const int n = min(min(max(p.n_path[b], 0), p.n), max(p.cache.rows - len, 0));
  if (tid < p.n) s_path[tid] = p.path[(int64_t)b * p.path_seq + tid];
  __syncthreads();
  const int ch = p.row_bytes / 16, per_head = n * ch;
  const int64_t total = (int64_t)2 * p.L * p.Hkv * per_head;
  const int esize = p.srow_bytes ? 1 : 2;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + tid; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int lh = (int)(i / per_head), r = (int)(i - (int64_t)lh * per_head), k = r / ch, c = r - k * ch;
    const int kv = lh & 1, h = (lh >> 1) % p.Hkv, l = (lh >> 1) / p.Hkv, node = s_path[k];
    if (node < 0 || node >= p.tree.rows) continue;
    const uint8_t* src = (kv ? p.tree.v : p.tree.k) +
                         esize * (b * p.tree.seq + l * p.t_layer + h * p.tree.head + node * p.tree.row) + 16 * c;
    uint8_t* dst = const_cast<uint8_t*>(kv ? p.cache.v : p.cache.k) +
                   esize * (b * p.cache.seq + l * p.c_layer + h * p.cache.head + (len + k) * p.cache.row) + 16 * c;
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
    if (c == 0 && p.srow_bytes) {
      const uint16_t* ss = (kv ? p.tree.vs : p.tree.ks) + b * p.tree.sseq + l * p.t_slayer + h * p.tree.shead +
                           node * p.tree.srow;
      uint16_t* sd = const_cast<uint16_t*>(kv ? p.cache.vs : p.cache.ks) + b * p.cache.sseq + l * p.c_slayer +
                     h * p.cache.shead + (len + k) * p.cache.srow;
      for (int e = 0; e < p.srow_bytes / 2; ++e) sd[e] = ss[e];
    }
  }
  if (p.new_lens != p.lens && blockIdx.x == 0 && tid == 0) p.new_lens[b] = len + n;
}
__global__ void __launch_bounds__(256) advance_kernel(const CommitParams p) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.B) return;
  const int len = max(p.lens[b], 0);
  p.new_lens[b] = len + min(min(max(p.n_path[b], 0), p.n), max(p.cache.rows - len, 0));
}

int pow2_at_least(int x) {
  int r = 1;
  while (r < x) r *= 2;
  return r;
}

}  // namespace

cudaError_t launch_token_probs(const TokenProbsParams& p, int n_sm, cudaStream_t st) {
  const int max_slice = p.top_k ? 32768 : kProbSlice;
  int C = pow2_at_least((p.V + max_slice - 1) / max_slice);
  if (C > 16) return cudaErrorInvalidValue;
  while (C < 8 && (int64_t)p.R * C < 2 * n_sm && p.V / (2 * C) >= 2048) C *= 2;
  while (C < 8 && p.V / C > 20480) C *= 2;  // two CTAs on an SM
  const int slice = (p.V + 4 * C - 1) / (4 * C) * 4;
  static SmemLimit lim_s, lim_k;
  if (p.top_k == 0) {
    const int smem = (slice + 4) * 4;
    cudaError_t e = lim_s.raise(softmax_rows_kernel, (kProbSlice + 8) * 4);
    if (e == cudaSuccess && C > 8)
      e = cudaFuncSetAttribute(softmax_rows_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e == cudaSuccess ? launch_cluster(softmax_rows_kernel, dim3(p.R * C), kProbThreads, C, smem, st, p) : e;
  }
  // the keys from the threshold on belong to at most top_k of the groups of 4 threads
  const int cand = kSampleMaxK * 4 * ((slice + kProbThreads - 1) / kProbThreads);
  TokenProbsParams q = p;
  q.cap = slice;
  cudaError_t e = lim_k.raise(topk_rows_kernel, 210 * 1024);
  if (e == cudaSuccess && C > 8)
    e = cudaFuncSetAttribute(topk_rows_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e == cudaSuccess
             ? launch_cluster(topk_rows_kernel, dim3(p.R * C), kProbThreads, C, (slice + 4 + cand) * 4, st, q)
             : e;
}

cudaError_t launch_verify_tree(const VerifyParams& p, int n_sm, cudaStream_t st) {
  if (p.targets) {
    verify_greedy_kernel<<<p.B, kTreeMaxNodes, 0, st>>>(p);
    return cudaGetLastError();
  }
  int C = 1;
  while (C < 8 && p.V / (2 * C) >= 2 * kVerThreads) C *= 2;
  return p.q ? launch_cluster(verify_kernel<true>, dim3(p.B * C), kVerThreads, C, 0, st, p)
             : launch_cluster(verify_kernel<false>, dim3(p.B * C), kVerThreads, C, 0, st, p);
}

cudaError_t launch_commit_tree(const CommitParams& p, cudaStream_t st) {
  const int64_t chunks = (int64_t)2 * p.L * p.Hkv * p.n * (p.row_bytes / 16);
  const int blocks = (int)((chunks + 255) / 256 < 4096 ? (chunks + 255) / 256 : 4096);
  commit_kernel<<<dim3(blocks, p.B), 256, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.new_lens == p.lens) {  // every copy has read the lengths before they advance
    advance_kernel<<<(p.B + 255) / 256, 256, 0, st>>>(p);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace llmq

// ---- C entries -------------------------------------------------------------------
using namespace llmq;

namespace {

int bad(int code, const char* fmt, const char* a = "", long long b = 0) {
  char msg[256];
  std::snprintf(msg, sizeof(msg), fmt, a, b);
  return op_error(code, msg);
}

int cuda_bad(cudaError_t e, const char* what) {
  char msg[256];
  std::snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return op_error(e == cudaErrorMemoryAllocation ? LLM_ERR_OOM : LLM_ERR_CUDA, msg);
}

// Status word of the tree attention's bounded waits, one per device.
__device__ int g_tree_status;

cudaError_t status_word(int dev, int** p) {
  static std::atomic<int*> known[64];
  *p = dev < 64 ? known[dev].load(std::memory_order_acquire) : nullptr;
  if (*p) return cudaSuccess;
  void* a = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&a, g_tree_status);
  if (e != cudaSuccess) return e;
  *p = static_cast<int*>(a);
  if (dev < 64) known[dev].store(*p, std::memory_order_release);
  return cudaSuccess;
}

// Checks of one call: the current device, and that every buffer is its memory.
struct Call {
  int dev = -1, n_sm = 0, rc = LLM_OK;
  cudaError_t e = cudaSuccess;  // reported by the first buffer's check, after those of sizes
  Call() {
    static std::atomic<int> sms[64];
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) {
      n_sm = dev < 64 ? sms[dev].load(std::memory_order_relaxed) : 0;
      if (!n_sm) {
        e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && dev < 64) sms[dev].store(n_sm, std::memory_order_relaxed);
      }
    }
  }
  bool device(const char* name, const void* p, size_t align) {
    if (rc) return false;
    if (!p) {
      rc = bad(LLM_ERR_INVALID_ARG, "%s is null", name);
      return false;
    }
    if (reinterpret_cast<uintptr_t>(p) % align) {
      rc = bad(LLM_ERR_INVALID_ARG, "%s is not aligned to %lld bytes", name, (long long)align);
      return false;
    }
    if (e != cudaSuccess) {
      rc = cuda_bad(e, "current device");
      return false;
    }
    cudaPointerAttributes a{};
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) cudaGetLastError();
    const bool dm = a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged;
    if (!dm || (a.type == cudaMemoryTypeDevice && a.device != dev)) {
      rc = bad(LLM_ERR_INVALID_ARG, "%s is not memory of the current device", name);
      return false;
    }
    return true;
  }
  bool need(bool ok, int code, const char* fmt, const char* a = "", long long b = 0) {
    if (!rc && !ok) rc = bad(code, fmt, a, b);
    return !rc;
  }
};

// Whether rows of `inner` elements at these (size, stride) steps are apart.
bool apart(int64_t inner, int n, const int64_t* size, const int64_t* stride) {
  int order[4] = {0, 1, 2, 3};
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if (stride[order[j]] < stride[order[i]]) std::swap(order[i], order[j]);
  int64_t extent = inner;
  for (int i = 0; i < n; ++i) {
    const int64_t s = size[order[i]], t = stride[order[i]];
    if (s <= 1) continue;
    if (t < extent) return false;
    extent += t * (s - 1);
  }
  return true;
}

bool check_view(Call& c, const llm_kv_view* v, const char* name) {
  if (!c.need(v != nullptr, LLM_ERR_INVALID_ARG, "%s is null", name)) return false;
  if (!c.need(v->dtype == LLM_BF16 || v->dtype == LLM_Q8G32, LLM_ERR_UNSUPPORTED,
              "%s: rows are bf16 or int8 with a scale per 32 values", name) ||
      !c.need(v->head_dim == 64 || v->head_dim == 128, LLM_ERR_UNSUPPORTED, "%s: head_dim %lld (64 or 128)", name,
              v->head_dim) ||
      !c.need(v->n_seq > 0 && v->n_layers > 0 && v->n_heads > 0 && v->rows >= 0 && v->n_seq <= 65535,
              LLM_ERR_INVALID_ARG, "%s: a size is not positive, or over 65535 sequences", name))
    return false;
  const bool q8 = v->dtype == LLM_Q8G32;
  const int64_t m = q8 ? 16 : 8, sm = v->head_dim / 32;
  if (!c.need(v->seq_stride >= 0 && v->layer_stride >= 0 && v->head_stride >= 0 && v->row_stride >= 0 &&
                  v->seq_stride % m == 0 && v->layer_stride % m == 0 && v->head_stride % m == 0 &&
                  v->row_stride % m == 0,
              LLM_ERR_INVALID_ARG, "%s: a stride is negative or no multiple of 16 bytes", name))
    return false;
  if (q8 && !c.need(v->scale_seq_stride >= 0 && v->scale_layer_stride >= 0 && v->scale_head_stride >= 0 &&
                    v->scale_row_stride >= 0 && v->scale_seq_stride % sm == 0 && v->scale_layer_stride % sm == 0 &&
                    v->scale_head_stride % sm == 0 && v->scale_row_stride % sm == 0,
                LLM_ERR_INVALID_ARG, "%s: a scale stride is negative or no multiple of a row's scales", name))
    return false;
  return true;
}

bool view_memory(Call& c, const llm_kv_view* v, const char* name) {
  if (v->rows == 0) return true;  // an empty cache has no rows to point at
  const size_t sm = 2 * (v->head_dim / 32);
  return c.device(name, v->k, 16) && c.device(name, v->v, 16) &&
         (v->dtype != LLM_Q8G32 || (c.device(name, v->k_scales, sm) && c.device(name, v->v_scales, sm)));
}

KvRows rows_of(const llm_kv_view& v) {
  KvRows r;
  r.k = static_cast<const uint8_t*>(v.k);
  r.v = static_cast<const uint8_t*>(v.v);
  r.ks = static_cast<const uint16_t*>(v.k_scales);
  r.vs = static_cast<const uint16_t*>(v.v_scales);
  r.seq = v.seq_stride;
  r.head = v.head_stride;
  r.row = v.row_stride;
  r.sseq = v.scale_seq_stride;
  r.shead = v.scale_head_stride;
  r.srow = v.scale_row_stride;
  r.rows = v.rows;
  return r;
}

int finish(cudaError_t e, const char* what) { return e == cudaSuccess ? LLM_OK : cuda_bad(e, what); }

}  // namespace

extern "C" {

int llm_tree_attention(const llm_tree_attention_args* a, void* cuda_stream) {
  Call c;
  if (!c.need(a != nullptr, LLM_ERR_INVALID_ARG, "the arguments are null")) return c.rc;
  if (!c.need(a->dtype == LLM_BF16 || a->dtype == LLM_F32, LLM_ERR_UNSUPPORTED, "queries are bf16 or f32")) return c.rc;
  if (!c.need(a->n_nodes >= 1 && a->n_nodes <= kTreeMaxNodes, LLM_ERR_UNSUPPORTED, "%sn_nodes %lld (1..64)", "",
              a->n_nodes) ||
      !c.need(a->n_seq >= 1, LLM_ERR_INVALID_ARG, "n_seq is not positive") ||
      !c.need(std::isfinite(a->scale), LLM_ERR_INVALID_ARG, "the scale is not finite") ||
      !check_view(c, a->cache, "cache"))
    return c.rc;
  const llm_kv_view &v = *a->cache, *t = a->tree;
  if (!c.need(a->n_heads > 0 && a->n_heads % v.n_heads == 0, LLM_ERR_INVALID_ARG,
              "n_heads is no multiple of the cache's heads") ||
      !c.need(v.n_seq >= a->n_seq && v.n_layers == 1, LLM_ERR_INVALID_ARG,
              "the cache view holds fewer sequences, or several layers") ||
      !c.need((int64_t)v.n_heads * ((int64_t)a->n_nodes * (a->n_heads / v.n_heads) / 16 + 1) <= 65535,
              LLM_ERR_UNSUPPORTED, "too many heads"))
    return c.rc;
  if (t && (!check_view(c, t, "tree") ||
            !c.need(t->dtype == v.dtype && t->head_dim == v.head_dim && t->n_heads == v.n_heads && t->n_layers == 1 &&
                        t->n_seq >= a->n_seq && t->rows >= a->n_nodes,
                    LLM_ERR_INVALID_ARG, "the tree's rows do not match the cache or the nodes")))
    return c.rc;
  const int64_t hd = v.head_dim, m = a->dtype == LLM_F32 ? 4 : 8;
  const int64_t size[3] = {a->n_seq, a->n_nodes, a->n_heads};
  for (int i = 0; i < 3; ++i)
    if (!c.need(a->q_strides[i] >= 0 && a->out_strides[i] >= 0 && a->q_strides[i] % m == 0 &&
                    a->out_strides[i] % m == 0,
                LLM_ERR_INVALID_ARG, "a stride of q or out is negative or no multiple of 16 bytes"))
      return c.rc;
  if (!c.need(apart(hd, 3, size, a->out_strides), LLM_ERR_INVALID_ARG, "rows of out overlap") ||
      !view_memory(c, a->cache, "cache") || (t && (!view_memory(c, t, "tree") || !c.device("mask", a->mask, 8))) ||
      !c.device("q", a->q, 16) || !c.device("out", a->out, 16) || !c.device("lens", a->lens, 4) ||
      (a->counts && !c.device("counts", a->counts, 4)))
    return c.rc;
  TreeAttnParams p{};
  p.q = a->q;
  p.out = a->out;
  p.q_seq = a->q_strides[0], p.q_node = a->q_strides[1], p.q_head = a->q_strides[2];
  p.o_seq = a->out_strides[0], p.o_node = a->out_strides[1], p.o_head = a->out_strides[2];
  p.cache = rows_of(v);
  if (t) p.tree = rows_of(*t);
  p.lens = a->lens;
  p.mask = a->mask;
  p.mask_seq = a->n_nodes;
  p.counts = a->counts;
  p.c = (float)((double)a->scale * 1.4426950408889634);
  if (std::fabs(p.c) < 1e-30f) p.c = 1e-30f;  // a scale of 0: every score below 2^-60, and c times -inf still -inf
  const cudaError_t es = status_word(c.dev, &p.status);
  if (es != cudaSuccess) return cuda_bad(es, "status word");
  p.B = a->n_seq;
  p.n = a->n_nodes;
  p.Hkv = v.n_heads;
  p.gq = a->n_heads / v.n_heads;
  return finish(launch_tree_attn(p, (int)hd, a->dtype == LLM_F32, v.dtype == LLM_Q8G32, c.n_sm,
                                 static_cast<cudaStream_t>(cuda_stream)),
                "tree attention launch");
}

int llm_tree_status(void* cuda_stream) {
  Call c;
  int *p = nullptr, st = 0;
  cudaError_t e = c.e != cudaSuccess ? c.e : status_word(c.dev, &p);
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&st, p, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && st) e = cudaMemsetAsync(p, 0, sizeof(int), s);
  if (e != cudaSuccess) return cuda_bad(e, "tree status");
  return st & ST_TIMEOUT ? bad(LLM_ERR_TIMEOUT, "a device-side wait of a tree attention exceeded its limit") : LLM_OK;
}

int llm_token_probs(const float* logits, int64_t logits_stride, float* probs, int64_t probs_stride, int32_t n_rows,
                    int32_t vocab, float temperature, int32_t top_k, float top_p, void* cuda_stream) {
  Call c;
  const double cc = 1.4426950408889634 / (double)temperature;
  if (!c.need(n_rows >= 1 && vocab >= 1, LLM_ERR_INVALID_ARG, "n_rows or vocab is not positive") ||
      !c.need(temperature > 0.f && std::isfinite(temperature) && cc <= 3e38, LLM_ERR_INVALID_ARG,
              "temperature must be finite and > 0 (the greedy choice needs no probabilities)") ||
      !c.need(top_k >= 0 && top_k <= kSampleMaxK, LLM_ERR_INVALID_ARG, "top_k must be in 0..64") ||
      !c.need(top_p > 0.f && top_p <= 1.f, LLM_ERR_INVALID_ARG, "top_p must be in (0, 1]") ||
      !c.need(top_k > 0 || top_p == 1.f, LLM_ERR_UNSUPPORTED, "top_p below 1 needs a top_k") ||
      !c.need(vocab <= (top_k ? 16 * 32768 : 16 * kProbSlice), LLM_ERR_UNSUPPORTED, "%svocab %lld is too large", "",
              vocab) ||
      !c.need((int64_t)n_rows * 16 <= 0x7FFFFFFF, LLM_ERR_UNSUPPORTED, "too many rows") ||
      !c.need(n_rows == 1 || probs_stride >= vocab, LLM_ERR_INVALID_ARG, "rows of probs overlap") ||
      !c.need(logits_stride >= 0, LLM_ERR_INVALID_ARG, "a stride is negative") || !c.device("logits", logits, 4) ||
      !c.device("probs", probs, 4))
    return c.rc;
  if (!c.need(static_cast<const void*>(logits) == probs ? n_rows == 1 || logits_stride == probs_stride
                                                        : probs + (int64_t)(n_rows - 1) * probs_stride + vocab <= logits ||
                                                              logits + (int64_t)(n_rows - 1) * logits_stride + vocab <= probs,
              LLM_ERR_INVALID_ARG, "probs overlaps logits (allowed: the same rows)"))
    return c.rc;
  TokenProbsParams p{};
  p.logits = logits;
  p.probs = probs;
  p.l_row = logits_stride;
  p.p_row = probs_stride;
  p.R = n_rows;
  p.V = vocab;
  p.c = (float)cc;
  p.top_k = top_k;
  p.top_p = top_p;
  return finish(launch_token_probs(p, c.n_sm, static_cast<cudaStream_t>(cuda_stream)), "token probabilities launch");
}

int llm_verify_tree(const llm_verify_tree_args* a, void* cuda_stream) {
  Call c;
  if (!c.need(a != nullptr, LLM_ERR_INVALID_ARG, "the arguments are null")) return c.rc;
  if (!c.need(a->n_nodes >= 1 && a->n_nodes <= kTreeMaxNodes, LLM_ERR_UNSUPPORTED, "%sn_nodes %lld (1..64)", "",
              a->n_nodes) ||
      !c.need(a->n_seq >= 1 && a->n_seq <= (1 << 20), LLM_ERR_INVALID_ARG, "n_seq is not in 1..2^20") ||
      !c.need((a->probs != nullptr) != (a->targets != nullptr), LLM_ERR_INVALID_ARG,
              "either probs or targets must be given") ||
      !c.need(!a->targets || !a->draft_probs, LLM_ERR_INVALID_ARG, "draft_probs need probs") ||
      !c.device("tokens", a->tokens, 4) || !c.device("parents", a->parents, 4) || !c.device("path", a->path, 4) ||
      !c.device("n_path", a->n_path, 4) || !c.device("next", a->next, 4) ||
      (a->counts && !c.device("counts", a->counts, 4)) || (a->targets && !c.device("targets", a->targets, 4)))
    return c.rc;
  if (a->probs &&
      (!c.need(a->vocab >= 1 && a->vocab <= (1 << 30), LLM_ERR_INVALID_ARG, "vocab is not in 1..2^30") ||
       !c.device("probs", a->probs, 4) || !c.device("uniforms", a->uniforms, 4) ||
       (a->draft_probs && !c.device("draft_probs", a->draft_probs, 4)) ||
       !c.need(a->probs_strides[0] >= 0 && a->probs_strides[1] >= 0 && a->draft_strides[0] >= 0 &&
                   a->draft_strides[1] >= 0,
               LLM_ERR_INVALID_ARG, "a stride is negative")))
    return c.rc;
  VerifyParams p{};
  p.tokens = a->tokens;
  p.parents = a->parents;
  p.counts = a->counts;
  p.u = a->uniforms;
  p.p = a->probs;
  p.q = a->draft_probs;
  p.p_seq = a->probs_strides[0], p.p_node = a->probs_strides[1];
  p.q_seq = a->draft_strides[0], p.q_node = a->draft_strides[1];
  p.targets = a->targets;
  p.path = a->path;
  p.n_path = a->n_path;
  p.next = a->next;
  p.B = a->n_seq;
  p.n = a->n_nodes;
  p.V = a->vocab;
  return finish(launch_verify_tree(p, c.n_sm, static_cast<cudaStream_t>(cuda_stream)), "verification launch");
}

int llm_commit_tree(const llm_kv_view* cache, const llm_kv_view* tree, int32_t n_seq, int32_t n_nodes,
                    const int32_t* lens, const int32_t* path, const int32_t* n_path, int32_t* new_lens,
                    void* cuda_stream) {
  Call c;
  if (!c.need(n_nodes >= 1 && n_nodes <= kTreeMaxNodes, LLM_ERR_UNSUPPORTED, "%sn_nodes %lld (1..64)", "", n_nodes) ||
      !c.need(n_seq >= 1, LLM_ERR_INVALID_ARG, "n_seq is not positive") || !check_view(c, cache, "cache") ||
      !check_view(c, tree, "tree") ||
      !c.need(cache->dtype == tree->dtype && cache->head_dim == tree->head_dim && cache->n_heads == tree->n_heads &&
                  cache->n_layers == tree->n_layers && cache->n_seq >= n_seq && tree->n_seq >= n_seq &&
                  tree->rows >= n_nodes,
              LLM_ERR_INVALID_ARG, "the tree's rows do not match the cache or the nodes") ||
      !c.need(new_lens == lens || new_lens + n_seq <= lens || lens + n_seq <= new_lens, LLM_ERR_INVALID_ARG,
              "new_lens overlaps lens (allowed: the same array)"))
    return c.rc;
  const int64_t size[4] = {cache->n_seq, cache->n_layers, cache->n_heads, cache->rows};
  const int64_t stride[4] = {cache->seq_stride, cache->layer_stride, cache->head_stride, cache->row_stride};
  const int64_t sstride[4] = {cache->scale_seq_stride, cache->scale_layer_stride, cache->scale_head_stride,
                              cache->scale_row_stride};
  const bool q8 = cache->dtype == LLM_Q8G32;
  if (!c.need(apart(cache->head_dim, 4, size, stride) && (!q8 || apart(cache->head_dim / 32, 4, size, sstride)),
              LLM_ERR_INVALID_ARG, "rows of the cache overlap") ||
      !view_memory(c, cache, "cache") || !view_memory(c, tree, "tree") || !c.device("lens", lens, 4) ||
      !c.device("path", path, 4) || !c.device("n_path", n_path, 4) || !c.device("new_lens", new_lens, 4))
    return c.rc;
  CommitParams p{};
  p.cache = rows_of(*cache);
  p.tree = rows_of(*tree);
  p.c_layer = cache->layer_stride, p.c_slayer = cache->scale_layer_stride;
  p.t_layer = tree->layer_stride, p.t_slayer = tree->scale_layer_stride;
  p.lens = lens;
  p.path = path;
  p.n_path = n_path;
  p.new_lens = new_lens;
  p.path_seq = n_nodes;
  p.B = n_seq;
  p.L = cache->n_layers;
  p.Hkv = cache->n_heads;
  p.n = n_nodes;
  p.row_bytes = cache->head_dim * (q8 ? 1 : 2);
  p.srow_bytes = q8 ? cache->head_dim / 16 : 0;
  return finish(launch_commit_tree(p, static_cast<cudaStream_t>(cuda_stream)), "commit launch");
}

}  // extern "C"
