// Token probabilities, draft verification and the commit of accepted rows, and
// the C entries of the tree-decoding operators (see tree.cuh).
#include <cooperative_groups.h>

#include <cmath>
#include <utility>

#include "common.cuh"
#include "op_call.cuh"
#include "sample_key.cuh"

namespace llmq {
namespace cg = cooperative_groups;

std::atomic<bool> g_expire_waits{false};

cudaError_t launch_tree_attn(const TreeAttnParams& p, int hd, bool f32, bool q8, int n_sm, cudaStream_t st) {
  return hd == 64 ? launch_tree_attn_64(p, f32, q8, n_sm, st) : launch_tree_attn_128(p, f32, q8, n_sm, st);
}

namespace {

// ---- sums that decide integers --------------------------------------------------
// A sum over a vocabulary picks a token, so it is carried far beyond fp32: as an
// unevaluated pair of floats (two-sums and fused products, ~2^-46 relative).
// This GPU has 64 times fewer fp64 than fp32 lanes: the same reductions in fp64
// took 10 us of a 20 us verification.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  const Two t = two_sum(a.h, b.h);
  const float l = __fadd_rn(t.l, __fadd_rn(a.l, b.l)), h = __fadd_rn(t.h, l);
  return {h, __fsub_rn(l, __fsub_rn(h, t.h))};
}
// the same without renormalising: for sums of many terms (|l| stays far below h)
__device__ __forceinline__ Two two_add(Two a, Two b) {
  const Two t = two_sum(a.h, b.h);
  return {t.h, __fadd_rn(t.l, __fadd_rn(a.l, b.l))};
}
__device__ __forceinline__ Two two_norm(Two a) {
  const float h = __fadd_rn(a.h, a.l);
  return {h, __fsub_rn(a.l, __fsub_rn(h, a.h))};
}
__device__ __forceinline__ Two two_prod(float a, float b) {
  const float h = __fmul_rn(a, b);
  return {h, __fmaf_rn(a, b, -h)};
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  const Two p = two_prod(a.h, b.h);
  const float l = __fadd_rn(p.l, __fadd_rn(__fmul_rn(a.h, b.l), __fmul_rn(a.l, b.h))), h = __fadd_rn(p.h, l);
  return {h, __fsub_rn(l, __fsub_rn(h, p.h))};
}
__device__ __forceinline__ bool operator<(Two a, Two b) {
  return a.h < b.h || (a.h == b.h && a.l < b.l);  // both normalised: |l| at most half a step of h
}
__device__ __forceinline__ Two two_recip(Two m) {  // one Newton step from the fp32 reciprocal
  const float r = __fdiv_rn(1.f, m.h);
  const float e = __fsub_rn(__fmaf_rn(-m.h, r, 1.f), __fmul_rn(m.l, r));
  const float l = __fmul_rn(r, e), h = __fadd_rn(r, l);
  return {h, __fsub_rn(l, __fsub_rn(h, r))};
}
__device__ __forceinline__ Two two_xor(Two v, int o) {
  return {__shfl_xor_sync(0xffffffffu, v.h, o), __shfl_xor_sync(0xffffffffu, v.l, o)};
}
template <int LANES>
__device__ __forceinline__ Two two_reduce(Two v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = two_add(v, two_xor(v, o));
  return two_norm(v);
}
__device__ __forceinline__ Two two_scan(Two v, int lane) {  // inclusive, over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two y = {__shfl_up_sync(0xffffffffu, v.h, o), __shfl_up_sync(0xffffffffu, v.l, o)};
    if (lane >= o) v = two_add(v, y);
  }
  return two_norm(v);
}

// ---- token probabilities -----------------------------------------------------
// p_j = 2^(c (l_j - m)) / sum over the kept tokens, c = log2(e) / T. A cluster
// owns a row: every CTA keeps its slice in shared memory, so the row is read
// once and written once; a CTA's (max, sum) or, with top_k, its sorted top_k
// candidates are all that crosses the cluster. A NaN counts as -inf, +inf as
// the largest finite value; a row without a finite logit is all zeros.
constexpr int kProbThreads = 512;

__device__ __forceinline__ float clean_logit(float x) { return x != x ? -INFINITY : fminf(x, 3.402823466e38f); }

// A slice of a row in global memory: [off, end) from a 16-byte boundary on,
// whole float4s [v0, v1), up to three floats before and after them.
struct Slice {
  int off, end, v0, v1, head, tail;
  __device__ Slice(const float* p, int n) {
    off = (int)((reinterpret_cast<uintptr_t>(p) >> 2) & 3);
    end = off + n;
    v0 = (off + 3) / 4;
    v1 = end / 4;
    head = min(4 * v0, end);
    tail = max(4 * v1, head);
  }
};

// The slice [p, p + n) to shared memory at the same alignment; f(x) maps a
// group of one or four values. Four 16-byte loads of a thread in flight.
template <typename F>
__device__ __forceinline__ void load_slice(float* sx, const float* p, const Slice& c, F f) {
  const float4* base = reinterpret_cast<const float4*>(p - c.off);
  constexpr int U = 4;
  for (int i0 = c.v0 + threadIdx.x; i0 < c.v1; i0 += U * kProbThreads) {
    float4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kProbThreads < c.v1) x[u] = __ldcs(base + i0 + u * kProbThreads);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kProbThreads < c.v1) {
        float v[4] = {clean_logit(x[u].x), clean_logit(x[u].y), clean_logit(x[u].z), clean_logit(x[u].w)};
        f(v);
        reinterpret_cast<float4*>(sx)[i0 + u * kProbThreads] = make_float4(v[0], v[1], v[2], v[3]);
      }
  }
  const int e = threadIdx.x < 4 ? c.off + (int)threadIdx.x : c.tail + (int)threadIdx.x - 4;
  if (threadIdx.x < 8 && (threadIdx.x < 4 ? e < c.head : e < c.end)) {
    float v[1] = {clean_logit(p[e - c.off])};
    f(v);
    sx[e] = v[0];
  }
}

struct ProbRange {  // slice of CTA `rank` of C: starts on a multiple of 4
  int a, n;
  __device__ ProbRange(int V, int rank, int C) {
    const int q = (V + 4 * C - 1) / (4 * C) * 4;
    a = min(V, q * rank);
    n = min(V, a + q) - a;
  }
};

// Shared -> global bulk copy (addresses 16-B aligned, bytes a multiple of 16).
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// Every token. Bulk copies bring the slice in two pieces and take it out again,
// so that the threads only compute, in place in shared memory, and three CTAs on
// an SM keep both directions of HBM busy: read and written once, 311 MB for 256 x
// 151936. Exponentials are taken once, against a reference instead of the row's
// maximum: the largest of the first piece. A CTA whose largest logit lies 2^60
// over its reference, or below it, takes its slice again against that one. 65.2 us (71 %
// of the copy rate); 512 threads 71.5, four pieces 66.2, one 70.6; 16 CTAs a row 75.6.
constexpr int kSoftThreads = 256;
constexpr int kPieces = 2;
static __device__ __noinline__ void wait_or_late(uint64_t* bar, uint32_t parity, int* status, uint32_t ns, int* late) {
  if (!mbar_wait(bar, parity, status, ns)) *late = 1;
}
__global__ void __launch_bounds__(kSoftThreads) softmax_rows_kernel(const TokenProbsParams p) {
  extern __shared__ __align__(16) float sx[];
  __shared__ __align__(8) uint64_t bars[kPieces];
  __shared__ float2 s_warp[kSoftThreads / 32];
  __shared__ float2 s_ms[16];
  __shared__ int s_late;  // a wait has run out
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31;
  auto started = cl.barrier_arrive();  // shared memory of another CTA: only once that CTA runs
  const ProbRange r(p.V, rank, C);
  const float* src = p.logits + (int64_t)row * p.l_row + r.a;
  float* dst = p.probs + (int64_t)row * p.p_row + r.a;
  const Slice sl(src, r.n);
  const int nv = max(sl.v1 - sl.v0, 0);
  auto piece = [&](int q) { return sl.v0 + (int)((int64_t)nv * q / kPieces); };
  if (tid == 0) {
    s_late = 0;
    for (int q = 0; q < kPieces; ++q) mbar_init(bars + q, 1 + p.wait.missing);
    mbar_fence_init();
  }
  pdl_wait();
  pdl_trigger();
  const uint64_t once = policy_evict_first();
  auto request = [&]() {
    for (int q = 0; q < kPieces; ++q) {
      const uint32_t bytes = 16 * (piece(q + 1) - piece(q));
      mbar_expect_tx(bars + q, bytes);
      if (bytes) bulk_g2s(sx + 4 * piece(q), src - sl.off + 4 * piece(q), bytes, bars + q, once);
    }
  };
  const int edge = tid < 4 ? sl.off + tid : sl.tail + tid - 4;  // this thread's float before or after the pieces
  const bool has_edge = tid < 8 && (tid < 4 ? edge < sl.head : edge < sl.end);
  float2 own = make_float2(-INFINITY, 0.f);  // (reference, sum) of the CTA
  // over the warps, in a fixed order, to every thread
  auto reduce = [&](float mx, float sum) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    __syncthreads();  // the last reduction has been read
    if (lane == 0) s_warp[tid >> 5] = make_float2(mx, sum);
    __syncthreads();
    float2 w = s_warp[lane & (kSoftThreads / 32 - 1)];
#pragma unroll
    for (int o = kSoftThreads / 64; o > 0; o >>= 1) {
      w.x = fmaxf(w.x, __shfl_xor_sync(0xffffffffu, w.x, o));
      w.y += __shfl_xor_sync(0xffffffffu, w.y, o);
    }
    return w;
  };
  float ref = 0.f;
  int turn = 0;
  auto landed = [&](int q) {
    if (!mbar_try_wait(bars + q, turn)) wait_or_late(bars + q, turn, p.status, p.wait.ns, &s_late);
  };
  for (; turn < 2; ++turn) {
    __syncthreads();  // the barriers are ready; a second turn: the slice has been read
    if (tid == 0) request();
    const float x_edge = has_edge ? clean_logit(src[edge - sl.off]) : -INFINITY;
    if (turn == 0) {
      float mx = x_edge;
      landed(0);
      for (int i = piece(0) + tid; i < piece(1); i += kSoftThreads) {
        const float4 x = reinterpret_cast<const float4*>(sx)[i];
        mx = fmaxf(mx, fmaxf(fmaxf(clean_logit(x.x), clean_logit(x.y)), fmaxf(clean_logit(x.z), clean_logit(x.w))));
      }
      mx = reduce(mx, 0.f).x;
      ref = mx == -INFINITY ? 0.f : mx;
    }
    float mx = x_edge, sum = 0.f;
    if (has_edge) {
      const float e = exp2f((x_edge - ref) * p.c);
      sx[edge] = e;
      sum += e;
    }
    for (int q = 0; q < kPieces; ++q) {
      landed(q);
#pragma unroll 2
      for (int i = piece(q) + tid; i < piece(q + 1); i += kSoftThreads) {
        float4 x = reinterpret_cast<const float4*>(sx)[i];
        x.x = clean_logit(x.x), x.y = clean_logit(x.y), x.z = clean_logit(x.z), x.w = clean_logit(x.w);
        mx = fmaxf(mx, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
        x.x = exp2f((x.x - ref) * p.c), x.y = exp2f((x.y - ref) * p.c);
        x.z = exp2f((x.z - ref) * p.c), x.w = exp2f((x.w - ref) * p.c);
        sum += (x.x + x.y) + (x.z + x.w);
        reinterpret_cast<float4*>(sx)[i] = x;
      }
    }
    const float2 w = reduce(mx, sum);
    own = make_float2(w.x == -INFINITY ? -INFINITY : ref, w.y);
    // (below it only where the first piece had none: small terms would be lost)
    if (turn == 1 || s_late || w.x == -INFINITY || (w.x >= ref && (w.x - ref) * p.c <= 60.f)) break;
    ref = w.x;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the slice is overwritten by bulk copies
  }
  if (s_late && tid == 0)  // no copy in flight outlives the CTA
    for (int q = 0; q < kPieces; ++q) landed(q);
  cl.barrier_wait(std::move(started));
  if (tid < C) cl.map_shared_rank(s_ms, tid)[rank] = own;  // to every rank
  cl.sync();  // after it no rank touches another's memory
  float M = -INFINITY, S = 0.f;
  for (int k = 0; k < C; ++k) M = fmaxf(M, s_ms[k].x);
  for (int k = 0; k < C; ++k)
    if (s_ms[k].x != -INFINITY) S += s_ms[k].y * exp2f((s_ms[k].x - M) * p.c);
  // 2^((own.x - M) c) / S in two factors: own terms reach 2^60, the largest rank's sum 2^77, so the whole may lie
  // below fp32's range where its products do not
  const int e2 = S > 0.f ? (int)(__float_as_uint(S) >> 23) - 127 : 0;
  const float h = S > 0.f && own.x != -INFINITY ? exp2f((own.x - M) * p.c * 0.5f) : 0.f;
  const float f1 = h * __uint_as_float((uint32_t)(127 - e2 / 2) << 23);
  const float f2 = h * __uint_as_float((uint32_t)(127 - (e2 - e2 / 2)) << 23) /
                   (S > 0.f ? __uint_as_float((__float_as_uint(S) & 0x007FFFFFu) | 0x3F800000u) : 1.f);
  if (has_edge) dst[edge - sl.off] = sx[edge] * f1 * f2;
  if ((int)((reinterpret_cast<uintptr_t>(dst) >> 2) & 3) == sl.off) {
    for (int q = 0; q < kPieces; ++q) {
#pragma unroll 2
      for (int i = piece(q) + tid; i < piece(q + 1); i += kSoftThreads) {
        float4 x = reinterpret_cast<const float4*>(sx)[i];
        x.x *= f1, x.y *= f1, x.z *= f1, x.w *= f1;
        x.x *= f2, x.y *= f2, x.z *= f2, x.w *= f2;
        reinterpret_cast<float4*>(sx)[i] = x;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      if (tid == 0) {
        const uint32_t bytes = 16 * (piece(q + 1) - piece(q));
        if (bytes) bulk_s2g(dst - sl.off + 4 * piece(q), sx + 4 * piece(q), bytes);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // written before the CTA ends
  } else {
    __syncthreads();
    for (int i = 4 * sl.v0 - sl.off + tid; i < 4 * sl.v1 - sl.off; i += kSoftThreads) dst[i] = sx[sl.off + i] * f1 * f2;
  }
}

// With top_k: 64-bit keys (order-preserving value, complement of the token id)
// make every logit's place unique, ties to the lower id. Of G = 128 groups of a
// CTA's threads the k-th largest group maximum is at most the CTA's k-th
// largest key, so the keys from it on, a few more than k, hold the CTA's top k;
// their ranks among themselves sort them. The sorted lists go to rank 0, which
// merges them by binary search, cuts the nucleus and writes every listed token;
// the other tokens are zeros that each CTA writes to its slice meanwhile
// (listed ones are marked there and left out). Bound by latency at few rows: 8.8 us
// for one row of 32000 tokens, top 40 (8 CTAs; a launch and three exchanges). Where the
// largest logits crowd into fewer groups than k, all of those groups' may be candidates,
// and the ranks quadratic: 9 ms for half of 151936 tokens.
constexpr int kProbGroups = 128;
constexpr int kFewCand = 768;

struct TopKShared {
  unsigned long long gmax[kProbGroups];
  unsigned long long few[kFewCand];               // the candidates' keys while they are few
  unsigned long long top[kSampleMaxK];            // this CTA's largest keys, sorted
  unsigned long long all[16][kSampleMaxK];        // rank 0: every rank's
  unsigned long long sorted[16 * kSampleMaxK];
  int n_all[16];
  int n_cand;
  unsigned long long thr;
};

__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u ^ 0x80000000u) : ~u);
}

__global__ void __launch_bounds__(kProbThreads) topk_rows_kernel(const TokenProbsParams p) {
  extern __shared__ __align__(16) float sx[];
  __shared__ TopKShared s;
  using u64 = unsigned long long;
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), row = blockIdx.x / C, tid = threadIdx.x;
  auto started = cl.barrier_arrive();
  pdl_wait();
  pdl_trigger();
  const ProbRange r(p.V, rank, C);
  const int K = min(p.top_k, p.V);
  int* cand = reinterpret_cast<int*>(sx + p.cap + 4);
  const float* src = p.logits + (int64_t)row * p.l_row + r.a;
  const Slice sl(src, r.n);
  load_slice(sx, src, sl, [](auto&) {});
  if (tid == 0) s.n_cand = 0;
  __syncthreads();
  auto key = [&](int i) {  // of slice element i; 0: a logit that is never kept
    const float x = sx[sl.off + i];
    return x == -INFINITY ? 0ull : ((u64)sample_key(x) << 32) | (uint32_t)(0x7FFFFFFF - (r.a + i));
  };
  u64 best = 0;
#pragma unroll 4
  for (int i = tid; i < r.n; i += kProbThreads) best = max(best, key(i));
  best = max(best, __shfl_xor_sync(0xffffffffu, best, 1));
  best = max(best, __shfl_xor_sync(0xffffffffu, best, 2));
  if ((tid & 3) == 0) s.gmax[tid >> 2] = best;
  __syncthreads();
  {  // the group maximum with K - 1 larger ones (group maxima differ, or are 0): four threads count for each
    const int gi = tid >> 2, part = tid & 3;
    int above = 0;
#pragma unroll
    for (int j = 0; j < kProbGroups / 4; ++j) {
      const int o = part + 4 * j;
      above += s.gmax[o] > best || (s.gmax[o] == best && o < gi);
    }
    above += __shfl_xor_sync(0xffffffffu, above, 1);
    above += __shfl_xor_sync(0xffffffffu, above, 2);
    if (part == 0 && above == K - 1) s.thr = best;
  }
  __syncthreads();
  const u64 thr = max(s.thr, 1ull);
#pragma unroll 4
  for (int i = tid; i < r.n; i += kProbThreads) {
    const u64 v = key(i);
    if (v >= thr) {
      const int at = atomicAdd(&s.n_cand, 1);
      cand[at] = i;
      if (at < kFewCand) s.few[at] = v;
    }
  }
  __syncthreads();
  // ranks among the candidates (keys are unique: the list's order does not matter)
  const int nc = s.n_cand;
  if (nc <= kFewCand) {
    for (int i = tid >> 2; i < ((nc + 7) & ~7); i += kProbThreads / 4) {  // whole warps take part
      const u64 v = i < nc ? s.few[i] : 0;
      int above = 0;
#pragma unroll 4
      for (int j = tid & 3; j < nc; j += 4) above += s.few[j] > v;
      above += __shfl_xor_sync(0xffffffffu, above, 1);
      above += __shfl_xor_sync(0xffffffffu, above, 2);
      if ((tid & 3) == 0 && i < nc && above < K) s.top[above] = v;
    }
  } else {
    for (int i = tid; i < nc; i += kProbThreads) {
      const u64 v = key(cand[i]);
      int above = 0;
      for (int j = 0; j < nc; ++j) above += key(cand[j]) > v;
      if (above < K) s.top[above] = v;
    }
  }
  cl.barrier_wait(std::move(started));
  __syncthreads();
  const int nt = min(nc, K);
  if (tid < nt) {
    const u64 v = s.top[tid];
    cl.map_shared_rank(&s.all[0][0], 0)[rank * kSampleMaxK + tid] = v;
    const int i = 0x7FFFFFFF - (int)(uint32_t)v - r.a;
    sx[sl.off + i] = NAN;  // listed: written by rank 0 (no other entry is NaN)
  }
  if (tid == 0) cl.map_shared_rank(s.n_all, 0)[rank] = nt;
  auto arrived = cl.barrier_arrive();
  __syncthreads();
  {
    float* dst = p.probs + (int64_t)row * p.p_row + r.a;
    const Slice d(dst, r.n);
    if (d.off == sl.off) {
      float4* base = reinterpret_cast<float4*>(dst - d.off);
      for (int i = d.v0 + tid; i < d.v1; i += kProbThreads) {
        const float4 x = reinterpret_cast<const float4*>(sx)[i];
        if (x.x == x.x && x.y == x.y && x.z == x.z && x.w == x.w) {
          __stcs(base + i, make_float4(0.f, 0.f, 0.f, 0.f));
        } else {
          float* e = reinterpret_cast<float*>(base + i);
          if (x.x == x.x) e[0] = 0.f;
          if (x.y == x.y) e[1] = 0.f;
          if (x.z == x.z) e[2] = 0.f;
          if (x.w == x.w) e[3] = 0.f;
        }
      }
      const int e = tid < 4 ? d.off + tid : d.tail + tid - 4;
      if (tid < 8 && (tid < 4 ? e < d.head : e < d.end) && sx[e] == sx[e]) dst[e - d.off] = 0.f;
    } else {
      for (int i = tid; i < r.n; i += kProbThreads)
        if (sx[sl.off + i] == sx[sl.off + i]) dst[i] = 0.f;
    }
  }
  cl.barrier_wait(std::move(arrived));
  if (rank != 0) return;  // nothing of another rank is read from here on
  int total = 0;
  for (int k = 0; k < C; ++k) total += s.n_all[k];
  const int n = min(total, K);
  for (int i = tid; i < C * kSampleMaxK; i += kProbThreads) {
    const int own = i / kSampleMaxK, j = i % kSampleMaxK;
    if (j >= s.n_all[own]) continue;
    const u64 v = s.all[own][j];
    int place = 0;
    for (int k0 = 0; k0 < C; k0 += 4) {  // four lists at a time: how many of each are larger
      int lo[4] = {0, 0, 0, 0};
#pragma unroll
      for (int step = kSampleMaxK; step > 0; step >>= 1)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int k = k0 + q, at = lo[q] + step;
          if (k < C && at <= s.n_all[k] && s.all[k][at - 1] > v) lo[q] = at;
        }
      place += (lo[0] + lo[1]) + (lo[2] + lo[3]);
    }
    s.sorted[place] = v;
  }
  __syncthreads();
  float* out = p.probs + (int64_t)row * p.p_row;
  if (tid < 32) {  // lane l: tokens l and l + 32 in order
    const float m = n > 0 ? key_value(s.sorted[0]) : 0.f;
    float e[2];
    Two cum[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = tid + 32 * h;
      e[h] = j < n ? exp2f((key_value(s.sorted[j]) - m) * p.c) : 0.f;
      cum[h] = two_scan({e[h], 0.f}, tid);
    }
    cum[1] = cum[1] + Two{__shfl_sync(0xffffffffu, cum[0].h, 31), __shfl_sync(0xffffffffu, cum[0].l, 31)};
    const Two tot = {__shfl_sync(0xffffffffu, cum[1].h, 31), __shfl_sync(0xffffffffu, cum[1].l, 31)};
    const Two limit = tot * Two{p.top_p, 0.f};
    bool in[2];
    float kept = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // kept while the mass ahead of it is below top_p
      in[h] = tid + 32 * h < n && (tid + 32 * h == 0 || cum[h] + Two{-e[h], 0.f} < limit);
      kept += in[h] ? e[h] : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) kept += __shfl_xor_sync(0xffffffffu, kept, o);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = tid + 32 * h;
      if (j < n) out[0x7FFFFFFF - (int)(uint32_t)s.sorted[j]] = in[h] ? e[h] / kept : 0.f;
    }
  } else {
    for (int j = n + tid - 32; j < total; j += kProbThreads - 32) out[0x7FFFFFFF - (int)(uint32_t)s.sorted[j]] = 0.f;
  }
}

// ---- draft verification ---------------------------------------------------------
constexpr int kVerThreads = 512;
template <int K>
struct Const {
  static constexpr int value = K;
};

struct VerShared {
  int tok[kTreeMaxNodes], path[kTreeMaxNodes];
  float u[kTreeMaxNodes], px[kTreeMaxNodes], qx[kTreeMaxNodes];
  unsigned long long child[kTreeMaxNodes];  // the nodes below each node
  unsigned long long take;      // the nodes that pass as the first tested child: u q < p
  Two mass[kTreeMaxNodes + 1];  // what k rejections left, in all
  Two inv[kTreeMaxNodes + 1];   // its reciprocal
  Two warp_sum[kVerThreads / 32];
  Two sums[2][16];              // every rank's slice sum, in two buffers used in turn
  Two scan[kVerThreads / 32];
  int first, last;
};

// What k rejections leave of p(j), unnormalised after the last one; a NaN
// probability counts as 0. One rejection (or none: q = 0) is exact. The general
// case is a call: inlined with the rest, the kernel's 200 KB of code, fetched
// once by every CTA, were what a small tree waited for.
__device__ __forceinline__ Two residual1(float p, float q) {
  q = fmaxf(q, 0.f);
  const float h = __fsub_rn(p, q);
  // (p >= q >= 0 where the difference counts: three operations are exact)
  return h > 0.f ? Two{h, __fsub_rn(__fsub_rn(p, h), q)} : Two{0.f, 0.f};
}
static __device__ __noinline__ Two residual_of(float p, float q, const Two* inv, int k) {
  Two r = {fmaxf(p, 0.f), 0.f};
  q = fmaxf(q, 0.f);
#pragma unroll 1
  for (int i = 0; i < k; ++i) {
    if (i > 0) r = r * inv[i];
    const Two d = r + Two{-q, 0.f};
    r = d.h > 0.f ? d : Two{0.f, 0.f};
  }
  return r;
}

// One cluster per sequence. Every CTA walks the tree on the same prefetched
// values, so the walk needs no communication; the vocabulary is read only for
// the masses of rejections that a later sibling needs, and once for the final
// draw: each rank sums its slice (a lane's loads of eight elements in flight),
// the ranks exchange their sums, and the rank, the warp's part and the token
// where the running sum passes u tot are found level by level. Bound by
// latency: launch, three dependent loads, one cluster exchange; 32 rows of
// 151936 p and q (39 MB) stream meanwhile: 14.5 us (40 % of the copy rate), p alone
// 13.6; with 2 and 4 CTAs a sequence instead of 8 22.5 and 19.1. One sequence over
// 32000 tokens is bound by the host's 6.5 us a call.
template <bool SOFT>  // SOFT: draft probabilities are given
__global__ void __launch_bounds__(kVerThreads) verify_kernel(const VerifyParams p) {
  __shared__ VerShared s;
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = kVerThreads / 32;
  using u64 = unsigned long long;
  const int V = p.V;
  int* path_out = p.path + (int64_t)b * p.n;
  const float* pb = p.p + (int64_t)b * p.p_seq;
  const float* qb = SOFT ? p.q + (int64_t)b * p.q_seq : nullptr;
  pdl_wait();
  pdl_trigger();
  // every node's test values at once
  int par = -1, tok = 0;
  float u = 0.f;
  if (tid < p.n) {
    const int64_t at = (int64_t)b * p.n + tid;
    if (tid) par = p.parents[at];
    tok = p.tokens[at];
    u = p.u[at];
  }
  const int cnt = p.counts ? min(max(p.counts[b], 0), p.n) : p.n;
  if (cnt == 0) {  // nothing is chosen (the same in every CTA of the cluster)
    if (rank == 0) {
      if (tid < p.n) path_out[tid] = -1;
      if (tid == 0) p.n_path[b] = 0, p.next[b] = -1;
    }
    return;
  }
  auto started = cl.barrier_arrive();  // shared memory of another CTA: only once that CTA runs
  if (tid < kTreeMaxNodes) s.child[tid] = 0;
  if (tid == 0) s.take = 0, s.path[0] = 0, s.mass[0] = {1.f, 0.f}, s.first = kVerThreads, s.last = -1;
  __syncthreads();
  if (tid < cnt) {
    const bool below = par >= 0 && par < tid, ok = below && tok >= 0 && tok < V;
    s.tok[tid] = tok;
    s.u[tid] = u;
    const float px = ok ? fmaxf(pb[(int64_t)par * p.p_node + tok], 0.f) : 0.f;
    const float qx = SOFT ? ok ? fmaxf(qb[(int64_t)par * p.q_node + tok], 0.f) : 1.f : 1.f;
    s.px[tid] = px;
    s.qx[tid] = qx;
    if (below) atomicOr(&s.child[par], 1ull << tid);
    if (two_prod(u, qx) < Two{px, 0.f}) atomicOr(&s.take, 1ull << tid);
  }
  __syncthreads();
  if constexpr (!SOFT) {  // an earlier sibling with the same token takes its probability
    if (tid > 0 && tid < cnt && par >= 0 && par < tid)
      for (u64 w = s.child[par] & ((1ull << tid) - 1); w; w &= w - 1)
        if (s.tok[__ffsll(w) - 1] == tok) s.px[tid] = 0.f;
    __syncthreads();
  }
  cl.barrier_wait(std::move(started));
  // warp `warp` owns elements w0 .. w1 of the row, 32 chunk of them but for the end
  const int chunk = (V + 32 * C * NW - 1) / (32 * C * NW);
  const int w0 = (int)min((int64_t)V, (int64_t)32 * chunk * (rank * NW + warp)), w1 = min(V, w0 + 32 * chunk);
  int turn = 0, cur = 0, n_path = 1, k = 0;  // k: rejections that count at `cur`
  const float *pr = nullptr, *qr = nullptr;
  u64 gone_bits = 0;     // !SOFT: which of this lane's elements (the first 64) are rejected tokens
  bool gone_far = false;  // and whether one beyond is
  auto rejected = [&](int j) {
#pragma unroll 1
    for (u64 w = s.child[cur]; w; w &= w - 1)
      if (s.tok[__ffsll(w) - 1] == j) return true;
    return false;
  };
  // this lane's part of it, after K (2: any number of) rejections
  auto sum = [&](auto kk) {
    constexpr int K = decltype(kk)::value;
    Two a[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 2
    for (int e = 0; e < chunk; e += 8) {
      float x[8], y[8];
      const int i0 = w0 + 32 * e + lane;
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const bool in = e + v < chunk && i0 + 32 * v < w1;
        x[v] = in ? __ldg(pr + i0 + 32 * v) : 0.f;
        if constexpr (K > 0) y[v] = in ? __ldg(qr + i0 + 32 * v) : 0.f;
      }
      if constexpr (!SOFT) {
        const uint32_t bits = e < 64 ? (uint32_t)(gone_bits >> e) : 0u;
#pragma unroll
        for (int v = 0; v < 8; ++v)
          if ((bits >> v) & 1) x[v] = 0.f;
        if (gone_far && e >= 64)
#pragma unroll 1
          for (int v = 0; v < 8; ++v)
            if (rejected(i0 + 32 * v)) x[v] = 0.f;
      }
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        if constexpr (K == 0) {
          const Two t = two_sum(a[v & 1].h, fmaxf(x[v], 0.f));
          a[v & 1] = {t.h, __fadd_rn(a[v & 1].l, t.l)};
        } else {
          a[v & 1] = two_add(a[v & 1], K == 1 ? residual1(x[v], y[v]) : residual_of(x[v], y[v], s.inv, k));
        }
      }
    }
    return two_add(a[0], a[1]);
  };
  // the sum over the row of `cur` after k rejections; leaves warp_sum and sums
  auto total = [&]() {
    pr = pb + (int64_t)cur * p.p_node;
    if constexpr (SOFT) {
      qr = qb + (int64_t)cur * p.q_node;
    } else {
      gone_bits = 0;
      gone_far = false;
#pragma unroll 1
      for (u64 w = s.child[cur]; w; w &= w - 1) {
        const int off = s.tok[__ffsll(w) - 1] - w0, e = off >> 5;
        if (off >= 0 && e < chunk && (off & 31) == lane) {
          if (e < 64) gone_bits |= 1ull << e;
          else gone_far = true;
        }
      }
    }
    Two d;
    if constexpr (SOFT) d = k == 0 ? sum(Const<0>{}) : k == 1 ? sum(Const<1>{}) : sum(Const<2>{});
    else d = sum(Const<0>{});
    d = two_reduce<32>(d);
    if (lane == 0) s.warp_sum[warp] = d;
    __syncthreads();
    if (warp == 0) {
      d = two_reduce<32>(lane < NW ? s.warp_sum[lane] : Two{0.f, 0.f});
      if (lane < C) cl.map_shared_rank(&s.sums[turn][0], lane)[rank] = d;
    }
    cl.sync();
    const Two t = two_reduce<16>((lane & 15) < C ? s.sums[turn][lane & 15] : Two{0.f, 0.f});
    turn ^= 1;  // the other ranks have left the other buffer before this call's barrier
    return t;
  };
  bool known = true;     // s.mass[k], s.inv[k] are set
  Two left = {1.f, 0.f}; // !SOFT: 1 less the probability of the rejected children
  Two tot;
  int no_mass = V - 1;   // the next token where nothing is left to draw from
  const u64 first_take = s.take;
  for (u64 w = s.child[0];;) {
#pragma unroll 1
    while (w && (!SOFT || known)) {  // as far as it goes without a sum
      const int i = __ffsll(w) - 1;
      w &= w - 1;
      bool take;
      if (k == 0) {
        take = (first_take >> i) & 1;
        if (!SOFT) left = two_sum(1.f, -s.px[i]);
      } else if constexpr (SOFT) {
        take = two_prod(s.u[i], s.qx[i]) * s.mass[k] < residual_of(s.px[i], s.qx[i], s.inv, k);
      } else {
        const float x = s.px[i];
        take = left * Two{s.u[i], 0.f} < Two{x, 0.f};
        left = left + Two{-x, 0.f};
      }
      if (take && i < cnt) {
        if (tid == 0) s.path[n_path] = i;
        cur = i;
        ++n_path;
        k = 0;
        w = s.child[i];
      } else {
        ++k;
        known = false;
      }
    }
    tot = total();
    if constexpr (!SOFT) {
      if (tot.h > 0.f || k == 0) break;
      // The children's tokens are the row's whole support (and fp32 probabilities that sum to less than 1 can all be
      // rejected). The rejection of the last one that has mass does not count: a later sibling with its token is
      // tested against the same mass, and it is what the next token is drawn from.
      int z = -1;
      left = {1.f, 0.f};  // less the tokens ahead of z
#pragma unroll 1
      for (u64 c = s.child[cur]; c; c &= c - 1) {
        const int i = __ffsll(c) - 1;
        if (s.px[i] > 0.f) {
          if (z >= 0) left = left + Two{-s.px[z], 0.f};
          z = i;
        }
      }
      if (z < 0) break;  // a row without mass
      no_mass = s.tok[z];
      int again = -1;
#pragma unroll 1
      for (u64 c = s.child[cur] & ~((2ull << z) - 1); c && again < 0; c &= c - 1) {
        const int i = __ffsll(c) - 1;
        if (s.tok[i] == no_mass && left * Two{s.u[i], 0.f} < Two{s.px[z], 0.f}) again = i;
      }
      if (again < 0) break;
      if (tid == 0) s.path[n_path] = again;
      cur = again;
      ++n_path;
      k = 0;
      w = s.child[cur];
      no_mass = V - 1;
      continue;
    }
    if (tot.h > 0.f || k == 0) {
      if (w == 0) break;  // no child is left: tot is what the next token is drawn from
      if (tid == 0) {
        s.inv[k] = two_recip(tot);
        s.mass[k] = tot;
      }
      __syncthreads();
    } else {
      --k;  // nothing was left: that rejection does not count (the mass of the one before it is known)
    }
    known = true;
  }
  const Two target = tot * Two{s.u[0], 0.f};
  // the rank where the running sum passes the target (every warp finds it from the same sums)
  const Two* sums = s.sums[turn ^ 1];
  Two mine = lane < C ? sums[lane] : Two{0.f, 0.f};
  Two incl = two_scan(mine, lane);
  unsigned over = __ballot_sync(0xffffffffu, mine.h > 0.f && target < incl), some = __ballot_sync(0xffffffffu, mine.h > 0.f);
  int owner = over ? __ffs(over) - 1 : 31 - __clz(some);  // none passes: the last with any mass (u beyond the sum's last bit)
  Two base = incl + Two{-mine.h, -mine.l};
  base = {__shfl_sync(0xffffffffu, base.h, max(owner, 0)), __shfl_sync(0xffffffffu, base.l, max(owner, 0))};
  if (rank == 0 && tid < p.n) path_out[tid] = tid < n_path ? s.path[tid] : -1;
  if (rank == 0 && tid == 0) {
    p.n_path[b] = n_path;
    if (owner < 0) p.next[b] = no_mass;
  }
  if (owner != rank) return;  // no rank reads or writes another's memory from here on
  mine = lane < NW ? s.warp_sum[lane] : Two{0.f, 0.f};
  incl = base + two_scan(mine, lane);
  over = __ballot_sync(0xffffffffu, mine.h > 0.f && target < incl);
  some = __ballot_sync(0xffffffffu, mine.h > 0.f);
  const int ow = over ? __ffs(over) - 1 : max(31 - __clz(some), 0);
  base = incl + Two{-mine.h, -mine.l};
  base = {__shfl_sync(0xffffffffu, base.h, ow), __shfl_sync(0xffffffffu, base.l, ow)};
  // that warp's 32 chunk elements, a run for each thread of the CTA
  const int o0 = (int)min((int64_t)V, (int64_t)32 * chunk * (rank * NW + ow)), o1 = min(V, o0 + 32 * chunk);
  const int run = (o1 - o0 + kVerThreads - 1) / kVerThreads;
  const int l0 = min(o1, o0 + tid * run), l1 = min(o1, l0 + run);
  constexpr int kRun = 4;  // elements kept in registers; longer runs (vocabularies beyond 512 K) are read twice
  u64 holes = 0;           // !SOFT: the rejected tokens of this run
  if constexpr (!SOFT)
    for (u64 w = s.child[cur]; w; w &= w - 1) {
      const int off = s.tok[__ffsll(w) - 1] - l0;
      if (off >= 0 && off < 64) holes |= 1ull << off;
    }
  float xs[kRun], ys[kRun];
#pragma unroll
  for (int e = 0; e < kRun; ++e) {
    xs[e] = l0 + e < l1 ? pr[l0 + e] : 0.f;
    ys[e] = SOFT && k && l0 + e < l1 ? qr[l0 + e] : 0.f;
  }
  auto element = [&](int e, float x, float y) {
    if constexpr (SOFT) return k < 2 ? residual1(x, y) : residual_of(x, y, s.inv, k);
    else return Two{(e < 64 ? (holes >> e) & 1 : rejected(l0 + e)) ? 0.f : fmaxf(x, 0.f), 0.f};
  };
  auto far = [&](int e) { return element(e, pr[l0 + e], SOFT && k ? qr[l0 + e] : 0.f); };
  Two acc = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < kRun; ++e) acc = two_add(acc, element(e, xs[e], ys[e]));  // (past the run: 0)
  for (int e = kRun; e < l1 - l0; ++e) acc = two_add(acc, far(e));
  acc = two_norm(acc);
  const Two upto = two_scan(acc, lane);
  if (lane == 31) s.scan[warp] = upto;
  __syncthreads();
  mine = lane < warp ? s.scan[lane] : Two{0.f, 0.f};
  base = base + two_reduce<32>(mine);
  incl = base + upto;
  // the first thread whose running sum passes the target; none: the last with any mass
  if (acc.h > 0.f) {
    if (target < incl) atomicMin(&s.first, tid);
    atomicMax(&s.last, tid);
  }
  __syncthreads();
  if (tid == (s.first < kVerThreads ? s.first : s.last)) {
    Two at = incl + Two{-acc.h, -acc.l};
    int pick = V - 1;
    bool done = false;
    auto step = [&](int e, Two x) {
      at = at + x;
      if (x.h > 0.f && !done) pick = l0 + e;
      done = done || (x.h > 0.f && target < at);
    };
#pragma unroll
    for (int e = 0; e < kRun; ++e)
      if (l0 + e < l1) step(e, element(e, xs[e], ys[e]));
    for (int e = kRun; e < l1 - l0 && !done; ++e) step(e, far(e));
    p.next[b] = pick;
  } else if (s.last < 0 && tid == 0) {
    p.next[b] = V - 1;
  }
}

// Greedy: a child is kept when it is the target's own choice after its parent.
__global__ void __launch_bounds__(kTreeMaxNodes) verify_greedy_kernel(const VerifyParams p) {
  __shared__ int tok[kTreeMaxNodes], par[kTreeMaxNodes], tgt[kTreeMaxNodes], path[kTreeMaxNodes];
  __shared__ int s_n;
  const int b = blockIdx.x, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
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
// cache row len + k = tree row path[k] for every layer, head, K and V. A thread
// owns 16 bytes of four rows (all loads before the stores): few threads carry
// enough bytes in flight, and the index arithmetic is small beside them. 32 x 9 rows
// of 28 layers, 8 heads x 128 (66 MB): 13.8 us, 71 % of the copy rate, launch included.
constexpr int kCommitRows = 4;
__global__ void __launch_bounds__(256) commit_kernel(const CommitParams p) {
  const int b = blockIdx.y, tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (p.status && *p.status) return;
  const int len = max(p.lens[b], 0);
  const int n = min(min(max(p.n_path[b], 0), p.n), max(p.cache.rows - len, 0));
  if (p.new_lens != p.lens && blockIdx.x == 0 && tid == 0) p.new_lens[b] = len + n;
  const int lch = p.row_bytes == 256 ? 4 : p.row_bytes == 128 ? 3 : 2;  // log2 of a row's 16-byte chunks
  const int c = tid & ((1 << lch) - 1), slots = 256 >> lch;
  const int rows = 2 * p.L * p.Hkv * n, first = blockIdx.x * kCommitRows * slots + (tid >> lch);
  if (first >= rows) return;
  const int esize = p.srow_bytes ? 1 : 2;
  int lh = first / n, k = first - lh * n;  // row first + u slots: (layer, head, K or V) lh, node k of the path
  const int step_lh = slots / n, step_k = slots - step_lh * n;
  uint4 x[kCommitRows];
  uint8_t* dst[kCommitRows];
#pragma unroll
  for (int u = 0; u < kCommitRows; ++u) {
    dst[u] = nullptr;
    if (first + u * slots < rows) {
      const int node = p.path[(int64_t)b * p.path_seq + k];
      if (node >= 0 && node < p.tree.rows) {
        const int kv = lh & 1, l = p.by_heads.div(lh >> 1), h = (lh >> 1) - l * p.Hkv;
        x[u] = *reinterpret_cast<const uint4*>(
            (kv ? p.tree.v : p.tree.k) +
            esize * (b * p.tree.seq + l * p.t_layer + h * p.tree.head + node * p.tree.row) + 16 * c);
        dst[u] = const_cast<uint8_t*>(kv ? p.cache.v : p.cache.k) +
                 esize * (b * p.cache.seq + l * p.c_layer + h * p.cache.head + (len + k) * p.cache.row) + 16 * c;
        if (c == 0 && p.srow_bytes) {
          const uint16_t* ss = (kv ? p.tree.vs : p.tree.ks) + b * p.tree.sseq + l * p.t_slayer + h * p.tree.shead +
                               node * p.tree.srow;
          uint16_t* sd = const_cast<uint16_t*>(kv ? p.cache.vs : p.cache.ks) + b * p.cache.sseq + l * p.c_slayer +
                         h * p.cache.shead + (len + k) * p.cache.srow;
#pragma unroll 1
          for (int e = 0; e < p.srow_bytes / 2; ++e) sd[e] = ss[e];
        }
      }
    }
    lh += step_lh;
    k += step_k;
    if (k >= n) k -= n, ++lh;
  }
#pragma unroll
  for (int u = 0; u < kCommitRows; ++u)
    if (dst[u]) *reinterpret_cast<uint4*>(dst[u]) = x[u];
}
__global__ void __launch_bounds__(256) advance_kernel(const CommitParams p) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (b >= p.B || (p.status && *p.status)) return;
  if (p.next) *p.tok = *p.argmax = *p.next;
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
  const int max_slice = p.top_k ? kProbTopSlice : kProbSlice;
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
    return e == cudaSuccess ? launch_cluster(softmax_rows_kernel, dim3(p.R * C), kSoftThreads, C, smem, st, p, p.pdl) : e;
  }
  // the keys from the threshold on belong to at most top_k of the groups of 4 threads
  const int cand = kSampleMaxK * 4 * ((slice + kProbThreads - 1) / kProbThreads);
  TokenProbsParams q = p;
  q.cap = slice;
  cudaError_t e = lim_k.raise(topk_rows_kernel, (kProbTopSlice + 4 + kSampleMaxK * 4 * kProbTopSlice / kProbThreads) * 4);
  if (e == cudaSuccess && C > 8)
    e = cudaFuncSetAttribute(topk_rows_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e == cudaSuccess
             ? launch_cluster(topk_rows_kernel, dim3(p.R * C), kProbThreads, C, (slice + 4 + cand) * 4, st, q, p.pdl)
             : e;
}

cudaError_t launch_verify_tree(const VerifyParams& p, int n_sm, cudaStream_t st) {
  if (p.targets) {
    return launch_cluster(verify_greedy_kernel, dim3(p.B), kTreeMaxNodes, 1, 0, st, p, p.pdl);
  }
  int C = 1;
  while (C < 8 && p.V / (2 * C) >= 2 * kVerThreads) C *= 2;
  return p.q ? launch_cluster(verify_kernel<true>, dim3(p.B * C), kVerThreads, C, 0, st, p, p.pdl)
             : launch_cluster(verify_kernel<false>, dim3(p.B * C), kVerThreads, C, 0, st, p, p.pdl);
}

cudaError_t launch_commit_tree(const CommitParams& p, cudaStream_t st) {
  const int64_t rows = (int64_t)2 * p.L * p.Hkv * p.n, per = kCommitRows * 256 / (p.row_bytes / 16);
  cudaError_t e = launch_cluster(commit_kernel, dim3((unsigned)((rows + per - 1) / per), p.B), 256, 1, 0, st, p, p.pdl);
  if (e == cudaSuccess && p.new_lens == p.lens)  // every copy has read the lengths before they advance
    e = launch_cluster(advance_kernel, dim3((p.B + 255) / 256), 256, 1, 0, st, p, p.pdl);
  return e;
}

}  // namespace llmq

// ---- C entries -------------------------------------------------------------------
using namespace llmq;

namespace llmq {

// Status word of the bounded waits, one per device.
static __device__ int g_tree_status;

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

bool attention_params(Call& c, const llm_tree_attention_args* a, TreeAttnParams& p) {
  if (!c.need(a->dtype == LLM_BF16 || a->dtype == LLM_F32, LLM_ERR_UNSUPPORTED, "queries are bf16 or f32")) return false;
  if (!c.need(a->n_nodes >= 1 && a->n_nodes <= kTreeMaxNodes, LLM_ERR_UNSUPPORTED, "%sn_nodes %lld (1..64)", "",
              a->n_nodes) ||
      !c.need(a->n_seq >= 1, LLM_ERR_INVALID_ARG, "n_seq is not positive") ||
      !c.need(std::isfinite(a->scale), LLM_ERR_INVALID_ARG, "the scale is not finite") ||
      !check_view(c, a->cache, "cache"))
    return false;
  const llm_kv_view &v = *a->cache, *t = a->tree;
  if (!c.need(a->n_heads > 0 && a->n_heads % v.n_heads == 0, LLM_ERR_INVALID_ARG,
              "n_heads is no multiple of the cache's heads") ||
      !c.need(v.n_seq >= a->n_seq && v.n_layers == 1, LLM_ERR_INVALID_ARG,
              "the cache view holds fewer sequences, or several layers") ||
      !c.need((int64_t)v.n_heads * ((int64_t)a->n_nodes * (a->n_heads / v.n_heads) / 16 + 1) <= 65535,
              LLM_ERR_UNSUPPORTED, "too many heads") ||
      !c.need((int64_t)a->n_nodes * (a->n_heads / v.n_heads) < 65536, LLM_ERR_UNSUPPORTED, "too many heads"))
    return false;
  if (t && (!check_view(c, t, "tree") ||
            !c.need(t->dtype == v.dtype && t->head_dim == v.head_dim && t->n_heads == v.n_heads && t->n_layers == 1 &&
                        t->n_seq >= a->n_seq && t->rows >= a->n_nodes,
                    LLM_ERR_INVALID_ARG, "the tree's rows do not match the cache or the nodes")))
    return false;
  const int64_t hd = v.head_dim, m = a->dtype == LLM_F32 ? 4 : 8;
  const int64_t size[3] = {a->n_seq, a->n_nodes, a->n_heads};
  for (int i = 0; i < 3; ++i)
    if (!c.need(a->q_strides[i] >= 0 && a->out_strides[i] >= 0 && a->q_strides[i] % m == 0 &&
                    a->out_strides[i] % m == 0,
                LLM_ERR_INVALID_ARG, "a stride of q or out is negative or no multiple of 16 bytes"))
      return false;
  if (!c.need(apart(hd, 3, size, a->out_strides), LLM_ERR_INVALID_ARG, "rows of out overlap") ||
      !view_memory(c, a->cache, "cache") || (t && (!view_memory(c, t, "tree") || !c.device("mask", a->mask, 8))) ||
      !c.device("q", a->q, 16) || !c.device("out", a->out, 16) || !c.device("lens", a->lens, 4) ||
      (a->counts && !c.device("counts", a->counts, 4)))
    return false;
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
  // a scale of 0: every score's difference times c below 2^-60, and c times -inf still -inf
  p.c = (float)std::fmin(std::fmax(std::fabs((double)a->scale) * 1.4426950408889634, 1e-30), 3e38);
  p.neg = a->scale < 0.f;
  const cudaError_t es = status_word(c.dev, &p.status);
  if (es != cudaSuccess) c.rc = cuda_bad(es, "status word");
  p.B = a->n_seq;
  p.n = p.nodes = a->n_nodes;
  p.Hkv = v.n_heads;
  p.gq = a->n_heads / v.n_heads;
  p.by_gq = FastDiv(p.gq);
  return c.rc == LLM_OK;
}

}  // namespace llmq

extern "C" {

int llm_tree_attention(const llm_tree_attention_args* a, void* cuda_stream) {
  Call c;
  TreeAttnParams p{};
  if (!c.need(a != nullptr, LLM_ERR_INVALID_ARG, "the arguments are null") || !attention_params(c, a, p)) return c.rc;
  return finish(launch_tree_attn(p, a->cache->head_dim, a->dtype == LLM_F32, a->cache->dtype == LLM_Q8G32, c.n_sm,
                                 static_cast<cudaStream_t>(cuda_stream)),
                "tree attention launch");
}

int llm_debug_expire_waits(int32_t on) {
  g_expire_waits.store(on != 0, std::memory_order_relaxed);
  return LLM_OK;
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
  return st & ST_TIMEOUT ? bad(LLM_ERR_TIMEOUT, "a device-side wait of a tree operator exceeded its limit") : LLM_OK;
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
      !c.need(vocab <= (top_k ? 16 * kProbTopSlice : 16 * kProbSlice), LLM_ERR_UNSUPPORTED, "%svocab %lld is too large", "",
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
  const cudaError_t es = status_word(c.dev, &p.status);
  if (es != cudaSuccess) return cuda_bad(es, "status word");
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
       !c.device("uniforms", a->uniforms, 4) || !c.device("probs", a->probs, 4) ||
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
      !c.need((int64_t)2 * cache->n_layers * cache->n_heads * n_nodes < (1ll << 31) &&
                  (int64_t)cache->n_layers * cache->n_heads * cache->n_heads < (1ll << 32),
              LLM_ERR_UNSUPPORTED,
              "too many layers and heads") ||
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
  // drafts kept in the cache's own rows (of the same layout) would be overwritten while others are read
  const int64_t ahead = (static_cast<const char*>(tree->k) - static_cast<const char*>(cache->k)) / (q8 ? 1 : 2);
  const bool alike = cache->seq_stride == tree->seq_stride && cache->layer_stride == tree->layer_stride &&
                     cache->head_stride == tree->head_stride && cache->row_stride == tree->row_stride;
  if (!c.need(!alike || cache->row_stride == 0 || ahead % cache->row_stride || ahead / cache->row_stride >= cache->rows ||
                  ahead / cache->row_stride <= -(int64_t)tree->rows,
              LLM_ERR_INVALID_ARG, "the tree's rows lie in the cache"))
    return c.rc;
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
  p.by_heads = FastDiv(p.Hkv);
  return finish(launch_commit_tree(p, static_cast<cudaStream_t>(cuda_stream)), "commit launch");
}

}  // extern "C"
