// The second part of the attention behind shared prefixes for few rows: a token's
// (or a small tree's) queries over its sequence's own rows and the tree's.
//
// At most eight query rows of a kv head meet keys that no other block reads, so
// the work is latency: a warp takes 16 keys at a time, its fragments straight
// from global memory in 16-byte loads, and no barrier stands between a load and
// the products.
//   S^T[keys][rows] = K Q^T     mma m16n8k16: A = K, a lane has 16-byte pieces of
//                               keys g and g + 8 (g = lane / 4), B = Q, of row g;
//                               which dims make up a step is free, so a piece's
//                               words are the steps' halves
//   P^T -> B                    8 x 8 transposed in registers
//   O^T[dims][rows] = V^T P^T   A = V^T from pieces of keys 2t, 2t + 1, 2t + 8,
//                               2t + 9 (t = lane % 4): pairs of keys by byte permutes
// Int8 rows: the codes are bf16 values as they are, a lane's piece lies in one block of 32
// dims; K's scales multiply the blocks' scores, V's the probabilities, per block.
// P in NP bf16 parts (16 bits for bf16 queries, 24 for fp32 ones, whose Q has
// three parts as well). A row's reference is renewed when a probability passes
// 2^60, so most steps have no reduction over lanes. The warps' results are joined
// in shared memory, then as those of the tree attention are.
//
// (tcgen05 instructions hold 128 rows, a tile's loads, barriers and tensor memory:
// about 7 us a CTA whatever its rows are, and two CTAs on an SM: 256 sequences of 32/4 heads x 64 with 1 to 300
// rows of their own take them 27 us, this kernel 13; DRAM at 28 %, issue slots 38 %, the rest is the loads' latency.)
#pragma once
#include "tree_attn.cuh"

namespace llmq {

template <int HD, bool F32, bool Q8>
struct Own {
  static constexpr int NT = 128, NW = NT / 32, N = 8;
  static constexpr int NQ = F32 ? 3 : 1, NP = F32 ? 3 : 2;
  // CTAs on an SM: warps hide the loads' latency better than loads ahead do (64 sequences x 8 kv heads x 128
  // behind 256 rows 21.3 us with 3, 15.0 with 4; loads a step ahead 21.5, steps by way of shared memory 24.5)
  static constexpr int kBlocks = HD == 64 ? (F32 ? 4 : 6) : F32 ? 2 : Q8 ? 3 : 4;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// bf16 values of four codes: bytes behind 2^23, less 2^23 + 128, hold at most eight bits
__device__ __forceinline__ void codes_bf16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  codes ^= 0x80808080u;
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(__byte_perm(codes, 0x4B000000u, 0x7440 + e));
  add2(x[0], x[1], x[0], x[1], -8388736.f, -8388736.f);
  add2(x[2], x[3], x[2], x[3], -8388736.f, -8388736.f);
  lo = __byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x7632);
  hi = __byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x7632);
}
__device__ __forceinline__ float max_of_keys(float x) {  // over the lanes of a row
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// The z-th of at most 256 sequences, by eighths of the longest cache, the longest first: blocks start in grid order
// (rising lengths, 256 x 4 x 64 and 128 x 8 x 128 of 16 .. 300 rows: 64 and 48 us in the order given, 59 and 39 longest
// first). Every warp finds it by itself.
__device__ __forceinline__ int nearly_longest(const int* lens, int B, int z, int lane) {
  constexpr int K = 8;
  int l[K], top = 0;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    l[k] = lane + 32 * k < B ? max(lens[lane + 32 * k], 0) : -1;
    top = max(top, l[k]);
  }
  const float f = 8.f / ((float)__reduce_max_sync(0xffffffffu, top) + 1.f);
  uint64_t n[2] = {0, 0};  // sequences of each eighth, in 16 bits
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int v = 7 - min((int)((float)l[k] * f), 7);
    if (l[k] >= 0) n[v >> 2] += 1ull << (16 * (v & 3));
    l[k] = l[k] >= 0 ? v : -1;
  }
  uint64_t to[2] = {n[0], n[1]};  // up to and with this lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t x = __shfl_up_sync(0xffffffffu, to[i], o);
      if (lane >= o) to[i] += x;
    }
  auto of = [](const uint64_t (&x)[2], int v) { return (int)((v & 4 ? x[1] : x[0]) >> (16 * (v & 3))) & 0xFFFF; };
  const uint64_t all[2] = {__shfl_sync(0xffffffffu, to[0], 31), __shfl_sync(0xffffffffu, to[1], 31)};
  int v = 0;
  for (; v < 7 && z >= of(all, v); ++v) z -= of(all, v);
  int left = z - (of(to, v) - of(n, v)), found = -1;  // of this lane's in that eighth
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (l[k] == v && left-- == 0) found = lane + 32 * k;
  const unsigned who = __ballot_sync(0xffffffffu, found >= 0);
  return __shfl_sync(0xffffffffu, found, __ffs(who) - 1);
}

template <int HD, bool F32, bool Q8>
__global__ void __launch_bounds__(Own<HD, F32, Q8>::NT, Own<HD, F32, Q8>::kBlocks) own_attn_kernel(const __grid_constant__ TreeAttnParams p) {
  using C = Own<HD, F32, Q8>;
  constexpr int NW = C::NW, N = C::N, NQ = C::NQ, NP = C::NP, NT = C::NT;
  constexpr int NC = HD / 32;  // 16-byte pieces of a row that a lane has
  __shared__ __align__(16) float s_o[NW][N][HD];
  __shared__ float2 s_ml[NW][N];
  __shared__ __align__(16) float so[N * HD];
  __shared__ float2 sml[N];
  __shared__ __align__(16) uint8_t s_in[kJoin<HD, N>];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_trigger();
  const int hkv = blockIdx.y, rank = blockIdx.x;
  const int b = !p.sorted ? blockIdx.z : p.B <= 64 ? nth_longest(p.lens, p.B, blockIdx.z, lane) : nearly_longest(p.lens, p.B, blockIdx.z, lane);
  const TreeBlock block(p, b);
  const int len = min(max(p.lens[b], 0), p.cache.rows), n_pre = (len + 15) / 16, n_all = n_pre + (p.tree.k ? 1 : 0);
  const int cnt = block.cnt, rows = cnt * p.gq, most = p.n * p.gq;
  uint32_t q[NQ][NC][4];  // row g
  {
    const int node = p.by_gq.div(g), h = hkv * p.gq + g - node * p.gq;
    const int64_t off = (int64_t)b * p.q_seq + (int64_t)node * p.q_node + (int64_t)h * p.q_head + 8 * t;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if constexpr (F32) {
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (g < most) {
          const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + off + 32 * i);
          const float4 lo = src[0], hi = src[1];
          x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = p.neg ? -x[e] : x[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t part[NQ];
          split_pack<NQ>(x[2 * e], x[2 * e + 1], part);
#pragma unroll
          for (int k = 0; k < NQ; ++k) q[k][i][e] = part[k];
        }
      } else {
        const uint4 w = g < most ? __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + off + 32 * i)) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t turn = p.neg ? 0x80008000u : 0u;
        q[0][i][0] = w.x ^ turn, q[0][i][1] = w.y ^ turn, q[0][i][2] = w.z ^ turn, q[0][i][3] = w.w ^ turn;
      }
    }
  }
  // what the lane's rows 2t and 2t + 1 see of the tree
  uint64_t sees[2] = {0, 0};
  if (p.tree.k)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (2 * t + e < most) sees[e] = p.mask[(int64_t)b * p.mask_seq + p.by_gq.div(2 * t + e)];

  if (rows == 0) {  // (in every CTA of the cluster)
    pdl_wait();     // the kernel ends after the first part's
    return;
  }
  if (p.S > 1) cluster_arrive();
  const int c0 = (int)((int64_t)n_all * rank / p.S), c1 = (int)((int64_t)n_all * (rank + 1) / p.S);
  float o[HD / 16][4];  // [16 dims]: (dim, row 2t), (dim, row 2t + 1), (next dim, ..)
#pragma unroll
  for (int i = 0; i < HD / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float m[2] = {kNone, kNone}, l[2] = {0.f, 0.f};
  // a step's keys
  constexpr int kSize = Q8 ? 1 : 2, kWords = Q8 ? 2 : 4;  // bytes of a value; words of a lane's eight
  uint32_t kw[2][NC][kWords], vw[4][Q8 ? NC : HD / 64][Q8 ? 1 : 4];
  uint32_t ks[2][Q8 ? HD / 64 : 1], vs[2][Q8 ? HD / 64 : 1];  // scales of keys g and g + 8, pairs of fp16
  auto load = [&](uint32_t (&w)[kWords], const uint8_t* at, bool there) {
    if constexpr (Q8) {
      const uint2 x = there ? __ldcg(reinterpret_cast<const uint2*>(at)) : make_uint2(0u, 0u);
      w[0] = x.x, w[1] = x.y;
    } else {
      const uint4 x = there ? __ldcg(reinterpret_cast<const uint4*>(at)) : make_uint4(0u, 0u, 0u, 0u);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
  };
  auto load_scales = [&](uint32_t (&s)[2][Q8 ? HD / 64 : 1], const KvRows& from, const uint16_t* of, int k0, int n) {
    const int64_t at = (int64_t)b * from.sseq + (int64_t)hkv * from.shead + (int64_t)k0 * from.srow;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < HD / 64; ++i)
        s[e][i] = g + 8 * e < n ? __ldcg(reinterpret_cast<const uint32_t*>(of + at + (g + 8 * e) * from.srow) + i) : 0u;
  };
  auto load_k = [&](int c) {
    const bool tree = c >= n_pre;
    const KvRows& from = tree ? p.tree : p.cache;
    const int k0 = tree ? 0 : 16 * c, n = tree ? cnt : len - k0;
    const uint8_t* at = from.k + ((int64_t)b * from.seq + (int64_t)hkv * from.head + (int64_t)k0 * from.row + 8 * t) * kSize;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < NC; ++i) load(kw[e][i], at + ((g + 8 * e) * from.row + 32 * i) * kSize, g + 8 * e < n);
    if constexpr (Q8) load_scales(ks, from, from.ks, k0, n);
  };
  auto load_v = [&](int c) {
    const bool tree = c >= n_pre;
    const KvRows& from = tree ? p.tree : p.cache;
    const int k0 = tree ? 0 : 16 * c, n = tree ? cnt : len - k0;
    const uint8_t* at = from.v + ((int64_t)b * from.seq + (int64_t)hkv * from.head + (int64_t)k0 * from.row + (Q8 ? 4 : 8) * g) * kSize;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = 2 * t + (e & 1) + 8 * (e >> 1);
      const uint8_t* row = at + key * from.row * kSize;
      if constexpr (Q8) {  // four codes of each block: the 16 dims of a product are of one
#pragma unroll
        for (int i = 0; i < NC; ++i) vw[e][i][0] = key < n ? __ldcg(reinterpret_cast<const uint32_t*>(row) + 8 * i) : 0u;
      } else {
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) load(vw[e][i], row + 128 * i, key < n);
      }
    }
    if constexpr (Q8) load_scales(vs, from, from.vs, k0, n);
  };
#pragma unroll
  for (int e = 0; e < 2; ++e)
    sees[e] = 2 * t + e < rows ? sees[e] & ((1ull << cnt) - 1) : 0;
#pragma unroll 1
  for (int c = c0 + warp; c < c1; c += NW) {
    const bool tree = c >= n_pre;
    const int n = tree ? cnt : len - 16 * c;  // keys of the step
    load_k(c);
    load_v(c);
    auto scale_of = [&](const uint32_t (&s)[2][Q8 ? HD / 64 : 1], int e, int block) {
      return __half2float(__ushort_as_half((uint16_t)(s[e][block / 2] >> (16 * (block & 1)))));
    };
    float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};  // (key g, rows 2t, 2t + 1), (key g + 8, ..)
    if constexpr (Q8) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        uint32_t a[2][4];
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) codes_bf16(kw[e][i][0], a[e][0], a[e][1]), codes_bf16(kw[e][i][1], a[e][2], a[e][3]);
#pragma unroll
        for (int k = NQ - 1; k >= 0; --k) {
          mma_16816(y, a[0][0], a[1][0], a[0][1], a[1][1], q[k][i][0], q[k][i][1]);
          mma_16816(y, a[0][2], a[1][2], a[0][3], a[1][3], q[k][i][2], q[k][i][3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = fmaf(y[e], scale_of(ks, e >> 1, i), s[e]);
      }
    } else {
#pragma unroll
      for (int k = NQ - 1; k >= 0; --k)  // the smallest part first
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          mma_16816(s, kw[0][i][0], kw[1][i][0], kw[0][i][1], kw[1][i][1], q[k][i][0], q[k][i][1]);
          mma_16816(s2, kw[0][i][2], kw[1][i][2], kw[0][i][3], kw[1][i][3], q[k][i][2], q[k][i][3]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = g + 8 * (e >> 1);
      s[e] += s2[e];
      if (key >= n || (tree && !(sees[e & 1] >> key & 1))) s[e] = -INFINITY;
    }
    float x[4];
    bool over = c == c0 + warp;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = ex2((s[e] - m[e & 1]) * p.c);
      over |= x[e] > 1152921504606846976.f;  // 2^60
    }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float top = max_of_keys(fmaxf(s[r], s[r + 2]));
        // (NaN or infinite scores alone: any reference does, the sum says what the row is)
        const unsigned odd = __ballot_sync(0xffffffffu, s[r] != s[r] || s[r + 2] != s[r + 2]) & (0x11111111u << t);
        float now = fmaxf(m[r], top < INFINITY ? top : kNone);
        if (now <= kNone && (odd || top == INFINITY)) now = 0.f;
        const float f = exp2f((m[r] - now) * p.c);
        m[r] = now;
        l[r] *= f;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) o[i][r] *= f, o[i][r + 2] *= f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = ex2((s[e] - m[e & 1]) * p.c);
    }
    l[0] += x[0] + x[2], l[1] += x[1] + x[3];
    uint32_t lo[NP], hi[NP];  // P^T: row g, keys 2t, 2t + 1 (+ 8)
    auto parts = [&](const float (&x)[4]) {
      split_pack<NP>(x[0], x[1], lo);
      split_pack<NP>(x[2], x[3], hi);
#pragma unroll
      for (int k = 0; k < NP; ++k) lo[k] = transposed(lo[k]), hi[k] = transposed(hi[k]);
    };
    // o[i] += V^T P^T of 16 dims, of which a lane has two of its keys' values in a word each
    auto product = [&](int i, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
      const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
      const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
      if constexpr (F32) {  // the products cut off where an add rounds: over many steps sums would come out low
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = NP - 1; k >= 0; --k) mma_16816(y, a0, a1, a2, a3, lo[k], hi[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] += y[e];
      } else {
#pragma unroll
        for (int k = 0; k < NP; ++k) mma_16816(o[i], a0, a1, a2, a3, lo[k], hi[k]);
      }
    };
    if constexpr (Q8) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = s[e] == -INFINITY ? 0.f : x[e] * scale_of(vs, e >> 1, i);  // (a scale may be infinite)
        parts(y);
        uint32_t v[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) codes_bf16(vw[e][i][0], v[e][0], v[e][1]);
        product(2 * i, v[0][0], v[1][0], v[2][0], v[3][0]);
        product(2 * i + 1, v[0][1], v[1][1], v[2][1], v[3][1]);
      }
    } else {
      parts(x);
      // Of the tree, infinities and NaNs have to stay away from the rows that do not see them: zeros in the
      // product, added to the others behind it.
      uint32_t odd = 0;
      auto bad = [](uint32_t v) {  // halves whose exponents are all ones
        return ((v & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((v & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
      };
      if (tree) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < HD / 64; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) odd |= bad(vw[e][i][w]);
        odd = __any_sync(0xffffffffu, odd);
      }
      if (odd) {
#pragma unroll 1
        for (int j = 0; j < cnt; ++j)
#pragma unroll
          for (int i = 0; i < HD / 64; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t mine = j & 1 ? vw[1][i][w] : vw[0][i][w];  // the lane t = j / 2 has it
              const uint32_t v = __shfl_sync(0xffffffffu, mine, (lane & 28) | (j >> 1)), is = bad(v);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((e & 2 ? is >> 16 : is & 0xFFFFu) && (sees[e & 1] >> j & 1))
                  o[4 * i + w][e] += __uint_as_float(e & 2 ? v & 0xFFFF0000u : v << 16);
            }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < HD / 64; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) vw[e][i][w] &= ~bad(vw[e][i][w]);
      }
#pragma unroll
      for (int i = 0; i < HD / 64; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) product(4 * i + w, vw[0][i][w], vw[1][i][w], vw[2][i][w], vw[3][i][w]);
    }
  }
  // ---- the warps' results joined
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
  if (lane < 4) s_ml[warp][2 * t] = make_float2(m[0], l[0]), s_ml[warp][2 * t + 1] = make_float2(m[1], l[1]);
#pragma unroll
  for (int i = 0; i < HD / 16; ++i) {
    const int d = Q8 ? 32 * (i / 2) + 4 * g + 2 * (i & 1) : 64 * (i / 4) + 8 * g + 2 * (i & 3);
#pragma unroll
    for (int r = 0; r < 2; ++r) *reinterpret_cast<float2*>(&s_o[warp][2 * t + r][d]) = make_float2(o[i][r], o[i][r + 2]);
  }
  __syncthreads();
#pragma unroll
  for (int i = tid; i < N * HD / 4; i += NT) {
    const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
    float M = kNone, L = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[w][r].x);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float2 ml = s_ml[w][r];
      const float f = ml.x <= kNone ? 0.f : ex2((ml.x - M) * p.c);
      const float4 y = *reinterpret_cast<const float4*>(&s_o[w][r][d]);
      L = fmaf(ml.y, f, L);
      a.x = fmaf(y.x, f, a.x), a.y = fmaf(y.y, f, a.y), a.z = fmaf(y.z, f, a.z), a.w = fmaf(y.w, f, a.w);
    }
    *reinterpret_cast<float4*>(so + r * HD + d) = a;
    if (d == 0) sml[r] = make_float2(M, L);
  }
  join_splits<HD, F32, N, NT>(p, so, sml, s_in, rank, b, hkv, 0, rows);
}

// Whether the own rows are this kernel's: at most eight query rows, and of bf16 rows of 128 dims a cache of at most
// 384, since the tree attention's tiles stream long ones faster (whole calls, this kernel / the tree attention's: 256
// sequences x 8 kv heads x 128 of 300 rows 104 / 134 us, 32 of 512 rows 23.5 / 21.8, of 1024 34 / 26; 128 x 4 x 64 of
// 2048 rows 41 / 47; 24 x 8 x 128 of 2000 int8 rows 50 / 62).
inline bool own_fits(const TreeAttnParams& p, int hd, bool q8) {
  return p.part == TreeAttnParams::kSecond && p.n * p.gq <= 8 && (hd == 64 || q8 || p.cache.rows <= 384);
}

template <int HD, bool F32, bool Q8>
cudaError_t launch_own(TreeAttnParams p, int n_sm, cudaStream_t st) {
  using C = Own<HD, F32, Q8>;
  // Splits of the keys: until the CTAs fill the SMs' places, while a CTA has 256 rows (32 x 8 x 128 of 2048 rows
  // 92 / 60 / 57 / 59 us for 1, 2, 4, 8; 128 x 4 x 64 of 2048 53 / 41 / 48 / 65).
  const int64_t clusters = (int64_t)p.Hkv * p.B;
  int S = 1;
  while (S < 8 && clusters * S < (int64_t)n_sm * C::kBlocks && p.cache.rows / (2 * S) >= 256) S *= 2;
  p.S = S;
  p.sorted = p.B > 1 && p.B <= 256 && p.cache.rows > 128;
  return launch_cluster(own_attn_kernel<HD, F32, Q8>, dim3(S, p.Hkv, p.B), C::NT, S, 0, st, p, p.pdl);
}

}  // namespace llmq
