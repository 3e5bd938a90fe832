// Tree attention over int8 rows with a scale per 32 values, on the tensor cores
// (the products, roles and references of tree_attn.cuh; what differs:)
// - Eight converter warps widen the codes, which TMA brings as they are, to bf16
//   (exact): four for the K tiles, four for the V tiles.
// - S^T of each group of 32 dims has columns of its own; the softmax thread, which
//   is one key, adds them with its key's scales: s = sum_g ks_g S_g.
// - A value's scale goes to the probabilities, p vs_g, so P has columns for every
//   group; of a 64-dim product's 128 rows, 32 belong to each of the two groups.
//   The sums of p itself are the threads' own (16 rows a block), added at the end.
// Codes are always finite and a row's scale meets only its own key's
// probabilities, so what a node does not see cannot reach it.
// Bound: conversion (a byte of HBM is two of shared memory written and read by the
// MMAs) and the MMAs' fetch of it, 24 x ~64 cycles a tile at 128 dims.
#pragma once
#include "tree_attn.cuh"

namespace llmq {

// Four int8 codes (a word) as two bf16 pairs, exactly: 128 + (c & 127) and
// 128 + (c & 128) are bf16 integers below 512 of the same step, and their
// difference is c.
__device__ __forceinline__ uint2 i8x4_to_bf16(uint32_t w) {
  uint32_t r[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t b = __byte_perm(w, 0u, h ? 0x4342 : 0x4140);  // bytes 2h, 2h+1 in the low halves' bytes
    const uint32_t a = (b & 0x007F007Fu) | 0x43004300u, s = (b & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&s));
    r[h] = *reinterpret_cast<const uint32_t*>(&d);
  }
  return make_uint2(r[0], r[1]);
}

template <int HD, bool F32, int G>
struct TreeQ8 {
  static constexpr int NB = 16, N = NB * G, BK = 128, H = HD / 64, NG = HD / 32;
  static constexpr int NQ = F32 ? 3 : 1, NP = F32 ? 3 : 2;
  static constexpr int NS = NQ * NB, NO = NP * NB;   // columns of a group's S and O of a block
  static constexpr int NSA = G * NS, NOA = G * NO;   // of all blocks: one product serves them
  static constexpr int NT = 32 * (4 * G + 8 + 2);
  static constexpr int kRaw = BK * HD, kConv = BK * HD * 2;              // bytes of a K or V tile: codes, bf16
  static constexpr int kAtoms = (2 * NOA + 63) / 64;                      // of 64 columns: P of the two groups of 64 dims
  static constexpr int kPUnit = BK * 128 * kAtoms, kP = H * kPUnit;
  static constexpr int kQ = NQ * N * HD * 2;
  static constexpr int kOffRow = 1024;
  static constexpr int kSmall = kOffRow + N * (8 + 4 + 16 + 8 + 4);
  static constexpr int kFixed = 2 * kConv + kP + kQ + kSmall + 1024;
  static constexpr int fit = (232448 - kFixed) / (2 * kRaw);
  static constexpr int R = fit < 4 ? fit : 4;                             // raw tiles of each of K and V
  static constexpr int kSmem = kFixed + 2 * R * kRaw;
  static constexpr int DB = NG * (2 * NSA + NOA) <= 512 ? 2 : 1;         // buffers of S: the scores are a tile ahead
  static constexpr int kUsed = NG * (DB * NSA + NOA);
  static constexpr int kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(R >= 2 && kUsed <= 512 && N * HD * 4 <= 2 * kConv && kMaxSplits * N * 4 <= kP, "fits");
};

template <int HD, bool F32, int G>
__global__ void __launch_bounds__(TreeQ8<HD, F32, G>::NT, 1) tree_attn_q8_kernel(const __grid_constant__ TreeAttnTcParams tp) {
  using C = TreeQ8<HD, F32, G>;
  constexpr int N = C::N, NT = C::NT, NB = C::NB, NQ = C::NQ, NP = C::NP, NG = C::NG, BK = C::BK, H = C::H, R = C::R;
  constexpr int NS = C::NS, NO = C::NO, NSA = C::NSA, NOA = C::NOA, DB = C::DB, kConvWarp = 4 * G, kTmaWarp = 4 * G + 8, kMmaWarp = 4 * G + 9;
  constexpr float kNone = -3e38f;
  extern __shared__ uint8_t sm_raw[];
  const TreeAttnParams& p = tp.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  uint8_t* sconv = sm;                        // K, V: [2][H][128 keys][128 B]
  uint8_t* sraw = sconv + 2 * C::kConv;       // [2][R] tiles of codes
  uint8_t* sp = sraw + 2 * R * C::kRaw;       // [H] P of two groups: columns [group][block][part][row]
  uint8_t* sq = sp + C::kP;                   // [H][G][NQ][NB][128 B]
  uint8_t* small = sq + C::kQ;
  uint64_t* bars = reinterpret_cast<uint64_t*>(small);
  uint64_t *raw_full = bars, *raw_empty = bars + 8, *conv_full = bars + 16, *conv_empty = bars + 18, *s_full = bars + 20,
           *p_full = bars + 22, *o_done = bars + 24, *drain = bars + 26;  // [2][4], then pairs
  volatile int* s_abort = reinterpret_cast<volatile int*>(small + 256);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(small + 264);
  uint64_t* smask = reinterpret_cast<uint64_t*>(small + 512);        // [64]
  uint64_t* srow = reinterpret_cast<uint64_t*>(small + C::kOffRow);  // [N]
  float* sm_m = reinterpret_cast<float*>(srow + N);                  // [N] references, negated
  float* sm_w = sm_m + N;                                            // [4][N]
  float2* sml = reinterpret_cast<float2*>(sm_w + 4 * N);             // [N]
  float* sfac = reinterpret_cast<float*>(sml + N);                   // [N]
  float* sw = reinterpret_cast<float*>(sp);                          // merge weights, when P is done with

  if (tid == 32 * kTmaWarp) {
    *s_abort = 0;
    for (int i = 0; i < 8; ++i) mbar_init(raw_full + i, 1), mbar_init(raw_empty + i, 128);
    mbar_fence_init();
  }
  pdl_wait();
  pdl_trigger();
  const int hkv = blockIdx.y % p.Hkv, m0 = (blockIdx.y / p.Hkv) * N, rank = blockIdx.x;
  const int b = p.sorted ? nth_longest(p.lens, p.B, blockIdx.z, lane) : blockIdx.z;
  const int len_b = p.lens[b], cnt_b = p.counts ? p.counts[b] : p.n;
  const int cnt = min(max(cnt_b, 0), p.n);
  if (m0 >= cnt * p.gq) return;  // no rows: the same in every CTA of the cluster
  const int len = min(max(len_b, 0), p.cache.rows);
  const int n_pre = (len + BK - 1) / BK, n_tiles = n_pre + (p.tree.k ? 1 : 0);
  const int t0 = (int)((int64_t)n_tiles * rank / p.S), t1 = (int)((int64_t)n_tiles * (rank + 1) / p.S), n_own = t1 - t0;
  auto request = [&](int t, int kv) {
    const int slot = t % R;
    const bool tree = t0 + t >= n_pre;
    uint64_t* bar = raw_full + 4 * kv + slot;
    mbar_expect_tx(bar, C::kRaw);
    tma_box(sraw + (kv * R + slot) * C::kRaw, kv ? (tree ? &tp.tv : &tp.cv) : (tree ? &tp.tk : &tp.ck), 0,
            tree ? 0 : (t0 + t) * BK, hkv * (tree ? tp.t_head : tp.c_head), b * (tree ? tp.t_seq : tp.c_seq), bar);
  };
  if (warp == kTmaWarp) {
    if (lane == 0)
#pragma unroll 1
      for (int i = 0; i < 2 * min(R, n_own); ++i) request(i >> 1, i & 1);
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(conv_full + i, 128), mbar_init(conv_empty + i, 1);
        mbar_init(s_full + i, 1);
      }
      mbar_init(p_full, 128 * G), mbar_init(o_done, 1), mbar_init(drain, 1);
      mbar_fence_init();
    }
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                 "r"((uint32_t)C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    const int th = tid, nth = 32 * (4 * G + 8);
    if (p.tree.k)
      for (int i = th; i < kTreeMaxNodes; i += nth) smask[i] = i < cnt ? p.mask[(int64_t)b * p.mask_seq + i] : 0;
#pragma unroll 1
    for (int i = th; i < N * (HD / 8); i += nth) {
      const int r = i / (HD / 8), ch = i % (HD / 8), node = p.by_gq.div(m0 + r), h = hkv * p.gq + m0 + r - node * p.gq;
      const int64_t off = (int64_t)b * p.q_seq + (int64_t)node * p.q_node + (int64_t)h * p.q_head + 8 * ch;
      uint8_t* dst = sq + (((ch / 8) * G + r / NB) * NQ * NB + r % NB) * 128 + 16 * ((ch & 7) ^ (r & 7));
      if constexpr (F32) {
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (node < cnt) {
          const float4 lo = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + off);
          const float4 hi = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + off + 4);
          x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
        }
        uint32_t part[4][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_pack<3>(x[2 * e], x[2 * e + 1], part[e]);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4*>(dst + k * NB * 128) = make_uint4(part[0][k], part[1][k], part[2][k], part[3][k]);
      } else {
        *reinterpret_cast<uint4*>(dst) = node < cnt
                                             ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + off)
                                             : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    for (int i = th; i < N; i += nth) sm_m[i] = -kNone;
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;  // S of buffer d, group q at columns (d NG + q) NSA; O of unit u at DB NG NSA + 2 u NOA
  uint64_t seen = 0;
  if (p.tree.k) {
    const uint64_t a = smask[lane] | smask[lane + 32];
    seen = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(a >> 32)) << 32) |
           __reduce_or_sync(0xffffffffu, (uint32_t)a);
    if (cnt < 64) seen &= (1ull << cnt) - 1;
  }

  if (warp == kTmaWarp) {
    if (lane == 0) {
      int i = 2 * min(R, n_own);
#pragma unroll 1
      for (; i < 2 * n_own; ++i) {
        const int t = i >> 1, kv = i & 1;
        if (!tc_wait(raw_empty + 4 * kv + t % R, (t / R - 1) & 1, s_abort, p.status)) break;
        request(t, kv);
      }
      if (*s_abort)  // leave no copy in flight
#pragma unroll 1
        for (int j = max(0, i - 2 * R); j < i; ++j) {
          const unsigned long long s0 = globaltimer();
          while (!mbar_try_wait(raw_full + 4 * (j & 1) + (j >> 1) % R, ((j >> 1) / R) & 1) &&
                 globaltimer() - s0 < kWaitLimitNs) {
          }
        }
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t base_i = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);
    constexpr uint32_t idesc_s = base_i | ((uint32_t)(NSA >> 3) << 17);
    constexpr uint32_t idesc_o = base_i | ((uint32_t)(2 * NOA >> 3) << 17) | (1u << 15) | (1u << 16);
    const uint32_t uq = smem_u32(sq), up = smem_u32(sp), uk = smem_u32(sconv), uv = uk + C::kConv;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    bool ok = true;
#pragma unroll 1
    for (int t = -DB; t < n_own && ok; ++t) {
      if (t >= 0) {
        ok = tc_wait_warp(p_full, t & 1, s_abort, p.status) && tc_wait_warp(conv_full + 1, t & 1, s_abort, p.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int u = 0; u < H; ++u) {
          // rows 64.. are whatever lies behind the unit: their products are not read
          const uint64_t da = tc_desc(uv + u * BK * 128, BK * 128, 1024, 2);
          const uint64_t dp = tc_desc(up + u * C::kPUnit, BK * 128, 1024, 2);
          if (elect_lane()) {
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
              tc_mma(tm + DB * NG * NSA + u * 2 * NOA, da + ks * (uint64_t)128, dp + ks * (uint64_t)128, idesc_o,
                     t > 0 || ks > 0);
          }
          __syncwarp();
        }
        tc_commit(conv_empty + 1);
        tc_commit(o_done);
      }
      if (t + DB < n_own) {  // S of tile t0 + t + DB, into the buffer just read
        const int x = DB == 2 ? t & 1 : 0;
        ok = tc_wait_warp(conv_full, (t + DB) & 1, s_abort, p.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int u = 0; u < H; ++u) {
          const uint64_t da = tc_desc(uk + u * BK * 128, 16, 1024, 2);
          const uint64_t dq = tc_desc(uq + u * NSA * 128, 16, 1024, 2);
          if (elect_lane()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma(tm + (x * NG + 2 * u + ks / 2) * NSA, da + 2 * ks, dq + 2 * ks, idesc_s, ks & 1);
          }
          __syncwarp();
        }
        tc_commit(conv_empty);
        tc_commit(s_full + x);
      }
    }
    if (!ok) {  // no MMA may outlive its operands
      tc_commit(drain);
      const unsigned long long s0 = globaltimer();
      while (!mbar_try_wait(drain, 0) && globaltimer() - s0 < kWaitLimitNs) {
      }
    }
  } else if (warp >= kConvWarp) {
    // ---- converters: thread = row of the K (kv 0) or V tile
    const int kv = (warp - kConvWarp) >> 2, r = (warp & 3) * 32 + lane;
    uint8_t* conv = sconv + kv * C::kConv + r * 128;
    const int sel = HD == 128 ? r & 7 : (r >> 1) & 3;
#pragma unroll 1
    for (int t = 0; t < n_own; ++t) {
      const int slot = t % R;
      tc_wait(raw_full + 4 * kv + slot, (t / R) & 1, s_abort, p.status);
      const uint8_t* raw = sraw + (kv * R + slot) * C::kRaw + r * HD;
      uint4 w[HD / 16];
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) w[c] = *reinterpret_cast<const uint4*>(raw + 16 * (c ^ sel));
      mbar_arrive(raw_empty + 4 * kv + slot);
      if (t > 0) tc_wait(conv_empty + kv, (t - 1) & 1, s_abort, p.status);
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) {
        const uint2 a = i8x4_to_bf16(w[c].x), d = i8x4_to_bf16(w[c].y), e = i8x4_to_bf16(w[c].z), f = i8x4_to_bf16(w[c].w);
        uint8_t* dst = conv + (c / 4) * BK * 128;
        *reinterpret_cast<uint4*>(dst + 16 * ((2 * (c & 3)) ^ (r & 7))) = make_uint4(a.x, a.y, d.x, d.y);
        *reinterpret_cast<uint4*>(dst + 16 * ((2 * (c & 3) + 1) ^ (r & 7))) = make_uint4(e.x, e.y, f.x, f.y);
      }
      fence_async_smem();
      mbar_arrive(conv_full + kv);
    }
  } else {
    // ---- softmax: thread = key
    const int g = warp >> 2, key = (warp & 3) * 32 + lane;
    uint32_t tS = tmem + ((uint32_t)(warp & 3) << 21) + g * NS;  // of group q: + q NSA
    const uint32_t tO = tmem + ((uint32_t)(warp & 3) << 21) + DB * NG * NSA + g * NO;  // of group q: + q NOA
    float* m = sm_m + g * NB;
    const float masked = p.c < 0.f ? INFINITY : -INFINITY;
    if (p.tree.k && key < NB) {
      const int node = p.by_gq.div(m0 + g * NB + key);
      srow[g * NB + key] = node < cnt ? smask[node] & seen : 0;
    }
    group_sync(g);
    const uint32_t* vis = reinterpret_cast<const uint32_t*>(srow + g * NB) + (warp & 1);
    auto sees = [&](int r) { return key < kTreeMaxNodes && ((vis[2 * r] >> lane) & 1); };
    auto valid_at = [&](int t) { return t >= n_pre ? key < kTreeMaxNodes && ((seen >> (key & 63)) & 1) : t * BK + key < len; };
    // this key's scales in tile t (0 where there is no such row): K's, then V's, two halves a word
    constexpr int NW = NG / 2;
    uint32_t sc[2 * NW];
    auto scales = [&](int t) {
#pragma unroll
      for (int i = 0; i < 2 * NW; ++i) sc[i] = 0;
      if (t < t1 && valid_at(t)) {
        const bool tree = t >= n_pre;
        const KvRows& rw = tree ? p.tree : p.cache;
        const int64_t off = (int64_t)b * rw.sseq + (int64_t)hkv * rw.shead + (int64_t)(tree ? key : t * BK + key) * rw.srow;
        if constexpr (NG == 4) {
          const uint2 a = __ldg(reinterpret_cast<const uint2*>(rw.ks + off)), d = __ldg(reinterpret_cast<const uint2*>(rw.vs + off));
          sc[0] = a.x, sc[1] = a.y, sc[2] = d.x, sc[3] = d.y;
        } else {
          sc[0] = __ldg(reinterpret_cast<const uint32_t*>(rw.ks + off));
          sc[1] = __ldg(reinterpret_cast<const uint32_t*>(rw.vs + off));
        }
      }
    };
    auto scale = [&](const uint32_t (&w)[2 * NW], int i) {
      return __half2float(__ushort_as_half((uint16_t)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu)));
    };
    scales(t0);
    float l[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) l[j] = 0.f;
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
      const bool tree = t >= n_pre, whole = !tree && (t + 1) * BK <= len, valid = valid_at(t);
      uint32_t own[2 * NW];
#pragma unroll
      for (int i = 0; i < 2 * NW; ++i) own[i] = sc[i];
      scales(t + 1);  // the next tile's are on their way meanwhile
      const int x = DB == 2 ? (t - t0) & 1 : 0;
      tc_wait(s_full + x, (DB == 2 ? (t - t0) >> 1 : t - t0) & 1, s_abort, p.status);
      tc_fence_after();
      if constexpr (DB == 2) tS = tmem + ((uint32_t)(warp & 3) << 21) + x * NG * NSA + g * NS;
      auto scores = [&](float (&s)[NB]) {
#pragma unroll
        for (int q = 0; q < NG; ++q) {
          float v[NQ][NB];
#pragma unroll
          for (int k = 0; k < NQ; ++k) tc_ld(v[k], tS + q * NSA + k * NB);
#pragma unroll
          for (int k = 0; k < NQ; ++k) tc_wait_ld(v[k]);
          const float f = scale(own, q);
#pragma unroll
          for (int j = 0; j < NB; j += 2) {
            float x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) x[i] = NQ == 3 ? v[0][j + i] + (v[1 % NQ][j + i] + v[2 % NQ][j + i]) : v[0][j + i];
            if (q == 0) mul2(s[j], s[j + 1], x[0], x[1], f);
            else fma2(s[j], s[j + 1], x[0], x[1], f, f);
          }
        }
      };
      if (t == t0) {  // the references: the score of the first key that a row sees
        float* first = reinterpret_cast<float*>(sp) + g * 64 * NB;  // [64][NB], where P comes to lie
        if (warp < 4 * g + (tree ? 2 : 1)) {
          float s[NB];
          scores(s);
          if (tree || lane == 0)
#pragma unroll
            for (int j = 0; j < NB; j += 4)
              *reinterpret_cast<float4*>(first + key * NB + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
        }
        group_sync(g);
        float y = INFINITY;
        if (key < NB) {
          const int j = tree ? __ffsll(srow[g * NB + key]) - 1 : 0;
          if (j >= 0) y = first[j * NB + key] * p.c;
          m[key] = fabsf(y) < 1e38f ? -y : -kNone;
        }
        // every block's first scores have been read: P may be written
        asm volatile("bar.sync %0, %1;" ::"r"(3), "n"(128 * G) : "memory");
      }
      uint8_t* prow = sp + key * 128;
      for (;;) {
        float s[NB];
        scores(s);
        if (tree) {
#pragma unroll
          for (int j = 0; j < NB; ++j)
            if (!sees(j)) s[j] = masked;
        } else if (!whole && !valid) {
#pragma unroll
          for (int j = 0; j < NB; ++j) s[j] = masked;
        }
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < NB; j += 4) {
          const float4 ref = *reinterpret_cast<const float4*>(m + j);
          float y[4] = {ref.x, ref.y, ref.z, ref.w};
          fma2(y[0], y[1], s[j], s[j + 1], p.c, p.c);
          fma2(y[2], y[3], s[j + 2], s[j + 3], p.c, p.c);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[j + i] = ex2(y[i]);
          top = fmaxf(top, fmaxf(fmaxf(s[j], s[j + 1]), fmaxf(s[j + 2], s[j + 3])));
        }
        if (group_any(g, top > 1152921504606846976.f)) {  // 2^60 past the references: renew them
          float z[NB];
          scores(z);
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const bool in = tree ? sees(j) : valid;
            float y = in ? z[j] * p.c : -INFINITY;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
            if (lane == 0) sm_w[(warp & 3) * N + g * NB + j] = y;
          }
          group_sync(g);
          if (key < NB) {
            const float* w = sm_w + g * NB + key;
            const float old = -m[key], now = fmaxf(fmaxf(fmaxf(w[0], w[N]), fmaxf(w[2 * N], w[3 * N])), old);
            m[key] = -now;
            sfac[g * NB + key] = old == now ? 1.f : exp2f(old - now);
          }
          group_sync(g);
#pragma unroll
          for (int j = 0; j < NB; ++j) l[j] *= sfac[g * NB + j];
          if (t > t0) {
            tc_wait(o_done, (t - t0 - 1) & 1, s_abort, p.status);
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < NO * NG; c0 += 16) {
              const uint32_t at = tO + (c0 / NO) * NOA + c0 % NO;
              float o[16];
              tc_ld(o, at);
              tc_wait_ld(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] *= sfac[g * NB + j];
              tc_st16(at, o);
            }
            tc_wait_st();
          }
          continue;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) l[j] += s[j];
        if (t > t0) tc_wait(o_done, (t - t0 - 1) & 1, s_abort, p.status);  // the last P V has read P
        // a masked key's scale may be anything: its probabilities stay 0
        float f[NG];
        bool odd = false;
#pragma unroll
        for (int q = 0; q < NG; ++q) {
          f[q] = scale(own, NG + q);
          odd |= !(fabsf(f[q]) <= 65504.f);
        }
        const bool any_odd = __any_sync(0xffffffffu, odd);
#pragma unroll
        for (int q = 0; q < NG; ++q) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t part[4][NP];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              float a, d;
              mul2(a, d, s[8 * h + j], s[8 * h + j + 1], f[q]);
              if (any_odd) a = s[8 * h + j] == 0.f ? 0.f : a, d = s[8 * h + j + 1] == 0.f ? 0.f : d;
              split_pack<NP>(a, d, part[j / 2]);
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
              const int chunk = ((q & 1) * NOA + g * NO + k * NB + 8 * h) / 8;
              *reinterpret_cast<uint4*>(prow + (q >> 1) * C::kPUnit + (chunk / 8) * BK * 128 + 16 * ((chunk & 7) ^ (key & 7))) =
                  make_uint4(part[0][k], part[1][k], part[2][k], part[3][k]);
            }
          }
        }
        break;
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(p_full);
    }
    // ---- O^T and the sums to shared memory, [row][dim]
    if (n_own > 0) tc_wait(o_done, (n_own - 1) & 1, s_abort, p.status);
    tc_fence_after();
    asm volatile("bar.sync %0, %1;" ::"r"(3), "n"(128 * G) : "memory");  // every block's MMAs have read the tiles
    float* so = reinterpret_cast<float*>(sm) + g * NB * HD;
    if ((warp & 3) < 2) {  // lanes 0..63: dims; the two warps' columns are their own group's
#pragma unroll 1
      for (int u = 0; u < H; ++u) {
        float o[NP][NB];
        if (n_own > 0) {
#pragma unroll
          for (int k = 0; k < NP; ++k) tc_ld(o[k], tO + (2 * u + (warp & 1)) * NOA + k * NB);
#pragma unroll
          for (int k = 0; k < NP; ++k) tc_wait_ld(o[k]);
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          float x = 0.f;
          if (n_own > 0)
#pragma unroll
            for (int k = NP - 1; k >= 0; --k) x += o[k][j];
          so[j * HD + 64 * u + key] = x;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      float x = l[j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) sm_w[(warp & 3) * N + g * NB + j] = x;
    }
    group_sync(g);
    if (key < NB) {
      const float* w = sm_w + g * NB + key;
      sml[g * NB + key] = make_float2(-m[key], (w[0] + w[N]) + (w[2 * N] + w[3 * N]));
    }
    tc_fence_before();
  }
  __syncwarp();
  join_splits<HD, F32, N, NT>(p, reinterpret_cast<float*>(sm), sml, sw, rank, b, hkv, m0, min(N, cnt * p.gq - m0));
  if (warp == kMmaWarp) {  // (freed last: see tree_attn_tc_kernel)
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)C::kCols));
  }
}

template <int HD, bool F32, int G>
cudaError_t launch_tree_q8_t(TreeAttnTcParams& tp, int n_sm, cudaStream_t st) {
  using C = TreeQ8<HD, F32, G>;
  const auto kern = tree_attn_q8_kernel<HD, F32, G>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(kern, C::kSmem, true);
  if (e != cudaSuccess) return e;
  TreeAttnParams& p = tp.p;
  const int m_tiles = (p.n * p.gq + C::N - 1) / C::N;
  const int64_t clusters = (int64_t)p.B * p.Hkv * m_tiles;
  const int tiles = (p.cache.rows + C::BK - 1) / C::BK + 1;
  int S = 1;
  while (S < kMaxSplits && S < tiles && clusters * S < n_sm) S *= 2;
  p.S = S;
  p.sorted = p.B > 1 && p.B <= 64;
  return launch_cluster(kern, dim3(S, p.Hkv * m_tiles, p.B), C::NT, S, C::kSmem, st, tp, p.pdl);
}

template <int HD>
cudaError_t launch_tree_q8(const TreeAttnParams& p, bool f32, int n_sm, cudaStream_t st) {
  TreeAttnTcParams tp;
  tp.p = p;
  if (!encode_all<HD, true>(tp)) return cudaErrorNotSupported;
  const int M = p.n * p.gq;
  // 16 rows a block; two blocks share the widened tiles where tensor memory holds both
  if (f32)
    return HD == 128 || M <= 16 ? launch_tree_q8_t<HD, true, 1>(tp, n_sm, st)
                                : launch_tree_q8_t<HD, true, HD == 64 ? 2 : 1>(tp, n_sm, st);
  return M <= 16 ? launch_tree_q8_t<HD, false, 1>(tp, n_sm, st) : launch_tree_q8_t<HD, false, 2>(tp, n_sm, st);
}

}  // namespace llmq
