// Tree attention over int8 rows with a scale per 32 values, on the tensor cores
// (the products, roles and references of tree_attn.cuh; what differs:)
// - Converter warps widen the codes, which TMA brings as they are, to bf16: four
//   for the K tiles (exact; into tensor memory, lane = key, as the product's A: a
//   fifth of the tile's shared memory traffic less), eight for the V tiles.
// - S^T of each group of 32 dims has columns of its own; the softmax thread, which
//   is one key, adds them with its key's scales: s = sum_g ks_g S_g.
// - A value is its code times its scale, 8 + 11 bits, in two bf16 parts (16 bits;
//   fp32 queries: three, exact), each a tile of its own. One part took 12 % less
//   time, with 1.42 times the error of an exactly rounded output. A form
//   with the scales in the probabilities, P for every group, took twice the time: the
//   softmax wrote four times as much, and three quarters of the product were not used.
// - The sums of p are the threads' own (16 rows a block), added at the end.
// A non-finite scale of a tree row is left out of the products and added at the
// end for the nodes that see the row.
// Bound: a tile takes ~3,500 cycles; widening V and P V take turns on its one buffer
// (1,500 and 1,000), and the ~250 KB that pass through shared memory (codes in and
// out, V's parts, the MMAs' fetches, P) are 1,900 of them. Giving the buffer back in
// two halves took 10 to 15 % more: all of it competes for the same bandwidth.
// 8 sequences x 13 nodes, 16/8 heads x 128 over 301..4099 rows 36.0 us, 16 % of the
// copy rate (bf16 rows are twice the bytes and wait for memory instead).
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

// Loads that stay where they are written, a tile ahead of their use (the
// compiler moves plain read-only ones down to it).
__device__ __forceinline__ uint2 ld_early2(const uint16_t* at) {
  uint2 w;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(at) : "memory");
  return w;
}
__device__ __forceinline__ uint32_t ld_early(const uint16_t* at) {
  uint32_t w;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w) : "l"(at) : "memory");
  return w;
}
__device__ __forceinline__ uint32_t ld_early_half(const uint16_t* at) {
  uint16_t w;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(w) : "l"(at) : "memory");
  return w;
}
// Four int8 codes times f as NP bf16 parts each: out[k] has part k of the four.
// (In bf16 arithmetic, c a rounded and the exact rest c a - hi + c b with a + b = f,
// it took fewer instructions and 8 % more time.)
template <int NP>
__device__ __forceinline__ void i8x4_scaled(uint32_t w, float f, uint2 (&out)[NP]) {
  w ^= 0x80808080u;
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + i));  // 2^23 + 128 + code
  uint32_t a[NP], b[NP];
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    sub2(x[i], x[i + 1], x[i], x[i + 1], 8388736.f, 8388736.f);
    mul2(x[i], x[i + 1], x[i], x[i + 1], f);
  }
  split_pack<NP>(x[0], x[1], a);
  split_pack<NP>(x[2], x[3], b);
#pragma unroll
  for (int k = 0; k < NP; ++k) out[k] = make_uint2(a[k], b[k]);
}

// A from tensor memory: lane = row, 16 bf16 of K a step in 8 columns
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

template <int HD, bool F32, int G>
struct TreeQ8 {
  static constexpr int NB = 16, N = NB * G, BK = 128, H = HD / 64, NG = HD / 32;
  static constexpr int NQ = F32 ? 3 : 1, NP = F32 ? 3 : 2;
  static constexpr int NS = NQ * NB, NO = NP * NB;   // columns of a group's S and O of a block
  static constexpr int NSA = G * NS, NOA = G * NO;   // of all blocks: one product serves them
  static constexpr int NT = 32 * (4 * G + 12 + 2);
  static constexpr int kRaw = BK * HD, kConv = BK * HD * 2;              // bytes of a K or V tile: codes, bf16
  static constexpr int kP = (NOA + 63) / 64 * BK * 128;                   // atoms of 64 columns
  static constexpr int kQ = NQ * N * HD * 2;
  static constexpr int kOffRow = 1024;
  static constexpr int kSmall = kOffRow + N * (8 + 4 + 16 + 8 + 4);
  static constexpr int PB = NP * kConv + 2 * kP + kQ + kSmall + 1024 + 4 * kRaw <= 232448 ? 2 : 1;  // buffers of P
  static constexpr int kFixed = NP * kConv + PB * kP + kQ + kSmall + 1024;
  static constexpr int fit = (232448 - kFixed) / (2 * kRaw);
  static constexpr int R = fit < 4 ? fit : 4;                             // raw tiles of each of K and V
  static constexpr int kSmem = kFixed + 2 * R * kRaw;
  static constexpr int kAtK = 2 * NG * NSA + NOA;                         // two buffers of S: the scores are a tile ahead
  static constexpr int kUsed = kAtK + HD / 2;                             // and the widened K tile
  static constexpr int kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(R >= 2 && kUsed <= 512 && G * 4096 <= kP, "fits");
  static_assert(tmem_fits(kSmem, kCols), "tensor memory of CTAs on an SM");
};

template <int HD, bool F32, int G>
__global__ void __launch_bounds__(TreeQ8<HD, F32, G>::NT, 1) tree_attn_q8_kernel(const __grid_constant__ TreeAttnTcParams tp) {
  using C = TreeQ8<HD, F32, G>;
  constexpr int N = C::N, NT = C::NT, NB = C::NB, NQ = C::NQ, NP = C::NP, NG = C::NG, BK = C::BK, H = C::H, R = C::R;
  constexpr int NS = C::NS, NO = C::NO, NSA = C::NSA, NOA = C::NOA, PB = C::PB;
  constexpr int kConvWarp = 4 * G, kTmaWarp = 4 * G + 12, kMmaWarp = 4 * G + 13;
  extern __shared__ uint8_t sm_raw[];
  const TreeAttnParams& p = tp.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  uint8_t* sconv = sm;                        // V's parts: [NP][H][128 keys][128 B]
  uint8_t* sraw = sconv + NP * C::kConv;      // [2][R] tiles of codes
  uint8_t* sp = sraw + 2 * R * C::kRaw;       // [PB] P: columns [block][part][row]
  uint8_t* sq = sp + PB * C::kP;                   // [H][G][NQ][NB][128 B]
  uint8_t* small = sq + C::kQ;
  uint64_t* bars = reinterpret_cast<uint64_t*>(small);
  uint64_t *raw_full = bars, *raw_empty = bars + 8, *conv_full = bars + 16, *conv_empty = bars + 18, *s_full = bars + 20,
           *p_full = bars + 22, *o_done = bars + 24, *drain = bars + 26;  // [2][4], then pairs
  unsigned long long* s_bad = reinterpret_cast<unsigned long long*>(small + 272);  // tree rows with a non-finite scale of V
  volatile int* s_abort = reinterpret_cast<volatile int*>(small + 256);
  volatile int* s_stop = reinterpret_cast<volatile int*>(small + 288);  // [G] a wait of the block's has failed
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(small + 264);
  uint64_t* smask = reinterpret_cast<uint64_t*>(small + 512);        // [64]
  uint64_t* srow = reinterpret_cast<uint64_t*>(small + C::kOffRow);  // [N]
  float* sm_m = reinterpret_cast<float*>(srow + N);                  // [N] references, negated
  float* sm_w = sm_m + N;                                            // [4][N]
  float2* sml = reinterpret_cast<float2*>(sm_w + 4 * N);             // [N]
  float* sfac = reinterpret_cast<float*>(sml + N);                   // [N]
  uint8_t* sjoin = sconv + N * HD * 4;                               // the other ranks' parts at the end
  static_assert(N * HD * 4 + kJoin<HD, N> <= NP * C::kConv, "room for them");

  if (tid == 32 * kTmaWarp) {
    s_abort[0] = 0, s_abort[kLimitAt] = p.wait.ns;
    *s_bad = 0;
    s_stop[0] = s_stop[1] = 0;
    for (int i = 0; i < 8; ++i) mbar_init(raw_full + i, 1), mbar_init(raw_empty + i, i < 4 ? 128 : 256);
    mbar_fence_init();
  }
  if (p.part != TreeAttnParams::kSecond) pdl_wait();
  pdl_trigger();
  const int hkv = blockIdx.y % p.Hkv, m0 = (blockIdx.y / p.Hkv) * N, rank = blockIdx.x;
  const int b = p.sorted ? nth_longest(p.lens, p.B, blockIdx.z, lane) : blockIdx.z;
  const int len_b = p.lens[b];
  const TreeBlock block(p, b);
  const int cnt = block.cnt;
  if (m0 >= cnt * p.gq) {  // no rows: the same in every CTA of the cluster
    if (p.part == TreeAttnParams::kSecond) pdl_wait();  // (the kernel ends after the first part's)
    return;
  }
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
        mbar_init(conv_full + i, i ? 256 : 128), mbar_init(conv_empty + i, 1);
        mbar_init(s_full + i, 1), mbar_init(p_full + i, 128 * G + p.wait.missing), mbar_init(o_done + i, 1);
      }
      mbar_init(drain, 1);
      mbar_fence_init();
    }
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                 "r"((uint32_t)C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    const int th = tid, nth = 32 * (4 * G + 12);
    if (p.tree.k)
      for (int i = th; i < kTreeMaxNodes; i += nth) smask[i] = i < cnt ? p.mask[(int64_t)b * p.mask_seq + i] : 0;
#pragma unroll 1
    for (int i = th; i < N * (HD / 8); i += nth) {
      const int r = i / (HD / 8), ch = i % (HD / 8), node = p.by_gq.div(m0 + r), h = hkv * p.gq + m0 + r - node * p.gq;
      const int64_t off = block.q_at(p, node) + (int64_t)h * p.q_head + 8 * ch;
      uint8_t* dst = sq + (((ch / 8) * G + r / NB) * NQ * NB + r % NB) * 128 + 16 * ((ch & 7) ^ (r & 7));
      if constexpr (F32) {
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (node < cnt) {
          const float4 lo = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + off);
          const float4 hi = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + off + 4);
          x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = p.neg ? -x[e] : x[e];
        }
        uint32_t part[4][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_pack<3>(x[2 * e], x[2 * e + 1], part[e]);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4*>(dst + k * NB * 128) = make_uint4(part[0][k], part[1][k], part[2][k], part[3][k]);
      } else {
        uint4 w = node < cnt ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + off)
                             : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t turn = p.neg ? 0x80008000u : 0u;
        w.x ^= turn, w.y ^= turn, w.z ^= turn, w.w ^= turn;
        *reinterpret_cast<uint4*>(dst) = w;
      }
    }
    for (int i = th; i < N; i += nth) sm_m[i] = -kNone;
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;  // S of buffer d, group q at columns (d NG + q) NSA; O behind them
  uint64_t seen = 0;
  if (p.tree.k) {
    const uint64_t a = smask[lane] | smask[lane + 32];
    seen = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(a >> 32)) << 32) |
           __reduce_or_sync(0xffffffffu, (uint32_t)a);
    if (cnt < 64) seen &= (1ull << cnt) - 1;
  }
  auto steps = [&](int t) {  // of 16 keys that hold a visible one (see tree_attn_tc_kernel)
    const int n = t0 + t >= n_pre ? 64 - __clzll((long long)seen) : min(BK, len - (t0 + t) * BK);
    return max(1, (n + 15) / 16);
  };

  int sent = 2 * min(R, n_own);  // by the TMA lane
  if (warp == kTmaWarp) {
    if (lane == 0) {
#pragma unroll 1
      for (int& i = sent; i < 2 * n_own; ++i) {
        const int t = i >> 1, kv = i & 1;
        if (!tc_wait(raw_empty + 4 * kv + t % R, (t / R - 1) & 1, s_abort, p.status)) break;
        request(t, kv);
      }
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t base_i = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);
    constexpr uint32_t idesc_s = base_i | ((uint32_t)(NSA >> 3) << 17);
    constexpr uint32_t idesc_o = base_i | ((uint32_t)(NOA >> 3) << 17) | (1u << 15) | (1u << 16);
    const uint32_t uq = smem_u32(sq), up = smem_u32(sp), uv = smem_u32(sconv);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    bool ok = true;
#pragma unroll 1
    for (int t = -2; t < n_own && ok; ++t) {
      if (t >= 0) {
        const int y = t % PB;
        ok = tc_wait_warp(p_full + y, (t / PB) & 1, s_abort, p.status) && tc_wait_warp(conv_full + 1, t & 1, s_abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const int n_steps = steps(t);
        const uint64_t dp = tc_desc(up + y * C::kP, BK * 128, 1024, 2);
#pragma unroll 1
        for (int k = NP - 1; k >= 0; --k) {  // the small part first: fewer steps cut off at the sum's own size
          // at 64 dims, rows 64.. are whatever lies behind the part: their products are not read
          const uint64_t da = tc_desc(uv + k * C::kConv, BK * 128, 1024, 2);
          if (elect_lane()) {
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
              if (ks < n_steps)
                tc_mma(tm + 2 * NG * NSA, da + ks * (uint64_t)128, dp + ks * (uint64_t)128, idesc_o, (!F32 && t > 0) || k < NP - 1 || ks > 0);
          }
          __syncwarp();
        }
        tc_commit(conv_empty + 1);
        tc_commit(o_done + y);
      }
      if (t + 2 < n_own) {  // S of tile t0 + t + 2, into the buffer just read
        const int x = t & 1;
        ok = tc_wait_warp(conv_full, t & 1, s_abort, p.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int u = 0; u < H; ++u) {
          const uint64_t dq = tc_desc(uq + u * NSA * 128, 16, 1024, 2);
          if (elect_lane()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ts(tm + (x * NG + 2 * u + ks / 2) * NSA, tm + C::kAtK + 32 * u + 8 * ks, dq + 2 * ks, idesc_s, ks & 1);
          }
          __syncwarp();
        }
        tc_commit(conv_empty);
        tc_commit(s_full + x);
      }
    }
  } else if (warp >= kConvWarp) {
    // ---- converters. K: thread = row; V: thread = half a row
    // A slot of codes is given back behind the proxy fence: the copy that fills it
    // next is of the other proxy, and an arrival alone does not order these reads
    // before it (without the fence, codes of four tiles on were met).
    const bool of_v = warp >= kConvWarp + 4;
    const int r = (warp & 3) * 32 + lane;
    const int sel = HD == 128 ? r & 7 : (r >> 1) & 3;
    if (!of_v) {
      const uint32_t tk = tmem + ((uint32_t)(warp & 3) << 21) + C::kAtK;
#pragma unroll 1
      for (int t = 0; t < n_own; ++t) {
        const int slot = t % R;
        tc_wait(raw_full + slot, (t / R) & 1, s_abort, p.status);
        const uint8_t* raw = sraw + slot * C::kRaw + r * HD;
        uint4 w[HD / 16];
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) w[c] = *reinterpret_cast<const uint4*>(raw + 16 * (c ^ sel));
        if (t > 0) tc_wait_together(conv_empty, (t - 1) & 1, s_abort, p.status);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < HD / 16; c += 2) {
          float x[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint2 v = i8x4_to_bf16((&w[c + i / 4].x)[i & 3]);
            x[2 * i] = __uint_as_float(v.x), x[2 * i + 1] = __uint_as_float(v.y);
          }
          tc_st16(tk + 8 * c, x);
        }
        tc_wait_st();
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(raw_empty + slot);
        mbar_arrive(conv_full);
      }
    } else {
      constexpr int NC = HD / 32;  // chunks of 16 codes a thread
      const int half = warp >= kConvWarp + 8;
      uint8_t* conv = sconv + (HD == 128 ? half * BK * 128 : 0) + r * 128;
      // the scales of the thread's codes (of one or two groups) in tile t: two halves a word
      auto scales = [&](int t) -> uint32_t {
        const bool tree = t >= n_pre;
        if (t >= t1 || !(tree ? r < kTreeMaxNodes && ((seen >> (r & 63)) & 1) : t * BK + r < len)) return 0;  // no such row
        const KvRows& rw = tree ? p.tree : p.cache;
        const uint16_t* at = rw.vs + (int64_t)b * rw.sseq + (int64_t)hkv * rw.shead + (int64_t)(tree ? r : t * BK + r) * rw.srow;
        return HD == 128 ? ld_early(at + 2 * half) : ld_early_half(at + half);
      };
      uint32_t next = scales(t0);
#pragma unroll 1
      for (int t = 0; t < n_own; ++t) {
        const int slot = t % R;
        uint32_t own = next;
        next = scales(t0 + t + 1);
        if (t0 + t >= n_pre) {  // the tree's
          const bool b0 = (own & 0x7C00u) == 0x7C00u, b1 = (own & 0x7C000000u) == 0x7C000000u;
          if (b0 || b1) atomicOr(s_bad, 1ull << r);
          own &= (b0 ? 0xFFFF0000u : ~0u) & (b1 ? 0xFFFFu : ~0u);
        }
        const float f0 = __half2float(__ushort_as_half((uint16_t)(own & 0xFFFFu)));
        const float f1 = HD == 128 ? __half2float(__ushort_as_half((uint16_t)(own >> 16))) : f0;
        tc_wait(raw_full + 4 + slot, (t / R) & 1, s_abort, p.status);
        const uint8_t* raw = sraw + (R + slot) * C::kRaw + r * HD;
        uint4 w[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) w[c] = *reinterpret_cast<const uint4*>(raw + 16 * ((half * NC + c) ^ sel));
        if (t > 0) tc_wait(conv_empty + 1, (t - 1) & 1, s_abort, p.status);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int at = 2 * ((half * NC + c) & 3);
          const float f = 2 * c < NC ? f0 : f1;
          uint2 x[4][NP];
          i8x4_scaled<NP>(w[c].x, f, x[0]), i8x4_scaled<NP>(w[c].y, f, x[1]);
          i8x4_scaled<NP>(w[c].z, f, x[2]), i8x4_scaled<NP>(w[c].w, f, x[3]);
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            *reinterpret_cast<uint4*>(conv + k * C::kConv + 16 * (at ^ (r & 7))) = make_uint4(x[0][k].x, x[0][k].y, x[1][k].x, x[1][k].y);
            *reinterpret_cast<uint4*>(conv + k * C::kConv + 16 * ((at + 1) ^ (r & 7))) = make_uint4(x[2][k].x, x[2][k].y, x[3][k].x, x[3][k].y);
          }
        }
        fence_async_smem();
        mbar_arrive(raw_empty + 4 + slot);
        mbar_arrive(conv_full + 1);
      }
    }
  } else {
    // ---- softmax: thread = key
    const int g = warp >> 2, key = (warp & 3) * 32 + lane;
    uint32_t tS = 0;  // S of block g, group 0; of group q: + q NSA
    const uint32_t tO = tmem + ((uint32_t)(warp & 3) << 21) + 2 * NG * NSA + g * NO;
    float* m = sm_m + g * NB;
    if (p.tree.k && key < NB) {
      const int node = p.by_gq.div(m0 + g * NB + key);
      srow[g * NB + key] = node < cnt ? smask[node] & seen : 0;
    }
    group_sync(g);
    auto row_bits = [&]() {  // bit r: row r of the block sees this thread's tree row
      return transpose_bits(key < kTreeMaxNodes && lane < NB
                                ? reinterpret_cast<const uint32_t*>(srow + g * NB + lane)[warp & 1]
                                : 0u,
                            lane);
    };
    auto valid_at = [&](int t) { return t >= n_pre ? key < kTreeMaxNodes && ((seen >> (key & 63)) & 1) : t * BK + key < len; };
    // this key's scales in tile t (0 where there is no such row), two halves a word
    constexpr int NW = NG / 2;
    uint32_t sc[NW];
    auto scales = [&](int t) {
#pragma unroll
      for (int i = 0; i < NW; ++i) sc[i] = 0;
      if (t < t1 && valid_at(t)) {
        const bool tree = t >= n_pre;
        const KvRows& rw = tree ? p.tree : p.cache;
        const int64_t off = (int64_t)b * rw.sseq + (int64_t)hkv * rw.shead + (int64_t)(tree ? key : t * BK + key) * rw.srow;
        if constexpr (NG == 4) {
          const uint2 a = ld_early2(rw.ks + off);
          sc[0] = a.x, sc[1 % NW] = a.y;
        } else {
          sc[0] = ld_early(rw.ks + off);
        }
      }
    };
    auto scale = [&](const uint32_t (&w)[NW], int i) {
      return __half2float(__ushort_as_half((uint16_t)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu)));
    };
    scales(t0);
    float l[NB], acc[F32 ? NB : 1];  // fp32: O of the tiles that have left tensor memory
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      l[j] = 0.f;
      if constexpr (F32) acc[j] = 0.f;
    }
    auto part_of = [&](float (&x)[NB]) {  // this thread's O, its parts added, the small ones first
      float o[NP][NB];
#pragma unroll
      for (int k = 0; k < NP; ++k) tc_ld(o[k], tO + k * NB);
#pragma unroll
      for (int k = 0; k < NP; ++k) tc_wait_ld(o[k]);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        x[j] = o[NP - 1][j];
#pragma unroll
        for (int k = NP - 2; k >= 0; --k) x[j] += o[k][j];
      }
    };
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
      const bool tree = t >= n_pre, whole = !tree && (t + 1) * BK <= len, valid = valid_at(t);
      uint32_t own[NW];
#pragma unroll
      for (int i = 0; i < NW; ++i) own[i] = sc[i];
      scales(t + 1);  // the next tile's are on their way meanwhile
      const int i_own = t - t0, x = i_own & 1, y = i_own % PB;
      const bool failed = !tc_wait_warp(s_full + x, (i_own >> 1) & 1, s_abort, p.status);
      tc_fence_after();
      tS = tmem + ((uint32_t)(warp & 3) << 21) + x * NG * NSA + g * NS;
      auto scores = [&](float (&s)[NB]) {
        constexpr int QS = F32 ? 1 : 2;
#pragma unroll
        for (int q0 = 0; q0 < NG; q0 += QS) {  // as many groups at a time as registers allow
          float v[QS][NQ][NB];
#pragma unroll
          for (int q = 0; q < QS; ++q)
#pragma unroll
            for (int k = 0; k < NQ; ++k) tc_ld(v[q][k], tS + (q0 + q) * NSA + k * NB);
#pragma unroll
          for (int q = 0; q < QS; ++q)
#pragma unroll
            for (int k = 0; k < NQ; ++k) tc_wait_ld(v[q][k]);
#pragma unroll
          for (int q = 0; q < QS; ++q) {
            const float f = scale(own, q0 + q);
#pragma unroll
            for (int j = 0; j < NB; j += 2) {
              float x[2];
#pragma unroll
              for (int i = 0; i < 2; ++i)
                x[i] = NQ == 3 ? v[q][0][j + i] + (v[q][1 % NQ][j + i] + v[q][2 % NQ][j + i]) : v[q][0][j + i];
              if (q0 + q == 0) mul2(s[j], s[j + 1], x[0], x[1], f);
              else fma2(s[j], s[j + 1], x[0], x[1], f, f);
            }
          }
        }
      };
      if (t == t0) {  // the references: the score of the first key that a row sees
        float* first = reinterpret_cast<float*>(sp) + g * 64 * NB;  // [64][NB], where P comes to lie
        if (!failed && warp < 4 * g + (tree ? 2 : 1)) {
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
          if (j >= 0) y = first[j * NB + key];
          m[key] = fabsf(y) < 1e38f ? -y : -kNone;
        }
        // every block's first scores have been read: P may be written
        asm volatile("bar.sync %0, %1;" ::"r"(3), "n"(128 * G) : "memory");
      }
      uint8_t* prow = sp + y * C::kP + key * 128;
      for (;;) {
        if (failed) {  // (see tree_attn_tc_kernel)
          group_any(g, true);
          s_stop[g] = 1;
          group_sync(g);
          goto stopped;
        }
        float s[NB];
        scores(s);
        if (tree) {
          const uint32_t bits = row_bits();
#pragma unroll
          for (int j = 0; j < NB; ++j)
            if (!((bits >> j) & 1)) s[j] = -INFINITY;
        } else if (!whole && !valid) {
#pragma unroll
          for (int j = 0; j < NB; ++j) s[j] = -INFINITY;
        }
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < NB; j += 4) {
          const float4 ref = *reinterpret_cast<const float4*>(m + j);
          float y[4] = {ref.x, ref.y, ref.z, ref.w};
          add2(y[0], y[1], y[0], y[1], s[j], s[j + 1]);
          add2(y[2], y[3], y[2], y[3], s[j + 2], s[j + 3]);
          mul2(y[0], y[1], y[0], y[1], p.c);
          mul2(y[2], y[3], y[2], y[3], p.c);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[j + i] = ex2(y[i]);
          top = fmaxf(top, fmaxf(fmaxf(s[j], s[j + 1]), fmaxf(s[j + 2], s[j + 3])));
        }
        if (group_any(g, top > 1152921504606846976.f)) {  // 2^60 past the references: renew them
          float z[NB];
          scores(z);
          const uint32_t bits = tree ? row_bits() : valid ? ~0u : 0u;
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const bool in = (bits >> j) & 1;
            float y = in ? z[j] : -INFINITY;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
            if (lane == 0) sm_w[(warp & 3) * N + g * NB + j] = y;
          }
          group_sync(g);
          if (s_stop[g]) goto stopped;
          if (key < NB) {
            const float* w = sm_w + g * NB + key;
            const float old = -m[key], now = fmaxf(fmaxf(fmaxf(w[0], w[N]), fmaxf(w[2 * N], w[3 * N])), old);
            m[key] = -now;
            sfac[g * NB + key] = old == now ? 1.f : exp2f((old - now) * p.c);
          }
          group_sync(g);
#pragma unroll
          for (int j = 0; j < NB; ++j) l[j] *= sfac[g * NB + j];
          if (t > t0) {
            tc_wait_together(o_done + (i_own - 1) % PB, ((i_own - 1) / PB) & 1, s_abort, p.status);
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < NO; c0 += 16) {
              float o[16];
              tc_ld(o, tO + c0);
              tc_wait_ld(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] *= sfac[g * NB + j];
              tc_st16(tO + c0, o);
            }
            tc_wait_st();
            if constexpr (F32)
#pragma unroll
              for (int j = 0; j < NB; ++j) acc[j] *= sfac[g * NB + j];
          }
          continue;
        }
#pragma unroll
        for (int j = 0; j < NB; j += 2) add2(l[j], l[j + 1], l[j], l[j + 1], s[j], s[j + 1]);
        if (i_own >= PB) tc_wait(o_done + y, (i_own / PB - 1) & 1, s_abort, p.status);  // the P V of this buffer's last tile
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t part[4][NP];
#pragma unroll
          for (int j = 0; j < 8; j += 2) split_pack<NP>(s[8 * h + j], s[8 * h + j + 1], part[j / 2]);
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            const int chunk = (g * NO + k * NB + 8 * h) / 8;
            *reinterpret_cast<uint4*>(prow + (chunk / 8) * BK * 128 + 16 * ((chunk & 7) ^ (key & 7))) =
                make_uint4(part[0][k], part[1][k], part[2][k], part[3][k]);
          }
        }
        break;
      }
      if constexpr (F32) {
        if (i_own > 0) {  // every tile: its P V, three times the steps of a bf16 tile's, starts anew
          tc_wait_together(o_done + (i_own - 1) % PB, ((i_own - 1) / PB) & 1, s_abort, p.status);
          tc_fence_after();
          float x[NB];
          part_of(x);
#pragma unroll
          for (int j = 0; j < NB; ++j) acc[j] += x[j];
        }
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(p_full + y);
    }
  stopped:
    // ---- O^T and the sums to shared memory, [row][dim]
    if (n_own > 0) tc_wait_together(o_done + (n_own - 1) % PB, ((n_own - 1) / PB) & 1, s_abort, p.status);
    tc_fence_after();
    asm volatile("bar.sync %0, %1;" ::"r"(3), "n"(128 * G) : "memory");  // every block's MMAs have read the tiles
    if (p.S > 1) cluster_arrive();
    float* so = reinterpret_cast<float*>(sm) + g * NB * HD;
    const bool have = n_own > 0 && !__any_sync(0xffffffffu, *s_abort);
    if (key < HD) {  // lanes are dims
      float x[NB];
      if (have) {
        part_of(x);
        if constexpr (F32)
#pragma unroll
          for (int j = 0; j < NB; ++j) x[j] += acc[j];
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) so[j * HD + key] = have ? x[j] : 0.f;
      const unsigned long long bad = *s_bad;
      if (bad && t1 == n_tiles) {  // tree values with non-finite scales, where they are seen
        const int64_t at = (int64_t)b * p.tree.seq + (int64_t)hkv * p.tree.head + key;
        const int64_t at_s = (int64_t)b * p.tree.sseq + (int64_t)hkv * p.tree.shead + key / 32;
#pragma unroll 1
        for (int r = 0; r < NB; ++r)
          for (uint64_t v = srow[g * NB + r] & bad; v; v &= v - 1) {
            const int j = __ffsll(v) - 1;
            const float f = __half2float(__ushort_as_half(p.tree.vs[at_s + j * p.tree.srow]));
            if (!(fabsf(f) <= 65504.f)) so[r * HD + key] += f * (float)reinterpret_cast<const int8_t*>(p.tree.v)[at + j * p.tree.row];
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
  if (warp >= kConvWarp && p.S > 1) cluster_arrive();
  join_splits<HD, F32, N, NT>(p, reinterpret_cast<float*>(sm), sml, sjoin, rank, block.seq, hkv, m0, min(N, cnt * p.gq - m0));
  if (warp >= kTmaWarp && *s_abort) {  // (see tree_attn_tc_kernel)
    const unsigned long long s0 = globaltimer();
    if (warp == kTmaWarp && lane == 0)
#pragma unroll 1
      for (int j = max(0, sent - 2 * R); j < sent; ++j)
        while (!mbar_try_wait(raw_full + 4 * (j & 1) + (j >> 1) % R, ((j >> 1) / R) & 1) &&
               globaltimer() - s0 < kWaitLimitNs) {
        }
    __syncwarp();
    if (warp == kMmaWarp) {
      tc_commit(drain);
      while (!mbar_try_wait(drain, 0) && globaltimer() - s0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  }
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
  const int m_tiles = (p.nodes * p.gq + C::N - 1) / C::N;
  const int64_t clusters = busy_clusters(p, m_tiles);
  const int tiles = (p.cache.rows + C::BK - 1) / C::BK + 1;
  static ClusterCount at_once;
  p.S = lone_splits(clusters, tiles, [&](int S) { return at_once.get(kern, S, C::NT, C::kSmem); });
  p.sorted = p.B > 1 && p.B <= 64;
  return launch_cluster(kern, dim3(p.S, p.Hkv * m_tiles, p.B), C::NT, p.S, C::kSmem, st, tp, p.pdl);
}

template <int HD>
cudaError_t launch_tree_q8(const TreeAttnParams& p, bool f32, int n_sm, cudaStream_t st) {
  TreeAttnTcParams tp;
  tp.p = p;
  if (!encode_all<HD, true>(tp)) return cudaErrorNotSupported;
  const int M = p.nodes * p.gq;
  // 16 rows a block; two blocks share the widened tiles where tensor memory holds both
  if (f32)
    return HD == 128 || M <= 16 ? launch_tree_q8_t<HD, true, 1>(tp, n_sm, st)
                                : launch_tree_q8_t<HD, true, HD == 64 ? 2 : 1>(tp, n_sm, st);
  return M <= 16 ? launch_tree_q8_t<HD, false, 1>(tp, n_sm, st) : launch_tree_q8_t<HD, false, 2>(tp, n_sm, st);
}

}  // namespace llmq
