// Attention of a tree of drafted tokens over the K/V cache.
//
// A sequence's n nodes (n <= 64) share its cached prefix; node i also sees the
// tree rows whose bits its mask sets. The gq query heads of a kv head and the
// n nodes form M = n gq query rows against the same keys (row r: node r / gq,
// head r % gq), so one pass over K and V serves all of them:
//   o_r = sum_j 2^(c s_rj - m_r) v_j / sum_j 2^(c s_rj - m_r),  s_rj = q_r . k_j,
// with c = scale log2(e) and the running maximum m_r and sum in fp32.
#pragma once
#include <cooperative_groups.h>

#include "attn_mma.cuh"
#include "tree.cuh"

namespace llmq {
namespace cg = cooperative_groups;

// 16-byte asynchronous copy; zeros where !ok (nothing is read then)
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}

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

// x as a sum of bf16 parts: part i is the rounding of what the earlier ones
// left, so two parts carry 16 bits of the mantissa and three all 24.
template <int N>
__device__ __forceinline__ void split_bf16(float x, float (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    part[i] = __bfloat162float(__float2bfloat16_rn(x));
    x -= part[i];
  }
}

// The mma.sync form: a CTA owns MT = 16 WM rows of a (sequence, kv head) and a
// range of key tiles; warp (wm, wk) scores rows 16 wm .. +15 against keys
// KW wk .. of every tile of BK keys. Tiles stream through a ring of cp.async
// stages (three tiles of 32 KB in flight keep HBM busy with two CTAs on an
// SM); every warp keeps its own running softmax state, so a tile costs one CTA
// barrier, and the WK states, then the cluster's S ranges of keys, merge at
// the end. fp32 queries enter as three bf16 parts (24 bits), their
// probabilities too; for bf16 queries, which are exact, the probabilities
// enter as two parts (relative error 2^-17, below the output's own rounding).
// int8 rows are widened to bf16 (exact) once per tile for all warps; a key
// group's scale multiplies its partial scores, a value group's scale the
// probabilities of that group's products.
template <int HD, bool F32, bool KV8, int WM, int WK>
struct TreeAttn {
  static constexpr int BK = HD == 64 ? 128 : 64, KW = BK / WK, NT = 32 * WM * WK, MT = 16 * WM;
  static constexpr int NQ = F32 ? 3 : 1, NP = F32 ? 3 : 2, NG = HD / 32, NST = 3;
  static constexpr int kTile = BK * HD;                               // elements of a K or V tile
  static constexpr int kStage = KV8 ? 2 * kTile + 4 * BK * NG : 4 * kTile;  // bytes
  static constexpr int kWork = KV8 ? 4 * kTile : 0;                   // widened K and V
  static constexpr int kRing = NST * kStage + kWork;
  static constexpr int kMerge = WK * MT * HD * 4;                     // over the ring, after the last tile
  static constexpr int kQ = NQ * MT * HD * 2;
  static constexpr int kOffQ = kRing > kMerge ? kRing : kMerge;
  static constexpr int kOffMl = kOffQ + kQ;                           // [WK][MT] (max, sum)
  static constexpr int kOffW = kOffMl + WK * MT * 8;                  // [16][MT] merge weights
  static constexpr int kOffMask = kOffW + 16 * MT * 4;                // [64] masks
  static constexpr int kOffNf = kOffMask + 8 * kTreeMaxNodes;         // [3][64][HD / 32] non-finite values
  static constexpr int kSmem = kOffNf + 3 * kTreeMaxNodes * NG * 4 + 16;
};

template <int HD, bool F32, bool KV8, int WM, int WK>
__global__ void __launch_bounds__(32 * WM * WK) tree_attn_kernel(const __grid_constant__ TreeAttnParams p) {
  using C = TreeAttn<HD, F32, KV8, WM, WK>;
  constexpr int BK = C::BK, KW = C::KW, NT = C::NT, MT = C::MT, NQ = C::NQ, NP = C::NP, NG = C::NG, NST = C::NST;
  constexpr int CH = HD / 8;  // 16-byte chunks of a bf16 row
  extern __shared__ __align__(128) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wm = warp / WK, wk = warp % WK;
  const int b = blockIdx.z, g = blockIdx.y % p.Hkv, m0 = (blockIdx.y / p.Hkv) * MT, rank = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int cnt = p.counts ? min(max(p.counts[b], 0), p.n) : p.n;
  if (m0 >= cnt * p.gq) return;  // no rows: the same in every CTA of the cluster
  const int len = min(max(p.lens[b], 0), p.cache.rows);
  const int n_pre = (len + BK - 1) / BK, n_tiles = n_pre + (p.tree.k ? 1 : 0);
  const int t0 = (int)((int64_t)n_tiles * rank / p.S), t1 = (int)((int64_t)n_tiles * (rank + 1) / p.S);
  uint16_t* sq = reinterpret_cast<uint16_t*>(sm + C::kOffQ);
  float2* sml = reinterpret_cast<float2*>(sm + C::kOffMl);
  float* sw = reinterpret_cast<float*>(sm + C::kOffW);
  uint64_t* smask = reinterpret_cast<uint64_t*>(sm + C::kOffMask);
  uint32_t* snf = reinterpret_cast<uint32_t*>(sm + C::kOffNf);
  int* s_any = reinterpret_cast<int*>(snf + 3 * kTreeMaxNodes * NG);

  const int64_t cb = (int64_t)b * p.cache.seq + (int64_t)g * p.cache.head;
  const int64_t tb = (int64_t)b * p.tree.seq + (int64_t)g * p.tree.head;
  const int64_t csb = (int64_t)b * p.cache.sseq + (int64_t)g * p.cache.shead;
  const int64_t tsb = (int64_t)b * p.tree.sseq + (int64_t)g * p.tree.shead;

  uint64_t seen = 0;  // tree rows that some node of the sequence sees: no other is read
  if (p.tree.k) {
    for (int i = tid; i < kTreeMaxNodes; i += NT) smask[i] = i < cnt ? p.mask[(int64_t)b * p.mask_seq + i] : 0;
    if (tid == 0) *s_any = 0;
    __syncthreads();
    const uint64_t a = smask[lane] | smask[lane + 32];
    seen = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(a >> 32)) << 32) |
           __reduce_or_sync(0xffffffffu, (uint32_t)a);
    if (cnt < 64) seen &= (1ull << cnt) - 1;
  }

  auto stage = [&](int t) {
    uint8_t* base = sm + (t % NST) * C::kStage;
    const bool tree = t >= n_pre;
    const KvRows& r = tree ? p.tree : p.cache;
    const int row0 = tree ? 0 : t * BK;
    const int64_t off = tree ? tb : cb, soff = tree ? tsb : csb;
    auto ok = [&](int row) { return tree ? row < kTreeMaxNodes && ((seen >> (row & 63)) & 1) : row0 + row < len; };
    if constexpr (KV8) {
      constexpr int C8 = HD / 16;
      for (int i = tid; i < 2 * BK * C8; i += NT) {
        const int kv = i >= BK * C8, j = i - kv * BK * C8, row = j / C8, ch = j % C8;
        const bool in = ok(row);
        const uint8_t* src = (kv ? r.v : r.k) + (in ? off + (int64_t)(row0 + row) * r.row + 16 * ch : 0);
        cp_async16_or_zero(base + kv * C::kTile + row * HD + 16 * (ch ^ (row & (C8 - 1))), src, in);
      }
      uint16_t* sc = reinterpret_cast<uint16_t*>(base + 2 * C::kTile);  // [2][BK][NG]
      for (int i = tid; i < 2 * BK; i += NT) {
        const int kv = i >= BK, row = i - kv * BK;
        uint16_t* dst = sc + i * NG;
        if (ok(row)) cp_async_small<2 * NG>(dst, (kv ? r.vs : r.ks) + soff + (int64_t)(row0 + row) * r.srow);
        else
#pragma unroll
          for (int e = 0; e < NG; ++e) dst[e] = 0;
      }
    } else {
      for (int i = tid; i < 2 * BK * CH; i += NT) {
        const int kv = i >= BK * CH, j = i - kv * BK * CH, row = j / CH, ch = j % CH;
        const bool in = ok(row);
        const uint8_t* src = (kv ? r.v : r.k) + (in ? 2 * (off + (int64_t)(row0 + row) * r.row + 8 * ch) : 0);
        cp_async16_or_zero(base + 2 * (kv * C::kTile + tile_off<HD, HD, true>(row, ch)), src, in);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) {
    if (t0 + i < t1) stage(t0 + i);
    cp_async_commit();
  }
  // the query rows as bf16 parts, in the tiles' permuted chunks
  for (int i = tid; i < MT * CH; i += NT) {
    const int r = i / CH, ch = i % CH, node = (m0 + r) / p.gq, h = g * p.gq + (m0 + r) % p.gq;
    const int64_t off = (int64_t)b * p.q_seq + (int64_t)node * p.q_node + (int64_t)h * p.q_head + 8 * ch;
    const int dst = tile_off<HD, HD, true>(r, ch);
    if constexpr (F32) {
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (node < cnt) {
        const float4 lo = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + off);
        const float4 hi = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + off + 4);
        x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
      }
      float part[8][3];
#pragma unroll
      for (int e = 0; e < 8; ++e) split_bf16<3>(x[e], part[e]);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint4*>(sq + k * MT * HD + dst) =
            make_uint4(pack_bf16x2(part[0][k], part[1][k]), pack_bf16x2(part[2][k], part[3][k]),
                       pack_bf16x2(part[4][k], part[5][k]), pack_bf16x2(part[6][k], part[7][k]));
    } else {
      *reinterpret_cast<uint4*>(sq + dst) =
          node < cnt ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + off)
                     : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  const int r8 = lane & 7, mi = lane >> 3, gr = lane >> 2, tq = lane & 3;
  const int node0 = (m0 + 16 * wm + gr) / p.gq, node1 = (m0 + 16 * wm + gr + 8) / p.gq;
  float o[HD / 8][4], mrun[2] = {-INFINITY, -INFINITY}, lrun[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < HD / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  for (int t = t0; t < t1; ++t) {
    cp_async_wait_group<NST - 2>();
    __syncthreads();  // the tile has landed for every thread, and its predecessor's slot is free
    if (t + NST - 1 < t1) stage(t + NST - 1);
    cp_async_commit();
    const bool tree = t >= n_pre;
    uint8_t* base = sm + (t % NST) * C::kStage;
    uint16_t* kt = reinterpret_cast<uint16_t*>(base);
    uint16_t* vt = kt + C::kTile;
    const uint16_t* sc = reinterpret_cast<const uint16_t*>(base + 2 * C::kTile);
    if constexpr (KV8) {
      constexpr int C8 = HD / 16;
      kt = reinterpret_cast<uint16_t*>(sm + NST * C::kStage);
      vt = kt + C::kTile;
      for (int i = tid; i < 2 * BK * C8; i += NT) {
        const int kv = i >= BK * C8, j = i - kv * BK * C8, row = j / C8, ch = j % C8;
        const uint4 w = *reinterpret_cast<const uint4*>(base + kv * C::kTile + row * HD + 16 * (ch ^ (row & (C8 - 1))));
        const uint2 a = i8x4_to_bf16(w.x), c = i8x4_to_bf16(w.y), d = i8x4_to_bf16(w.z), e = i8x4_to_bf16(w.w);
        *reinterpret_cast<uint4*>(kt + kv * C::kTile + tile_off<HD, HD, true>(row, 2 * ch)) = make_uint4(a.x, a.y, c.x, c.y);
        *reinterpret_cast<uint4*>(kt + kv * C::kTile + tile_off<HD, HD, true>(row, 2 * ch + 1)) =
            make_uint4(d.x, d.y, e.x, e.y);
      }
      __syncthreads();
    } else if (tree) {
      // a value that is not finite must not reach the nodes that do not see
      // it (0 * inf is NaN): it becomes 0 here and is added to the rows that
      // do see it at the end
      for (int i = tid; i < 3 * kTreeMaxNodes * NG; i += NT) snf[i] = 0;
      __syncthreads();
      for (int i = tid; i < kTreeMaxNodes * HD; i += NT) {
        const int row = i / HD, d = i % HD;
        uint16_t* x = vt + tile_off<HD, HD, true>(row, d >> 3) + (d & 7);
        if ((*x & 0x7F80u) == 0x7F80u) {
          const int kind = (*x & 0x7Fu) ? 2 : *x >> 15;
          atomicOr(snf + (kind * kTreeMaxNodes + row) * NG + (d >> 5), 1u << (d & 31));
          *x = 0;
          *s_any = 1;
        }
      }
      __syncthreads();
    }
    const int k0 = KW * wk;
    float s[KW / 8][4];
#pragma unroll
    for (int j = 0; j < KW / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
    const int lim = tree ? kTreeMaxNodes : len - t * BK;  // rows of the tile that exist
    if (k0 < lim) {
      if constexpr (KV8) {
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
          float sg[KW / 8][4];
#pragma unroll
          for (int j = 0; j < KW / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sg[j][e] = 0.f;
#pragma unroll
          for (int ks = 2 * gg; ks < 2 * gg + 2; ++ks) {
            uint32_t qf[NQ][4];
#pragma unroll
            for (int k = 0; k < NQ; ++k)
              ldsm_x4(qf[k], sq + k * MT * HD + tile_off<HD, HD, true>(16 * wm + 8 * (mi & 1) + r8, 2 * ks + (mi >> 1)));
#pragma unroll
            for (int j = 0; j < KW / 8; j += 2) {
              uint32_t kb[4];
              ldsm_x4(kb, kt + tile_off<HD, HD, true>(k0 + 8 * j + 8 * (mi >> 1) + r8, 2 * ks + (mi & 1)));
#pragma unroll
              for (int k = NQ - 1; k >= 0; --k) {
                mma_bf16_16816(sg[j], qf[k], kb[0], kb[1]);
                mma_bf16_16816(sg[j + 1], qf[k], kb[2], kb[3]);
              }
            }
          }
#pragma unroll
          for (int j = 0; j < KW / 8; ++j) {
            const float s0 = __half2float(__ushort_as_half(sc[(k0 + 8 * j + 2 * tq) * NG + gg]));
            const float s1 = __half2float(__ushort_as_half(sc[(k0 + 8 * j + 2 * tq + 1) * NG + gg]));
            s[j][0] = fmaf(sg[j][0], s0, s[j][0]);
            s[j][1] = fmaf(sg[j][1], s1, s[j][1]);
            s[j][2] = fmaf(sg[j][2], s0, s[j][2]);
            s[j][3] = fmaf(sg[j][3], s1, s[j][3]);
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          uint32_t qf[NQ][4];
#pragma unroll
          for (int k = 0; k < NQ; ++k)
            ldsm_x4(qf[k], sq + k * MT * HD + tile_off<HD, HD, true>(16 * wm + 8 * (mi & 1) + r8, 2 * ks + (mi >> 1)));
#pragma unroll
          for (int j = 0; j < KW / 8; j += 2) {
            uint32_t kb[4];
            ldsm_x4(kb, kt + tile_off<HD, HD, true>(k0 + 8 * j + 8 * (mi >> 1) + r8, 2 * ks + (mi & 1)));
#pragma unroll
            for (int k = NQ - 1; k >= 0; --k) {
              mma_bf16_16816(s[j], qf[k], kb[0], kb[1]);
              mma_bf16_16816(s[j + 1], qf[k], kb[2], kb[3]);
            }
          }
        }
      }
      const bool whole = !tree && k0 + KW <= lim;
      const uint64_t v0 = tree ? (node0 < cnt ? smask[node0] : 0) & seen : 0;
      const uint64_t v1 = tree ? (node1 < cnt ? smask[node1] : 0) & seen : 0;
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < KW / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[j][e] * p.c;
          if (!whole) {
            const int key = k0 + 8 * j + 2 * tq + (e & 1);
            const bool in = tree ? key < kTreeMaxNodes && (((e < 2 ? v0 : v1) >> (key & 63)) & 1) : key < lim;
            x = in ? x : -INFINITY;
          }
          s[j][e] = x;
          mx[e >> 1] = fmaxf(mx[e >> 1], x);
        }
      float mnew[2], f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        mnew[h] = fmaxf(mrun[h], mx[h]);
        f[h] = mrun[h] == mnew[h] ? 1.f : exp2f(mrun[h] - mnew[h]);
      }
      if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          o[i][0] *= f[0];
          o[i][1] *= f[0];
          o[i][2] *= f[1];
          o[i][3] *= f[1];
        }
        lrun[0] *= f[0];
        lrun[1] *= f[1];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mrun[h] = mnew[h];
        if (mnew[h] == -INFINITY) mnew[h] = 0.f;  // nothing seen yet: every 2^-inf below is 0
      }
#pragma unroll
      for (int j = 0; j < KW / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[j][e] = exp2f(s[j][e] - mnew[e >> 1]);
          lrun[e >> 1] += s[j][e];
        }
#pragma unroll
      for (int c = 0; c < KW / 16; ++c) {
        const int kr = k0 + 16 * c;
        if constexpr (KV8) {
          const uint16_t* vsc = sc + BK * NG;
#pragma unroll
          for (int gg = 0; gg < NG; ++gg) {
            float pp[8][NP];
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // i: n-tile half (i / 4) and element
              const int key = kr + 8 * (i >> 2) + 2 * tq + (i & 1);
              const float w = __half2float(__ushort_as_half(vsc[key * NG + gg]));
              const float x = s[2 * c + (i >> 2)][i & 3];
              split_bf16<NP>(x == 0.f ? 0.f : x * w, pp[i]);  // a masked row's scale may be anything
            }
            uint32_t pa[NP][4];
#pragma unroll
            for (int k = 0; k < NP; ++k) {
              pa[k][0] = pack_bf16x2(pp[0][k], pp[1][k]);
              pa[k][1] = pack_bf16x2(pp[2][k], pp[3][k]);
              pa[k][2] = pack_bf16x2(pp[4][k], pp[5][k]);
              pa[k][3] = pack_bf16x2(pp[6][k], pp[7][k]);
            }
#pragma unroll
            for (int nt = 4 * gg; nt < 4 * gg + 4; nt += 2) {
              uint32_t vb[4];
              ldsm_x4_t(vb, vt + tile_off<HD, HD, true>(kr + 8 * (mi & 1) + r8, nt + (mi >> 1)));
#pragma unroll
              for (int k = NP - 1; k >= 0; --k) {
                mma_bf16_16816(o[nt], pa[k], vb[0], vb[1]);
                mma_bf16_16816(o[nt + 1], pa[k], vb[2], vb[3]);
              }
            }
          }
        } else {
          float pp[8][NP];
#pragma unroll
          for (int i = 0; i < 8; ++i) split_bf16<NP>(s[2 * c + (i >> 2)][i & 3], pp[i]);
          uint32_t pa[NP][4];
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            pa[k][0] = pack_bf16x2(pp[0][k], pp[1][k]);
            pa[k][1] = pack_bf16x2(pp[2][k], pp[3][k]);
            pa[k][2] = pack_bf16x2(pp[4][k], pp[5][k]);
            pa[k][3] = pack_bf16x2(pp[6][k], pp[7][k]);
          }
#pragma unroll
          for (int nt = 0; nt < HD / 8; nt += 2) {
            uint32_t vb[4];
            ldsm_x4_t(vb, vt + tile_off<HD, HD, true>(kr + 8 * (mi & 1) + r8, nt + (mi >> 1)));
#pragma unroll
            for (int k = NP - 1; k >= 0; --k) {
              mma_bf16_16816(o[nt], pa[k], vb[0], vb[1]);
              mma_bf16_16816(o[nt + 1], pa[k], vb[2], vb[3]);
            }
          }
        }
      }
    }
    if constexpr (KV8) __syncthreads();  // the widened tile has been read
  }
  cp_async_wait_all();
  // non-finite tree values, to the rows that see them (the rank with the tree
  // tile, one warp of the WK that share the rows)
  if (!KV8 && p.tree.k && t0 < t1 && t1 == n_tiles && wk == 0 && *s_any) {
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const int node = h ? node1 : node0;
      uint64_t v = node < cnt ? smask[node] & seen : 0;
      while (v) {
        const int j = __ffsll(v) - 1;
        v &= v - 1;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = 8 * i + 2 * tq + e;
            const float bad[3] = {INFINITY, -INFINITY, NAN};
#pragma unroll
            for (int kind = 0; kind < 3; ++kind)
              if ((snf[(kind * kTreeMaxNodes + j) * NG + (d >> 5)] >> (d & 31)) & 1) {
                if (h) o[i][2 + e] += bad[kind];
                else o[i][e] += bad[kind];
              }
          }
      }
    }
  }
  // ---- the WK warps of each row -> the CTA's state -> the cluster's
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    lrun[h] += __shfl_xor_sync(0xffffffffu, lrun[h], 1);
    lrun[h] += __shfl_xor_sync(0xffffffffu, lrun[h], 2);
  }
  __syncthreads();  // the ring is free
  float* so = reinterpret_cast<float*>(sm);  // [WK][MT][HD]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 16 * wm + gr + 8 * h;
    float* dst = so + (wk * MT + r) * HD + 2 * tq;
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) *reinterpret_cast<float2*>(dst + 8 * i) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
    if (tq == 0) sml[wk * MT + r] = make_float2(mrun[h], lrun[h]);
  }
  __syncthreads();
  for (int r = tid; r < MT; r += NT) {  // weights of the WK states, the CTA's (max, sum) in their place
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) M = fmaxf(M, sml[w * MT + r].x);
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const float2 ml = sml[w * MT + r];
      const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      sw[w * MT + r] = f;
      L += ml.y * f;
    }
    sml[r] = make_float2(M, L);
  }
  __syncthreads();
  for (int i = tid; i < MT * HD / 4; i += NT) {
    const int r = i / (HD / 4);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const float4 x = reinterpret_cast<const float4*>(so + w * MT * HD)[i];
      const float f = sw[w * MT + r];
      // a state without keys has weight 0 and o = 0
      a.x = fmaf(x.x, f, a.x), a.y = fmaf(x.y, f, a.y), a.z = fmaf(x.z, f, a.z), a.w = fmaf(x.w, f, a.w);
    }
    reinterpret_cast<float4*>(so)[i] = a;
  }
  cg::cluster_group cl = cg::this_cluster();
  if (p.S > 1) cl.sync();
  else __syncthreads();
  for (int r = tid; r < MT; r += NT) {
    float M = -INFINITY, L = 0.f;
    for (int k = 0; k < p.S; ++k) M = fmaxf(M, cl.map_shared_rank(sml, k)[r].x);
    for (int k = 0; k < p.S; ++k) {
      const float2 ml = cl.map_shared_rank(sml, k)[r];
      const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
      sw[k * MT + r] = f;
      L += ml.y * f;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;  // nothing seen: 0
    for (int k = 0; k < p.S; ++k) sw[k * MT + r] *= inv;
  }
  __syncthreads();
  const int n4 = MT * HD / 4, i0 = (int)((int64_t)n4 * rank / p.S), i1 = (int)((int64_t)n4 * (rank + 1) / p.S);
  for (int i = i0 + tid; i < i1; i += NT) {
    const int r = i / (HD / 4), node = (m0 + r) / p.gq, h = g * p.gq + (m0 + r) % p.gq;
    if (node >= cnt) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < p.S; ++k) {
      const float4 x = reinterpret_cast<const float4*>(cl.map_shared_rank(so, k))[i];
      const float f = sw[k * MT + r];
      a.x = fmaf(x.x, f, a.x), a.y = fmaf(x.y, f, a.y), a.z = fmaf(x.z, f, a.z), a.w = fmaf(x.w, f, a.w);
    }
    const int64_t off = (int64_t)b * p.o_seq + (int64_t)node * p.o_node + (int64_t)h * p.o_head + 4 * (i % (HD / 4));
    if constexpr (F32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + off) = a;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + off) =
          make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
  if (p.S > 1) cl.sync();  // a CTA's shared memory lives until every rank has read it
}

template <int HD, bool F32, bool KV8, int WM, int WK>
cudaError_t launch_tree_attn_t(TreeAttnParams p, int n_sm, cudaStream_t st) {
  using C = TreeAttn<HD, F32, KV8, WM, WK>;
  const auto kern = tree_attn_kernel<HD, F32, KV8, WM, WK>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(kern, C::kSmem);
  if (e != cudaSuccess) return e;
  const int m_tiles = (p.n * p.gq + C::MT - 1) / C::MT;
  const int64_t clusters = (int64_t)p.B * p.Hkv * m_tiles;
  const int tiles = (p.cache.rows + C::BK - 1) / C::BK + 1;
  int S = 1;
  while (S < 8 && S < tiles && clusters * S < 4 * n_sm) S *= 2;
  p.S = S;
  return launch_cluster(kern, dim3(S, p.Hkv * m_tiles, p.B), C::NT, S, C::kSmem, st, p);
}

template <int HD, bool F32, bool KV8>
cudaError_t launch_tree_attn_m(const TreeAttnParams& p, int n_sm, cudaStream_t st) {
  const int M = p.n * p.gq;
  if (M <= 16) return launch_tree_attn_t<HD, F32, KV8, 1, 4>(p, n_sm, st);
  if (M <= 32) return launch_tree_attn_t<HD, F32, KV8, 2, 4>(p, n_sm, st);
  return launch_tree_attn_t<HD, F32, KV8, 4, 2>(p, n_sm, st);
}

template <int HD>
cudaError_t launch_tree_attn_hd(const TreeAttnParams& p, bool f32, bool q8, int n_sm, cudaStream_t st) {
  if (f32) return q8 ? launch_tree_attn_m<HD, true, true>(p, n_sm, st) : launch_tree_attn_m<HD, true, false>(p, n_sm, st);
  return q8 ? launch_tree_attn_m<HD, false, true>(p, n_sm, st) : launch_tree_attn_m<HD, false, false>(p, n_sm, st);
}

}  // namespace llmq
