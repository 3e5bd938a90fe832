// Attention of many query rows over bf16 K/V rows that they all see: the first part
// of prefix_attention where a group has more rows than the tree attention's
// kernels take at once (see TreeAttnParams::Part).
//
// Rows (a group's sequences x nodes x query heads of a kv head) are the long side here,
// so the products run untransposed, a tile of 128 rows against 128 keys:
//   S [128 rows x 128 keys] = Q K_tile^T        (both K-major, from shared memory)
//   O [128 rows x dims]    += P V_tile          (P from tensor memory, V as TMA lays it down)
// A CTA takes two tiles of rows over the same keys, 64 keys (a block) at a time; a tile
// has three blocks of scores in tensor memory at 64 dims, two at 128 (O takes the rest), so that
// scores are made while the block before them becomes probabilities, which come to lie
// over them. A thread is a row: its scores, reference and sum are its own. The
// reference is the first block's maximum and is renewed only when a block's
// probabilities pass 2^60 (bf16 and fp32 keep their precision over that range), so O is
// hardly ever touched between products. Four softmax warps for each tile, one that
// issues Q K and one that issues P V: beside the softmax a wait takes 150 cycles even when it
// is over, and a warp that issued both was the slowest (1,250 cycles a block).
// P is rounded to bf16 (8 bits): the outputs' error is 1.41 times what rounding them
// to bf16 gives. Two parts of it would make half as many matrix operations more.
//
// Work: the (group, kv head, 256 rows, key tile) units in one row are cut into equal
// ranges, one for each CTA, so that every SM has the same number whatever the sizes of the
// groups; the pieces of a row tile (max_parts at most) are joined by the second part.
//
// Measured: 256 sequences of 32/4 heads x 64 behind 16384 rows 49 us of the call's 64 (34.4 GFLOP, 700 TFLOP/s). Bound by
// the softmax warps: about 1,000 cycles for a block of 128 rows x 64 keys (exponentials alone 512 for the two tiles) and 400 between blocks,
// tensor pipe 33 % and issue slots 44 % busy; 16 softmax warps instead of 8 gained nothing.
#pragma once
#include "tree_attn_q8.cuh"

namespace llmq {

constexpr int kWideRows = 256;       // query rows of a CTA
constexpr int kWideGroups = 1024;    // most groups
// Pieces that a row tile may be cut into, of all n heads rows: few rows need them to fill the SMs, many have
// tiles enough, and their pieces would be memory (8, 4, 1 piece, us a call, 32/4 heads x 64: 2048 rows behind 8192 26 / 54 /
// 95, 8192 behind 16384 62 / 105 / 191, 14336 behind 4096 45 / 47 / 65, 32768 87 / 85 / 84, 57344 132 / 129 / 142).
inline int wide_parts(int64_t rows) { return rows <= 10240 ? 8 : rows <= 40960 ? 4 : 1; }

template <int HD>
struct Wide {
  static constexpr int H = HD / 64, BK = 128, KB = 64;            // keys of a tile in shared memory, of a block
  static constexpr int NBUF = HD == 64 ? 3 : 2;                   // blocks of scores of a row tile
  static constexpr int kMmaWarp = 8, kTmaWarp = 12, NT = 416;
  static constexpr int kTile = 128 * HD * 2, kUnit = 128 * 128;  // bytes of 128 rows of Q, K or V; of 64 dims of them
  static constexpr int NST = HD == 64 ? 4 : 2;                   // K tiles in flight, and V tiles
  static constexpr int kOffCum = 512, kOffGroup = kOffCum + 4 * (kWideGroups + 4), kSmall = kOffGroup + 12 * kWideGroups;
  static constexpr int kSmem = 2 * kTile + 2 * NST * kTile + kSmall + 1024;
  static_assert(kSmem <= 232448 && tmem_fits(kSmem, 512), "shared memory");
  static constexpr int kAtO = 2 * NBUF * KB;                      // columns: S of tile t, buffer x at (t NBUF + x) KB; then O
  static_assert(kAtO + 2 * HD <= 512, "tensor memory");
};

struct WideParams {
  CUtensorMap k, v;
  TreeAttnParams p;
  int head, seq;        // 0 where a stride is 0, else 1
  bool whole;           // max_parts too few for cuts: ranges of row tiles
};

__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]),
      "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]),
      "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void st_global8(float* at, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
               "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// What a CTA has to do, one stretch of keys of a row tile after the other.
struct WideSegment {
  int g, hkv, row0, rows, k0, k1, len;  // group; rows row0 .. of the group; key tiles k0 .. k1 - 1 of the prefix's len rows
  int first, piece, pieces;             // the group's first sequence; which piece of the row tile, of how many
};
struct WideGroup {
  int first, rows, len;  // its first sequence, query rows of a kv head, prefix rows
  __device__ int key_tiles() const { return (len + 127) / 128; }
  __device__ int row_tiles() const { return (rows + kWideRows - 1) / kWideRows; }
};
struct WidePlan {
  const TreeAttnParams& p;
  const uint32_t* cum;      // [G + 1] units before a group
  const WideGroup* groups;  // [G]
  bool whole;
  uint32_t U, N, pos, end;
  // a b / c, of 32 bits; a 64-bit quotient takes some hundred cycles
  __device__ static uint32_t muldiv(uint32_t a, uint32_t b, uint32_t c) {
    return __umulhi(a, b) ? (uint32_t)((uint64_t)a * b / c) : a * b / c;
  }
  __device__ WidePlan(const TreeAttnParams& p_, const uint32_t* cum_, const WideGroup* groups_, bool whole_, int kt_max)
      : p(p_), cum(cum_), groups(groups_), whole(whole_) {
    U = cum[p.B];
    N = min(gridDim.x, U);
    if (!whole && U > 0) N = max((uint32_t)min((uint64_t)N, (uint64_t)U * (p.max_parts - 2) / kt_max), 1u);  // no row tile in more pieces
    pos = blockIdx.x < N ? muldiv(U, blockIdx.x, N) : 0;
    end = blockIdx.x < N ? muldiv(U, blockIdx.x + 1, N) : 0;
  }
  __device__ int cta_of(uint32_t u) const {  // ((u + 1) N - 1) / U
    return __umulhi(u + 1, N) ? (int)(((uint64_t)(u + 1) * N - 1) / U) : (int)(((u + 1) * N - 1) / U);
  }
  __device__ bool next(WideSegment& s) {
    if (pos >= end) return false;
    int lo = 0, hi = p.B - 1;  // the last group that starts at or before pos and is not empty
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (cum[mid] <= pos) lo = mid;
      else hi = mid - 1;
    }
    const WideGroup x = groups[lo];
    const uint32_t kt = x.key_tiles(), rt = x.row_tiles(), per = whole ? 1 : kt, off = pos - cum[lo], q = off / per;
    s.g = lo, s.first = x.first, s.len = x.len;
    s.hkv = q / rt;
    s.row0 = (q - s.hkv * rt) * kWideRows;
    s.rows = min(x.rows - s.row0, kWideRows);
    const uint32_t start = cum[lo] + q * per;
    s.k0 = whole ? 0 : off - q * kt;
    s.k1 = whole ? kt : min(kt, s.k0 + end - pos);
    s.piece = whole ? 0 : (int)blockIdx.x - cta_of(start);
    s.pieces = whole ? 1 : cta_of(start + kt - 1) - cta_of(start) + 1;
    pos += whole ? 1 : s.k1 - s.k0;
    return true;
  }
};

template <int HD>
__global__ void __launch_bounds__(Wide<HD>::NT, 1) wide_attn_kernel(const __grid_constant__ WideParams wp) {
  using C = Wide<HD>;
  constexpr int H = C::H, NST = C::NST, BK = C::BK, KB = C::KB, NBUF = C::NBUF;
  extern __shared__ uint8_t sm_raw[];
  const TreeAttnParams& p = wp.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  uint8_t* sq = sm;                       // [2][H][128 rows][128 B]
  uint8_t* sring = sq + 2 * C::kTile;     // [K, V][NST][H][128 keys][128 B]
  uint8_t* small = sring + 2 * NST * C::kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(small);
  uint64_t *full = bars, *empty = bars + 8, *q_full = bars + 16, *s_full = bars + 18, *p_full = bars + 24, *o_done = bars + 30,
           *drain = bars + 36;  // [K, V][4], [K, V][4], [2], then [2][3]
  volatile int* s_abort = reinterpret_cast<volatile int*>(small + 304);  // (12 ints: see tc_wait_long)
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(small + 352);
  int* s_kt = reinterpret_cast<int*>(small + 356);   // most key tiles of a group
  int* s_none = reinterpret_cast<int*>(small + 360);  // a group without prefix rows
  uint32_t* cum = reinterpret_cast<uint32_t*>(small + C::kOffCum);
  WideGroup* groups = reinterpret_cast<WideGroup*>(small + C::kOffGroup);
  if (tid == 0) {
    s_abort[0] = 0, s_abort[kLimitAt] = p.wait.ns;
    for (int i = 0; i < 8; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 2);
    for (int i = 0; i < 2; ++i) mbar_init(q_full + i, 128);
    for (int i = 0; i < 6; ++i)
      mbar_init(s_full + i, 1), mbar_init(p_full + i, 128 + p.wait.missing), mbar_init(o_done + i, 1);
    mbar_init(drain, 4);
    mbar_fence_init();
  }
  pdl_wait();
  pdl_trigger();
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else if (warp == C::kTmaWarp) {  // units before each group
    uint32_t before = 0;
    int most = 1, begun = 0;
    bool none = false;
    for (int g0 = 0; g0 < p.B; g0 += 32) {
      // No group begins before one ahead of it, whatever `starts` says: the groups are apart, so that their units
      // stay within 32 bits and their rows within the queries'
      const int g = g0 + lane;
      int from = g < p.B ? min(max(p.starts[g], 0), p.all) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) from = max(from, __shfl_up_sync(0xffffffffu, from, o));
      from = max(from, begun);
      begun = __shfl_sync(0xffffffffu, from, 31);
      WideGroup own{0, 0, 0};
      if (g < p.B) {
        own.first = from;
        own.rows = (max(min(p.starts[g + 1], p.all), from) - from) * p.n * p.gq;
        own.len = min(max(p.lens[g], 0), p.cache.rows);
        groups[g] = own;
      }
      const int kt = own.key_tiles();
      uint32_t u = kt > 0 ? (uint32_t)own.row_tiles() * (wp.whole ? 1 : kt) * p.Hkv : 0u, x = u;
      if (u) most = max(most, kt);
      none |= own.rows > 0 && kt == 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (g < p.B) cum[g] = before + x - u;
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    none = __any_sync(0xffffffffu, none);
    if (lane == 0) cum[p.B] = before, *s_kt = most, *s_none = none;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  if (*s_none)
    for (int g = 0; g < p.B; ++g) {
      const WideGroup x = groups[g];
      if (x.len == 0)
        for (int i = blockIdx.x * C::NT + tid; i < x.rows * p.Hkv; i += gridDim.x * C::NT)
          p.part_n[(int64_t)x.first * p.n * p.Hkv * p.gq + i] = 0;
    }
  WidePlan plan(p, cum, groups, wp.whole, *s_kt);
  WideSegment seg{};
  // Key tiles are counted over all segments. K and V have rings of their own: a warp
  // that waits for some tiles of a ring waits for all of them, in order, since a wait for a
  // phase whose predecessor is not over is over at once. (So the warps that issue wait for
  // tiles, those of row tiles without rows too, and the softmax warps, which pass over
  // such segments, never do.)
  uint32_t base = 0;  // key tiles of the segments before
  auto landed = [&](int kv, uint32_t i) { return tc_wait_warp(full + 4 * kv + i % NST, (i / NST) & 1, s_abort, p.status); };
  auto blocks = [&]() { return min(2 * (seg.k1 - seg.k0), (seg.len - seg.k0 * BK + KB - 1) / KB); };
  uint32_t sent[2] = {0, 0};  // by the TMA lane
  if (warp == C::kTmaWarp) {
    if (lane == 0) {
      bool ok = true;
      while (ok && plan.next(seg)) {
        const int n = seg.k1 - seg.k0;
#pragma unroll 1
        for (int j = 0; j < 2 * n && ok; ++j) {  // K0 K1 V0 K2 V1 .. V
          const int kv = j > 0 && (!(j & 1) || j == 2 * n - 1), k = j == 2 * n - 1 ? n - 1 : kv ? j / 2 - 1 : (j + 1) / 2;
          const uint32_t i = base + k, slot = i % NST;
          uint64_t* bar = full + 4 * kv + slot;
          if (i >= (uint32_t)NST) ok = tc_wait(empty + 4 * kv + slot, (i / NST - 1) & 1, s_abort, p.status);
          if (!ok) break;
          mbar_expect_tx(bar, C::kTile);
#pragma unroll
          for (int u = 0; u < H; ++u)
            tma_box(sring + (kv * NST + slot) * C::kTile + u * C::kUnit, kv ? &wp.v : &wp.k, 64 * u, (seg.k0 + k) * BK,
                    seg.hkv * wp.head, seg.g * wp.seq, bar);
          sent[kv] = i + 1;
        }
        base += n;
      }
    }
  } else if (warp >= C::kMmaWarp) {
    // ---- products of row tile t: Q K, or P V
    constexpr uint32_t base_i = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);  // fp32 += bf16 x bf16, 128 rows
    constexpr uint32_t idesc_s = base_i | ((uint32_t)(KB >> 3) << 17);
    constexpr uint32_t idesc_o = base_i | ((uint32_t)(HD >> 3) << 17) | (1u << 16);  // V is MN-major
    const int t = warp & 1;
    const bool values = warp >= C::kMmaWarp + 2;
    const uint32_t ur = smem_u32(sring) + (values ? NST * C::kTile : 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t tS = tm + t * NBUF * KB, tO = tm + C::kAtO + t * HD;
    const uint64_t da = tc_desc(smem_u32(sq) + t * C::kTile, 16, 1024, 2);
    bool ok = true;
    uint32_t n_seg = 0, done = 0;  // segments, blocks so far
    while (ok && plan.next(seg)) {
      const int n = seg.k1 - seg.k0, nb = blocks();
      if (t * 128 >= seg.rows) {  // no rows: the tiles are given back as they come
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          ok = landed(values, base + j);
          if (ok && lane == 0) mbar_arrive(empty + 4 * values + (base + j) % NST);
        }
        base += n;
        continue;
      }
      if (!values) {
        ok = tc_wait_warp(q_full + t, n_seg & 1, s_abort, p.status);
        ++n_seg;
#pragma unroll 1
        for (int j = 0; j < nb && ok; ++j) {
          const uint32_t b = done + j, x = b % NBUF, i = base + (j >> 1), slot = i % NST;
          if (!(j & 1)) ok = landed(0, i);
          // into the buffer of the block NBUF before: its P V is done (of the segment before, all are)
          if (j >= NBUF) ok = ok && tc_wait_warp(o_done + 3 * t + x, (b / NBUF - 1) & 1, s_abort, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t db = tc_desc(ur + slot * C::kTile + (j & 1) * KB * 128, 16, 1024, 2);
          if (elect_lane()) {
#pragma unroll
            for (int u = 0; u < H; ++u)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)  // 16 dims: 32 bytes further
                tc_mma(tS + x * KB, da + (u * C::kUnit >> 4) + 2 * ks, db + (u * C::kUnit >> 4) + 2 * ks, idesc_s, u > 0 || ks > 0);
          }
          __syncwarp();
          tc_commit(s_full + 3 * t + x);
          if ((j & 1) || j == nb - 1) tc_commit(empty + slot);
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < nb && ok; ++j) {
          const uint32_t b = done + j, x = b % NBUF, i = base + (j >> 1), slot = i % NST;
          if (!(j & 1)) ok = landed(1, i);
          if (!ok) break;
          const int left = seg.len - seg.k0 * BK - j * KB;  // keys from this block on
          if (left < KB) {  // V rows that are not there become zeros: 0 times whatever lies there need not be 0
            // (both row tiles' warps write them, the same; the tile goes back only when both have multiplied it)
#pragma unroll 1
            for (int c = lane; c < (KB - left) * (HD / 8); c += 32) {
              const int row = (j & 1) * KB + left + c / (HD / 8), ch = c % (HD / 8);
              *reinterpret_cast<uint4*>(sring + (NST + slot) * C::kTile + (ch / 8) * C::kUnit + row * 128 + 16 * (ch & 7)) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
            __syncwarp();
          }
          ok = tc_wait_warp(p_full + 3 * t + x, (b / NBUF) & 1, s_abort, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t db = tc_desc(ur + slot * C::kTile + (j & 1) * KB * 128, C::kUnit, 1024, 2);
          if (elect_lane()) {
#pragma unroll
            for (int ks = 0; ks < KB / 16; ++ks)  // 16 keys: 8 columns of P, 2 KB of V further
              tc_mma_ts(tO, tS + x * KB + 8 * ks, db + ks * (uint64_t)128, idesc_o, j > 0 || ks > 0);
          }
          __syncwarp();
          tc_commit(o_done + 3 * t + x);
          if ((j & 1) || j == nb - 1) tc_commit(empty + 4 + slot);
        }
      }
      done += nb;
      base += n;
    }
  } else {
    // ---- softmax: thread = row of tile t
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t tS0 = tmem + lanes + t * NBUF * KB, tO = tmem + lanes + C::kAtO + t * HD;
    uint32_t done = 0;  // blocks so far
    bool ok = true;
    auto pv_done = [&](uint32_t b) { return tc_wait_warp(o_done + 3 * t + b % NBUF, (b / NBUF) & 1, s_abort, p.status); };
    while (ok && plan.next(seg)) {
      const int nb = blocks();
      if (t * 128 >= seg.rows) continue;
      const int row = seg.row0 + t * 128 + r, node = p.by_gq.div(row), h = seg.hkv * p.gq + row - node * p.gq;
      const bool there = t * 128 + r < seg.rows;
      {  // Q: 128-byte rows of 64 dims, chunks permuted as by TMA's 128-byte swizzle
        const int s = p.by_n.div(node);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (int64_t)(seg.first + s) * p.q_seq +
                                                          (int64_t)(node - s * p.n) * p.q_node + (int64_t)h * p.q_head);
        const uint32_t turn = p.neg ? 0x80008000u : 0u;
        uint8_t* dst = sq + t * C::kTile + r * 128;
#pragma unroll
        for (int ch = 0; ch < HD / 8; ++ch) {
          uint4 w = there ? src[ch] : make_uint4(0u, 0u, 0u, 0u);
          w.x ^= turn, w.y ^= turn, w.z ^= turn, w.w ^= turn;
          *reinterpret_cast<uint4*>(dst + (ch / 8) * C::kUnit + 16 * ((ch & 7) ^ (r & 7))) = w;
        }
        fence_async_smem();
        mbar_arrive(q_full + t);
      }
      float ref = -kNone, l = 0.f;  // the reference, negated; the sum of the probabilities
#pragma unroll 1
      for (int j = 0; j < nb; ++j) {
        const uint32_t blk = done + j, x = blk % NBUF, tS = tS0 + x * KB;
        const int left = seg.len - seg.k0 * BK - j * KB;  // keys from this block on
        ok = tc_wait_warp(s_full + 3 * t + x, (blk / NBUF) & 1, s_abort, p.status);
        if (!ok) break;
        tc_fence_after();
        float a[32], b[32];
        auto load = [&]() {
          tc_ld(a, tS);
          tc_ld(b, tS + 32);
          tc_wait_ld(a);
          tc_wait_ld(b);
          if (left < KB)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (i >= left) a[i] = -INFINITY;
              if (32 + i >= left) b[i] = -INFINITY;
            }
        };
        auto highest = [&]() {
          float m = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; ++i) m = fmaxf(m, fmaxf(a[i], b[i]));
          return m;
        };
        load();
        if (j == 0) {
          const float m = highest();
          ref = fabsf(m) < 1e38f ? -m : -kNone;
        }
        uint32_t pk[KB / 2];
        float sum;
        for (;;) {
          float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            add2(a[i], a[i + 1], a[i], a[i + 1], ref, ref);
            add2(b[i], b[i + 1], b[i], b[i + 1], ref, ref);
            mul2(a[i], a[i + 1], a[i], a[i + 1], p.c);
            mul2(b[i], b[i + 1], b[i], b[i + 1], p.c);
            a[i] = ex2(a[i]), a[i + 1] = ex2(a[i + 1]);
            b[i] = ex2(b[i]), b[i + 1] = ex2(b[i + 1]);
            add2(s0, s1, s0, s1, a[i], a[i + 1]);
            add2(s2, s3, s2, s3, b[i], b[i + 1]);
            pk[i / 2] = pack_bf16x2(a[i], a[i + 1]);
            pk[16 + i / 2] = pack_bf16x2(b[i], b[i + 1]);
          }
          sum = (s0 + s1) + (s2 + s3);
          const bool over = sum > 1152921504606846976.f;  // 2^60
          if (!__any_sync(0xffffffffu, over)) break;
          // renew the references of the warp's rows; rescale O and the sums
          load();
          const float old = -ref, now = fmaxf(highest(), old), f = !over || old == now ? 1.f : exp2f((old - now) * p.c);
          if (over && now > old) ref = -now;
          l *= f;
          if (j > 0) {
            ok = pv_done(blk - 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 16) {
              float o[16];
              tc_ld(o, tO + c0);
              tc_wait_ld(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f;
              tc_st16(tO + c0, o);
            }
            tc_wait_st();
          }
        }
        if (!ok) break;
        l += sum;
        tc_st32(tS, pk);
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + 3 * t + x);
      }
      if (!ok) break;
      done += nb;
      // (one phase of a buffer at a time: the last but one of each is over when its scores have come)
      for (int k = min(nb, NBUF); k > 0 && ok; --k) ok = pv_done(done - k);
      if (!ok) break;
      tc_fence_after();
      const int64_t at = ((int64_t)seg.first * p.n + node) * (p.Hkv * p.gq) + h;
      const float f = l == 0.f ? 0.f : 1.f / l;
      float* out = p.part_o + (seg.piece * p.part_rows + at) * HD;
#pragma unroll
      for (int c0 = 0; c0 < HD; c0 += 32) {
        float a[32];
        tc_ld(a, tO + c0);
        tc_wait_ld(a);
#pragma unroll
        for (int i = 0; i < 32; ++i) a[i] *= f;
        if (there)
#pragma unroll
          for (int i = 0; i < 32; i += 8) st_global8(out + c0 + i, a + i);
      }
      if (there) {
        p.part_ml[seg.piece * p.part_rows + at] = make_float2(-ref, l);
        if (seg.piece == 0) p.part_n[at] = seg.pieces;
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  __syncthreads();
  if (*s_abort) {  // no copy and no product in flight outlives the CTA
    const unsigned long long s0 = globaltimer();
    if (warp == C::kTmaWarp && lane == 0)
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv)
#pragma unroll 1
        for (uint32_t j = sent[kv] > (uint32_t)NST ? sent[kv] - NST : 0; j < sent[kv]; ++j)
          while (!mbar_try_wait(full + 4 * kv + j % NST, (j / NST) & 1) && globaltimer() - s0 < kWaitLimitNs) {
          }
    __syncwarp();
    if (warp >= C::kMmaWarp && warp < C::kTmaWarp) {
      tc_commit(drain);  // of a warp's own products
      while (!mbar_try_wait(drain, 0) && globaltimer() - s0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
    __syncthreads();
  }
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

template <int HD>
cudaError_t launch_wide(const TreeAttnParams& p, int n_sm, cudaStream_t st) {
  WideParams wp;
  wp.p = p;
  wp.head = p.cache.head != 0, wp.seq = p.cache.seq != 0;
  wp.whole = p.max_parts < 3;
  if (!encode_rows<HD, false>(&wp.k, p.cache.k, p.cache, p.B, p.Hkv) || !encode_rows<HD, false>(&wp.v, p.cache.v, p.cache, p.B, p.Hkv))
    return cudaErrorNotSupported;
  const auto kern = wide_attn_kernel<HD>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(kern, Wide<HD>::kSmem);
  return e == cudaSuccess ? launch_cluster(kern, dim3(n_sm), Wide<HD>::NT, 1, Wide<HD>::kSmem, st, wp, p.pdl) : e;
}

}  // namespace llmq
