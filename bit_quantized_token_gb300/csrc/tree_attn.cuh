// Attention of a tree of drafted tokens over bf16 K/V rows.
//
// A sequence's n nodes (n <= 64) share its cached prefix; node i also sees the
// tree rows whose bits its mask sets. The gq query heads of a kv head and the
// n nodes form M = n gq query rows against the same keys (row r: node r / gq,
// head r % gq), so one pass over K and V serves all of them:
//   o_r = sum_j 2^(c (s_rj - m_r)) v_j / sum_j 2^(c (s_rj - m_r)),  s_rj = q_r . k_j,
// with c = |scale| log2(e) (a negative scale turns the queries' signs), the
// references m_r and the sums in fp32. A reference is a score: c s - m, one
// operation less, has no reference within 2^60 of a row's largest once that passes
// 2^30, where fp32 steps by 128.
//
// The products run transposed, so that the few query rows are the narrow side:
//   S^T [128 keys x N rows] = K_tile Q^T     (A = the K tile as TMA lays it down, K-major)
//   O^T [dims x N rows]    += V_tile^T P^T   (A = the V tile, read MN-major; B = P, [key][row])
// A thread of a softmax warp is one key: it reads its scores from tensor
// memory, turns them into probabilities and writes them as a row of P, so no
// exchange between threads is needed. Instead of the running maximum, a
// reference within 2^60 of it does: it starts as the first key's scores and is
// renewed (and O rescaled) only when a score passes it by more than 2^60; bf16
// and fp32 keep their relative precision over that range.
// A tile is read as units of 128 keys x 64 dims (16 KB, one TMA box, 128-byte
// swizzle): K and V units stream through one ring. Of each P V product's 128
// rows the upper 64 read ones instead of V, so lanes 64.. hold the sums of P.
// fp32 operands are parts in bf16 (24 bits in three, 16 in two): the parts of Q
// and of P are columns of their own in one product each, so that A, whose fetch
// from shared memory (4 KB, ~64 cycles) bounds these narrow products, is fetched
// once; the sums over the parts are formed on the way out. So are the rows of
// all G blocks: a block is what four softmax warps take, not a product.
// Warp roles: 4 softmax warps per block of NB rows, one TMA warp, one warp that
// issues every MMA. What a softmax waits for overlaps the other CTA on the SM,
// where shared and tensor memory let two fit; S and P have two buffers where that
// costs no second CTA, and the scores are then a tile ahead.
// Measured (GB300): 32 sequences x 8 nodes, 16/8 heads x 128 over 512..2048 rows
// 36.6 us, 70 % of the copy rate: what two CTAs' rings hold on their way to an SM.
// 16 x 64 nodes, 32/4 heads x 64 over 1024..8192 rows 85.5 us: a tile's chain from
// scores to probabilities to P V (3,200 cycles, two CTAs an SM) and the uneven last
// CTAs. 16 fp32 nodes over 4097 rows 13.0 us and one over 256 rows 5.9: start, a few
// tiles, join.
#pragma once
#include <cuda.h>

#include <cooperative_groups.h>

#include <algorithm>

#include "attn_mma.cuh"
#include "tree.cuh"

namespace llmq {
namespace cg = cooperative_groups;

struct TreeAttnTcParams {
  CUtensorMap ck, cv, tk, tv;  // cache and tree rows: [seq][head][row][dim], boxes of 128 rows x 64 dims
  TreeAttnParams p;
  // 0 where a stride is 0 (all sequences, or heads, share the rows), else 1: TMA takes no stride of 0
  int c_seq, c_head, t_seq, t_head;
};

constexpr int kMaxSplits = 16;  // CTAs of a cluster
constexpr float kNone = -3.402823466e38f;  // a row's reference before any visible score
// For fp32 queries, tiles that O adds up in tensor memory. An MMA cuts its sum off
// where an add would round, so long sums come out low: 1e-6 of the output after 8
// tiles and 8e-6 after 125 (int8, three parts of V: 3e-6 and 1e-5), against 2e-7 for
// sums that round. Every two tiles (int8: each) the sums go to registers, which
// round: 4e-7, at 0.5 us of 12.3 (16 nodes over 4097 rows).
constexpr int kTogether = 2;

// Whether CTAs that take tensor memory, each with this shared memory and these columns, find their columns wherever
// an SM's 228 KB (a CTA's own and 1 KB) hold them together: at most two share an SM, and one of more than half of the
// columns shares it with none. So an allocation never waits for a CTA that waits for its kernel (a cluster that
// gathers, a second part that waits for the first).
constexpr bool tmem_fits(int smem, int cols) {
  constexpr int kSm = 228 * 1024, kOwn = 1024, kThird = kSm / 3;
  return smem + kOwn > kThird && (cols <= 256 || smem + kOwn + kThird >= kSm);
}

template <int HD, bool F32, int NB, int G>
struct TreeTc {
  static constexpr int N = NB * G, BK = 128, H = HD / 64;
  // Parts of the queries, of P. One part of P (8 bits) where a CTA takes 128 rows: the outputs' error is 0.0024 of
  // their size, with two parts 0.0017, what rounding them to bf16 gives. Two parts would leave one CTA on an SM at 64
  // dims (16 x 64 nodes over 1024..8192 rows 86 -> 87 us, 32 x 16 over 512..4096 34 -> 45) and do not fit tensor
  // memory at 128 (64 rows a CTA instead: 105 -> 113 and 112 -> 251 us for 2 and 4 query heads a kv head).
  static constexpr int NQ = F32 ? 3 : 1, NP = F32 ? 3 : (N > 64 ? 1 : 2);
  static constexpr int NS = NQ * NB, NO = NP * NB;                        // columns of a block's S, of its O (64 dims)
  static constexpr int NSA = G * NS, NOA = G * NO;                        // of all blocks
  static constexpr int NT = 32 * (4 * G + 2);
  static constexpr int kUnit = BK * 128;                                  // bytes: 64 dims of a K or V tile
  static constexpr int kRowP = NOA >= 48 ? 128 : 2 * NOA;                 // bytes of a key's row of a P atom (64 columns)
  static constexpr int kP = BK * kRowP * ((NOA + 63) / 64);               // bytes of P
  static constexpr int kQ = NQ * N * HD * 2, kOnes = 2048;
  static constexpr int kOffRow = 1024;                                   // of the small arrays: [N] row masks
  static constexpr int kSmall = kOffRow + N * (8 + 4 + 16 + 8 + 4) + 3 * kTreeMaxNodes * (HD / 32) * 4;
  static constexpr int kRest = kQ + kOnes + kSmall + 1024;
  static constexpr int kOut = N * HD * 4;                                // fp32 results, over the ring at the end
  static constexpr int kLimit = 232448, kHalf = 115712;                  // shared memory of a CTA alone, of two on an SM
  // a tile's K and V units and, of 64 dims, the next K unit must fit
  static constexpr int kLeast = H == 1 ? 3 : 4, kMin = kLeast > kOut / kUnit ? kLeast : kOut / kUnit;
  static constexpr bool two1 = kRest + kP + kMin * kUnit <= kHalf && NSA + H * NOA <= 256;
  static constexpr bool two2 = kRest + 2 * kP + kMin * kUnit <= kHalf && 2 * NSA + H * NOA <= 256;
  static constexpr bool one2 = kRest + 2 * kP + kMin * kUnit <= kLimit && 2 * NSA + H * NOA <= 512;
  static constexpr int DB = two2 || (!two1 && one2) ? 2 : 1;             // buffers of S and P
  static constexpr bool two = DB == 2 ? two2 : two1;                     // CTAs on an SM
  static constexpr int kFixed = kRest + DB * kP;
  static constexpr int fit = ((two ? kHalf : kLimit) - kFixed) / kUnit;
  static constexpr int NST = fit < 12 ? fit : 12;
  static constexpr int kSmem = NST * kUnit + kFixed;
  static_assert(NST >= kMin, "shared memory");
  static constexpr int kUsed = DB * NSA + H * NOA;                       // S, and O of every 64 dims
  static_assert(kUsed <= 512, "tensor memory");
  static constexpr int kCols = kUsed <= 32 ? 32 : kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(tmem_fits(kSmem, kCols), "tensor memory of CTAs on an SM");
};

// A warp's bounded wait with one answer for all lanes.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status);
__device__ __forceinline__ bool tc_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return __all_sync(0xffffffffu, tc_wait(bar, parity, abort_flag, status));
}
// A bounded wait: past the limit the CTA's abort flag and the device's status
// word are set, and from kGraceNs later on every wait of the CTA that is not over
// fails at once, so that the loops end and no barrier is missed. (In the time of grace
// what is in flight lands.) A block of softmax warps one of whose waits for scores has
// failed agrees on it by its barriers and leaves its loop (an arrival out of turn can
// find fewer pending than a warp brings, which faults); the MMA warp issues nothing
// behind a failed wait, and a wait that ends with the flag set has failed too: the
// converters of int8 rows go on and may let phases complete out of turn. A poll is
// over within kPollNs of its look at the flag, long before that. In a CTA with the
// flag set the MMA warp and the TMA lane wait at the end for all that they have
// issued; without it the other warps' waits were for the same.
// (A call: the kernel's code is fetched anew by every CTA, and short ones wait for it.)
constexpr unsigned long long kGraceNs = 200000;
constexpr uint32_t kPollNs = 20000;
constexpr int kLimitAt = 3, kAbortAt = 10;  // ints from the flag on: the limit in ns, the time when the flag was set
static __device__ __noinline__ bool tc_wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  volatile unsigned long long* aborted = reinterpret_cast<volatile unsigned long long*>(abort_flag + kAbortAt);
  unsigned long long start = 0;
  for (uint32_t i = 0;; ++i) {
    const int set = *abort_flag;
    uint32_t over;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(over)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kPollNs)
        : "memory");
    if (over) return set == 0;
    if (set) {
      if (globaltimer() > *aborted + kGraceNs) return false;
    } else if ((i & 63) == 63) {
      const unsigned long long t = globaltimer();
      if (start == 0) {
        start = t;
      } else if (t - start > (uint32_t)abort_flag[kLimitAt]) {
        *aborted = t;
        __threadfence_block();
        *abort_flag = 1;
        atomicOr(status, ST_TIMEOUT);
      }
    }
  }
}
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return mbar_try_wait(bar, parity) || tc_wait_long(bar, parity, abort_flag, status);
}
// By all lanes of a warp, which go on converged: the tensor memory accesses behind
// such a wait are the warp's together, and a wait can end for some lanes first.
__device__ __forceinline__ void tc_wait_together(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  tc_wait(bar, parity, abort_flag, status);
  __syncwarp();
}
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x, int row, int head, int seq,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(row), "r"(head), "r"(seq), "r"(smem_u32(bar))
      : "memory");
}
// The MMA warp runs converged, so that addresses stay in uniform registers, and
// one elected lane (always the same of a full warp) issues.
__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      :
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  if (elect_lane())
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// Shared memory matrix descriptor: start, leading and stride byte offsets in
// 16-byte units; swizzle 2: 128 B, 4: 64 B, 6: 32 B.
__device__ __forceinline__ uint64_t tc_desc(uint32_t start, uint32_t lbo, uint32_t sbo, uint64_t swizzle) {
  return (uint64_t)((start & 0x3FFFF) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         (1ull << 46) | (swizzle << 61);
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// W columns of this warp's 32 lanes, one lane per thread
template <int W>
__device__ __forceinline__ void tc_ld(float (&v)[W], uint32_t addr) {
  static_assert(W == 16 || W == 32, "columns");
  if constexpr (W == 16)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(addr));
  else
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
                 : "r"(addr));
}
// Waits for the loads; the values pass through, so that no use of them moves ahead of the wait.
template <int W>
__device__ __forceinline__ void tc_wait_ld(float (&v)[W]) {
  if constexpr (W == 16)
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]) : : "memory");
  else
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]) : : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// a, b as NP bf16 pairs whose sums carry 8 NP bits
template <int NP>
__device__ __forceinline__ void split_pack(float a, float b, uint32_t (&part)[NP]) {
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    part[k] = pack_bf16x2(a, b);
    if (k + 1 < NP) sub2(a, b, a, b, __uint_as_float(part[k] << 16), __uint_as_float(part[k] & 0xFFFF0000u));
  }
}
// Bit j of lane i's word becomes bit i of lane j's: halves of ever smaller blocks change places.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, int lane) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const uint32_t low = 0xFFFFFFFFu / ((1u << m) + 1);  // the bits whose index has not m
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, m);
    x = lane & m ? (x & ~low) | ((y & ~low) >> m) : (x & low) | ((y & low) << m);
  }
  return x;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// the 128 threads of softmax group g (named barriers 1..G)
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(g + 1) : "memory"); }
__device__ __forceinline__ bool group_any(int g, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(g + 1)
      : "memory");
  return r != 0;
}

// The sequence with the z-th longest cache of at most 64 (every warp finds it by
// itself): blocks start in grid order, and starting the long sequences first
// leaves the short ones to fill the end.
__device__ __forceinline__ int nth_longest(const int* lens, int B, int z, int lane) {
  const int a = lane < B ? lens[lane] : -1, c = lane + 32 < B ? lens[lane + 32] : -1;
  int ra = 0, rc = 0;  // sequences ahead of this lane's two
  for (int j = 0; j < min(B, 32); ++j) {
    const int o = __shfl_sync(0xffffffffu, a, j);
    ra += o > a || (o == a && j < lane);
    rc += o >= c;
  }
  for (int j = 32; j < B; ++j) {
    const int o = __shfl_sync(0xffffffffu, c, j - 32);
    ra += o > a;
    rc += o > c || (o == c && j < lane + 32);
  }
  const unsigned ha = __ballot_sync(0xffffffffu, lane < B && ra == z);
  const unsigned hc = __ballot_sync(0xffffffffu, lane + 32 < B && rc == z);
  return ha ? __ffs(ha) - 1 : 31 + __ffs(hc);
}

// A block's sequence of queries (the first of several) and its nodes.
struct TreeBlock {
  int seq, cnt;
  __device__ TreeBlock(const TreeAttnParams& p, int b) {
    if (p.part == TreeAttnParams::kFirst) {
      seq = min(max(p.starts[b], 0), p.all);
      cnt = (min(max(p.starts[b + 1], seq), p.all) - seq) * p.n;
    } else {
      seq = b;
      const int c = p.counts ? p.counts[b] : p.n;
      cnt = min(max(c, 0), p.n);
    }
  }
  // offset of a node's queries
  __device__ __forceinline__ int64_t q_at(const TreeAttnParams& p, int node) const {
    const int s = p.part == TreeAttnParams::kFirst ? p.by_n.div(node) : 0;
    return (int64_t)(seq + s) * p.q_seq + (int64_t)(node - s * p.n) * p.q_node;
  }
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// The cluster's S key ranges joined (S a power of two, so it divides N). so: a
// rank's unnormalised O [N][HD], sml its (reference, sum) per row. Rank q owns the
// rows from q share on: every rank stores its part of them into q's `in`
// ([S][share] rows, their (reference, sum), room for weights: kJoin bytes), and q
// adds the parts from its own shared memory. (Loads from the other ranks took a
// round trip for the weights and one for the parts, and a barrier more.) With S >
// 1 every thread has arrived once (cluster_arrive) when its CTA's part of `in` was free.
// In an attention of two parts the owner writes them out, or joins its row with the
// first part's, which it waits for here: the kernels overlap until then.
template <int HD, int N>
constexpr int kJoin = N * HD * 4 + N * (12 + 4 * TreeAttnParams::kMaxParts);
template <int HD, bool F32, int N, int NT>
__device__ __forceinline__ void join_splits(const TreeAttnParams& p, const float* so, const float2* sml, uint8_t* in,
                                            int rank, int b, int hkv, int m0, int rows) {
  constexpr int R4 = HD / 4;
  const int tid = threadIdx.x, S = p.S, share = (rows + S - 1) / S;
  const float4* part = reinterpret_cast<const float4*>(so);  // [S][share][R4]
  const float2* ml = sml;                                    // [S][share]
  float* sw = reinterpret_cast<float*>(in + N * HD * 4 + N * 8);
  float* sw_first = sw + N;                                  // [pieces][share] of the first part
  // row m0 + r of the block (its nodes follow one another): index of its (sequence, node, head) in part_ml
  auto part_at = [&](int row) {
    const int node = p.by_gq.div(row);
    return ((int64_t)b * p.n + node) * (p.Hkv * p.gq) + hkv * p.gq + row - node * p.gq;
  };
  const bool second = p.part == TreeAttnParams::kSecond;
  if (second) pdl_wait();
  const bool first_has = second && b >= p.starts[0] && b < p.starts[p.G];
  __syncthreads();
  if (S > 1) {
    cg::cluster_group cl = cg::this_cluster();
    float4* in4 = reinterpret_cast<float4*>(in);
    float2* in_ml = reinterpret_cast<float2*>(in + N * HD * 4);
    const uint32_t inv = (65535 + share) / share;  // r / share = r inv >> 16 (r and share at most 128)
    cluster_wait();
#pragma unroll 4
    for (int i = tid; i < rows * R4; i += NT) {
      const int r = i / R4, q = r * inv >> 16;
      cl.map_shared_rank(in4, q)[(rank * share + r - q * share) * R4 + i % R4] = part[i];
    }
    for (int r = tid; r < rows; r += NT) {
      const int q = r * inv >> 16;
      cl.map_shared_rank(in_ml, q)[rank * share + r - q * share] = sml[r];
    }
    cluster_arrive();
    cluster_wait();  // every part is here, and no rank touches another's memory from here on
    part = in4, ml = in_ml;
  }
  const int own = min(share, rows - rank * share);  // (none: 0 or less)
  // no visible score (NaN scores alone leave no reference either, but a NaN sum, which has to count)
  auto none = [](float2 ml) { return ml.x <= kNone && ml.y == ml.y; };
  for (int r = tid; r < own; r += NT) {
    float M = ml[r].x, L = 0.f;
    for (int k = 1; k < S; ++k) M = fmaxf(M, ml[k * share + r].x);
    for (int k = 0; k < S; ++k) {
      const float2 x = ml[k * share + r];
      const float w = none(x) ? 0.f : ex2((x.x - M) * p.c);
      L = fmaf(x.y, w, L);
      sw[k * share + r] = w;
    }
    float f = L == 0.f ? 0.f : 1.f / L;  // nothing seen: 0
    if (p.part == TreeAttnParams::kFirst) {
      const int64_t at = part_at(m0 + rank * share + r);
      p.part_ml[at] = make_float2(M, L);
      p.part_n[at] = 1;
    }
    if (second) {
      const int64_t at = part_at(m0 + rank * share + r);
      const int n = first_has ? __ldcg(p.part_n + at) : 0;
      float2 o[TreeAttnParams::kMaxParts];
      float top = M, sum = 0.f;
#pragma unroll
      for (int k = 0; k < TreeAttnParams::kMaxParts; ++k) {
        o[k] = k < n && k < p.max_parts ? __ldcg(p.part_ml + k * p.part_rows + at) : make_float2(kNone, 0.f);
        top = fmaxf(top, o[k].x);
      }
      const float own_w = none(make_float2(M, L)) ? 0.f : ex2((M - top) * p.c);
#pragma unroll
      for (int k = 0; k < TreeAttnParams::kMaxParts; ++k) {
        o[k].y = none(o[k]) ? 0.f : ex2((o[k].x - top) * p.c) * o[k].y;
        sum += o[k].y;
      }
      sum = fmaf(own_w, L, sum);
      f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int k = 0; k < TreeAttnParams::kMaxParts; ++k)
        if (k < p.max_parts) sw_first[k * share + r] = o[k].y * f;
      f *= own_w;
    }
    for (int k = 0; k < S; ++k) sw[k * share + r] *= f;
  }
  __syncthreads();
#pragma unroll 2
  for (int i = tid; i < own * R4; i += NT) {
    const int r = i / R4, row = m0 + rank * share + r, node = p.by_gq.div(row), h = hkv * p.gq + row - node * p.gq;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < S; ++k) {
      const float4 x = part[k * share * R4 + i];
      const float f = sw[k * share + r];
      a.x = fmaf(x.x, f, a.x), a.y = fmaf(x.y, f, a.y), a.z = fmaf(x.z, f, a.z), a.w = fmaf(x.w, f, a.w);
    }
    if (p.part == TreeAttnParams::kFirst) {
      reinterpret_cast<float4*>(p.part_o)[part_at(row) * R4 + i % R4] = a;
      continue;
    }
    if (first_has) {
      const float4* o = reinterpret_cast<const float4*>(p.part_o) + part_at(row) * R4 + i % R4;
#pragma unroll 4
      for (int k = 0; k < p.max_parts; ++k) {
        const float f = sw_first[k * share + r];
        const float4 x = f != 0.f ? __ldcg(o + k * p.part_rows * R4) : make_float4(0.f, 0.f, 0.f, 0.f);
        a.x = fmaf(x.x, f, a.x), a.y = fmaf(x.y, f, a.y), a.z = fmaf(x.z, f, a.z), a.w = fmaf(x.w, f, a.w);
      }
    }
    const int64_t off = (int64_t)b * p.o_seq + (int64_t)node * p.o_node + (int64_t)h * p.o_head + 4 * (i % R4);
    if constexpr (F32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + off) = a;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + off) =
          make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

template <int HD, bool F32, int NB, int G>
__global__ void __launch_bounds__(TreeTc<HD, F32, NB, G>::NT, TreeTc<HD, F32, NB, G>::two ? 2 : 1) tree_attn_tc_kernel(
    const __grid_constant__ TreeAttnTcParams tp) {
  using C = TreeTc<HD, F32, NB, G>;
  constexpr int N = C::N, NT = C::NT, NST = C::NST, NQ = C::NQ, NP = C::NP, NG = HD / 32, BK = C::BK, H = C::H, DB = C::DB;
  extern __shared__ uint8_t sm_raw[];
  const TreeAttnParams& p = tp.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* sm = sm_raw + ((1024 - (smem_u32(sm_raw) & 1023)) & 1023);
  uint8_t* sring = sm;
  uint8_t* sp = sring + NST * C::kUnit;   // [DB] P: [atom of 64 columns][key][kRowP], columns [block][part][row]
  uint8_t* sq = sp + DB * C::kP;          // [H][G][NQ][NB][128 B]
  uint8_t* sones = sq + C::kQ;
  uint8_t* small = sones + C::kOnes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(small);
  uint64_t *full = bars, *empty = bars + 12, *s_full = bars + 24, *p_full = bars + 26, *o_done = bars + 28, *drain = bars + 30;
  volatile int* s_abort = reinterpret_cast<volatile int*>(small + 256);
  int* s_any = reinterpret_cast<int*>(small + 260);
  volatile int* s_stop = reinterpret_cast<volatile int*>(small + 288);  // [G] a wait of the block's has failed
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(small + 264);
  uint64_t* smask = reinterpret_cast<uint64_t*>(small + 512);          // [64]
  uint64_t* srow = reinterpret_cast<uint64_t*>(small + C::kOffRow);    // [N] what each row sees of the tree
  float* sm_m = reinterpret_cast<float*>(srow + N);             // [N] references, negated
  float* sm_w = sm_m + N;                                       // [4][N]
  float2* sml = reinterpret_cast<float2*>(sm_w + 4 * N);        // [N]
  float* sfac = reinterpret_cast<float*>(sml + N);              // [N] rescaling of O and the sums
  uint32_t* snf = reinterpret_cast<uint32_t*>(sfac + N);        // [3][64][NG]
  // the other ranks' parts at the end: behind this one's in the ring, or over P
  constexpr bool in_ring = C::kOut + kJoin<HD, N> <= NST * C::kUnit;
  uint8_t* sjoin = in_ring ? sring + C::kOut : sp;
  static_assert(in_ring || kJoin<HD, N> <= DB * C::kP + C::kQ, "room for the other ranks' parts");

  // TMA: the units in the order in which the MMAs release them
  if (tid == 4 * G * 32) {
    s_abort[0] = 0, s_abort[kLimitAt] = p.wait.ns;
    *s_any = 0;
    s_stop[0] = s_stop[1] = 0;
    for (int i = 0; i < NST; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 1);
    mbar_fence_init();
  }
  if (p.part != TreeAttnParams::kSecond) pdl_wait();  // nothing before this touches global memory
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
  const int t0 = (int)((int64_t)n_tiles * rank / p.S), t1 = (int)((int64_t)n_tiles * (rank + 1) / p.S);
  const int n_own = t1 - t0, n_units = 2 * H * n_own;
  // The ring's order, in halves (K or V) of the CTA's tiles: K0 K1 V0 K2 V1 ..
  auto k_unit = [&](int t) { return H * (t == 0 ? 0 : 2 * t - 1); };
  auto v_unit = [&](int t) { return H * (t == n_own - 1 ? 2 * t + 1 : 2 * t + 2); };
  auto request = [&](int i) {
    const int j = i / H, u = i % H, slot = i % NST;
    const bool val = j > 0 && (!(j & 1) || j == 2 * n_own - 1);
    const int t = t0 + (j == 2 * n_own - 1 ? n_own - 1 : val ? j / 2 - 1 : (j + 1) / 2);
    const bool tree = t >= n_pre;
    const CUtensorMap* map = val ? (tree ? &tp.tv : &tp.cv) : (tree ? &tp.tk : &tp.ck);
    mbar_expect_tx(full + slot, C::kUnit);
    tma_box(sring + slot * C::kUnit, map, 64 * u, tree ? 0 : t * BK, hkv * (tree ? tp.t_head : tp.c_head),
            b * (tree ? tp.t_seq : tp.c_seq), full + slot);
  };
  if (warp == 4 * G) {  // the ring's barriers are this warp's own: the first units are on their way at once
    if (lane == 0)
#pragma unroll 1
      for (int i = 0; i < NST && i < n_units; ++i) request(i);
  } else if (warp == 4 * G + 1) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) mbar_init(s_full + i, 1), mbar_init(p_full + i, 128 * G + p.wait.missing);
      mbar_init(o_done, 1), mbar_init(o_done + 1, 1);
      mbar_init(drain, 1);
      mbar_fence_init();
    }
    __syncwarp();
    // (after pdl_wait: held earlier, it could be what the kernel before this one is waiting for. A second part takes
    // it while the first still may: both find room on an SM, see tmem_fits)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                 "r"((uint32_t)C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    // the query rows' bf16 parts, 128-byte rows of 64 dims, chunks permuted as by TMA's 128-byte swizzle
    if (p.tree.k)
      for (int i = tid; i < kTreeMaxNodes; i += 128 * G)
        smask[i] = i < cnt ? p.mask[(int64_t)b * p.mask_seq + i] : 0;
#pragma unroll 4
    for (int i = tid; i < N * (HD / 8); i += 128 * G) {
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
    for (int i = tid; i < C::kOnes / 16; i += 128 * G)
      reinterpret_cast<uint4*>(sones)[i] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    if (p.tree.k && t1 == n_tiles)
      for (int i = tid; i < 3 * kTreeMaxNodes * NG; i += 128 * G) snf[i] = 0;
    for (int i = tid; i < N; i += 128 * G) sm_m[i] = -kNone;
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;  // S of block g and buffer d at columns (d G + g) NS, O of 64 dims u at DB G NS + (u G + g) NO
  uint64_t seen = 0;              // tree rows that some node sees
  if (p.tree.k) {
    const uint64_t a = smask[lane] | smask[lane + 32];
    seen = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(a >> 32)) << 32) |
           __reduce_or_sync(0xffffffffu, (uint32_t)a);
    if (cnt < 64) seen &= (1ull << cnt) - 1;
  }
  // Steps of 16 keys of own tile t that hold a visible one: P is 0 behind them.
  auto steps = [&](int t) {
    const int n = t0 + t >= n_pre ? 64 - __clzll((long long)seen) : min(BK, len - (t0 + t) * BK);
    return max(1, (n + 15) / 16);
  };

  // P V of own tile t. With two buffers a barrier for each: a wait for the last but one, once it has handed
  // over the last one's P, would otherwise come too late when both are over, and see the phase behind them.
  auto pv_bar = [&](int t) { return o_done + (DB == 2 ? t & 1 : 0); };
  auto pv_parity = [&](int t) { return (uint32_t)(DB == 2 ? t >> 1 : t) & 1; };

  int sent = min(NST, n_units);  // by the TMA lane
  if (warp == 4 * G) {
    if (lane == 0) {
      for (int& i = sent; i < n_units; ++i) {
        if (!tc_wait(empty + i % NST, (i / NST - 1) & 1, s_abort, p.status)) break;
        request(i);
      }
    }
  } else if (warp == 4 * G + 1) {
    // ---- MMA: commits release units and publish scores
    constexpr uint32_t base_i = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);  // fp32 += bf16 x bf16, 128 rows
    constexpr uint32_t idesc_s = base_i | ((uint32_t)(C::NSA >> 3) << 17);
    constexpr uint32_t idesc_o = base_i | ((uint32_t)(C::NOA >> 3) << 17) | (1u << 15) | (1u << 16);  // A and B MN-major
    constexpr uint64_t swp = C::kRowP == 128 ? 2 : (C::kRowP == 64 ? 4 : 6);
    constexpr uint32_t step_p = 16 * C::kRowP, sbo_p = 8 * C::kRowP;
    const uint32_t uq = smem_u32(sq), up = smem_u32(sp), ur = smem_u32(sring), uo = smem_u32(sones);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    bool ok = true;
#pragma unroll 1
    for (int t = -DB; t < n_own && ok; ++t) {
      const int x = DB == 2 ? t & 1 : 0;
      if (t >= 0) ok = tc_wait_warp(p_full + x, (DB == 2 ? t >> 1 : t) & 1, s_abort, p.status);
      // S of tile t0 + t + DB goes into the buffer just read. With one buffer it
      // is first: the softmax goes on with it while O is brought up to date
      // (16 x 64 nodes over 1024..8192 rows: 91.4 us so, 99.8 with it second).
#pragma unroll
      for (int first = 1; first >= 0; --first) {
        if ((first == 1) == (DB == 1)) {
          if (t + DB >= n_own) continue;
#pragma unroll 1
          for (int u = 0; u < H; ++u) {
            const int i = k_unit(t + DB) + u, slot = i % NST;
            ok = ok && tc_wait_warp(full + slot, (i / NST) & 1, s_abort, p.status);
            if (!ok) break;
            tc_fence_after();
            const uint64_t da = tc_desc(ur + slot * C::kUnit, 16, 1024, 2);
            const uint64_t dq = tc_desc(uq + u * C::NSA * 128, 16, 1024, 2);
            if (elect_lane()) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)  // 16 dims: 32 bytes further
                tc_mma(tm + x * C::NSA, da + 2 * ks, dq + 2 * ks, idesc_s, u > 0 || ks > 0);
            }
            __syncwarp();
            tc_commit(empty + slot);
          }
          if (ok) tc_commit(s_full + x);
        } else if (t >= 0) {  // O += V^T P^T of tile t0 + t, from buffer x
          const int n_steps = steps(t);
#pragma unroll 1
          for (int u = 0; u < H; ++u) {
            const int i = v_unit(t) + u, slot = i % NST;
            ok = ok && tc_wait_warp(full + slot, (i / NST) & 1, s_abort, p.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t v = ur + slot * C::kUnit;
            // the second 64 rows of V are the ones: a fixed place, so the leading offset falls as the start rises
            const uint64_t da = tc_desc(v, uo - v, 1024, 2);
            const uint64_t dp = tc_desc(up + x * C::kP, BK * 128, sbo_p, swp);
            if (elect_lane()) {
#pragma unroll
              for (int ks = 0; ks < BK / 16; ++ks)  // 16 keys: 2 KB further
                if (ks < n_steps)
                  tc_mma(tm + DB * C::NSA + u * C::NOA, da + ks * (uint64_t)128 - ((uint64_t)(ks * 128) << 16),
                         dp + (ks * step_p >> 4), idesc_o, (F32 ? t % kTogether : t) > 0 || ks > 0);
            }
            __syncwarp();
            tc_commit(empty + slot);
          }
          if (ok) tc_commit(o_done + x);
        }
      }
    }
  } else {
    // ---- softmax: thread = key
    const int g = warp >> 2, key = (warp & 3) * 32 + lane;
    uint32_t tS = tmem + ((uint32_t)(warp & 3) << 21) + g * C::NS;
    const uint32_t tO = tmem + ((uint32_t)(warp & 3) << 21) + DB * C::NSA + g * C::NO;  // of 64 dims u: + u NOA
    float* m = sm_m + g * NB;  // the references, negated
    if (p.tree.k)
      for (int r = key; r < NB; r += 128) {
        const int node = p.by_gq.div(m0 + g * NB + r);
        srow[g * NB + r] = node < cnt ? smask[node] & seen : 0;
      }
    group_sync(g);
    constexpr int W = NB >= 32 && NQ == 1 ? 32 : 16;
    auto load = [&](float (&v)[NQ][W], int c0) {
#pragma unroll
      for (int k = 0; k < NQ; ++k) tc_ld(v[k], tS + k * NB + c0);
    };
    auto ready = [&](float (&v)[NQ][W]) {  // waits, and adds the parts, the small ones first
#pragma unroll
      for (int k = 0; k < NQ; ++k) tc_wait_ld(v[k]);
      if constexpr (NQ == 3)
#pragma unroll
        for (int j = 0; j < W; ++j) v[0][j] += v[1][j] + v[2][j];
    };
    float acc[F32 ? H : 1][16];  // fp32: O of the tiles that have left tensor memory
    static_assert(!F32 || NB == 16, "a thread's sums");
    auto part_of = [&](float (&x)[16], uint32_t at) {  // this thread's O, its parts added, the small ones first
      float v[NP][16];
#pragma unroll
      for (int k = 0; k < NP; ++k) tc_ld(v[k], at + k * NB);
#pragma unroll
      for (int k = 0; k < NP; ++k) tc_wait_ld(v[k]);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[j] = v[NP - 1][j];
#pragma unroll
        for (int k = NP - 2; k >= 0; --k) x[j] += v[k][j];
      }
    };
    if constexpr (F32)
#pragma unroll
      for (int u = 0; u < H; ++u)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[u][j] = 0.f;
    for (int t = t0; t < t1; ++t) {
      const bool tree = t >= n_pre, whole = !tree && (t + 1) * BK <= len;
      const bool valid = tree ? key < kTreeMaxNodes && ((seen >> (key & 63)) & 1) : t * BK + key < len;
      const int x = DB == 2 ? (t - t0) & 1 : 0;
      const bool failed = !tc_wait_warp(s_full + x, (DB == 2 ? (t - t0) >> 1 : t - t0) & 1, s_abort, p.status);
      tc_fence_after();
      if constexpr (DB == 2) tS = tmem + ((uint32_t)(warp & 3) << 21) + x * C::NSA + g * C::NS;
      // tree: whether row r of the block sees this thread's tree row
      uint32_t rv[(NB + 31) / 32] = {};
      if (tree)
#pragma unroll
        for (int r0 = 0; r0 < NB; r0 += 32)
          rv[r0 / 32] = transpose_bits(key < kTreeMaxNodes && r0 + lane < NB
                                           ? reinterpret_cast<const uint32_t*>(srow + g * NB + r0 + lane)[warp & 1]
                                           : 0u,
                                       lane);
      auto sees = [&](int r) { return (((NB > 32 && r >= 32 ? rv[NB / 32 - (NB >= 32)] : rv[0]) >> (r & 31)) & 1) != 0; };
      if (t == t0) {  // the references: the score of the first key that a row sees (renewed below if not finite)
        float* first = reinterpret_cast<float*>(sp + x * C::kP) + g * 64 * NB;  // [64][NB], where P comes to lie
        static_assert(64 * N * 4 <= C::kP, "room for the first scores");
        if (!failed && warp < 4 * g + (tree ? 2 : 1))
#pragma unroll 1
          for (int c0 = 0; c0 < NB; c0 += W) {
            float v[NQ][W];
            load(v, c0);
            ready(v);
            if (tree || lane == 0)
#pragma unroll
              for (int j = 0; j < W; j += 4)
                *reinterpret_cast<float4*>(first + key * NB + c0 + j) =
                    make_float4(v[0][j], v[0][j + 1], v[0][j + 2], v[0][j + 3]);
          }
        group_sync(g);
        float y = INFINITY;
        if (key < NB) {  // a thread per row (NB <= 128)
          const int j = tree ? __ffsll(srow[g * NB + key]) - 1 : 0;
          if (j >= 0) y = first[j * NB + key];
          m[key] = fabsf(y) < 1e38f ? -y : -kNone;
        }
        // every block's first scores have been read: P may be written
        asm volatile("bar.sync %0, %1;" ::"r"(3), "n"(128 * G) : "memory");
      }
      uint8_t* prow = sp + x * C::kP + key * C::kRowP;
      const int sel = C::kRowP == 128 ? key & 7 : (C::kRowP == 64 ? (key >> 1) & 3 : (key >> 2) & 1);
      for (;;) {
        if (failed) {  // the block's other warps learn of it where they would renew their references
          group_any(g, true);
          s_stop[g] = 1;
          group_sync(g);
          goto stopped;
        }
        // probabilities with the references as they are; the largest excess over them
        uint32_t top = 0;  // of P's first parts, two at a time
        auto take = [&](float (&v)[NQ][W], int c0) {
          float(&s)[W] = v[0];
          if (tree) {
#pragma unroll
            for (int j = 0; j < W; ++j)
              if (!sees(c0 + j)) s[j] = -INFINITY;
          } else if (!whole && !valid) {
#pragma unroll
            for (int j = 0; j < W; ++j) s[j] = -INFINITY;
          }
          uint32_t part[W / 8][4][NP];
#pragma unroll
          for (int h = 0; h < W / 8; ++h)
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
              const float4 ref = *reinterpret_cast<const float4*>(m + c0 + 8 * h + j);
              float y[4] = {ref.x, ref.y, ref.z, ref.w};
              add2(y[0], y[1], y[0], y[1], s[8 * h + j], s[8 * h + j + 1]);
              add2(y[2], y[3], y[2], y[3], s[8 * h + j + 2], s[8 * h + j + 3]);
              mul2(y[0], y[1], y[0], y[1], p.c);
              mul2(y[2], y[3], y[2], y[3], p.c);
              split_pack<NP>(ex2(y[0]), ex2(y[1]), part[h][j / 2]);
              split_pack<NP>(ex2(y[2]), ex2(y[3]), part[h][j / 2 + 1]);
              top = max_bf16x2(top, max_bf16x2(part[h][j / 2][0], part[h][j / 2 + 1][0]));
            }
          // one buffer of P: the last P V has read it (with two, that of this buffer came before these scores)
          if (DB == 1 && c0 == 0 && t > t0) tc_wait(pv_bar(t - t0 - 1), pv_parity(t - t0 - 1), s_abort, p.status);
#pragma unroll
          for (int h = 0; h < W / 8; ++h)
#pragma unroll
            for (int k = 0; k < NP; ++k) {
              const int chunk = (g * C::NO + k * NB + c0 + 8 * h) / 8;
              *reinterpret_cast<uint4*>(prow + (chunk / 8) * BK * 128 + 16 * ((chunk & 7) ^ sel)) =
                  make_uint4(part[h][0][k], part[h][1][k], part[h][2][k], part[h][3][k]);
            }
        };
        float va[NQ][W], vb[NQ][W];  // the next columns load while these are worked on
        load(va, 0);
#pragma unroll 1
        for (int c0 = 0; c0 < NB; c0 += 2 * W) {
          ready(va);
          if (c0 + W < NB) load(vb, c0 + W);
          take(va, c0);
          if (c0 + W < NB) {
            ready(vb);
            if (c0 + 2 * W < NB) load(va, c0 + 2 * W);
            take(vb, c0 + W);
          }
        }
        constexpr float kLimit = 1152921504606846976.f;  // 2^60
        const bool over = __uint_as_float(top << 16) > kLimit || __uint_as_float(top & 0xFFFF0000u) > kLimit;
        if (!group_any(g, over)) break;
        // renew the references: the maxima per warp, then over the four; rescale O and the sums
#pragma unroll 1
        for (int c0 = 0; c0 < NB; c0 += W) {
          float v[NQ][W];
          load(v, c0);
          ready(v);
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const bool in = tree ? sees(c0 + j) : valid;
            float y = in ? v[0][j] : -INFINITY;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
            if (lane == 0) sm_w[(warp & 3) * N + g * NB + c0 + j] = y;
          }
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
        if (t > t0) {
          tc_wait_together(pv_bar(t - t0 - 1), pv_parity(t - t0 - 1), s_abort, p.status);  // the last P V is in O
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < C::NO * H; c0 += 16) {
            const uint32_t at = tO + (c0 / C::NO) * C::NOA + c0 % C::NO;
            float s[16];
            tc_ld(s, at);
            tc_wait_ld(s);
#pragma unroll
            for (int j = 0; j < 16; ++j) s[j] *= sfac[g * NB + (c0 + j) % NB];
            tc_st16(at, s);
          }
          tc_wait_st();
          if constexpr (F32)
#pragma unroll
            for (int u = 0; u < H; ++u)
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[u][j] *= sfac[g * NB + j];
        }
      }
      if constexpr (F32) {
        if (t > t0 && (t - t0) % kTogether == 0) {  // the next P V starts anew
          tc_wait_together(pv_bar(t - t0 - 1), pv_parity(t - t0 - 1), s_abort, p.status);
          tc_fence_after();
#pragma unroll
          for (int u = 0; u < H; ++u) {
            float x[16];
            part_of(x, tO + u * C::NOA);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[u][j] += x[j];
          }
        }
      }
      if (!whole) {
        // V rows that are not there become zeros, non-finite tree values too (noted for the
        // rows that see them), in the steps that are multiplied. After the last P V, so that
        // the slot's last unit has been read and its barrier is in this unit's phase.
        if (t > t0) tc_wait(pv_bar(t - t0 - 1), pv_parity(t - t0 - 1), s_abort, p.status);
        for (int u = 0; u < H; ++u) {
          const int i = v_unit(t - t0) + u;
          tc_wait(full + i % NST, (i / NST) & 1, s_abort, p.status);
        }
        const int r0 = tree ? 0 : len - t * BK, n_chunks = (16 * steps(t - t0) - r0) * (HD / 8);
#pragma unroll 1
        for (int i = tid; i < n_chunks; i += 128 * G) {
          const int row = r0 + i / (HD / 8), c = i % (HD / 8), slot = (v_unit(t - t0) + c / 8) % NST;
          uint4* at = reinterpret_cast<uint4*>(sring + slot * C::kUnit + row * 128 + 16 * ((c & 7) ^ (row & 7)));
          if (!tree || !((seen >> row) & 1)) {
            *at = make_uint4(0u, 0u, 0u, 0u);
            continue;
          }
          const uint4 w = *at;
          uint32_t inf = 0;  // whether an exponent is all ones
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v = (&w.x)[j] & 0x7F807F80u;
            inf |= (v & 0xFFFFu) == 0x7F80u || (v >> 16) == 0x7F80u;
          }
          if (inf) {
            uint16_t* e = reinterpret_cast<uint16_t*>(at);
#pragma unroll 1
            for (int j = 0; j < 8; ++j)
              if ((e[j] & 0x7F80u) == 0x7F80u) {
                const int kind = (e[j] & 0x7Fu) ? 2 : e[j] >> 15, d = 8 * c + j;
                atomicOr(snf + (kind * kTreeMaxNodes + row) * NG + (d >> 5), 1u << (d & 31));
                e[j] = 0;
              }
            *s_any = 1;
          }
        }
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(p_full + x);
    }
  stopped:
    // ---- O^T and the sums to shared memory, [row][dim]
    if (n_own > 0) tc_wait_together(pv_bar(n_own - 1), pv_parity(n_own - 1), s_abort, p.status);
    tc_fence_after();
    // every block's last MMAs have read the ring and P before any block writes over them
    asm volatile("bar.sync %0, %1;" ::"r"(3), "n"(128 * G) : "memory");
    if (p.S > 1) cluster_arrive();
    float* so = reinterpret_cast<float*>(sm) + g * NB * HD;
    const bool have = t0 < t1 && !__any_sync(0xffffffffu, *s_abort);
#pragma unroll(F32 ? H : 1)
    for (int c0 = 0; c0 < NB * H; c0 += 16) {
      const int u = c0 / NB, r0 = c0 % NB;
      float x[16];
      if (have) {
        part_of(x, tO + u * C::NOA + r0);
        if constexpr (F32)
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] += acc[u][j];
      }
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (!have) x[j] = 0.f;
        if (key < 64) so[(r0 + j) * HD + 64 * u + key] = x[j];
        sum = lane == j ? x[j] : sum;
      }
      // the lanes from 64 on all hold the sums: lane j of the third warp keeps row j's
      if (u == 0 && (warp & 3) == 2 && lane < 16) sml[g * NB + r0 + lane] = make_float2(-m[r0 + lane], sum);
    }
    if (p.tree.k && have && t1 == n_tiles && *s_any && key < 64) {  // non-finite tree values, where they are seen
      for (int d = key; d < HD; d += 64)
        for (int r = 0; r < NB; ++r)
          for (uint64_t v = srow[g * NB + r]; v; v &= v - 1) {
            const int j = __ffsll(v) - 1;
            const float bad[3] = {INFINITY, -INFINITY, NAN};
#pragma unroll
            for (int kind = 0; kind < 3; ++kind)
              if ((snf[(kind * kTreeMaxNodes + j) * NG + (d >> 5)] >> (d & 31)) & 1) so[r * HD + d] += bad[kind];
          }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (warp >= 4 * G && p.S > 1) cluster_arrive();
  join_splits<HD, F32, N, NT>(p, reinterpret_cast<float*>(sm), sml, sjoin, rank, block.seq, hkv, m0, min(N, cnt * p.gq - m0));
  if (warp >= 4 * G && *s_abort) {  // no copy and no product in flight outlives the CTA
    const unsigned long long s0 = globaltimer();
    if (warp == 4 * G && lane == 0)
#pragma unroll 1
      for (int j = max(0, sent - NST); j < sent; ++j)
        while (!mbar_try_wait(full + j % NST, (j / NST) & 1) && globaltimer() - s0 < kWaitLimitNs) {
        }
    __syncwarp();
    if (warp == 4 * G + 1) {
      tc_commit(drain);
      while (!mbar_try_wait(drain, 0) && globaltimer() - s0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  }
  // Freed last: no two CTAs that hold and that wait for tensor memory share an
  // SM (see tmem_fits), so a CTA that holds it while its cluster gathers cannot
  // keep a peer waiting.
  if (warp == 4 * G + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)C::kCols));
  }
}

// cuTensorMapEncodeTiled, looked up once; null where the driver has none.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled tensor_map_encoder() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// The map of one K or V tensor [seq][head][row][dim] of bf16 or int8.
template <int HD, bool Q8>
bool encode_rows(CUtensorMap* map, const uint8_t* base, const KvRows& r, int B, int heads) {
  const EncodeTiled enc = tensor_map_encoder();
  if (!enc) return false;
  if (r.seq == 0) B = 1;
  if (r.head == 0) heads = 1;
  const int64_t row = r.rows > 1 ? r.row : HD;
  const int64_t head = heads > 1 ? r.head : row * r.rows, seq = B > 1 ? r.seq : head * heads;
  const cuuint64_t dims[4] = {(cuuint64_t)HD, (cuuint64_t)r.rows, (cuuint64_t)heads, (cuuint64_t)B};
  const int64_t size = Q8 ? 1 : 2;
  const cuuint64_t strides[3] = {(cuuint64_t)(row * size), (cuuint64_t)(head * size), (cuuint64_t)(seq * size)};
  const cuuint32_t box[4] = {Q8 ? HD : 64, 128, 1, 1}, step[4] = {1, 1, 1, 1};
  return enc(map, Q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint8_t*>(base),
             dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             Q8 && HD == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <int HD, bool Q8>
bool encode_all(TreeAttnTcParams& tp) {
  const TreeAttnParams& p = tp.p;
  tp.c_seq = p.cache.seq != 0, tp.c_head = p.cache.head != 0, tp.t_seq = p.tree.seq != 0, tp.t_head = p.tree.head != 0;
  if (p.cache.rows > 0 && !(encode_rows<HD, Q8>(&tp.ck, p.cache.k, p.cache, p.B, p.Hkv) &&
                            encode_rows<HD, Q8>(&tp.cv, p.cache.v, p.cache, p.B, p.Hkv)))
    return false;
  return p.tree.k == nullptr || (encode_rows<HD, Q8>(&tp.tk, p.tree.k, p.tree, p.B, p.Hkv) &&
                                 encode_rows<HD, Q8>(&tp.tv, p.tree.v, p.tree, p.B, p.Hkv));
}

// Splits of a cluster's keys where a CTA has an SM to itself: least waves of
// clusters (those of 8 and 16 leave SMs of a processing cluster over) times a CTA's
// tiles and its start and join, about five tiles' time. Measured, us for 1, 2, 4,
// 8, 16: 64 clusters of 33 bf16 tiles 61 / 40 / 51; int8, 8 of 33 66 / 41 / 29 / 23 / 33,
// 16 of 129 221 / 119 / 68 / 77 / 76, 24 of 72 83 / 50 / 33 / 41 / 61.
template <typename AtOnce>
int lone_splits(int64_t clusters, int tiles, AtOnce at_once) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= kMaxSplits && s <= tiles; s *= 2) {
    const int n = at_once(s);
    if (n <= 0) continue;
    const int64_t t = (clusters + n - 1) / n * ((tiles + s - 1) / s + 5);
    if (t < least) least = t, best = s;
  }
  return best;
}

// Clusters of a launch (but for their splits) that have rows. Of groups that share the sequences, most blocks of
// the grid have none: it is as wide as if any one of them had all.
inline int64_t busy_clusters(const TreeAttnParams& p, int m_tiles) {
  return (int64_t)p.Hkv * (p.part == TreeAttnParams::kFirst ? m_tiles + p.B - 1 : (int64_t)p.B * m_tiles);
}

template <int HD, bool F32, int NB, int G>
cudaError_t launch_tree_tc_t(TreeAttnTcParams& tp, int n_sm, cudaStream_t st) {
  using C = TreeTc<HD, F32, NB, G>;
  const auto kern = tree_attn_tc_kernel<HD, F32, NB, G>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(kern, C::kSmem, true);
  if (e != cudaSuccess) return e;
  TreeAttnParams& p = tp.p;
  const int m_tiles = (p.nodes * p.gq + C::N - 1) / C::N;
  const int64_t clusters = busy_clusters(p, m_tiles);
  const int tiles = (p.cache.rows + C::BK - 1) / C::BK + 1;
  int S = 1;
  if constexpr (C::two) {
    // Split the keys until every SM has a CTA, and to fill both places while 16
    // tiles are left for each: more splits cost their merges
    // (32 sequences x 8 kv heads, 17 tiles: 37 / 39 / 45 us for 1 / 2 / 3; 16 x 4 x 4 row
    // tiles, 65 tiles: 104 / 85 / 94 / 102 for 1 to 4; 32 clusters of 34 fp32 tiles 12.3 /
    // 12.1 / 24 for 4 / 8 / 16).
    // The first of two parts: two tiles or more a CTA and eight splits at most, since the second part's CTAs want
    // places too (16 sequences of 2 rows, 8 kv heads x 128 behind 4096 rows: 16.0 / 21.8 us for 8 / 16; 32 of them
    // behind 512 12.5 / 12.4 / 15.2 for 2, 4, 8; 8 of 8 rows, 4 x 64 behind 2048 11.3 / 17.2 for 8 / 16).
    const int most = p.part == TreeAttnParams::kFirst ? std::min(8, (tiles + 1) / 2) : std::min(kMaxSplits, tiles);
    while ((p.part == TreeAttnParams::kFirst ? 2 * S <= most : S < most) && (clusters * S < n_sm || (clusters * S < 2 * n_sm && tiles / (2 * S) >= 16))) S *= 2;
  } else {
    static ClusterCount at_once;
    S = lone_splits(clusters, tiles, [&](int s) { return at_once.get(kern, s, C::NT, C::kSmem); });
  }
  p.S = S;
  p.sorted = p.B > 1 && p.B <= 64;
  return launch_cluster(kern, dim3(S, p.Hkv * m_tiles, p.B), C::NT, S, C::kSmem, st, tp, p.pdl);
}

// bf16 rows
template <int HD>
cudaError_t launch_tree_tc(const TreeAttnParams& p, bool f32, int n_sm, cudaStream_t st) {
  TreeAttnTcParams tp;
  tp.p = p;
  if (!encode_all<HD, false>(tp)) return cudaErrorNotSupported;
  // Rows of a CTA: as many as there are (K and V are read once for them), in two
  // blocks once there are 32 (one block's softmax overlaps the other's MMAs); but
  // fewer while the clusters, split eight ways, would leave SMs without a CTA
  // (16 nodes x 8 heads over 4097 rows, fp32: 16 / 32 rows 12.1 / 14.2 us).
  // 128 rows at most (16 x 64 nodes over 1024..8192 rows: 32 / 64 / 128 rows 155 / 147 /
  // 85 us): 256 would fill tensor memory and leave one CTA on an SM.
  const int M = p.nodes * p.gq, most = f32 ? 32 : 128;
  int N = 16;
  while (N < M && N < most) N *= 2;
  while (N > 16 && busy_clusters(p, (M + N - 1) / N) * 8 < n_sm) N /= 2;
  if (f32)
    return N == 16 ? launch_tree_tc_t<HD, true, 16, 1>(tp, n_sm, st) : launch_tree_tc_t<HD, true, 16, 2>(tp, n_sm, st);
  return N == 16   ? launch_tree_tc_t<HD, false, 16, 1>(tp, n_sm, st)
         : N == 32 ? launch_tree_tc_t<HD, false, 16, 2>(tp, n_sm, st)
         : N == 64 ? launch_tree_tc_t<HD, false, 32, 2>(tp, n_sm, st)
                   : launch_tree_tc_t<HD, false, 64, 2>(tp, n_sm, st);
}

}  // namespace llmq
