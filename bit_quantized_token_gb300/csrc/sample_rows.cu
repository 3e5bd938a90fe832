// The next token of every row of logits, under the row's own options and from a
// given uniform number (see serve.cuh).
//
// Tokens in order, the largest logit first, equal ones by id; w_j = 2^(-Y_j), Y_j =
// (l_0 - l_j) log2(e) / T. Every option keeps a prefix of that order: the first
// top_k; of those the shortest whose mass reaches top_p of theirs; the w_j of at least
// min_p. The token is the first one whose cumulative mass passes u times the kept
// one's. So nothing is sorted but what lies around the borders:
//   1. a histogram over -l log2(e) / T, 32 buckets an octave (finer for high
//      temperatures): the count and the mass of every bucket, in one pass, whose
//      window hangs on the largest of the first logits;
//   2. from the running sums below the row's largest logit, the few buckets in which
//      the borders can lie (the border of one option moves the next one's by a
//      bucket's mass at most);
//   3. a second pass brings their tokens, some hundreds, to the first CTA, which
//      sorts them and finds all borders exactly.
// A window that turns out too low, or too narrow, or buckets that hold more than
// kSampleList tokens around the borders (flat rows), are set again from the row's exact
// range, once. Rows that still have more there (crowds of equal logits) take the long
// way: each border by three digits of the logits' keys, over all tokens (256 x 151936
// 2.9 ms). So do rows whose largest logit is 32768 octaves or more from 0 (1.5 ms).
//
// Masses decide integers, so they are integers: a term is a number of 2^-34 steps
// below its bucket's largest, from the exact product of logit and temperature in a
// pair of floats and then in fixed point; sums have 2^-44 steps, in 64 bits, whatever
// their order. Terms below 2^-4 of the largest have their place in the bucket in fp32,
// whose roundings (of the place, of the polynomial, of their product: 11, 16 and 16 of
// those steps, with the rest 45) leave them 28 bits. They are of either sign: over
// rows of normal logits a border is off by 2^-35 of the row's mass, of bf16 ones by
// 2^-34, of thousands of equal ones in the tail by 2^-30. Of 150,000 borders, one draw
// in some 10^5 .. 10^6 falls on another side than with exact sums; fp32 sums would lose one draw
// in 2,000, and fp64 has 1/64 of fp32's lanes here.
//
// Measured at temperature 0.8 and top-p 0.95: 1 x 32000 15.8 us (of which the CTAs' exchanges and the sort of some
// hundred entries about 12), 32 x 151936 37.5, 256 x 151936 130 (rows of mixed options 38, temperatures 0.7 and 1 with
// min-p 144): two passes of some 70 instructions a warp's 32 logits, 64 % of the issue slots, HBM at 25 %. The second
// pass reads memory again (156 MB of rows and 129 MB of L2). A form
// that kept the logits in shared memory, and so took up to 16 CTAs a row, needed 391 us for the last.
#include <cooperative_groups.h>

#include "common.cuh"
#include "op_call.cuh"
#include "sample_key.cuh"
#include "serve.cuh"

namespace llmq {
namespace cg = cooperative_groups;
namespace {

using u64 = unsigned long long;
constexpr int kSampNT = 512;
constexpr int kSampB = 2048;           // buckets below the row's largest logit: 64 octaves (fewer, finer ones)
constexpr int kSampTable = 2 * kSampB; // a CTA's buckets, by their number modulo the table
constexpr int kSampPer = kSampB / kSampNT;
constexpr int kSampMaxSlice = 180000;
constexpr int kSampU = 8;               // loads of a thread in flight
constexpr float kLargest = 3.402823466e38f;  // what an infinite logit counts as
constexpr int kSortRegs = 4;            // entries of a thread that are sorted in registers

__constant__ const u64 kRoot32[32] = {  // 2^(63 - j/32)
    0x8000000000000000ull, 0x7D41D96DB915019Dull, 0x7A92BE8A92436616ull, 0x77F25CCDEE6D7AE6ull,
    0x75606373EE921C97ull, 0x72DC8373BE41A454ull, 0x70666F76154A7089ull, 0x6DFDDBCBED791BABull,
    0x6BA27E656B4EB57Aull, 0x69540EC8F895722Dull, 0x6712460A8FC24072ull, 0x64DCDEC3371793D1ull,
    0x62B39508AA836D6Full, 0x6096266533384A2Bull, 0x5E8451CFAC061B5Full, 0x5C7DD7A3B17DCF75ull,
    0x5A827999FCEF3242ull, 0x5891FAC0E95612C8ull, 0x56AC1F752150A563ull, 0x54D0AD5A753E077Cull,
    0x52FF6B54D8A89C75ull, 0x513821818624B40Cull, 0x4F7A993048D088D7ull, 0x4DC69CDCEAA72A9Cull,
    0x4C1BF828C6DC54B8ull, 0x4A7A77D47F7B84B1ull, 0x48E1E9B9D588E19Bull, 0x47521CC5A2E6A9E0ull,
    0x45CAE0F1F545EB73ull, 0x444C0740496D4294ull, 0x42D561B3E6243D8Aull, 0x4166C34C5615D0ECull};


struct SampShared {
  union {
    struct {                     // this CTA's histogram
      uint32_t lo[kSampTable];   // how far its terms lie below a bucket's largest, in 2^-34 steps, added up
      uint32_t hi[kSampTable];   // their number (18 bits), carries of lo (14 bits: a term's is below 2^28.5)
    };
    uint32_t h[3][kSampB];       // the long way's: sums of the terms' low and high words, counts
    struct {
      u64 local[kSampleList];    // entries of this CTA; later, on the first, the list's running masses
      uint32_t start[kSampB];    // first entry of a bucket
      uint16_t bucket[kSampleList];
    };
  };
  u64 mass[kSampB];              // running sums over the buckets, inclusive
  uint32_t count[kSampB];
  u64 list[kSampleList];         // of the first CTA: every CTA's entries, (key, complement of the id)
  uint8_t flag[kSampB];          // the bucket is gathered
  u64 best[16];                  // greedy: every CTA's largest (key, complement of the id)
  float4 range[16];              // of every CTA: largest logit, least in its window, largest outside, first bucket
  u64 warp64[kSampNT / 32];
  uint32_t warp32[kSampNT / 32];
  float3 warpf[kSampNT / 32];
  int found;
  uint32_t total, n_local, n_list, base;
  // the options
  float ch, cl, u;               // log2(e) / T
  double y_min;                  // -log2(min_p)
  u64 p_fix;                     // top_p in 2^-64 steps; 0: off
  int top_k, greedy, by_m;       // by_m: min_p leaves something out
  // answers
  u64 res_mass[3];
  uint32_t res_rank[2];
  u64 key;
};

struct Term {
  int b;       // bucket
  uint32_t q;  // place in it, 2^-32 steps
};
// The long way's: Y = (m - l) log2(e) / T in 32 buckets an octave. False: no weight (2^-64 and below).
__device__ __forceinline__ bool term_of(float l, float m, float ch, float cl, Term& t) {
  const float d = __fsub_rn(m, l), bb = __fsub_rn(d, m);
  const float dl = __fsub_rn(__fsub_rn(m, __fsub_rn(d, bb)), __fadd_rn(l, bb));  // m - l = d + dl, exactly
  const float p = __fmul_rn(d, ch), y = __fmul_rn(p, 32.f);
  if (!(y < (float)kSampB + 1.f)) return false;
  float e = __fmaf_rn(d, ch, -p);
  e = __fmaf_rn(d, cl, e);
  e = __fmaf_rn(dl, ch, e);
  const float fl = floorf(y);
  const long long q = (long long)__float2uint_rn((y - fl) * 4294967296.f) + __float2int_rn(e * 137438953472.f);
  t.b = (int)fl + (int)(q >> 32);  // (the remainder may take it past a border)
  t.q = (uint32_t)q;
  return t.b >= 0 && t.b < kSampB;
}
// -l log2(e) / T in S buckets an octave (ch, cl times S), |y| below 2^22: the bucket's number and place.
__device__ __forceinline__ Term place_of(float l, float chS, float clS) {
  const float p = __fmul_rn(-l, chS), fl = floorf(p);
  float e = __fmaf_rn(-l, chS, -p);
  e = __fmaf_rn(-l, clS, e);
  const long long q = (long long)__float2uint_rn((p - fl) * 4294967296.f) + __float2int_rn(e * 4294967296.f);
  return {(int)fl + (int)(q >> 32), (uint32_t)q};
}
// 2^37 (1 - 2^-z) for the place q of a bucket: z - z^2/2 + z^3/6 - .. in fixed point
__device__ __forceinline__ uint32_t below37(uint32_t q, int fine) {
  const uint32_t z = __umulhi(q, 2977044472u) >> fine;  // 2^37 ln(2) / S: below 2^31.5
  uint32_t a = ~__umulhi(z, 26843546u);                 // 1 - z/5
  a = ~__umulhi(z >> 7, a);                             // 1 - z/4 ..
  a = ~__umulhi(__umulhi(z, 44739243u), a);
  a = ~__umulhi(z >> 6, a);
  return __umulhi(z, a);
}
__device__ __forceinline__ uint32_t below(uint32_t q, int fine) { return (below37(q, fine) + 4) >> 3; }
// a 2^-34 steps of the largest term of bucket b, in 2^-44 steps of the largest of bucket 0
__device__ __forceinline__ u64 weight_of(u64 a, int b, int fine) {
  a <<= 10;
  if (fine) {
    const int lo = b & ((1 << fine) - 1);
    if (lo) a = __umul64hi(a, ((1ull << 37) - below37((uint32_t)lo << (32 - fine), 0)) << 27);
    b >>= fine;
  }
  const u64 r = __umul64hi(a, kRoot32[b & 31]);
  const int s = (b >> 5) - 1;
  return s < 0 ? r << 1 : s == 0 ? r : (r + (1ull << (s - 1))) >> s;
}
__device__ __forceinline__ u64 weight_of(const Term& t, int fine) { return weight_of((1ull << 34) - below(t.q, fine), t.b, fine); }
__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
__device__ __forceinline__ u64 shfl_up64(u64 v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

// Inclusive sums over the CTA's threads.
__device__ __forceinline__ void scan2(u64& a, uint32_t& c, SampShared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = shfl_up64(a, o);
    const uint32_t y = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) a += x, c += y;
  }
  if (lane == 31) s.warp64[warp] = a, s.warp32[warp] = c;
  __syncthreads();
  u64 x = lane < warp ? s.warp64[lane & 15] : 0;
  uint32_t y = lane < warp ? s.warp32[lane & 15] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
  }
  a += x, c += y;
  __syncthreads();  // the warps' sums have been read
}

// ceil(mass f 2^-64)
__device__ __forceinline__ u64 ceil_part(u64 mass, u64 f) { return __umul64hi(mass, f) + (mass * f != 0); }
// The first of kSampB rising values at which f holds (kSampB: none), by a warp.
template <typename F>
__device__ __forceinline__ int first_at(F f) {
  const int lane = threadIdx.x & 31;
  constexpr int Q = kSampB / 32;
  const unsigned c = __ballot_sync(0xffffffffu, f(Q * lane + Q - 1));
  if (!c) return kSampB;
  const int at = Q * (__ffs(c) - 1);
  static_assert(Q == 64, "two a lane");
  const bool odd = f(at + 2 * lane + 1), even = f(at + 2 * lane);
  const int l = __ffs(__ballot_sync(0xffffffffu, odd)) - 1;
  return at + 2 * l + !__shfl_sync(0xffffffffu, even, l);
}

// Entries e 512 + tid in v[e], sorted from the largest on (bitonic; n2, a power of two, from 32 on, or 512 E with
// E > 1: those that are not 0). buf: room for 512 E.
template <int E>
__device__ __forceinline__ void sort_list(u64 (&v)[kSortRegs], u64* buf, int n2) {
  const int tid = threadIdx.x;
#pragma unroll 1
  for (int k = 2; k <= n2; k *= 2)
#pragma unroll 1
    for (int j = k / 2; j > 0; j /= 2) {
      if (E > 1 && j >= kSampNT) {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int f = e + 1; f < E; ++f)
            if ((e ^ f) == j / kSampNT && (v[e] < v[f]) == (((e * kSampNT) & k) == 0)) {
              const u64 x = v[e];
              v[e] = v[f], v[f] = x;
            }
        continue;
      }
      u64 o[E];
      if (j >= 32) {
#pragma unroll
        for (int e = 0; e < E; ++e) buf[e * kSampNT + tid] = v[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = buf[e * kSampNT + (tid ^ j)];
        __syncthreads();
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = (u64)__shfl_xor_sync(0xffffffffu, v[e], j);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool larger = (((e * kSampNT + tid) & k) == 0) == ((tid & j) == 0);  // keeps the larger one
        v[e] = (o[e] > v[e]) == larger ? o[e] : v[e];
      }
    }
}

// The same for more, N of them, in shared memory (a function of its own: with eight entries a thread
// the ordinary way's registers spilled, 2 us of every call).
__device__ __noinline__ void sort_long(u64* list, const u64* in, int N) {
  const int tid = threadIdx.x;
#pragma unroll 1
  for (int i = tid; i < kSampleList; i += kSampNT) list[i] = i < N ? in[i] : 0;
  __syncthreads();
#pragma unroll 1
  for (int k = 2; k <= kSampleList; k *= 2)
#pragma unroll 1
    for (int j = k / 2; j > 0; j /= 2) {
#pragma unroll 1
      for (int i = tid; i < kSampleList / 2; i += kSampNT) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;  // pairs of places that differ in the bit j
        const u64 x = list[lo], y = list[hi];
        if ((x < y) == ((lo & k) == 0)) list[lo] = y, list[hi] = x;
      }
      __syncthreads();
    }
}

// The long way: the borders of top_k (or all tokens), top_p and the draw in turn, each by
// three digits of the keys from the top, over all tokens. m: the row's largest logit.
// (A function of its own, so that the ordinary way has its registers to itself.)
__device__ __noinline__ void sample_crowd(const SampleRowsParams& p, SampShared& s, float m) {
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31;
  const int first = rank * p.slice, n = max(min(p.V - first, p.slice), 0);
  const float* src = p.logits + (int64_t)row * p.stride + first;
  const float ch = s.ch, cl_ = s.cl;
  const bool by_k = s.top_k > 0, by_p = s.p_fix != 0, by_m = s.by_m;
  const u64 u_fix = __float2ull_rn(s.u * 18446744073709551616.f);
  auto logit = [&](int i) {
    const float l = i < n ? src[i] : -INFINITY;
    return l != l ? -INFINITY : fminf(l, kLargest);
  };
  if (tid == 0) s.key = by_m ? (u64)(s.y_min * 137438953472.0) : 0ull;  // of 32 buckets an octave, from the largest logit
  cl.sync();
  const int bm = by_m ? (int)min(s.key >> 32, (u64)kSampB) : kSampB;
  const uint32_t qm = (uint32_t)s.key;
  uint32_t kept = 0;
  u64 mass = 0;
  uint32_t key = 0, above = 0, equal = 0;  // a border's key, tokens above it and of it
  u64 mass_above = 0, each = 0;            // mass above it, and of one token of it
#pragma unroll 1
  for (int turn = 0; turn < 3; ++turn) {
    if (turn == 1 && !by_p) continue;
    if (turn == 0 ? !by_k : turn == 2 && by_m) {  // tokens and mass of all, or that min_p keeps
      u64 a = 0;
      uint32_t c = 0;
#pragma unroll 1
      for (int i0 = tid; i0 < n; i0 += 4 * kSampNT) {
        float l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) l[e] = logit(i0 + e * kSampNT);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          Term t;
          if (term_of(l[e], m, ch, cl_, t) && (turn == 0 || t.b < bm || (t.b == bm && t.q <= qm)))
            a += weight_of(t, 0), ++c;
        }
      }
      scan2(a, c, s);
      if (tid == kSampNT - 1) s.list[0] = a, s.list[1] = c;
      cl.sync();
      a = 0, c = 0;
      for (int k = 0; k < C; ++k) {
        const u64* o = cl.map_shared_rank(s.list, k);
        a += o[0], c += (uint32_t)o[1];
      }
      if (turn == 0 || c < kept) kept = c, mass = a;
      cl.sync();
      if (turn == 0) continue;
    }
    // found is where the count (turn 0) or the mass (1) reaches the target, or the mass passes it (2)
    const u64 target = turn == 0 ? (u64)s.top_k : turn == 1 ? ceil_part(mass, s.p_fix) : __umul64hi(mass, u_fix);
    auto over = [&](u64 m_, uint32_t n_) { return turn == 0 ? n_ >= target : turn == 1 ? m_ >= target : m_ > target; };
    // A digit's bins are few and full (the highest one is the exponent), so a warp's terms of one bin are added
    // first, for up to four bins
    auto put = [&](bool in, uint32_t bin, u64 w) {
      unsigned left = __ballot_sync(0xffffffffu, in);
      auto add = [&](u64 w, uint32_t n_) {
        const uint32_t lo32 = (uint32_t)w, old = atomicAdd(&s.h[0][bin], lo32);
        atomicAdd(&s.h[1][bin], (uint32_t)(w >> 32) + (old + lo32 < old));
        atomicAdd(&s.h[2][bin], n_);
      };
#pragma unroll 1
      for (int r = 0; r < 4 && left; ++r) {
        const int leader = __ffs(left) - 1;
        const uint32_t one = __shfl_sync(0xffffffffu, bin, leader);
        const unsigned same = __ballot_sync(0xffffffffu, in && bin == one);
        const bool mine = in && bin == one;
        const uint32_t lo = __reduce_add_sync(0xffffffffu, mine ? (uint32_t)w & 0x3FFFFFu : 0u);
        const uint32_t hi = __reduce_add_sync(0xffffffffu, mine ? (uint32_t)(w >> 22) : 0u);  // (below 2^27)
        if (lane == leader) add(((u64)hi << 22) + lo, __popc(same));
        left &= ~same;
      }
      if (left >> lane & 1) add(w, 1u);
    };
    key = above = 0, mass_above = 0;
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bins = level == 2 ? 1024 : 2048;
      const uint32_t prefix_mask = level == 0 ? 0u : level == 1 ? 0xFFE00000u : 0xFFFFFC00u;
      for (int i = tid; i < 3 * kSampB; i += kSampNT) (&s.h[0][0])[i] = 0;
      if (tid == 0) s.found = -1;
      __syncthreads();
#pragma unroll 1
      for (int i0 = tid; i0 - lane < n; i0 += 4 * kSampNT) {
        float l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) l[e] = logit(i0 + e * kSampNT);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          Term t;
          const uint32_t k = sample_key(l[e]);
          const bool in = (k & prefix_mask) == key && term_of(l[e], m, ch, cl_, t);
          const u64 w = in ? weight_of(t, 0) : 0;
          put(in, (k >> shift) & (bins - 1), w);
        }
      }
      cl.sync();
      // a CTA adds up its share of the bins, in descending order, for all
      const int share = bins / C;
      for (int i = tid; i < share; i += kSampNT) {
        const int j = rank * share + i, bin = bins - 1 - j;
        u64 w = 0;
        uint32_t c = 0;
#pragma unroll 8
        for (int k = 0; k < C; ++k) {
          const uint32_t(*h)[kSampB] = cl.map_shared_rank(&s.h[0], k);
          w += ((u64)h[1][bin] << 32) + h[0][bin];
          c += h[2][bin];
        }
        for (int k = 0; k < C; ++k) {
          cl.map_shared_rank(s.mass, k)[j] = w;
          cl.map_shared_rank(s.count, k)[j] = c;
        }
      }
      cl.sync();
      u64 a[kSampPer], sum = 0;
      uint32_t c[kSampPer], cnt = 0;
#pragma unroll
      for (int i = 0; i < kSampPer; ++i) {
        const int j = kSampPer * tid + i;
        a[i] = j < bins ? s.mass[j] : 0, c[i] = j < bins ? s.count[j] : 0;
        sum += a[i], cnt += c[i];
      }
      u64 up = sum;
      uint32_t nup = cnt;
      scan2(up, nup, s);
      if (tid == kSampNT - 1) s.total = nup;
      __syncthreads();
      up -= sum, nup -= cnt;
      // the first non-empty bin over the target; if there is none, the last non-empty one
#pragma unroll
      for (int i = 0; i < kSampPer; ++i) {
        const bool was = over(mass_above + up, above + nup), is = over(mass_above + up + a[i], above + nup + c[i]);
        const bool last = nup + c[i] == s.total && !is;
        if (c[i] && !was && (is || last)) {
          s.found = bins - 1 - (kSampPer * tid + i);
          s.res_mass[0] = mass_above + up;
          s.res_rank[0] = above + nup;
          s.res_rank[1] = c[i];
        }
        up += a[i], nup += c[i];
      }
      __syncthreads();
      key |= (uint32_t)max(s.found, 0) << shift;
      mass_above = s.res_mass[0], above = s.res_rank[0], equal = s.res_rank[1];
      __syncthreads();  // the result has been read; the sums are of the next level's only behind its first cluster barrier
    }
    Term t;
    each = 0;
    if (term_of(key_float(key), m, ch, cl_, t)) each = weight_of(t, 0);
    if (turn == 0) {
      kept = (uint32_t)min(target, (u64)(above + equal));
      mass = mass_above + (u64)(kept - above) * each;
    } else if (turn == 1) {
      const u64 more = target > mass_above ? target - mass_above : 0;
      const uint32_t j = each ? (uint32_t)min(max((more + each - 1) / each, 1ull), (u64)equal) : equal;
      if (above + j < kept) kept = above + j, mass = mass_above + j * each;
    }
  }
  const u64 target = __umul64hi(mass, u_fix);
  uint32_t j = each && target > mass_above ? (uint32_t)min((target - mass_above) / each, (u64)(equal - 1)) : 0u;
  if (above + j >= kept) j = kept > above ? kept - above - 1 : 0;
  // the j-th token of that key, by id: the CTAs hold ascending ids, their passes too
  int owner = 0;
  for (; owner < C - 1; ++owner) {
    const uint32_t c = cl.map_shared_rank(&s.h[0], owner)[2][key & 1023u];
    if (j < c) break;
    j -= c;
  }
  cl.sync();  // no CTA's shared memory is read from here on
  if (rank != owner) return;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kSampNT) {
    const float l = logit(i0 + tid);
    const bool hit = l != -INFINITY && sample_key(l) == key;
    u64 unused = 0;
    uint32_t c = hit;
    scan2(unused, c, s);
    if (hit && c == j + 1) {
      p.tokens[row] = first + i0 + tid;
      if (p.probs) p.probs[row] = (float)each / (float)mass;
    }
    if (tid == kSampNT - 1) s.total = c;
    __syncthreads();
    if (j < s.total) return;
    j -= s.total;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kSampNT, 2) sample_rows_kernel(const __grid_constant__ SampleRowsParams p) {
  extern __shared__ __align__(16) uint8_t sm_raw[];
  SampShared& s = *reinterpret_cast<SampShared*>(sm_raw);
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto started = cl.barrier_arrive();  // shared memory of another CTA: only once that CTA runs
  auto clear = [&]() {
    uint4* h = reinterpret_cast<uint4*>(s.lo);
    for (int i = tid; i < 2 * kSampTable / 4; i += kSampNT) h[i] = make_uint4(0u, 0u, 0u, 0u);
  };
  clear();
  pdl_wait();
  pdl_trigger();
  const int first = rank * p.slice, n = max(min(p.V - first, p.slice), 0);
  const float* src = p.logits + (int64_t)row * p.stride + first;
  float cur[kSampU];
  auto load = [&](float (&x)[kSampU], int i0) {
    if (i0 + kSampU * kSampNT <= n) {
#pragma unroll
      for (int e = 0; e < kSampU; ++e) x[e] = __ldg(src + i0 + e * kSampNT + tid);
    } else {
#pragma unroll
      for (int e = 0; e < kSampU; ++e) x[e] = i0 + e * kSampNT + tid < n ? __ldg(src + i0 + e * kSampNT + tid) : -INFINITY;
    }
  };
  load(cur, 0);
  if (tid == kSampNT - 1) {
    const float T = p.temperature ? p.temperature[row] : 1.f, P = p.top_p ? p.top_p[row] : 1.f;
    const float mp = p.min_p ? p.min_p[row] : 0.f, u = p.u[row];
    const double c = 1.4426950408889634 / (double)T;
    s.greedy = !(T > 0.f) || c > 3e38;
    s.ch = (float)c;
    s.cl = (float)(c - (double)s.ch);
    s.u = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;
    s.top_k = p.top_k ? max(p.top_k[row], 0) : 0;
    s.p_fix = P < 1.f ? max(__float2ull_rn(fmaxf(P, 0.f) * 18446744073709551616.f), 1ull) : 0;
    s.y_min = mp > 0.f ? -log2((double)fminf(mp, 1.f)) : 64.0;
    s.by_m = s.y_min < 63.0;
  }
  // over the CTA: largest, least, largest
  auto reduce3 = [&](float3 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x = fmaxf(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
      v.y = fminf(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
      v.z = fmaxf(v.z, __shfl_xor_sync(0xffffffffu, v.z, o));
    }
    __syncthreads();  // (the last reduction has been read; the options are there)
    if (lane == 0) s.warpf[warp] = v;
    __syncthreads();
    v = s.warpf[lane & 15];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      v.x = fmaxf(v.x, __shfl_xor_sync(0xffffffffu, v.x, o));
      v.y = fminf(v.y, __shfl_xor_sync(0xffffffffu, v.y, o));
      v.z = fmaxf(v.z, __shfl_xor_sync(0xffffffffu, v.z, o));
    }
    return v;
  };
  float top = -INFINITY;
#pragma unroll
  for (int e = 0; e < kSampU; ++e) top = fmaxf(top, cur[e]);
  top = reduce3(make_float3(top, INFINITY, -INFINITY)).x;
  const float ch = s.ch, cl_ = s.cl;
  if (s.greedy) {
    float mx = -INFINITY;
    int at = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kSampU * kSampNT) {
      float next[kSampU];
      load(next, i0 + kSampU * kSampNT);
#pragma unroll
      for (int e = 0; e < kSampU; ++e) {
        if (cur[e] > mx && mx < kLargest) mx = fminf(cur[e], kLargest), at = i0 + e * kSampNT + tid;
        cur[e] = next[e];
      }
    }
    u64 best = mx == -INFINITY ? 0 : ((u64)sample_key(mx) << 32) | (uint32_t)~(first + at);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, (u64)__shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) s.warp64[warp] = best;
    __syncthreads();
    for (int w = 0; w < kSampNT / 32; ++w) best = max(best, s.warp64[w]);
    cl.barrier_wait(std::move(started));
    if (tid == 0) cl.map_shared_rank(s.best, 0)[rank] = best;
    cl.sync();
    if (rank == 0 && tid == 0) {
      for (int k = 0; k < C; ++k) best = max(best, s.best[k]);
      p.tokens[row] = best ? (int)~(uint32_t)best : -1;
      if (p.probs) p.probs[row] = best ? 1.f : 0.f;
    }
    return;
  }
  // ---- the histogram
  // High temperatures: buckets as fine as lets the window take 40 above and below the
  // first logits' largest (the second time, the row's own range).
  int fine = 0;
  while (fine < 15 && 40.f * ch * (float)(64 << fine) < (float)kSampB) ++fine;
  float m = top;  // the row's largest, at last
  float S, chS, clS, lo_y, hi_y;
  Term tm;        // its place
  bool window, crowd = false;
  const bool by_p = s.p_fix != 0, by_m = s.by_m;
  bool by_k;
  const u64 u_fix = __float2ull_rn(s.u * 18446744073709551616.f);
  uint32_t n_all;
  u64 all;
  auto mass_to = [&](int b) { return b < 0 ? 0ull : s.mass[min(b, kSampB - 1)]; };
  auto count_to = [&](int b) { return b < 0 ? 0u : s.count[min(b, kSampB - 1)]; };
  int bk = -4, bm, bl, bh, pl, ph = -4;
  uint32_t qm;
#pragma unroll 1
  for (int turn = 0;; ++turn) {
    S = (float)(32 << fine), chS = ch * S, clS = cl_ * S;
    // buckets [from, from + kSampTable): half of them above the reference
    window = fabsf(m * chS) < 2090000.f;  // (else, and for no reference: nothing is in it)
    const float ref = floorf(-m * chS), from = ref - (turn ? 2.f : (float)kSampB);
    lo_y = window ? from + 1.f : INFINITY, hi_y = window ? from + (float)(kSampTable - 1) : -INFINITY;
    const float small = ref + 4.f * S;  // 2^-4 of the reference and less
    const float kap = 0.693147181f / S, k1 = kap * 17179869184.f, k2 = -0.5f * kap * k1, k3 = kap * kap / 6.f * k1, k4 = kap * kap * kap / -24.f * k1;
    float3 r = make_float3(-INFINITY, INFINITY, -INFINITY);  // the largest, the least in the window, the largest outside
    auto put = [&](int b, uint32_t D) {
      b &= kSampTable - 1;
      const uint32_t old = atomicAdd(&s.lo[b], D);
      atomicAdd(&s.hi[b], old + D < old ? 262145u : 1u);
    };
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kSampU * kSampNT) {
      float next[kSampU];
      load(next, i0 + kSampU * kSampNT);
#pragma unroll
      for (int e = 0; e < kSampU; e += 2) {
        const float l[2] = {cur[e], cur[e + 1]};
        float y[2], z[2], nr[2], fl[2], D[2];
        mul2(y[0], y[1], l[0], l[1], -chS);
        z[0] = -y[0], z[1] = -y[1];
        fma2(z[0], z[1], l[0], l[1], -chS, -chS);
        fma2(z[0], z[1], l[0], l[1], -clS, -clS);       // what the product lost
        add2(nr[0], nr[1], y[0], y[1], -0.5f, -0.5f);
        add2(nr[0], nr[1], nr[0], nr[1], 12582912.f, 12582912.f);  // the floor, or one less where y is whole
        sub2(fl[0], fl[1], nr[0], nr[1], 12582912.f, 12582912.f);
        sub2(y[0], y[1], y[0], y[1], fl[0], fl[1]);
        add2(z[0], z[1], z[0], z[1], y[0], y[1]);       // the place in the bucket
        D[0] = k3, D[1] = k3;
        fma2(D[0], D[1], z[0], z[1], k4, k4);
        float q[2] = {k2, k2};
        fma2(q[0], q[1], D[0], D[1], z[0], z[1]);
        D[0] = k1, D[1] = k1;
        fma2(D[0], D[1], q[0], q[1], z[0], z[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          r.x = fmaxf(r.x, l[i]);
          if (!(fl[i] >= lo_y && fl[i] < hi_y)) {
            r.z = fmaxf(r.z, l[i]);
          } else {
            if (fine) r.y = fminf(r.y, l[i]);
            // (near the bucket's ends the remainder decides which)
            if (fl[i] < small || z[i] < 1e-6f || z[i] > 0.999999f) {
              const Term p = place_of(l[i], chS, clS);
              put(p.b, below(p.q, fine));
            } else {
              put(__float_as_int(nr[i]) - 0x4B400000, __float2uint_rn(D[i] * z[i]));
            }
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kSampU; ++e) cur[e] = next[e];
    }
    r = reduce3(r);
    if (turn == 0) cl.barrier_wait(std::move(started));
    if (tid < C) cl.map_shared_rank(s.range, tid)[rank] = make_float4(r.x, r.y, r.z, window ? from : -1e9f);
    cl.sync();
    float least = INFINITY, out = -INFINITY;
    m = -INFINITY;
    for (int k = 0; k < C; ++k) {
      const float4 o = s.range[k];
      m = fmaxf(m, o.x), least = fminf(least, o.y), out = fmaxf(out, o.z);
    }
    if (m == -INFINITY) {
      if (rank == 0 && tid == 0) {
        p.tokens[row] = -1;
        if (p.probs) p.probs[row] = 0.f;
      }
      return;
    }
    if (m == INFINITY) m = kLargest;
    // logits of weight (2^-63 and more) that the buckets below the largest miss
    // (an infinite one is outside, and the difference times 0 at an infinite temperature says nothing)
    const bool missed = out > m || (m - out) * ch < 63.f || (fine > 0 && (m - least) * chS >= (float)(kSampB - 2));
    // (the long way too where bucket numbers come near 2^21, what the floor in fp32 and the window hold)
    crowd = !(fabsf(m * ch) < 32768.f) || (missed && turn == 1);
    if (crowd) break;
    if (!missed) {
      // ---- the CTAs' buckets from the largest logit's on, added up
      tm = place_of(m, chS, clS);
      if (tid == 0)  // the place up to which min_p keeps, behind the largest logit's
        s.key = tm.q + (by_m ? (u64)(s.y_min * (double)S * 4294967296.0) : 0ull);
      if (tid == 0) s.total = s.n_local = s.n_list = 0;
      const int share = kSampB / C;
      for (int i = tid; i < share; i += kSampNT) {
        const int j = rank * share + i, b = tm.b + j;
        u64 D = 0;
        uint32_t c = 0;
#pragma unroll 8
        for (int k = 0; k < C; ++k) {
          const int at = b - (int)s.range[k].w;
          if (at >= 0 && at < kSampTable) {
            const SampShared& o = *cl.map_shared_rank(&s, k);
            const uint32_t lo = o.lo[b & (kSampTable - 1)], hi = o.hi[b & (kSampTable - 1)];
            D += ((u64)(hi >> 18) << 32) + lo;
            c += hi & 0x3FFFFu;
          }
        }
        const u64 w = c ? weight_of(((u64)c << 34) - D, j, fine) : 0;
        for (int k = 0; k < C; ++k) {
          cl.map_shared_rank(s.mass, k)[j] = w;
          cl.map_shared_rank(s.count, k)[j] = c;
        }
      }
      cl.sync();
      // ---- running sums over the buckets; where the borders can be
      {
        u64 a[kSampPer], sum = 0;
        uint32_t c[kSampPer], cnt = 0;
#pragma unroll
        for (int i = 0; i < kSampPer; ++i) {
          a[i] = sum += s.mass[kSampPer * tid + i];
          c[i] = cnt += s.count[kSampPer * tid + i];
        }
        u64 up = sum;
        uint32_t nup = cnt;
        scan2(up, nup, s);
#pragma unroll
        for (int i = 0; i < kSampPer; ++i) {
          s.mass[kSampPer * tid + i] = up - sum + a[i];
          s.count[kSampPer * tid + i] = nup - cnt + c[i];
        }
      }
      __syncthreads();
      all = s.mass[kSampB - 1];
      n_all = s.count[kSampB - 1];
      by_k = s.top_k > 0 && (uint32_t)s.top_k < n_all;
      const u64 m_at = s.key;
      bm = by_m ? (int)min(m_at >> 32, (u64)kSampB) : kSampB, qm = (uint32_t)m_at;
      pl = -1;
      u64 k_lo = all, k_hi = all;
      if (by_k) {
        const uint32_t k = s.top_k;
        bk = first_at([&](int b) { return s.count[b] >= k; });
        k_lo = mass_to(bk - 1), k_hi = mass_to(bk);
      }
      u64 lo = k_lo, hi = k_hi;  // of the kept mass
      if (by_p) {
        const u64 tl = __umul64hi(k_lo, s.p_fix), th = __umul64hi(k_hi, s.p_fix) + 2;
        pl = first_at([&](int b) { return s.mass[b] >= tl; });
        ph = min(first_at([&](int b) { return s.mass[b] >= th; }), by_k ? bk : kSampB - 1);
        pl = min(pl, ph);
        lo = min(lo, mass_to(pl - 1)), hi = min(hi, mass_to(ph));
      }
      if (by_m) lo = min(lo, mass_to(bm - 1)), hi = min(hi, mass_to(bm));
      {
        const u64 tl = __umul64hi(lo, u_fix), th = __umul64hi(hi, u_fix) + 2;
        bl = min(first_at([&](int b) { return s.mass[b] > tl; }), kSampB - 1);
        bh = min(first_at([&](int b) { return s.mass[b] > th; }), kSampB - 1);
      }
      {
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < kSampPer; ++i) {
          const int b = kSampPer * tid + i;
          const bool in = b == bk || (by_p && b >= pl && b <= ph) || (by_m && b == bm) || (b >= bl && b <= bh);
          s.flag[b] = in;
          if (in) mine += count_to(b) - count_to(b - 1);
        }
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0 && mine) atomicAdd(&s.total, mine);
        __syncthreads();
        crowd = s.total > (uint32_t)kSampleList;
        if (!crowd || turn == 1) break;
      }
    }
    // once more, from the exact range (finer buckets too, if that is what it takes): the least logit of any weight
    float3 low = make_float3(0.f, INFINITY, 0.f);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kSampU * kSampNT) {
      load(cur, i0);
#pragma unroll
      for (int e = 0; e < kSampU; ++e)
        if ((m - cur[e]) * ch < 63.f) low.y = fminf(low.y, cur[e]);
    }
    low = reduce3(low);
    cl.sync();  // every CTA has read the ranges
    if (tid < C) cl.map_shared_rank(s.range, tid)[rank] = make_float4(0.f, low.y, 0.f, 0.f);
    cl.sync();
    for (int k = 0; k < C; ++k) low.y = fminf(low.y, s.range[k].y);
    const float wide = (m - low.y) * ch;
    const int was = fine;
    fine = 0;
    while (fine < 15 && wide * (float)(64 << fine) < (float)(kSampB - 4) && fabsf(m * ch) * (float)(64 << fine) < 1048576.f)
      ++fine;
    if (crowd && fine <= was) break;
    clear();
    cl.sync();
    load(cur, 0);
  }
  if (crowd) {
    sample_crowd(p, s, m);
    return;
  }
  // ---- the second pass: their tokens to the first CTA
  // (from the end on: what was read last is in L2 still, where the rows together are larger)
  // the gathered buckets, a little wider (y is within 2^-24 of its size, and as much again for the ratio's lower part, of the
  // exact place, and these numbers are rounded too): the draw's, top_p's, and the others'
  const float b0 = (float)tm.b, aside = 0.01f + fabsf(b0) * 2.4e-7f, g0 = fmaxf(b0 + (float)bl - aside, lo_y), g1 = fminf(b0 + (float)bh + 1.f + aside, hi_y);
  const float g2 = fmaxf(b0 + (float)pl - aside, lo_y), g3 = by_p ? fminf(b0 + (float)ph + 1.f + aside, hi_y) : -INFINITY;
  const int other = by_k && by_m ? min(bk, bm) : by_k ? bk : bm, others = by_k && by_m ? max(bk, bm) : other;
  const float g4 = fmaxf(b0 + (float)other - aside, lo_y), g5 = by_k || by_m ? fminf(b0 + (float)others + 1.f + aside, hi_y) : -INFINITY;
  constexpr int step = kSampU * kSampNT;
  const int last = n > 0 ? (n - 1) / step * step : -1;
  if (last >= 0) load(cur, last);
#pragma unroll 1
  for (int i0 = last; i0 >= 0; i0 -= step) {
    float next[kSampU];
    if (i0 > 0) load(next, i0 - step);
#pragma unroll
    for (int e = 0; e < kSampU; ++e) {
      const float y = __fmul_rn(-cur[e], chS);
      if ((y >= g0 && y < g1) || (y >= g2 && y < g3) || (y >= g4 && y < g5)) {
        const int j = place_of(cur[e], chS, clS).b - tm.b;
        if (j >= 0 && j < kSampB && s.flag[j])
          s.local[atomicAdd(&s.n_local, 1u)] =
              ((u64)sample_key(cur[e]) << 32) | (uint32_t)~(first + i0 + e * kSampNT + tid);
      }
    }
#pragma unroll
    for (int e = 0; e < kSampU; ++e) cur[e] = next[e];
  }
  __syncthreads();
  if (C > 1) {
    if (tid == 0 && s.n_local) s.base = atomicAdd(cl.map_shared_rank(&s.n_list, 0), s.n_local);
    __syncthreads();
    u64* list0 = cl.map_shared_rank(s.list, 0);
    for (uint32_t i = tid; i < s.n_local; i += kSampNT) list0[s.base + i] = s.local[i];
    cl.sync();
    if (rank != 0) return;
  }
  const u64* in = C > 1 ? s.list : s.local;
  const int N = C > 1 ? s.n_list : s.n_local;
  int E = 1, n2 = 32;
  while (E * kSampNT < N) E *= 2;
  while (n2 < N) n2 *= 2;
  if (E > kSortRegs) {
    sort_long(s.list, in, N);
  } else {
    u64 v[kSortRegs];
#pragma unroll
    for (int e = 0; e < kSortRegs; ++e) v[e] = e * kSampNT + tid < N ? in[e * kSampNT + tid] : 0;
    __syncthreads();
    if (E == 1) sort_list<1>(v, s.list, n2);
    else if (E == 2) sort_list<2>(v, s.list, n2);
    else sort_list<4>(v, s.list, n2);
#pragma unroll
    for (int e = 0; e < kSortRegs; ++e)
      if (e < E) s.list[e * kSampNT + tid] = v[e];  // read by this thread alone
  }
  // masses, running sums and first entries of the buckets
  auto entry = [&](u64 v) {
    Term t = place_of(key_float((uint32_t)(v >> 32)), chS, clS);
    t.b -= tm.b;
    return t;
  };
  u64 carry = 0;
#pragma unroll 1
  for (int j = tid; j < E * kSampNT; j += kSampNT) {
    const u64 v = s.list[j];
    Term t = {-1, 0u};
    u64 g = 0;  // up to and with an entry: first of the list, then of the row
    if (v) {
      t = entry(v);
      g = weight_of(t, fine);
      s.bucket[j] = (uint16_t)t.b;
    }
    uint32_t none = 0;
    scan2(g, none, s);
    if (tid == kSampNT - 1) s.res_mass[0] = g;
    s.local[j] = g + carry;
    __syncthreads();
    carry += s.res_mass[0];
    if (v && (j == 0 || s.bucket[j - 1] != t.b)) s.start[t.b] = j;
    __syncthreads();
  }
  // the masses that top_k, top_p and min_p keep
  if (tid == 0) {
    s.res_mass[0] = s.res_mass[1] = all;
    s.res_mass[2] = by_m ? mass_to(bm - 1) : all;  // or more, of min_p's own bucket
  }
  __syncthreads();
  // up to and with entry j, of bucket b. An entry's weight is rounded and a bucket's mass is not the sum of them to the
  // last bit: its last entry ends where it does, so that a border found between two buckets is found here too
  auto row_mass = [&](int j, int b) {
    const int f = s.start[b];
    const u64 end = mass_to(b);
    return j + 1 == N || s.bucket[j + 1] != b ? end : min(mass_to(b - 1) + s.local[j] - (f ? s.local[f - 1] : 0ull), end);
  };
#pragma unroll 1
  for (int j = tid; j < N; j += kSampNT) {
    const Term t = entry(s.list[j]);
    const u64 g = row_mass(j, t.b);
    if (by_k && count_to(t.b - 1) + (uint32_t)(j - s.start[t.b]) + 1 == (uint32_t)s.top_k) s.res_mass[0] = g;
    if (by_m && t.b == bm && t.q <= qm) atomicMax(&s.res_mass[2], g);
  }
  __syncthreads();
  if (by_p) {
    const u64 target = ceil_part(s.res_mass[0], s.p_fix);
#pragma unroll 1
    for (int j = tid; j < N; j += kSampNT) {
      const int b = s.bucket[j];
      if (b < pl) continue;
      const u64 g = row_mass(j, b);
      if (g >= target) atomicMin(&s.res_mass[1], g);
    }
    __syncthreads();
  }
  const u64 mass = min(min(s.res_mass[0], s.res_mass[1]), s.res_mass[2]), target = __umul64hi(mass, u_fix);
  if (tid == 0) s.found = max(N, 1) - 1;
  __syncthreads();
#pragma unroll 1
  for (int j = tid; j < N; j += kSampNT) {
    const int b = s.bucket[j];
    if (b >= bl && row_mass(j, b) > target) atomicMin(&s.found, j);
  }
  __syncthreads();
  if (tid == 0) {
    const u64 v = s.list[s.found];
    const Term t = entry(v);
    p.tokens[row] = (int)~(uint32_t)v;
    if (p.probs)
      p.probs[row] = (float)((1ull << 34) - below(t.q, fine)) * exp2f(-(float)t.b / S) * 1024.f / (float)mass;
  }
}

}  // namespace

cudaError_t launch_sample_rows(SampleRowsParams& p, int n_sm, cudaStream_t st) {
  // CTAs of a row: a CTA's fixed work (about 12 us) pays for as many logits as can be, so as many as
  // have an SM each, with 1000 logits or more, or two on an SM for slices of 32768 and more; at most
  // 180000 (the histogram's counts). Measured, us for 1, 2, 4, 8, 16: 1 x 32000 26 / 21 / 17 / 15 / 15,
  // 32 x 32000 30 / 23 / 18 / 25 / 43, 32 x 151936 86 / 54 / 37 / 35 / 57, 64 x 151936 89 / 53 / 46 / 57 / 99,
  // 256 x 151936 135 / 139 / 156 / 205 / 357.
  const auto more = [&](int C) {
    const int64_t ctas = (int64_t)2 * p.R * C;
    return (p.V + C - 1) / C > kSampMaxSlice || (ctas <= n_sm && p.V / (2 * C) >= 1000) || (ctas <= 2 * n_sm && p.V / C >= 32768);
  };
  int C = 1;
  while (C < 16 && more(C)) C *= 2;
  p.slice = (p.V + C - 1) / C;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(sample_rows_kernel, (int)sizeof(SampShared), true);
  return e == cudaSuccess ? launch_cluster(sample_rows_kernel, dim3(p.R * C), kSampNT, C, sizeof(SampShared), st, p, p.pdl) : e;
}

}  // namespace llmq

// ---- C entry ----------------------------------------------------------------------
using namespace llmq;

extern "C" int llm_sample_tokens(const llm_sample_args* a, void* cuda_stream) {
  Call c;
  if (!c.need(a != nullptr, LLM_ERR_INVALID_ARG, "the arguments are null") ||
      !c.need(a->n_rows >= 1 && a->vocab >= 1, LLM_ERR_INVALID_ARG, "n_rows or vocab is not positive") ||
      !c.need(a->vocab <= 1 << 19, LLM_ERR_UNSUPPORTED, "%svocab %lld is too large", "", a->vocab) ||
      !c.need((int64_t)a->n_rows * 16 <= 0x7FFFFFFF, LLM_ERR_UNSUPPORTED, "too many rows") ||
      !c.need(a->logits_stride >= 0, LLM_ERR_INVALID_ARG, "a stride is negative") || !c.device("logits", a->logits, 4) ||
      !c.device("uniforms", a->uniforms, 4) || !c.device("tokens", a->tokens, 4) ||
      (a->temperature && !c.device("temperature", a->temperature, 4)) || (a->top_k && !c.device("top_k", a->top_k, 4)) ||
      (a->top_p && !c.device("top_p", a->top_p, 4)) || (a->min_p && !c.device("min_p", a->min_p, 4)) ||
      (a->probs && !c.device("probs", a->probs, 4)))
    return c.rc;
  SampleRowsParams p{};
  p.logits = a->logits;
  p.stride = a->logits_stride;
  p.u = a->uniforms, p.temperature = a->temperature, p.top_p = a->top_p, p.min_p = a->min_p;
  p.top_k = a->top_k;
  p.tokens = a->tokens;
  p.probs = a->probs;
  p.R = a->n_rows, p.V = a->vocab;
  return finish(launch_sample_rows(p, c.n_sm, static_cast<cudaStream_t>(cuda_stream)), "sampling launch");
}
