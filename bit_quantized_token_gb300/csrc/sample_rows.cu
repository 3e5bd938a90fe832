// The next token of every row of logits, under the row's own options and from a
// given uniform number (see serve.cuh).
//
// Tokens in order, the largest logit first, equal ones by id; w_j = 2^(-Y_j), Y_j =
// (l_0 - l_j) log2(e) / T. Every option keeps a prefix of that order: the first
// top_k; of those the shortest whose mass reaches top_p of theirs; the w_j of at least
// min_p. The token is the first one whose cumulative mass passes u times the kept
// one's. So nothing is sorted but what lies around the borders:
//   1. a cluster holds a row in registers, read once; its largest logit;
//   2. a histogram over Y (32 buckets an octave, 64 octaves; finer for high
//      temperatures): the count and the mass of every bucket;
//   3. from their running sums, the few buckets in which the borders can lie (the
//      border of one option moves the next one's by a bucket's mass at most);
//   4. their tokens, some hundreds, to the first CTA, which sorts them and finds all
//      borders exactly.
// Rows that put more than kSampleList tokens into those buckets (all logits alike,
// crowds of equal ones) take the long way: each border by three digits of the
// logits' keys, over all tokens.
//
// Masses decide integers, so they are integers: a term is 2^-37 steps below its
// bucket's largest, computed from the logit's exact distance in pairs of floats and
// then in fixed point; sums have 2^-44 steps, in 64 bits, whatever their order. A
// border is off by less than 2^-36 of the row's mass: of 150,000 borders, one draw in
// some 10^5 .. 10^6 falls on another side than with exact sums. fp32 sums would lose one draw in
// 2,000, fp64 has 1/64 of fp32's lanes here.
#include <cooperative_groups.h>

#include "common.cuh"
#include "op_call.cuh"
#include "sample_key.cuh"
#include "serve.cuh"

namespace llmq {
namespace cg = cooperative_groups;
namespace {

using u64 = unsigned long long;
constexpr int kSampNT = 512, kSampB = 2048;  // threads; buckets of the histogram (in fours of a thread)
constexpr int kSampPer = kSampB / kSampNT;

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
  u64 mass[kSampB];         // running sums over the buckets, inclusive
  uint32_t count[kSampB];
  union {
    uint32_t h[3][kSampB];  // this CTA's histogram: sums of D, counts (low half) and carries of D (high half)
    struct {
      u64 local[kSampleList];   // entries of this CTA; later, on the first, the list's running masses
      uint32_t start[kSampB];   // first entry of a bucket
    };
  };
  u64 list[kSampleList];    // of the first CTA: every CTA's entries, (key, complement of the id)
  uint8_t flag[kSampB];     // 1: the bucket is gathered; 2: it or a neighbour
  u64 best[16];             // every CTA's largest (key, complement of the id)
  float least[16];
  u64 warp64[kSampNT / 32];
  uint32_t warp32[kSampNT / 32];
  float fwarp[kSampNT / 32];
  int found[2];
  uint32_t total, n_local, n_list, base;
  // the options
  float ch, cl, u;
  double y_min;             // -log2(min_p), or infinite
  u64 p_fix;                // top_p in 2^-64 steps; 0: off
  int top_k, greedy;
  // the first CTA's answers
  u64 res_mass[3];
  uint32_t res_rank[3];
  u64 key;
};

struct Term {
  int b;       // bucket
  uint32_t q;  // place in it, 2^-32 steps
};

// Y in S = 32 << fine buckets an octave. False: no weight (2^-64 and below).
__device__ __forceinline__ bool term_of(float l, float m, float ch, float cl, float S, Term& t) {
  const float d = __fsub_rn(m, l), bb = __fsub_rn(d, m);
  const float dl = __fsub_rn(__fsub_rn(m, __fsub_rn(d, bb)), __fadd_rn(l, bb));  // m - l = d + dl, exactly
  const float p = __fmul_rn(d, ch), y = __fmul_rn(p, S);
  if (!(y < (float)kSampB + 1.f)) return false;
  float e = __fmaf_rn(d, ch, -p);
  e = __fmaf_rn(d, cl, e);
  e = __fmaf_rn(dl, ch, e);
  const float fl = floorf(y);
  const long long q = (long long)__float2uint_rn((y - fl) * 4294967296.f) + __float2int_rn(e * S * 4294967296.f);
  t.b = (int)fl + (int)(q >> 32);  // (the remainder may take it past a border)
  t.q = (uint32_t)q;
  return t.b >= 0 && t.b < kSampB;
}
// 2^37 (1 - 2^-z) for the place q of a bucket: z - z^2/2 + z^3/6 - .. in fixed point
__device__ __forceinline__ uint32_t below(uint32_t q, int fine) {
  const uint32_t z = __umulhi(q, 2977044472u) >> fine;  // 2^37 ln(2) / S: below 2^31.5
  uint32_t a = ~__umulhi(z, 26843546u);                 // 1 - z/5
  a = ~__umulhi(z >> 7, a);                             // 1 - z/4 ..
  a = ~__umulhi(__umulhi(z, 44739243u), a);
  a = ~__umulhi(z >> 6, a);
  return __umulhi(z, a);
}
// a 2^-37 steps of the largest term of bucket b, in 2^-44 steps of the row's largest
__device__ __forceinline__ u64 weight_of(u64 a, int b, int fine) {
  if (fine) {
    const int lo = b & ((1 << fine) - 1);
    if (lo) {
      const uint32_t f = below((uint32_t)lo << (32 - fine), 0);
      a = __umul64hi(a << 7, ((1ull << 37) - f) << 27) >> 7;
    }
    b >>= fine;
  }
  const u64 r = __umul64hi(a << 7, kRoot32[b & 31]);
  const int s = (b >> 5) - 1;
  return s < 0 ? r << 1 : s == 0 ? r : (r + (1ull << (s - 1))) >> s;
}
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

template <int KPT>
__global__ void __launch_bounds__(kSampNT, KPT <= 20 ? 2 : 1) sample_rows_kernel(const SampleRowsParams p) {
  extern __shared__ __align__(16) uint8_t sm_raw[];
  SampShared& s = *reinterpret_cast<SampShared*>(sm_raw);
  cg::cluster_group cl = cg::this_cluster();
  const int C = cl.num_blocks(), rank = cl.block_rank(), row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto started = cl.barrier_arrive();  // shared memory of another CTA: only once that CTA runs
  for (int i = tid; i < 2 * kSampB; i += kSampNT) (&s.h[0][0])[i] = 0;
  if (tid == 0) s.n_local = s.n_list = s.total = 0;
  pdl_wait();
  pdl_trigger();
  // ---- the row, its largest logit
  const int first = rank * p.slice, n = min(p.V - first, p.slice);
  const float* src = p.logits + (int64_t)row * p.stride + first;
  float x[KPT];
#pragma unroll
  for (int e = 0; e < KPT; ++e) x[e] = e * kSampNT + tid < n ? __ldcs(src + e * kSampNT + tid) : -INFINITY;
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
    s.y_min = mp > 0.f ? -log2((double)fminf(mp, 1.f)) : 1e30;
  }
  float mx = -INFINITY;
  int at = 0;
#pragma unroll
  for (int e = 0; e < KPT; ++e) {
    x[e] = x[e] != x[e] ? -INFINITY : fminf(x[e], 3.402823466e38f);
    if (x[e] > mx) mx = x[e], at = e;
  }
  u64 best = mx == -INFINITY ? 0 : ((u64)sample_key(mx) << 32) | (uint32_t)~(first + at * kSampNT + tid);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, (u64)__shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) s.warp64[warp] = best;
  __syncthreads();
  best = s.warp64[lane & 15];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) best = max(best, (u64)__shfl_xor_sync(0xffffffffu, best, o));
  const float ch = s.ch, cl_ = s.cl;
  const bool hot = ch < 0.72f && !s.greedy;  // T above 2: the row may need finer buckets
  float least = INFINITY;
  if (hot) {
    const float from = best ? key_float((uint32_t)(best >> 32)) - 64.f / ch : -INFINITY;
#pragma unroll
    for (int e = 0; e < KPT; ++e)
      if (x[e] >= from && x[e] != -INFINITY) least = fminf(least, x[e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    if (lane == 0) s.fwarp[warp] = least;
    __syncthreads();
    least = s.fwarp[lane & 15];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
  }
  cl.barrier_wait(std::move(started));
  if (tid < C) {
    cl.map_shared_rank(s.best, tid)[rank] = best;
    cl.map_shared_rank(s.least, tid)[rank] = least;
  }
  cl.sync();
  for (int k = 0; k < C; ++k) best = max(best, s.best[k]), least = fminf(least, s.least[k]);
  if (best == 0 || s.greedy) {
    if (rank == 0 && tid == 0) {
      p.tokens[row] = best ? (int)~(uint32_t)best : -1;
      if (p.probs) p.probs[row] = best ? 1.f : 0.f;
    }
    return;
  }
  const float m = key_float((uint32_t)(best >> 32));
  int fine = 0;
  if (hot) {
    const float span = fminf(64.f, __fmul_rn(__fsub_rn(m, least), ch));
    while (fine < 15 && span * (float)(64 << fine) < (float)(kSampB - 2)) ++fine;
  }
  const float S = (float)(32 << fine);
  // ---- the histogram
#pragma unroll
  for (int e = 0; e < KPT; ++e) {
    Term t;
    if (term_of(x[e], m, ch, cl_, S, t)) {
      const uint32_t D = below(t.q, fine), old = atomicAdd(&s.h[0][t.b], D);
      atomicAdd(&s.h[1][t.b], old + D < old ? 65537u : 1u);
    }
  }
  cl.sync();
  {
    const int share = kSampB / C;
    for (int i = tid; i < share; i += kSampNT) {
      const int b = rank * share + i;
      u64 D = 0;
      uint32_t c = 0;
#pragma unroll 4
      for (int k = 0; k < C; ++k) {
        const uint32_t(*h)[kSampB] = cl.map_shared_rank(&s.h[0], k);
        const uint32_t lo = h[0][b], hi = h[1][b];
        D += ((u64)(hi >> 16) << 32) + lo;
        c += hi & 0xFFFFu;
      }
      const u64 w = c ? weight_of(((u64)c << 37) - D, b, fine) : 0;
      for (int k = 0; k < C; ++k) {
        cl.map_shared_rank(s.mass, k)[b] = w;
        cl.map_shared_rank(s.count, k)[b] = c;
      }
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
  const u64 all = s.mass[kSampB - 1];
  const uint32_t n_all = s.count[kSampB - 1];
  auto mass_to = [&](int b) { return b < 0 ? 0ull : s.mass[min(b, kSampB - 1)]; };
  auto count_to = [&](int b) { return b < 0 ? 0u : s.count[min(b, kSampB - 1)]; };
  // the first buckets at which two rising conditions hold (kSampB: none)
  auto find = [&](auto f, auto g, int& bf, int& bg) {
    if (tid == 0) s.found[0] = s.found[1] = kSampB;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSampPer; ++i) {
      const int b = kSampPer * tid + i;
      if (f(b) && (b == 0 || !f(b - 1))) s.found[0] = b;
      if (g(b) && (b == 0 || !g(b - 1))) s.found[1] = b;
    }
    __syncthreads();
    bf = s.found[0], bg = s.found[1];
    __syncthreads();
  };
  const bool by_k = s.top_k > 0 && (uint32_t)s.top_k < n_all, by_p = s.p_fix != 0;
  const double y_min = s.y_min * (double)S;
  const bool by_m = y_min < (double)kSampB;
  const int bm = by_m ? (int)y_min : kSampB;
  const uint32_t qm = by_m ? (uint32_t)fmin((y_min - (double)bm) * 4294967296.0, 4294967295.0) : 0;
  int bk = -1, pl = -1, ph = -2, bl, bh;
  u64 k_lo = all, k_hi = all;
  if (by_k) {
    const uint32_t k = s.top_k;
    int unused;
    find([&](int b) { return s.count[b] >= k; }, [&](int) { return false; }, bk, unused);
    k_lo = mass_to(bk - 1), k_hi = mass_to(bk);
  }
  u64 lo = k_lo, hi = k_hi;  // of the kept mass
  if (by_p) {
    const u64 tl = __umul64hi(k_lo, s.p_fix), th = __umul64hi(k_hi, s.p_fix) + 2;
    find([&](int b) { return s.mass[b] >= tl; }, [&](int b) { return s.mass[b] >= th; }, pl, ph);
    ph = min(ph, by_k ? bk : kSampB - 1);
    pl = min(pl, ph);
    lo = min(lo, mass_to(pl - 1)), hi = min(hi, mass_to(ph));
  }
  if (by_m) lo = min(lo, mass_to(bm - 1)), hi = min(hi, mass_to(bm));
  const u64 u_fix = __float2ull_rn(s.u * 18446744073709551616.f);
  {
    const u64 tl = __umul64hi(lo, u_fix), th = __umul64hi(hi, u_fix) + 2;
    find([&](int b) { return s.mass[b] > tl; }, [&](int b) { return s.mass[b] > th; }, bl, bh);
    bl = min(bl, kSampB - 1), bh = min(bh, kSampB - 1);
  }
  {
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kSampPer; ++i) {
      const int b = kSampPer * tid + i;
      auto in = [&](int d) {  // bucket b within d of one that is gathered
        return abs(b - bk) <= d || (pl >= 0 && b >= pl - d && b <= ph + d) || (by_m && abs(b - bm) <= d) || (b >= bl - d && b <= bh + d);
      };
      s.flag[b] = (in(0) ? 1 : 0) | (in(1) ? 2 : 0);
      if (in(0)) mine += count_to(b) - count_to(b - 1);
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0 && mine) atomicAdd(&s.total, mine);
  }
  __syncthreads();
  if (s.total <= (uint32_t)kSampleList) {
    // ---- their tokens to the first CTA
    float mo = m;
    asm volatile("" : "+f"(mo));  // (the terms anew: kept from the histogram they would not fit the registers)
#pragma unroll
    for (int e = 0; e < KPT; ++e) {
      const float y = (mo - x[e]) * ch * S;
      if (y < (float)kSampB + 1.f && (s.flag[min((int)y, kSampB - 1)] & 2)) {
        Term t;
        if (term_of(x[e], mo, ch, cl_, S, t) && (s.flag[t.b] & 1))
          s.local[atomicAdd(&s.n_local, 1u)] = ((u64)sample_key(x[e]) << 32) | (uint32_t)~(first + e * kSampNT + tid);
      }
    }
    __syncthreads();
    if (tid == 0 && s.n_local) s.base = atomicAdd(cl.map_shared_rank(&s.n_list, 0), s.n_local);
    __syncthreads();
    u64* list0 = cl.map_shared_rank(s.list, 0);
    for (uint32_t i = tid; i < s.n_local; i += kSampNT) list0[s.base + i] = s.local[i];
    cl.sync();
    if (rank != 0) return;
    const int N = s.n_list;
    int n2 = 2;
    while (n2 < N) n2 *= 2;
    for (int i = N + tid; i < n2; i += kSampNT) s.list[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int k = 2; k <= n2; k *= 2)  // bitonic, descending
#pragma unroll 1
      for (int j = k / 2; j > 0; j /= 2) {
        for (int i = tid; i < n2 / 2; i += kSampNT) {
          const int a = 2 * i - (i & (j - 1)), b = a + j;
          const u64 va = s.list[a], vb = s.list[b];
          if ((va < vb) == ((a & k) == 0)) s.list[a] = vb, s.list[b] = va;
        }
        __syncthreads();
      }
    // masses and running sums of the list: a thread has the entries kListPer tid ..
    constexpr int kListPer = kSampleList / kSampNT;
    u64 w[kListPer], sum = 0;
    Term t[kListPer];
    uint32_t none = 0;
#pragma unroll
    for (int i = 0; i < kListPer; ++i) {
      const int j = kListPer * tid + i;
      w[i] = 0;
      t[i].b = -1, t[i].q = 0;
      if (j < N && term_of(key_float((uint32_t)(s.list[j] >> 32)), m, ch, cl_, S, t[i]))
        w[i] = weight_of((1ull << 37) - below(t[i].q, fine), t[i].b, fine);
      sum += w[i];
    }
    u64 up = sum;
    scan2(up, none, s);
    up -= sum;
#pragma unroll
    for (int i = 0; i < kListPer; ++i) {
      s.local[kListPer * tid + i] = up += w[i];
      const int j = kListPer * tid + i;
      if (j < N) {
        Term before;
        before.b = -1;
        if (j > 0) term_of(key_float((uint32_t)(s.list[j - 1] >> 32)), m, ch, cl_, S, before);
        if (before.b != t[i].b) s.start[t[i].b] = j;
      }
    }
    if (tid < 3) s.res_rank[tid] = 0xFFFFFFFFu, s.res_mass[tid] = all;
    if (tid == 0) s.key = 0;
    __syncthreads();
    u64 G[kListPer];       // mass up to and with the entry
    uint32_t place[kListPer];  // its place in the row's order, from 1
#pragma unroll
    for (int i = 0; i < kListPer; ++i) {
      const int j = kListPer * tid + i;
      G[i] = 0, place[i] = 0;
      if (j < N) {
        const int f = s.start[t[i].b];
        G[i] = mass_to(t[i].b - 1) + s.local[j] - (f ? s.local[f - 1] : 0ull);
        place[i] = count_to(t[i].b - 1) + (uint32_t)(j - f) + 1;
        if (by_k && place[i] == (uint32_t)s.top_k) s.res_rank[0] = place[i], s.res_mass[0] = G[i];
      }
    }
    __syncthreads();
    if (by_p) {
      const u64 target = ceil_part(s.res_mass[0], s.p_fix);
#pragma unroll
      for (int i = 0; i < kListPer; ++i)
        if (place[i] && G[i] >= target && t[i].b >= pl) atomicMin(&s.res_rank[1], place[i]);
    }
    if (by_m) {  // the last one that min_p keeps, in its bucket or before it
      if (tid == 0) s.res_rank[2] = count_to(bm - 1), s.res_mass[2] = mass_to(bm - 1);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kListPer; ++i)
        if (place[i] && t[i].b == bm && t[i].q <= qm) atomicMax(&s.res_rank[2], place[i]);
    }
    __syncthreads();
    if (by_p || by_m) {
#pragma unroll
      for (int i = 0; i < kListPer; ++i) {
        if (by_p && place[i] && place[i] == s.res_rank[1]) s.res_mass[1] = G[i];
        if (by_m && place[i] && t[i].b == bm && place[i] == s.res_rank[2]) s.res_mass[2] = G[i];
      }
    }
    __syncthreads();
    uint32_t kept = n_all;
    u64 mass = all;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (s.res_rank[i] < kept) kept = s.res_rank[i], mass = s.res_mass[i];
    const u64 target = __umul64hi(mass, u_fix);
#pragma unroll
    for (int i = 0; i < kListPer; ++i)  // keys fall along the list: the first one over the target is the largest
      if (place[i] && place[i] <= kept && G[i] > target && t[i].b >= bl) atomicMax(&s.key, s.list[kListPer * tid + i]);
    __syncthreads();
    if (tid == 0) {
      const u64 k = s.key ? s.key : best;
      Term t0;
      term_of(key_float((uint32_t)(k >> 32)), m, ch, cl_, S, t0);
      p.tokens[row] = (int)~(uint32_t)k;
      if (p.probs)
        p.probs[row] = (float)((1ull << 37) - below(t0.q, fine)) * exp2f(-(float)t0.b / S) * 128.f / (float)mass;
    }
    return;
  }
  // ---- the long way: the borders of top_k (or all tokens), top_p and the draw in
  // turn, each by three digits of the keys from the top, over all tokens (read
  // again: registers held through here would cost the short way)
  auto logit = [&](int i) {
    const float l = i < n ? src[i] : -INFINITY;
    return l != l ? -INFINITY : fminf(l, 3.402823466e38f);
  };
  cl.sync();
  uint32_t kept = 0;
  u64 mass = 0;
  uint32_t key = 0, above = 0, equal = 0;  // a border's key, tokens above it and of it
  u64 mass_above = 0, each = 0;            // mass above it, and of one token of it
#pragma unroll 1
  for (int turn = 0; turn < 3; ++turn) {
    if (turn == 1 && !by_p) continue;
    if (turn == 2 && by_m) {  // tokens and mass that min_p keeps
      u64 a = 0;
      uint32_t c = 0;
#pragma unroll 1
      for (int i = tid; i < n; i += kSampNT) {
        Term t;
        if (term_of(logit(i), m, ch, cl_, S, t) && (t.b < bm || (t.b == bm && t.q <= qm)))
          a += weight_of((1ull << 37) - below(t.q, fine), t.b, fine), ++c;
      }
      scan2(a, c, s);
      if (tid == kSampNT - 1) s.list[0] = a, s.list[1] = c;
      cl.sync();
      a = 0, c = 0;
      for (int k = 0; k < C; ++k) {
        const u64* o = cl.map_shared_rank(s.list, k);
        a += o[0], c += (uint32_t)o[1];
      }
      if (c < kept) kept = c, mass = a;
      cl.sync();
    }
    // found is where the count (turn 0) or the mass (1) reaches the target, or the mass passes it (2)
    const u64 target = turn == 0 ? (by_k ? (u64)s.top_k : (u64)n_all) : turn == 1 ? ceil_part(mass, s.p_fix) : __umul64hi(mass, u_fix);
    auto over = [&](u64 m_, uint32_t n_) { return turn == 0 ? n_ >= target : turn == 1 ? m_ >= target : m_ > target; };
    key = above = 0, mass_above = 0;
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bins = level == 2 ? 1024 : 2048;
      const uint32_t prefix_mask = level == 0 ? 0u : level == 1 ? 0xFFE00000u : 0xFFFFFC00u;
      for (int i = tid; i < 3 * kSampB; i += kSampNT) (&s.h[0][0])[i] = 0;
      if (tid == 0) s.found[0] = -1;
      __syncthreads();
#pragma unroll 1
      for (int i = tid; i < n; i += kSampNT) {
        Term t;
        const float l = logit(i);
        const uint32_t k = sample_key(l);
        if ((k & prefix_mask) == key && term_of(l, m, ch, cl_, S, t)) {
          const u64 w = weight_of((1ull << 37) - below(t.q, fine), t.b, fine);
          const uint32_t bin = (k >> shift) & (bins - 1), lo32 = (uint32_t)w, old = atomicAdd(&s.h[0][bin], lo32);
          atomicAdd(&s.h[1][bin], (uint32_t)(w >> 32) + (old + lo32 < old));
          atomicAdd(&s.h[2][bin], 1u);
        }
      }
      cl.sync();
      // every CTA adds all of them up; a thread has four bins of the descending order
      u64 a[kSampPer], sum = 0;
      uint32_t c[kSampPer], cnt = 0;
#pragma unroll
      for (int i = 0; i < kSampPer; ++i) {
        const int bin = bins - 1 - (kSampPer * tid + i);
        a[i] = 0, c[i] = 0;
        if (bin >= 0)
          for (int k = 0; k < C; ++k) {
            const uint32_t(*h)[kSampB] = cl.map_shared_rank(&s.h[0], k);
            a[i] += ((u64)h[1][bin] << 32) + h[0][bin];
            c[i] += h[2][bin];
          }
        sum += a[i], cnt += c[i];
      }
      u64 up = sum;
      uint32_t nup = cnt;
      scan2(up, nup, s);
      up -= sum, nup -= cnt;
      // the first non-empty bin over the target; past everything (by rounding), the last non-empty one
#pragma unroll
      for (int i = 0; i < kSampPer; ++i) {
        const bool was = over(mass_above + up, above + nup), is = over(mass_above + up + a[i], above + nup + c[i]);
        const bool last = above + nup + c[i] == (level == 0 ? n_all : above + equal) && !is;
        if (c[i] && !was && (is || last)) {
          s.found[0] = bins - 1 - (kSampPer * tid + i);
          s.res_mass[0] = mass_above + up;
          s.res_rank[0] = above + nup;
          s.res_rank[1] = c[i];
        }
        up += a[i], nup += c[i];
      }
      __syncthreads();
      key |= (uint32_t)max(s.found[0], 0) << shift;
      mass_above = s.res_mass[0], above = s.res_rank[0], equal = s.res_rank[1];
      cl.sync();  // every CTA has read the histograms (the last turn's stay) and the result
    }
    Term t;
    each = 0;
    if (term_of(key_float(key), m, ch, cl_, S, t)) each = weight_of((1ull << 37) - below(t.q, fine), t.b, fine);
    if (turn == 0) {
      kept = (uint32_t)target;
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

template <int KPT>
cudaError_t launch_sample_t(SampleRowsParams& p, int C, cudaStream_t st) {
  const auto kern = sample_rows_kernel<KPT>;
  static SmemLimit limit;
  const cudaError_t e = limit.raise(kern, (int)sizeof(SampShared), true);
  return e == cudaSuccess ? launch_cluster(kern, dim3(p.R * C), kSampNT, C, sizeof(SampShared), st, p, p.pdl) : e;
}

}  // namespace

cudaError_t launch_sample_rows(SampleRowsParams& p, int n_sm, cudaStream_t st) {
  // CTAs of a row: so many that a thread holds 20 logits at most (two CTAs on an SM; V up to
  // 163840 with 16), and for few rows as many as have 1024 logits each.
  int C = 1;
  while (C < 16 && (p.V + C - 1) / C > 20 * kSampNT) C *= 2;
  while (C < 16 && (int64_t)p.R * C < n_sm && p.V / (2 * C) >= 1024) C *= 2;
  p.slice = (p.V + C - 1) / C;
  const int per = (p.slice + kSampNT - 1) / kSampNT;
  return per <= 8 ? launch_sample_t<8>(p, C, st) : per <= 20 ? launch_sample_t<20>(p, C, st)
         : per <= 64 ? launch_sample_t<64>(p, C, st) : cudaErrorInvalidValue;
}

}  // namespace llmq

// ---- C entry ----------------------------------------------------------------------
using namespace llmq;

extern "C" int llm_sample_tokens(const llm_sample_args* a, void* cuda_stream) {
  Call c;
  if (!c.need(a != nullptr, LLM_ERR_INVALID_ARG, "the arguments are null") ||
      !c.need(a->n_rows >= 1 && a->vocab >= 1, LLM_ERR_INVALID_ARG, "n_rows or vocab is not positive") ||
      !c.need(a->vocab <= 16 * 64 * kSampNT, LLM_ERR_UNSUPPORTED, "%svocab %lld is too large", "", a->vocab) ||
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
