// New tokens' K and V rows into a cache, with the norms and the rotation of
// their q and k heads, and cached rows back out as values (see serve.cuh).
#include <type_traits>

#include "common.cuh"
#include "op_call.cuh"
#include "serve.cuh"

namespace llmq {
namespace {

// ---- append --------------------------------------------------------------------
// A head of q or k: x / sqrt(mean(x^2) + eps) w (with a norm), then the pairs
// (i, i + hd/2) or (2i, 2i + 1) turned by position times freq_i. A group of hd/16
// lanes holds a row, a lane eight dims of the first half and the same eight of the
// second: both kinds of pairs lie in one lane, 32 neighbouring dims in four, and
// the norm is a sum over the group. Everything is fp32 and rounded once, into
// the outputs' type.
//
// Angles: the turn of a position is kept modulo 1 in 64-bit fixed point, so that
// position times turn wraps where an angle would and no position is too far (the
// table's 2^-50 of a turn grows with the position: 2^-30 at 2^20). The quadrant is
// taken off in integers; sincospi sees at most a quarter of a half turn.
//
// Int8 rows: per 32 values a scale fp16(amax / 127) and codes round(x / scale),
// halves away from zero, clamped to +-127, decided in fp32: the cache's own
// format and roundings. A scale past fp16's range saturates (values beyond 8.3e6
// become the largest that the row can hold), a NaN makes its 32 values NaN.
//
// Bound by HBM and its own instructions for many tokens (8192 of 16/8 heads x 128 in bf16, norms and rotation:
// 29 us, 4.6 TB/s, into int8 rows 42; a lane that held four neighbouring dims instead took 74; packed products of two
// values no less), by the launch for few (one token of 32/4 heads x 64 2.2 us, 32 of 16/8 heads x 128 into int8 rows 4.0).
// Seven CTAs on an SM, in 72 registers: 30.9 / 27.8 / 27.7 / 33.0 us with the compiler's 80, 72, 64 and 48.
constexpr int kAppendThreads = 128;

// eight values, of which the loads come before any use
struct Eight {
  uint4 w[2];
  __device__ __forceinline__ void load(const void* base, int64_t at, bool f32) {
    if (f32) {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
      w[0] = s[0], w[1] = s[1];
    } else {
      w[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    }
  }
  __device__ __forceinline__ void get(float* x, bool f32) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (f32) {
        x[e] = __uint_as_float((&w[0].x)[e]), x[4 + e] = __uint_as_float((&w[1].x)[e]);
      } else {
        x[2 * e] = __uint_as_float((&w[0].x)[e] << 16), x[2 * e + 1] = __uint_as_float((&w[0].x)[e] & 0xFFFF0000u);
      }
    }
  }
};
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void store4(void* base, int64_t at, const float* x, bool f32) {
  if (f32)
    *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
}

__device__ __forceinline__ void store8(void* base, int64_t at, const float* x, bool f32) {
  if (f32) {
    store4(base, at, x, true);
    store4(base, at + 4, x + 4, true);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
        make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
  }
}

// cos and sin of `angle` 2^-64 turns
__device__ __forceinline__ float2 turn_of(uint64_t angle) {
  const uint32_t hi = (uint32_t)(angle >> 32);
  const uint32_t quad = (hi + 0x20000000u) >> 30;                         // the nearest quarter turn
  const float r = (float)(int)(hi - (quad << 30)) * 4.656612873e-10f;     // 2^-31: half turns, within +-1/4
  float s, c;
  sincospif(r, &s, &c);
  const float a = quad & 1 ? s : c, b = quad & 1 ? c : s;
  return make_float2((quad + 1) & 2 ? -a : a, quad & 2 ? -b : b);
}

template <int HD, bool Q8, bool F32>
__global__ void __launch_bounds__(kAppendThreads, 7) append_kv_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = HD / 16, RPW = 32 / LPR;  // lanes of a row, rows of a warp
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, c = lane % LPR;
  const int heads = p.Hq + 2 * p.Hkv, per = RPW * p.passes, slices = (heads + per - 1) / per;
  const int64_t w = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(w / slices), h0 = (int)(w - (int64_t)t * slices) * per + lane / LPR;
  if (t >= p.T) return;
  // a pass's row: q heads, then k heads, then v heads
  Eight lo, hi;
  auto row_of = [&](int j, int& kind, int& hh) {
    const int h = h0 + j * RPW;
    kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
    hh = kind == 0 ? h : (h - p.Hq) - (kind - 1) * p.Hkv;
    return h < heads && j < p.passes;
  };
  auto load = [&](int j) {
    int kind, hh;
    if (row_of(j, kind, hh)) {
      const void* src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
      const int64_t at = t * (kind == 0 ? p.q_tok : kind == 1 ? p.k_tok : p.v_tok) +
                         hh * (kind == 0 ? p.q_head : kind == 1 ? p.k_head : p.v_head) + 8 * c;
      lo.load(src, at, F32);
      hi.load(src, at + HD / 2, F32);
    } else {
      lo.w[0] = lo.w[1] = hi.w[0] = hi.w[1] = make_uint4(0u, 0u, 0u, 0u);
    }
  };
  load(0);  // on its way while the angles are computed
  const int seq = p.seqs[t], row = p.rows[t];
  const bool kept = seq >= 0 && seq < p.n_seq && row >= 0 && row < p.cache.rows;
  float2 cs[8];
  if (p.rotate) {
    const int64_t pos = p.positions ? p.positions[t] : row;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = p.neox ? 8 * c + e : (e < 4 ? 4 * c + e : HD / 4 + 4 * c + e - 4);
      cs[e] = turn_of((uint64_t)pos * p.freq[i]);
    }
  }
#pragma unroll 1
  for (int j = 0; j < p.passes; ++j) {
    int kind, hh;
    const bool in = row_of(j, kind, hh);
    float x[16];
    lo.get(x, F32);
    hi.get(x + 8, F32);
    load(j + 1);
    const float* wn = kind == 0 ? p.q_norm : kind == 1 ? p.k_norm : nullptr;
    if (p.q_norm || p.k_norm) {  // (by the whole warp: its rows may be of different kinds)
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (wn && in) {
        const float inv = rsqrtf(fmaf(ss, 1.0f / HD, p.eps));
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 a = __ldg(reinterpret_cast<const float4*>(wn + (e & 8 ? HD / 2 : 0) + 8 * c + (e & 4)));
          x[e] *= inv * a.x, x[e + 1] *= inv * a.y, x[e + 2] *= inv * a.z, x[e + 3] *= inv * a.w;
        }
      }
    }
    if (p.rotate && kind < 2) {
      auto turned = [&](float& a, float& b, float2 cs_) {
        const float a0 = a;
        a = a0 * cs_.x - b * cs_.y;
        b = a0 * cs_.y + b * cs_.x;
      };
      if (p.neox) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turned(x[e], x[e + 8], cs[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) turned(x[2 * e], x[2 * e + 1], cs[e]);
      }
    }
    if (in && kind == 0) {
      const int64_t at = t * p.o_tok + hh * p.o_head + 8 * c;
      store8(p.q_out, at, x, p.out_f32);
      store8(p.q_out, at + HD / 2, x + 8, p.out_f32);
    }
    uint8_t* base = const_cast<uint8_t*>(kind == 2 ? p.cache.v : p.cache.k);
    const int64_t at = (int64_t)seq * p.cache.seq + (int64_t)hh * p.cache.head + (int64_t)row * p.cache.row;
    if constexpr (!Q8) {
      if (in && kind > 0 && kept) {
        store8(base, at + 8 * c, x, false);
        store8(base, at + HD / 2 + 8 * c, x + 8, false);
      }
    } else if (__any_sync(0xffffffffu, in && kind > 0)) {
      uint2 word[2];
      uint16_t sc[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {  // of either half: four lanes hold 32 neighbouring dims
        uint32_t top = 0;            // of the sizes as integers: a NaN's is above all others
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[8 * g + e]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float amax = __uint_as_float(top);
        const __half dh = __float2half_rn(top > 0x7F800000u ? amax : fminf(amax / 127.0f, 65504.f));
        const float dq = __half2float(dh);
        uint32_t codes[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float cf = dq == 0.f ? 0.f : fminf(fmaxf(roundf(x[8 * g + e] / dq), -127.f), 127.f);
          codes[e / 4] |= ((uint32_t)(int)cf & 0xFFu) << (8 * (e & 3));
        }
        word[g] = make_uint2(codes[0], codes[1]);
        sc[g] = __half_as_ushort(dh);
      }
      if (in && kind > 0 && kept) {
        *reinterpret_cast<uint2*>(base + at + 8 * c) = word[0];
        *reinterpret_cast<uint2*>(base + at + HD / 2 + 8 * c) = word[1];
        if ((c & 3) == 0) {
          uint16_t* s = const_cast<uint16_t*>(kind == 2 ? p.cache.vs : p.cache.ks) + (int64_t)seq * p.cache.sseq +
                        (int64_t)hh * p.cache.shead + (int64_t)row * p.cache.srow;
          s[c / 4] = sc[0];
          s[HD / 64 + c / 4] = sc[1];
        }
      }
    }
  }
}

// ---- read ----------------------------------------------------------------------
// A lane takes eight values of a K row and of the V row beside it (one index for both: the
// index arithmetic of every row by itself took half of the issue slots) and writes 16 bytes,
// or 32, of each output; two such pairs of a thread in flight. Rows run over (token, head) of
// a layer, so that neighbouring ones write neighbouring outputs. A token whose sequence
// or row is out of range reads zeros.
//
// Bound by HBM: 4099 tokens x 28 layers x 8 heads x 128 of int8 rows to bf16 124 us (5.8 TB/s, 85 % of
// a copy's; 121 / 124 / 139 with one, two and four pairs in flight, but fp32 231 / 217 / 230), of bf16 rows
// 136 us (6.9 TB/s); by the launch for few: 37 tokens x 22 layers x 4 heads x 64, bf16 to fp32, 2.4 us.
constexpr int kReadThreads = 256, kReadRows = 2;

// the values of eight bf16 or, times f, of eight codes (0 times an infinite scale is NaN, as in a product)
template <bool Q8>
__device__ __forceinline__ void values_of(float* y, uint4 x, float f) {
  if constexpr (Q8) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {  // bytes behind 2^23, less 2^23 + 128
      const uint32_t codes = (e < 4 ? x.x : x.y) ^ 0x80808080u;
      y[e] = __uint_as_float(__byte_perm(codes, 0x4B000000u, 0x7440 + (e & 3)));
      y[e + 1] = __uint_as_float(__byte_perm(codes, 0x4B000000u, 0x7441 + (e & 3)));
      add2(y[e], y[e + 1], y[e], y[e + 1], -8388736.f, -8388736.f);
      mul2(y[e], y[e + 1], y[e], y[e + 1], f);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[2 * e] = __uint_as_float((&x.x)[e] << 16);
      y[2 * e + 1] = __uint_as_float((&x.x)[e] & 0xFFFF0000u);
    }
  }
}

template <int HD, bool Q8>
__global__ void __launch_bounds__(kReadThreads) read_kv_kernel(const ReadParams p) {
  constexpr int LPR = HD / 8, RPB = kReadThreads / LPR;  // lanes of a row; rows of a block's pass
  pdl_wait();
  pdl_trigger();
  const int c = threadIdx.x % LPR, l = blockIdx.y, n = p.T * p.H;
  const int64_t first = (int64_t)blockIdx.x * RPB * kReadRows + threadIdx.x / LPR;
  uint4 x[kReadRows][2];
  float f[kReadRows][2];
  int64_t to[kReadRows];
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const int64_t i = first + u * RPB;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) x[u][kv] = make_uint4(0u, 0u, 0u, 0u), f[u][kv] = 0.f;
    to[u] = -1;
    if (i >= n) continue;
    const int t = p.by_heads.div((int)i), h = (int)i - t * p.H;
    to[u] = l * p.o_layer + (int64_t)t * p.o_tok + h * p.o_head + 8 * c;
    const int seq = p.seqs[t], row = p.rows[t];
    if (seq < 0 || seq >= p.n_seq || row < 0 || row >= p.cache.rows) continue;
    const int64_t at = (int64_t)seq * p.cache.seq + l * p.layer + h * p.cache.head + (int64_t)row * p.cache.row + 8 * c;
    if constexpr (!Q8) {
      x[u][0] = __ldcs(reinterpret_cast<const uint4*>(p.cache.k + 2 * at));
      x[u][1] = __ldcs(reinterpret_cast<const uint4*>(p.cache.v + 2 * at));
    } else {
      const uint2 k = __ldcs(reinterpret_cast<const uint2*>(p.cache.k + at)), v = __ldcs(reinterpret_cast<const uint2*>(p.cache.v + at));
      x[u][0].x = k.x, x[u][0].y = k.y, x[u][1].x = v.x, x[u][1].y = v.y;
      const int64_t s = (int64_t)seq * p.cache.sseq + l * p.slayer + h * p.cache.shead + (int64_t)row * p.cache.srow + c / 4;
      f[u][0] = __half2float(__ushort_as_half(p.cache.ks[s]));
      f[u][1] = __half2float(__ushort_as_half(p.cache.vs[s]));
    }
  }
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    if (to[u] < 0) continue;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      void* out = kv ? p.v : p.k;
      if (!Q8 && !p.f32) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + to[u]) = x[u][kv];
      } else {
        float y[8];
        values_of<Q8>(y, x[u][kv], f[u][kv]);
        store8(out, to[u], y, p.f32);
      }
    }
  }
}

}  // namespace

cudaError_t launch_append_kv(AppendParams& p, int hd, bool q8, int n_sm, cudaStream_t st) {
  const int rpw = 512 / hd, heads = p.Hq + 2 * p.Hkv, groups = (heads + rpw - 1) / rpw;
  // One pass a warp while there are fewer than six warps an SM; a warp that takes more rows of its token computes the
  // token's angles once for them (with 80 registers, 8192 tokens of 16/8 heads x 128: 61 / 40 / 32 / 30 us with 1, 2, 4, 8 passes, 512: 6.1
  // / 5.7 / 4.7 / 6.0, 64: 2.8 / 3.3 / 4.1 / 5.9).
  const int64_t per = (int64_t)p.T * groups / (6 * (int64_t)n_sm);
  p.passes = (int)(per < 1 ? 1 : per < groups ? per : groups);
  const int64_t warps = (int64_t)p.T * ((heads + rpw * p.passes - 1) / (rpw * p.passes));
  const dim3 grid((unsigned)((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32)));
  const auto of_type = [&](auto f32) {
    constexpr bool F32 = decltype(f32)::value;
    return hd == 64 ? (q8 ? append_kv_kernel<64, true, F32> : append_kv_kernel<64, false, F32>)
                    : (q8 ? append_kv_kernel<128, true, F32> : append_kv_kernel<128, false, F32>);
  };
  const auto kern = p.f32 ? of_type(std::true_type()) : of_type(std::false_type());
  return launch_cluster(kern, grid, kAppendThreads, 1, 0, st, p, p.pdl);
}

cudaError_t launch_read_kv(const ReadParams& p, int hd, bool q8, cudaStream_t st) {
  const int64_t rows = (int64_t)p.T * p.H, per = (int64_t)kReadRows * kReadThreads * 8 / hd;
  const auto kern = hd == 64 ? (q8 ? read_kv_kernel<64, true> : read_kv_kernel<64, false>)
                             : (q8 ? read_kv_kernel<128, true> : read_kv_kernel<128, false>);
  return launch_cluster(kern, dim3((unsigned)((rows + per - 1) / per), p.L), kReadThreads, 1, 0, st, p, p.pdl);
}

}  // namespace llmq

// ---- C entries -------------------------------------------------------------------
using namespace llmq;

namespace {

// The turns of base^(-2i/hd) radians a position, in 2^-64 turns. Powers of one
// root by its binary powers: six calls of pow, each power within 2^-50.
void turns_of(double theta, int hd, uint64_t* freq) {
  double root[6];
  for (int k = 0; k < 6; ++k) root[k] = std::pow(theta, -2.0 * (1 << k) / hd);
  for (int i = 0; i < hd / 2; ++i) {
    double f = 0.15915494309189533577;  // 1 / (2 pi)
    for (int k = 0; k < 6; ++k)
      if (i >> k & 1) f *= root[k];
    f -= std::floor(f);  // (a base below 1/(2 pi) turns more than once)
    const double x = std::nearbyint(f * 18446744073709551616.0);
    freq[i] = x >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(x);
  }
}

bool strides_ok(Call& c, const int64_t* s, int n, int64_t m, const char* name) {
  for (int i = 0; i < n; ++i)
    if (!c.need(s[i] >= 0 && s[i] % m == 0 && s[i] < (1ll << 38), LLM_ERR_INVALID_ARG,
                "a stride of %s is negative, over 2^38 or no multiple of 16 bytes", name))
      return false;
  return true;
}

bool view_apart(const llm_kv_view& v) {
  const int64_t size[4] = {v.n_seq, v.n_layers, v.n_heads, v.rows};
  const int64_t stride[4] = {v.seq_stride, v.layer_stride, v.head_stride, v.row_stride};
  const int64_t sstride[4] = {v.scale_seq_stride, v.scale_layer_stride, v.scale_head_stride, v.scale_row_stride};
  return apart(v.head_dim, 4, size, stride) && (v.dtype != LLM_Q8G32 || apart(v.head_dim / 32, 4, size, sstride));
}

}  // namespace

extern "C" {

int llm_append_kv(const llm_append_kv_args* a, void* cuda_stream) {
  Call c;
  if (!c.need(a != nullptr, LLM_ERR_INVALID_ARG, "the arguments are null")) return c.rc;
  if (!c.need((a->dtype == LLM_BF16 || a->dtype == LLM_F32) && (a->out_dtype == LLM_BF16 || a->out_dtype == LLM_F32),
              LLM_ERR_UNSUPPORTED, "q, k, v and q_out are bf16 or f32") ||
      !c.need(a->n_tokens >= 1 && a->n_tokens <= (1 << 24), LLM_ERR_INVALID_ARG, "n_tokens is not in 1..2^24") ||
      !check_view(c, a->cache, "cache"))
    return c.rc;
  const llm_kv_view& v = *a->cache;
  if (!c.need(v.n_layers == 1, LLM_ERR_INVALID_ARG, "the cache view has several layers") ||
      !c.need(a->n_heads >= 0 && a->n_heads <= 4096 && v.n_heads <= 4096, LLM_ERR_UNSUPPORTED, "too many heads") ||
      !c.need((a->n_heads > 0) == (a->q != nullptr), LLM_ERR_INVALID_ARG, "n_heads and q do not match") ||
      !c.need(a->rope_theta == 0.0 || (a->rope_theta > 0.0 && std::isfinite(a->rope_theta)), LLM_ERR_INVALID_ARG,
              "rope_theta is not positive and finite (0: no rotation)") ||
      // (a base near 0 turns so fast that 64 bits of theta^(-2i/hd) leave nothing of its fraction)
      !c.need(a->rope_theta == 0.0 || a->rope_theta >= 1.0 / 1024, LLM_ERR_UNSUPPORTED, "rope_theta is below 2^-10") ||
      !c.need(a->rope_neox == 0 || a->rope_neox == 1, LLM_ERR_INVALID_ARG, "rope_neox must be 0 or 1") ||
      !c.need(!(a->q_norm || a->k_norm) || (a->norm_eps > 0.f && std::isfinite(a->norm_eps)), LLM_ERR_INVALID_ARG,
              "norm_eps is not positive"))
    return c.rc;
  const int64_t m = a->dtype == LLM_F32 ? 4 : 8, mo = a->out_dtype == LLM_F32 ? 4 : 8;
  const int64_t size[2] = {a->n_tokens, a->n_heads};
  if (!strides_ok(c, a->k_strides, 2, m, "k") || !strides_ok(c, a->v_strides, 2, m, "v") ||
      (a->q && (!strides_ok(c, a->q_strides, 2, m, "q") || !strides_ok(c, a->out_strides, 2, mo, "q_out") ||
                !c.need(apart(v.head_dim, 2, size, a->out_strides), LLM_ERR_INVALID_ARG, "rows of q_out overlap") ||
                !c.need(a->q_out != a->q || (a->dtype == a->out_dtype && a->q_strides[0] == a->out_strides[0] &&
                                             a->q_strides[1] == a->out_strides[1]),
                        LLM_ERR_INVALID_ARG, "q_out is q with another type or strides"))) ||
      !c.need(view_apart(v), LLM_ERR_INVALID_ARG, "rows of the cache overlap") || !view_memory(c, a->cache, "cache") ||
      !c.device("k", a->k, 16) || !c.device("v", a->v, 16) || !c.device("seqs", a->seqs, 4) ||
      !c.device("rows", a->rows, 4) || (a->positions && !c.device("positions", a->positions, 4)) ||
      (a->q && (!c.device("q", a->q, 16) || !c.device("q_out", a->q_out, 16))) ||
      (a->q_norm && !c.device("q_norm", a->q_norm, 16)) || (a->k_norm && !c.device("k_norm", a->k_norm, 16)))
    return c.rc;
  AppendParams p{};
  p.q = a->q, p.k = a->k, p.v = a->v, p.q_out = a->q_out;
  p.q_tok = a->q_strides[0], p.q_head = a->q_strides[1];
  p.k_tok = a->k_strides[0], p.k_head = a->k_strides[1];
  p.v_tok = a->v_strides[0], p.v_head = a->v_strides[1];
  p.o_tok = a->out_strides[0], p.o_head = a->out_strides[1];
  p.cache = rows_of(v);
  p.seqs = a->seqs, p.rows = a->rows, p.positions = a->positions;
  p.q_norm = a->q ? a->q_norm : nullptr, p.k_norm = a->k_norm;
  p.eps = a->norm_eps;
  p.T = a->n_tokens, p.Hq = a->q ? a->n_heads : 0, p.Hkv = v.n_heads, p.n_seq = v.n_seq;
  p.rotate = a->rope_theta > 0.0;
  p.neox = a->rope_neox;
  p.f32 = a->dtype == LLM_F32, p.out_f32 = a->out_dtype == LLM_F32;
  if (p.rotate) turns_of(a->rope_theta, v.head_dim, p.freq);
  return finish(launch_append_kv(p, v.head_dim, v.dtype == LLM_Q8G32, c.n_sm, static_cast<cudaStream_t>(cuda_stream)),
                "append launch");
}

int llm_read_kv(const llm_kv_view* cache, int32_t n_tokens, const int32_t* seqs, const int32_t* rows, int32_t out_dtype,
                void* k, void* v, const int64_t* out_strides, void* cuda_stream) {
  Call c;
  if (!c.need(out_dtype == LLM_BF16 || out_dtype == LLM_F32, LLM_ERR_UNSUPPORTED, "k and v are read as bf16 or f32") ||
      !c.need(n_tokens >= 1, LLM_ERR_INVALID_ARG, "n_tokens is not positive") || !check_view(c, cache, "cache") ||
      !c.need(cache->n_layers <= 65535, LLM_ERR_UNSUPPORTED, "too many layers") ||
      !c.need((int64_t)n_tokens * cache->n_heads * cache->n_heads < (1ll << 32) && (int64_t)n_tokens * cache->n_heads < (1ll << 31),
              LLM_ERR_UNSUPPORTED, "too many tokens and heads") ||
      !c.need(out_strides != nullptr, LLM_ERR_INVALID_ARG, "out_strides is null") ||
      !strides_ok(c, out_strides, 3, out_dtype == LLM_F32 ? 4 : 8, "k and v"))
    return c.rc;
  const int64_t size[3] = {cache->n_layers, n_tokens, cache->n_heads};
  if (!c.need(apart(cache->head_dim, 3, size, out_strides), LLM_ERR_INVALID_ARG, "rows of the outputs overlap") ||
      !c.need(k != v || !k, LLM_ERR_INVALID_ARG, "k and v are the same memory") ||
      !view_memory(c, cache, "cache") || !c.device("seqs", seqs, 4) || !c.device("rows", rows, 4) ||
      !c.device("k", k, 16) || !c.device("v", v, 16))
    return c.rc;
  ReadParams p{};
  p.cache = rows_of(*cache);
  p.layer = cache->layer_stride, p.slayer = cache->scale_layer_stride;
  p.seqs = seqs, p.rows = rows;
  p.k = k, p.v = v;
  p.o_layer = out_strides[0], p.o_tok = out_strides[1], p.o_head = out_strides[2];
  p.T = n_tokens, p.L = cache->n_layers, p.H = cache->n_heads, p.n_seq = cache->n_seq;
  p.by_heads = FastDiv(p.H);
  p.f32 = out_dtype == LLM_F32;
  return finish(launch_read_kv(p, cache->head_dim, cache->dtype == LLM_Q8G32, static_cast<cudaStream_t>(cuda_stream)),
                "read launch");
}

}  // extern "C"
