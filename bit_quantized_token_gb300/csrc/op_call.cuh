// What the C entries of the operators on the caller's own tensors share: the
// checks of a call's arguments and its errors (llm_last_error(NULL)).
#pragma once
#include <cuda.h>

#include <cmath>
#include <cstdio>
#include <utility>

#include "llmq.h"
#include "tree.cuh"

namespace llmq {

inline int bad(int code, const char* fmt, const char* a = "", long long b = 0) {
  char msg[256];
  std::snprintf(msg, sizeof(msg), fmt, a, b);
  return op_error(code, msg);
}

inline int cuda_bad(cudaError_t e, const char* what) {
  char msg[256];
  std::snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return op_error(e == cudaErrorMemoryAllocation ? LLM_ERR_OOM : LLM_ERR_CUDA, msg);
}

// cuMemGetAddressRange, looked up once; null where the driver has none.
using AddressRange = CUresult (*)(CUdeviceptr*, size_t*, CUdeviceptr);
inline AddressRange address_range() {
  static const AddressRange fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<AddressRange>(f);
  }();
  return fn;
}

// Checks of one call: the current device, and that every buffer is its memory.
struct Call {
  int dev = -1, n_sm = 0, rc = LLM_OK;
  cudaError_t e = cudaSuccess;  // reported by the first buffer's check, after those of sizes
  static constexpr int kRanges = 4;
  uintptr_t lo[kRanges] = {}, size[kRanges] = {};  // the allocations of the last buffers looked up
  int n_ranges = 0;
  Call() {
    static std::atomic<int> sms[64];
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) {
      n_sm = dev < 64 ? sms[dev].load(std::memory_order_relaxed) : 0;
      if (!n_sm) {
        e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && dev < 64) sms[dev].store(n_sm, std::memory_order_relaxed);
      }
    }
  }
  bool device(const char* name, const void* p, size_t align) {
    if (rc) return false;
    if (!p) {
      rc = bad(LLM_ERR_INVALID_ARG, "%s is null", name);
      return false;
    }
    if (reinterpret_cast<uintptr_t>(p) % align) {
      rc = bad(LLM_ERR_INVALID_ARG, "%s is not aligned to %lld bytes", name, (long long)align);
      return false;
    }
    if (e != cudaSuccess) {
      rc = cuda_bad(e, "current device");
      return false;
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    for (int i = 0; i < kRanges; ++i)
      if (at - lo[i] < size[i]) return true;  // in the allocation of a buffer before: a pool's tensors share some
    cudaPointerAttributes a{};
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) cudaGetLastError();
    const bool dm = a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged;
    if (!dm || (a.type == cudaMemoryTypeDevice && a.device != dev)) {
      rc = bad(LLM_ERR_INVALID_ARG, "%s is not memory of the current device", name);
      return false;
    }
    CUdeviceptr base = 0;
    size_t n = 0;
    const auto range = address_range();
    if (range && range(&base, &n, static_cast<CUdeviceptr>(at)) == CUDA_SUCCESS) {
      lo[n_ranges % kRanges] = base;
      size[n_ranges++ % kRanges] = n;
    }
    return true;
  }
  bool need(bool ok, int code, const char* fmt, const char* a = "", long long b = 0) {
    if (!rc && !ok) rc = bad(code, fmt, a, b);
    return !rc;
  }
};

// Whether rows of `inner` elements at these (size, stride) steps are apart.
inline bool apart(int64_t inner, int n, const int64_t* size, const int64_t* stride) {
  int order[4] = {0, 1, 2, 3};
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if (stride[order[j]] < stride[order[i]]) std::swap(order[i], order[j]);
  int64_t extent = inner;
  for (int i = 0; i < n; ++i) {
    const int64_t s = size[order[i]], t = stride[order[i]];
    if (s <= 1) continue;
    if (t < extent) return false;
    extent += t * (s - 1);
  }
  return true;
}

inline bool check_view(Call& c, const llm_kv_view* v, const char* name) {
  if (!c.need(v != nullptr, LLM_ERR_INVALID_ARG, "%s is null", name)) return false;
  if (!c.need(v->dtype == LLM_BF16 || v->dtype == LLM_Q8G32, LLM_ERR_UNSUPPORTED,
              "%s: rows are bf16 or int8 with a scale per 32 values", name) ||
      !c.need(v->head_dim == 64 || v->head_dim == 128, LLM_ERR_UNSUPPORTED, "%s: head_dim %lld (64 or 128)", name,
              v->head_dim) ||
      !c.need(v->n_seq > 0 && v->n_layers > 0 && v->n_heads > 0 && v->rows >= 0 && v->n_seq <= 65535,
              LLM_ERR_INVALID_ARG, "%s: a size is not positive, or over 65535 sequences", name))
    return false;
  const bool q8 = v->dtype == LLM_Q8G32;
  const int64_t m = q8 ? 16 : 8, sm = v->head_dim / 32;
  if (!c.need(v->seq_stride >= 0 && v->layer_stride >= 0 && v->head_stride >= 0 && v->row_stride >= 0 &&
                  v->seq_stride % m == 0 && v->layer_stride % m == 0 && v->head_stride % m == 0 &&
                  v->row_stride % m == 0,
              LLM_ERR_INVALID_ARG, "%s: a stride is negative or no multiple of 16 bytes", name) ||
      !c.need(v->rows <= 1 || v->row_stride > 0, LLM_ERR_INVALID_ARG, "%s: the row stride is 0", name) ||
      !c.need(v->seq_stride < (1ll << 38) && v->layer_stride < (1ll << 38) && v->head_stride < (1ll << 38) &&
                  v->row_stride < (1ll << 38),
              LLM_ERR_UNSUPPORTED, "%s: a stride of 2^38 elements or more", name))
    return false;
  if (q8 && !c.need(v->scale_seq_stride >= 0 && v->scale_layer_stride >= 0 && v->scale_head_stride >= 0 &&
                    v->scale_row_stride >= 0 && v->scale_seq_stride % sm == 0 && v->scale_layer_stride % sm == 0 &&
                    v->scale_head_stride % sm == 0 && v->scale_row_stride % sm == 0,
                LLM_ERR_INVALID_ARG, "%s: a scale stride is negative or no multiple of a row's scales", name))
    return false;
  return true;
}

inline bool view_memory(Call& c, const llm_kv_view* v, const char* name) {
  if (v->rows == 0) return true;  // an empty cache has no rows to point at
  const size_t sm = 2 * (v->head_dim / 32);
  return c.device(name, v->k, 16) && c.device(name, v->v, 16) &&
         (v->dtype != LLM_Q8G32 || (c.device(name, v->k_scales, sm) && c.device(name, v->v_scales, sm)));
}

inline KvRows rows_of(const llm_kv_view& v) {
  KvRows r;
  r.k = static_cast<const uint8_t*>(v.k);
  r.v = static_cast<const uint8_t*>(v.v);
  r.ks = static_cast<const uint16_t*>(v.k_scales);
  r.vs = static_cast<const uint16_t*>(v.v_scales);
  r.seq = v.seq_stride;
  r.head = v.head_stride;
  r.row = v.row_stride;
  r.sseq = v.scale_seq_stride;
  r.shead = v.scale_head_stride;
  r.srow = v.scale_row_stride;
  r.rows = v.rows;
  return r;
}

inline int finish(cudaError_t e, const char* what) { return e == cudaSuccess ? LLM_OK : cuda_bad(e, what); }

// The checks of llm_tree_attention's arguments, and the kernel's from them.
bool attention_params(Call& c, const llm_tree_attention_args* a, TreeAttnParams& p);

}  // namespace llmq
