// What the sampler and the token probabilities share.
#pragma once
#include <cstdint>

namespace llmq {

constexpr int kSampleMaxK = 64;

// Order-preserving key of a float: a larger value has a larger key (-0 as +0).
__device__ __forceinline__ uint32_t sample_key(float x) {
  uint32_t b = __float_as_uint(x);
  if (b == 0x80000000u) b = 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

}  // namespace llmq
