// Router logits as keys that order them (shared by the expert layer and the routing of prompts).
#pragma once

#include "mx4_launch.hpp"

namespace i8mm {

__device__ __forceinline__ float moe_logit(const void* p, int type, int64_t i) {
  if (type == kMxF32) return static_cast<const float*>(p)[i];
  if (type == kMxF16) return static_cast<float>(static_cast<const _Float16*>(p)[i]);
  return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}

// Order-preserving map of fp32 to unsigned: -inf to 0 (an expert that is off), any NaN to
// the greatest.
__device__ __forceinline__ unsigned moe_key(float v) {
  const unsigned b = __builtin_bit_cast(unsigned, v);
  if (v != v) return 0xffffffffu;
  if (b == 0xff800000u) return 0u;
  const unsigned z = b == 0x80000000u ? 0u : b;  // -0 ties with +0
  return z ^ (z >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float moe_unkey(unsigned k) {
  if (k == 0xffffffffu) return __builtin_nanf("");
  return __builtin_bit_cast(float, k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

}  // namespace i8mm
