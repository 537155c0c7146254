// Gate arithmetic of the block operators, on the device.
#pragma once

#include "common.h"

namespace ret {

constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(g) and 1 - sigmoid(g), each to its own digits: with e = exp(-g), a =
// 1 / (1 + e), and 1 - a = e a where a is the larger of the two, else by
// subtraction (e overflows there, or its reciprocal is less than the least
// normal number, which the hardware's makes 0). The exponent's product is
// rounded relative to |g|, so that the smaller of the two is off by up to about
// (|g| + 8) roundings of 2^-24; they add up to 1 but for two. A NaN stays one in
// both.
__device__ __forceinline__ void sigmoid_pair(float g, float& a, float& one_less) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * g);
  a = __builtin_amdgcn_rcpf(1.0f + e);
  one_less = g < 0.0f ? 1.0f - a : e * a;
}

// e^g and 1 - e^g. Near 0 the difference is the series' own, g (1 + g / 2 (1 +
// g / 3 (1 + g / 4))), whose next term is below g^4 / 120, 2^-22.9 of it at
// 1/16: 1 - a would have a's rounding, 2^-24 / |g| of it.
__device__ __forceinline__ void exp_pair(float g, float& a, float& one_less) {
  a = __builtin_amdgcn_exp2f(kLog2e * g);
  const float series = fmaf(fmaf(fmaf(g, 1.0f / 24, 1.0f / 6), g, 0.5f), g, 1.0f);
  one_less = __builtin_fabsf(g) < 0.0625f ? -g * series : 1.0f - a;
}

// Workgroup barrier that orders LDS accesses only: outstanding global loads
// and stores stay in flight across it.
__device__ __forceinline__ void lds_only_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace ret
