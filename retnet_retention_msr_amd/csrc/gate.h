// Gate arithmetic of the block operators, on the device.
#pragma once

#include "common.h"

namespace ret {

constexpr float kLog2e = 1.4426950408889634f;

// sigmoid(g) and 1 - sigmoid(g), each to a few units in the last place: with
// e = exp(-|g|) the smaller of the two is e / (1 + e) and the larger its
// complement, so 1 - a keeps its digits where a is near 1. Holds for +-inf.
__device__ __forceinline__ void sigmoid_pair(float g, float& a, float& one_less) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(g));
  const float small = e * __builtin_amdgcn_rcpf(1.0f + e);
  const float large = 1.0f - small;
  a = g >= 0.0f ? large : small;
  one_less = g >= 0.0f ? small : large;
}

}  // namespace ret
