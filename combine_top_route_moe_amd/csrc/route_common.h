// What the routing kernels share: lane movements, the ranking of a logit, a
// slot's weight.
#pragma once

#include "common.h"

namespace moe {

// One DPP lane movement within each row of 16 lanes (every lane active).
template <int kCtrl>
__device__ __forceinline__ int row16_dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, kCtrl, 0xF, 0xF, false);
}

// Sum of x over lanes 0 .. n-1 (n <= 64, the same in every lane), read lane
// by lane in ascending order: no LDS traffic.
__device__ __forceinline__ double sum_lanes_below(double x, int n) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  double s = 0.0;
  for (int k = 0; k < n; ++k) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, k);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), k);
    s += __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
  }
  return s;
}

// A NaN logit ranks as -inf: it can never hide a real candidate from the
// argmax (every comparison with a NaN is false) and the order stays total.
__device__ __forceinline__ float rank_value(float x) { return x != x ? -__builtin_inff() : x; }

// exp(l - l_max) in double, with an l equal to l_max counting exp(0) even
// when both are infinite (inf - inf would be NaN): the limit of the softmax
// as the infinite logits grow, and for finite logits the same value.
__device__ __forceinline__ double weight_term(float l, float lmax) {
  return l == lmax ? 1.0 : exp((double)l - (double)lmax);
}

}  // namespace moe
