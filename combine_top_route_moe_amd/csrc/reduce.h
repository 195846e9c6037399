// Reductions over a wave, and a row of values as E4M3 codes.
#pragma once

#include "common.h"

namespace moe {

// One DPP lane movement within each row of 16 lanes (every lane of the row
// active): 0xB1 and 0x4E swap lanes within a quad, 0x141 mirrors each half
// row, 0x140 the row, so that after the four every lane has met its whole row.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false);
}
template <int kCtrl>
__device__ __forceinline__ float dpp16(float v) {
  return __uint_as_float(dpp16<kCtrl>(__float_as_uint(v)));
}

__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  v = max(v, dpp16<0xB1>(v));
  v = max(v, dpp16<0x4E>(v));
  v = max(v, dpp16<0x141>(v));
  return max(v, dpp16<0x140>(v));
}

__device__ __forceinline__ float row16_sum_f32(float v) {
  v += dpp16<0xB1>(v);
  v += dpp16<0x4E>(v);
  v += dpp16<0x141>(v);
  return v + dpp16<0x140>(v);
}

__device__ __forceinline__ float row16_top_f32(float v) {
  v = fmaxf(v, dpp16<0xB1>(v));
  v = fmaxf(v, dpp16<0x4E>(v));
  v = fmaxf(v, dpp16<0x141>(v));
  return fmaxf(v, dpp16<0x140>(v));
}

__device__ __forceinline__ float lane_f32(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Over the whole wave (every lane active), the result in every lane: the rows of
// 16, then row 0 into 1 and 2 into 3, then both into row 3, read from its last lane.
__device__ __forceinline__ float wave_sum_f32(float v) {
  v = row16_sum_f32(v);
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xA, 0xF, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xC, 0xF, false));
  return lane_f32(v, 63);
}
__device__ __forceinline__ float wave_top_f32(float v) {
  v = row16_top_f32(v);
  int b = __float_as_int(v);
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, 0x142, 0xA, 0xF, false)));
  b = __float_as_int(v);
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, 0x143, 0xC, 0xF, false)));
  return lane_f32(v, 63);
}

// E4M3 codes of 8 values (already divided by the scale and clamped), packed
// low byte first.
__device__ __forceinline__ uint2 e4m3x8(const float* r) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(r[4 * h], r[4 * h + 1], 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(r[4 * h + 2], r[4 * h + 3], p, true);
    w[h] = (uint32_t)p;
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace moe
