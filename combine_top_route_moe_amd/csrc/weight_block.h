// One expert-weight fragment as the few-row kernels stream it: 16 weight
// rows x one 128-wide block of the reduction dimension, in registers, for
// every weight format, and its conversion to the four bf16 MFMA operands
// (16 x 32 each) that the block holds.
//
// Lane l holds row l % 16; piece p = 0..3 covers columns 32 p + 8 (l / 16)
// .. +8 of the block.  Column tiles (64 weight rows, four fragments) and
// their order are those of the packed layouts in the header.
#pragma once

#include "gemm_common.h"

namespace moe {

// E8M0 byte -> the float32 power of two 2^(byte - 127) (byte 0: 2^-127, a
// subnormal)
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// 8 E2M1 codes (one dword, code j in bits 4j) times the power of two s, as
// bf16: exact (2 significant bits), one conversion instruction per pair.
__device__ __forceinline__ bf16x8_t dequant8_mxfp4(uint32_t c, float s) {
  const u32x4_t w = {
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))};
  return __builtin_bit_cast(bf16x8_t, w);
}

// 8 E2M1 codes times the float32 scale S: bf16(fl32(code * S)), the NVFP4
// fake-quant's value.
__device__ __forceinline__ bf16x8_t dequant8_nvfp4(uint32_t c, float S) {
  const f32x2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0) * S;
  const f32x2_t v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1) * S;
  const f32x2_t v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2) * S;
  const f32x2_t v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3) * S;
  const u32x4_t w = {__builtin_bit_cast(uint32_t, __builtin_convertvector(v0, bf16x2_t)),
                     __builtin_bit_cast(uint32_t, __builtin_convertvector(v1, bf16x2_t)),
                     __builtin_bit_cast(uint32_t, __builtin_convertvector(v2, bf16x2_t)),
                     __builtin_bit_cast(uint32_t, __builtin_convertvector(v3, bf16x2_t))};
  return __builtin_bit_cast(bf16x8_t, w);
}

// 8 E4M3 codes times the float32 scale s: bf16(fl32(code * s)), the FP8
// fake-quant's value.
__device__ __forceinline__ bf16x8_t dequant8_fp8(u32x2_t c, float s) {
  const f32x2_t v0 = __builtin_amdgcn_cvt_pk_f32_fp8(c.x, false) * s;
  const f32x2_t v1 = __builtin_amdgcn_cvt_pk_f32_fp8(c.x, true) * s;
  const f32x2_t v2 = __builtin_amdgcn_cvt_pk_f32_fp8(c.y, false) * s;
  const f32x2_t v3 = __builtin_amdgcn_cvt_pk_f32_fp8(c.y, true) * s;
  const u32x4_t w = {__builtin_bit_cast(uint32_t, __builtin_convertvector(v0, bf16x2_t)),
                     __builtin_bit_cast(uint32_t, __builtin_convertvector(v1, bf16x2_t)),
                     __builtin_bit_cast(uint32_t, __builtin_convertvector(v2, bf16x2_t)),
                     __builtin_bit_cast(uint32_t, __builtin_convertvector(v3, bf16x2_t))};
  return __builtin_bit_cast(bf16x8_t, w);
}

// One weight matrix stack [G, N, Kdim] in a packed format, as the kernels
// take it (device pointers; scales and tensor_scale as the format needs).
struct WMat {
  const void* w;
  const void* scales;
  const float* tensor_scale;
};

// NT: weights read once per call stream past the caches.
template <bool NT, typename V>
__device__ __forceinline__ V stream_load(const V* p) {
  if constexpr (NT)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}

// A fragment's stream over the reduction dimension: load(kb) fetches block
// kb's registers, operand(p) converts piece p.  g: expert, ct: column tile,
// f: fragment within it, n_ct: column tiles, nkb: Kdim / 128, row0: the
// fragment's first weight row (for the FP8 tile scales).
template <int FMT>
struct WStream;

template <>
struct WStream<MOE_W_BF16> {
  struct Block {
    u32x4_t v[4];
    __device__ __forceinline__ bf16x8_t operand(int p) const {
      return __builtin_bit_cast(bf16x8_t, v[p]);
    }
  };
  const u32x4_t* base;
  int stride;   // 16-byte units between K-steps
  __device__ __forceinline__ void init(const WMat& m, int g, int ct, int f, int n_ct, int nkb,
                                       int /*row0*/, int lane) {
    stride = n_ct * 256;
    base = static_cast<const u32x4_t*>(m.w) + ((int64_t)g * nkb * 4 * n_ct + ct) * 256 + f * 64 + lane;
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Block& b, int kb) const {
#pragma unroll
    for (int p = 0; p < 4; ++p) b.v[p] = stream_load<NT>(base + (int64_t)(4 * kb + p) * stride);
  }
};

template <>
struct WStream<MOE_W_FP8> {
  struct Block {
    u32x2_t v[4];
    float s;
    __device__ __forceinline__ bf16x8_t operand(int p) const { return dequant8_fp8(v[p], s); }
  };
  const u32x2_t* base;
  const float* sc;
  int stride;
  __device__ __forceinline__ void init(const WMat& m, int g, int ct, int f, int n_ct, int nkb,
                                       int row0, int lane) {
    stride = n_ct * 256;
    base = static_cast<const u32x2_t*>(m.w) + ((int64_t)g * nkb * 4 * n_ct + ct) * 256 + f * 64 + lane;
    sc = static_cast<const float*>(m.scales) + ((int64_t)g * (n_ct / 2) + row0 / 128) * nkb;
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Block& b, int kb) const {
#pragma unroll
    for (int p = 0; p < 4; ++p) b.v[p] = stream_load<NT>(base + (int64_t)(4 * kb + p) * stride);
    b.s = sc[kb];
  }
};

// 4-bit codes: a lane's 16 bytes are its whole 32 weights of the block
// (dword p is piece p); its scales one dword, byte p for piece p.
template <>
struct WStream<MOE_W_MXFP4> {
  struct Block {
    u32x4_t v;
    uint32_t s;
    __device__ __forceinline__ bf16x8_t operand(int p) const {
      return dequant8_mxfp4(v[p], e8m0_to_f32((s >> (8 * p)) & 0xffu));
    }
  };
  const u32x4_t* base;
  const uint32_t* sc;
  int stride;   // fragments between K-blocks
  __device__ __forceinline__ void init(const WMat& m, int g, int ct, int f, int n_ct, int nkb,
                                       int /*row0*/, int lane) {
    stride = n_ct * 4;
    const int64_t frag = ((int64_t)g * nkb * n_ct + ct) * 4 + f;
    base = static_cast<const u32x4_t*>(m.w) + frag * 64 + lane;
    sc = static_cast<const uint32_t*>(m.scales) + frag * 16 + (lane & 15);
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Block& b, int kb) const {
    const int64_t o = (int64_t)kb * stride;
    b.v = stream_load<NT>(base + o * 64);
    b.s = stream_load<NT>(sc + o * 16);
  }
};

template <>
struct WStream<MOE_W_NVFP4> {
  struct Block {
    u32x4_t v;
    uint32_t s;
    float g;
    __device__ __forceinline__ bf16x8_t operand(int p) const {
      const float b = p == 0   ? __builtin_amdgcn_cvt_f32_fp8((int)s, 0)
                      : p == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)s, 1)
                      : p == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)s, 2)
                               : __builtin_amdgcn_cvt_f32_fp8((int)s, 3);
      return dequant8_nvfp4(v[p], b * g);
    }
  };
  const u32x4_t* base;
  const uint32_t* sc;
  float g;
  int stride;
  __device__ __forceinline__ void init(const WMat& m, int grp, int ct, int f, int n_ct, int nkb,
                                       int /*row0*/, int lane) {
    stride = n_ct * 4;
    const int64_t frag = ((int64_t)grp * nkb * n_ct + ct) * 4 + f;
    base = static_cast<const u32x4_t*>(m.w) + frag * 64 + lane;
    sc = static_cast<const uint32_t*>(m.scales) + frag * 32 + (lane >> 5) * 16 + (lane & 15);
    g = m.tensor_scale[grp];
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Block& b, int kb) const {
    const int64_t o = (int64_t)kb * stride;
    b.v = stream_load<NT>(base + o * 64);
    b.s = stream_load<NT>(sc + o * 32);
    b.g = g;
  }
};

}  // namespace moe
