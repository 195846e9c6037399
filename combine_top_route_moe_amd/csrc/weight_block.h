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

// 8 E2M1 codes (one dword, code j in bits 4j) times the power of two s, as
// bf16: exact (2 significant bits), one conversion instruction per pair.  It
// reads only the exponent field of s, so that an E8M0 byte shifted there is
// its scale, 0 meaning 2^-127 (checked on the GPU for all codes and bytes).
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

// A raw buffer over `bytes` bytes at the wave-uniform address p (loads past
// them give 0), and loads from it at a uniform byte offset plus one per lane.
// The whole address but the lane's offset stays in scalar registers: with
// plain pointers the compiler keeps a 64-bit vector address per load of the
// unrolled loops and spills.  NT: what is read once per call streams past the
// caches (aux bit 1).
typedef __amdgpu_buffer_rsrc_t buffer_t;
__device__ __forceinline__ buffer_t uniform_buffer(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
template <bool NT>
__device__ __forceinline__ u32x4_t load_b128(buffer_t r, uint32_t lane_off, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)lane_off, (int)off, NT ? 2 : 0);
}
template <bool NT>
__device__ __forceinline__ u32x2_t load_b64(buffer_t r, uint32_t lane_off, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b64(r, (int)lane_off, (int)off, NT ? 2 : 0);
}
template <bool NT>
__device__ __forceinline__ uint32_t load_b32(buffer_t r, uint32_t lane_off, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, (int)lane_off, (int)off, NT ? 2 : 0);
}

// One weight matrix stack [G, N, Kdim] in a packed format, as the kernels
// take it (device pointers; scales and tensor_scale as the format needs).
struct WMat {
  const void* w;
  const void* scales;
  const float* tensor_scale;
};

// The stream of a column tile's fragments f0, f0 + 1, .. over the reduction
// dimension: load(block, kb, f) fetches K-block kb of fragment f0 + f, and
// Block::operand(p) converts piece p.  g: expert, ct: column tile, n_ct:
// column tiles, nkb: Kdim / 128.  For w13 `up0` is the first weight row of
// the tile's up half, whose fragments are 2 and 3 (FP8: the other tile scale).
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
  buffer_t buf;
  uint32_t stride, off;   // bytes between K-steps; the lane's
  __device__ __forceinline__ void init(const WMat& m, int g, int ct, int f0, int n_ct, int nkb,
                                       int /*row0*/, int /*up0*/, int lane) {
    stride = n_ct * 4096;
    const int64_t matrix = (int64_t)nkb * 4 * stride, at = ct * 4096 + f0 * 1024;
    buf = uniform_buffer(static_cast<const char*>(m.w) + g * matrix + at, matrix - at);
    off = (uint32_t)lane * 16u;
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Block& b, int kb, int f, bool /*up*/ = false) const {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      b.v[p] = load_b128<NT>(buf, off + f * 1024, (4 * kb + p) * stride);
  }
};

template <>
struct WStream<MOE_W_FP8> {
  struct Block {
    u32x2_t v[4];
    float s;
    __device__ __forceinline__ bf16x8_t operand(int p) const { return dequant8_fp8(v[p], s); }
  };
  buffer_t buf;
  const float* sc;
  const float* sc_up;
  uint32_t stride, off;
  __device__ __forceinline__ void init(const WMat& m, int g, int ct, int f0, int n_ct, int nkb,
                                       int row0, int up0, int lane) {
    stride = n_ct * 2048;
    const int64_t matrix = (int64_t)nkb * 4 * stride, at = ct * 2048 + f0 * 512;
    buf = uniform_buffer(static_cast<const char*>(m.w) + g * matrix + at, matrix - at);
    off = (uint32_t)lane * 8u;
    const float* s = static_cast<const float*>(m.scales) + (int64_t)g * (n_ct / 2) * nkb;
    sc = s + (int64_t)(row0 / 128) * nkb;
    sc_up = s + (int64_t)(up0 / 128) * nkb;
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Block& b, int kb, int f, bool up = false) const {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      b.v[p] = load_b64<NT>(buf, off + f * 512, (4 * kb + p) * stride);
    b.s = up ? sc_up[kb] : sc[kb];
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
      return dequant8_mxfp4(v[p], __uint_as_float(((s >> (8 * p)) & 0xffu) << 23));
    }
  };
  buffer_t buf, sbuf;
  uint32_t stride;   // code bytes between K-blocks (scales: 1/16 of them)
  uint32_t off, soff;
  __device__ __forceinline__ void init(const WMat& m, int g, int ct, int f0, int n_ct, int nkb,
                                       int /*row0*/, int /*up0*/, int lane) {
    stride = n_ct * 4096;
    const int64_t matrix = (int64_t)nkb * stride, at = ct * 4096 + f0 * 1024;
    buf = uniform_buffer(static_cast<const char*>(m.w) + g * matrix + at, matrix - at);
    sbuf = uniform_buffer(static_cast<const char*>(m.scales) + (g * matrix + at) / 16,
                          (matrix - at) / 16);
    off = (uint32_t)lane * 16u;
    soff = (uint32_t)(lane & 15) * 4u;
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Block& b, int kb, int f, bool /*up*/ = false) const {
    b.v = load_b128<NT>(buf, off + f * 1024, kb * stride);
    b.s = load_b32<NT>(sbuf, soff + f * 64, kb * (stride / 16));
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
  buffer_t buf, sbuf;
  float g;
  uint32_t stride;   // code bytes between K-blocks (scales: 1/8 of them)
  uint32_t off, soff;
  __device__ __forceinline__ void init(const WMat& m, int grp, int ct, int f0, int n_ct, int nkb,
                                       int /*row0*/, int /*up0*/, int lane) {
    stride = n_ct * 4096;
    const int64_t matrix = (int64_t)nkb * stride, at = ct * 4096 + f0 * 1024;
    buf = uniform_buffer(static_cast<const char*>(m.w) + grp * matrix + at, matrix - at);
    sbuf = uniform_buffer(static_cast<const char*>(m.scales) + (grp * matrix + at) / 8,
                          (matrix - at) / 8);
    off = (uint32_t)lane * 16u;
    soff = (uint32_t)((lane >> 5) * 16 + (lane & 15)) * 4u;
    g = m.tensor_scale[grp];
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Block& b, int kb, int f, bool /*up*/ = false) const {
    b.v = load_b128<NT>(buf, off + f * 1024, kb * stride);
    b.s = load_b32<NT>(sbuf, soff + f * 128, kb * (stride / 8));
    b.g = g;
  }
};

}  // namespace moe
