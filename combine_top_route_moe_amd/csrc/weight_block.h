// Expert weights as a wave streams them: fragments of 16 weight rows x one
// 128-wide block of the reduction dimension, in registers, for every weight
// format, and their conversion to the four bf16 MFMA operands (16 x 32 each)
// that a fragment's block holds.
//
// Lane l holds row l % 16; piece p = 0..3 covers columns 32 p + 8 (l / 16)
// .. +8 of the block.  Column tiles (64 weight rows, four fragments) and
// their order are those of the packed layouts in the header.
#pragma once

#include "gemm_common.h"

namespace moe {

// Workgroups of 256 threads that one launch can have (2^32 threads).
constexpr int64_t kMaxGrid = 1 << 24;

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

// One weight matrix stack [G, N, Kdim] in a packed format, as the kernels
// take it (device pointers; scales and tensor_scale as the format needs).
struct WMat {
  const void* w;
  const void* scales;
  const float* tensor_scale;
};

// The stream of a column tile's fragments f0 .. f0 + NF - 1 (GU, a w13 tile
// with NF < 4: NF / 2 gate fragments and the matching up ones, two on) over
// the reduction dimension: load(t, kb) fetches K-block kb into a Tile, and
// Tile::operand(f, p) converts piece p of fragment f.  g: expert, ct: column
// tile, n_ct: column tiles, nkb: Kdim / 128; row0, up0: the tile's first weight
// row, and of a w13 tile's up half.
constexpr int frag_of(bool gu, int nf, int f) { return gu && f >= nf / 2 ? f - nf / 2 + 2 : f; }

template <int FMT, int NF, bool GU>
struct WStream;

template <int NF, bool GU>
struct WStream<MOE_W_BF16, NF, GU> {
  struct Tile {
    u32x4_t v[NF][4];
    __device__ __forceinline__ bf16x8_t operand(int f, int p) const {
      return __builtin_bit_cast(bf16x8_t, v[f][p]);
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
  __device__ __forceinline__ void load(Tile& t, int kb) const {
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        t.v[f][p] = load_b128<NT>(buf, off + frag_of(GU, NF, f) * 1024, (4 * kb + p) * stride);
  }
};

template <int NF, bool GU>
struct WStream<MOE_W_FP8, NF, GU> {
  struct Tile {
    u32x2_t v[NF][4];
    float s[2];   // gate (or all), up
    __device__ __forceinline__ bf16x8_t operand(int f, int p) const {
      return dequant8_fp8(v[f][p], s[GU && f >= NF / 2]);
    }
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
  __device__ __forceinline__ void load(Tile& t, int kb) const {
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        t.v[f][p] = load_b64<NT>(buf, off + frag_of(GU, NF, f) * 512, (4 * kb + p) * stride);
    t.s[0] = sc[kb];
    t.s[1] = GU ? sc_up[kb] : t.s[0];
  }
};

// 4-bit codes, whole column tiles: a lane's 16 bytes per fragment are its 32
// weights of the block (dword p is piece p), its scales of the four fragments
// one more 16 bytes (dword f, byte p).
template <bool GU>
struct WStream<MOE_W_MXFP4, 4, GU> {
  struct Tile {
    u32x4_t v[4];
    u32x4_t s;
    __device__ __forceinline__ bf16x8_t operand(int f, int p) const {
      return dequant8_mxfp4(v[f][p], __uint_as_float(((s[f] >> (8 * p)) & 0xffu) << 23));
    }
  };
  buffer_t buf, sbuf;
  uint32_t stride;   // code bytes between K-blocks (scales: 1/16 of them)
  uint32_t off, soff;
  __device__ __forceinline__ void init(const WMat& m, int g, int ct, int /*f0*/, int n_ct, int nkb,
                                       int /*row0*/, int /*up0*/, int lane) {
    stride = 4096;
    const int64_t matrix = (int64_t)nkb * n_ct * 4096, at = (int64_t)ct * nkb * 4096;
    buf = uniform_buffer(static_cast<const char*>(m.w) + g * matrix + at, matrix - at);
    sbuf = uniform_buffer(static_cast<const char*>(m.scales) + (g * matrix + at) / 16,
                          (matrix - at) / 16);
    off = (uint32_t)lane * 16u;
    soff = (uint32_t)(lane & 15) * 16u;
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Tile& t, int kb) const {
#pragma unroll
    for (int f = 0; f < 4; ++f) t.v[f] = load_b128<NT>(buf, off + f * 1024, kb * stride);
    t.s = load_b128<NT>(sbuf, soff, kb * (stride / 16));
  }
};

template <bool GU>
struct WStream<MOE_W_NVFP4, 4, GU> {
  struct Tile {
    u32x4_t v[4];
    u32x4_t s;
    float g;
    __device__ __forceinline__ bf16x8_t operand(int f, int p) const {
      const int q = (int)s[f];
      const float b = p == 0   ? __builtin_amdgcn_cvt_f32_fp8(q, 0)
                      : p == 1 ? __builtin_amdgcn_cvt_f32_fp8(q, 1)
                      : p == 2 ? __builtin_amdgcn_cvt_f32_fp8(q, 2)
                               : __builtin_amdgcn_cvt_f32_fp8(q, 3);
      return dequant8_nvfp4(v[f][p], b * g);
    }
  };
  buffer_t buf, sbuf;
  float g;
  uint32_t stride;   // code bytes between K-blocks (scales: 1/8 of them)
  uint32_t off, soff;
  __device__ __forceinline__ void init(const WMat& m, int grp, int ct, int /*f0*/, int n_ct,
                                       int nkb, int /*row0*/, int /*up0*/, int lane) {
    stride = 4096;
    const int64_t matrix = (int64_t)nkb * n_ct * 4096, at = (int64_t)ct * nkb * 4096;
    buf = uniform_buffer(static_cast<const char*>(m.w) + grp * matrix + at, matrix - at);
    sbuf = uniform_buffer(static_cast<const char*>(m.scales) + (grp * matrix + at) / 8,
                          (matrix - at) / 8);
    off = (uint32_t)lane * 16u;
    soff = (uint32_t)((lane >> 5) * 16 + (lane & 15)) * 16u;
    g = m.tensor_scale[grp];
  }
  template <bool NT = true>
  __device__ __forceinline__ void load(Tile& t, int kb) const {
#pragma unroll
    for (int f = 0; f < 4; ++f) t.v[f] = load_b128<NT>(buf, off + f * 1024, kb * stride);
    t.s = load_b128<NT>(sbuf, soff, kb * (stride / 8));
    t.g = g;
  }
};

}  // namespace moe
