// The dense product on E4M3 codes: y = x W^T with a float32 scale per row and
// 128 columns of x and per 128 x 128 tile of W,
//   y[m, n] = sum_b sx[b, m] sw[n / 128, b] (sum over the 128 columns k of
//             block b of qx[m, k] qw[n, k]).
// One v_mfma_scale_f32_16x16x128_f8f6f4 gives a block's code products of 16 x
// 16 outputs, which one multiply-add per output scales into a float32 sum.
// The weights are the MFMA's A operand (its rows), 16 rows of x its columns: a
// lane then holds four outputs of one row of x, so that the row's scale times
// the tile's is one number per lane and block, and the four lie side by side
// in y.
//
// Packed weights: 16 x 128 tiles of 2 KB, for each 16 rows of W one block
// after another (a wave's stream through K is contiguous); in a tile, half h =
// 0, 1 and lane l = 0..63 the 16 codes of row l % 16, columns 64 h + 16 (l /
// 16) .. +16: both halves are one operand, whichever way it is fetched.
#include "gemm_common.h"
#include "reduce.h"

namespace moe {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t operand(const u32x4_t& lo, const u32x4_t& hi) {
  return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ f32x4_t mfma_codes(const i32x8_t& a, const i32x8_t& b) {
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 127, 0, 127);
}

// Four outputs side by side of one row; `some` of them lie in the matrix.
template <bool F32>
__device__ __forceinline__ void store4(void* y, int64_t at, const f32x4_t& v, int some, bool wide) {
  if (F32) {
    float* p = static_cast<float*>(y) + at;
    if (wide) {
      *reinterpret_cast<f32x4_t*>(p) = v;
    } else {
      for (int q = 0; q < 4; ++q)
        if (q < some) p[q] = v[q];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(y) + at;
    if (wide) {
      *reinterpret_cast<u32x2_t*>(p) = u32x2_t{
          __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{v[0], v[1]}, bf16x2_t)),
          __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{v[2], v[3]}, bf16x2_t))};
    } else {
      for (int q = 0; q < 4; ++q)
        if (q < some) p[q] = (uint16_t)f32_to_bf16(v[q]);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows: a workgroup owns 16 rows of W and 16 MT rows of x; its waves take
// the blocks of K in turn and add up through LDS, in order.  Bound by the
// weights' bytes, which are read once, straight into the operand's registers.
template <int MT, int NW, int PF, bool F32>
__global__ void __launch_bounds__(NW * kWave) linear_rows_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t sstride, int64_t M,
    const uint8_t* __restrict__ wq, const float* __restrict__ wsc, int N, int nkb, void* __restrict__ y) {
  __shared__ f32x4_t red[NW][MT][kWave];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ct = blockIdx.x;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const int64_t K = (int64_t)nkb * 128;
  const uint8_t* xr[MT];
  const float* sr[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = min(m0 + 16 * j + (lane & 15), M - 1);   // rows past the end re-read the last
    xr[j] = x + m * K + 16 * (lane >> 4);
    sr[j] = xs + m;
  }
  const u32x4_t* wp = reinterpret_cast<const u32x4_t*>(wq) + (int64_t)ct * nkb * 128 + lane;
  const float* sw = wsc + (int64_t)(ct / 8) * nkb;

  u32x4_t wlo[PF], whi[PF];
  auto fill = [&](int slot, int b) {
    const u32x4_t* p = wp + (int64_t)min(b, nkb - 1) * 128;
    wlo[slot] = __builtin_nontemporal_load(p);
    whi[slot] = __builtin_nontemporal_load(p + kWave);
  };
  f32x4_t acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < PF; ++s) fill(s, w + NW * s);
  for (int b0 = w; b0 < nkb; b0 += NW * PF) {
#pragma unroll
    for (int s = 0; s < PF; ++s) {
      const int b = b0 + NW * s;
      if (b < nkb) {
        const float scale = sw[b];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const u32x4_t* p = reinterpret_cast<const u32x4_t*>(xr[j] + (int64_t)b * 128);
          const f32x4_t t = mfma_codes(operand(wlo[s], whi[s]), operand(p[0], p[4]));
          const float c = sr[j][b * sstride] * scale;
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[j][q] = __builtin_fmaf(t[q], c, acc[j][q]);
        }
      }
      fill(s, b + NW * PF);
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) red[w][j][lane] = acc[j];
  __syncthreads();
  const int n = ct * 16 + 4 * (lane >> 4);
  for (int j = w; j < MT; j += NW) {
    f32x4_t v = red[0][j][lane];
#pragma unroll
    for (int i = 1; i < NW; ++i) {
      const f32x4_t a = red[i][j][lane];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += a[q];
    }
    const int64_t m = m0 + 16 * j + (lane & 15);
    if (m < M && n < N) store4<F32>(y, m * N + n, v, N - n, (N & 3) == 0);
  }
}

// ---------------------------------------------------------------------------
// Packing: one workgroup per 128 x 128 tile of W [N, K], through LDS, so that
// the transposed order costs no more than the plain one.
template <bool QUANT, bool TRANS>
__global__ void __launch_bounds__(256) pack_linear_kernel(
    const uint16_t* __restrict__ wide, const uint8_t* __restrict__ codes, const float* __restrict__ scales,
    int N, int K, uint8_t* __restrict__ packed, float* __restrict__ packed_scales) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[128][144];
  __shared__ float top[4];
  const int nb = blockIdx.y, kb = blockIdx.x, n_nb = gridDim.y, n_kb = gridDim.x;
  const int64_t row0 = (int64_t)nb * 128;
  float s;
  if (QUANT) {
    uint4 v[8];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = threadIdx.x + 256 * i, r = c >> 4;
      v[i] = row0 + r < N ? reinterpret_cast<const uint4*>(wide + (row0 + r) * K + kb * 128)[c & 15]
                          : make_uint4(0, 0, 0, 0);
      float f[8];
      unpack8(v[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
    }
    m = wave_top_f32(m);
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
    __syncthreads();
    s = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) / 448.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = threadIdx.x + 256 * i;
      float f[8];
      unpack8(v[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = s > 0.0f ? fminf(fmaxf(f[j] / s, -448.0f), 448.0f) : 0.0f;
      *reinterpret_cast<uint2*>(&tile[c >> 4][8 * (c & 15)]) = e4m3x8(f);
    }
  } else {
    s = scales[(int64_t)nb * n_kb + kb];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = threadIdx.x + 256 * i, r = c >> 3;
      *reinterpret_cast<uint4*>(&tile[r][16 * (c & 7)]) =
          row0 + r < N ? reinterpret_cast<const uint4*>(codes + (row0 + r) * K + kb * 128)[c & 7]
                       : make_uint4(0, 0, 0, 0);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) packed_scales[TRANS ? (int64_t)kb * n_nb + nb : (int64_t)nb * n_kb + kb] = s;
  // the tile's 8 x 128 units of 16 bytes: rows 16 i + l % 16 (of W or of W^T)
  const int64_t blk = TRANS ? nb : kb, blocks = TRANS ? n_nb : n_kb;
  const int64_t ct0 = (TRANS ? (int64_t)kb : (int64_t)nb) * 8;
  const int64_t tiles = TRANS ? K / 16 : (N + 15) / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = threadIdx.x + 256 * i, sub = u >> 7, h = (u >> 6) & 1, l = u & 63;
    if (ct0 + sub >= tiles) continue;
    const int r = 16 * sub + (l & 15), c = 64 * h + 16 * (l >> 4);
    uint4 out;
    if (TRANS) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = tile[c + 4 * j][r] | tile[c + 4 * j + 1][r] << 8 | tile[c + 4 * j + 2][r] << 16 |
               (uint32_t)tile[c + 4 * j + 3][r] << 24;
      out = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      out = *reinterpret_cast<const uint4*>(&tile[r][c]);
    }
    reinterpret_cast<uint4*>(packed)[((ct0 + sub) * blocks + blk) * 128 + h * 64 + l] = out;
  }
}

int launch_pack_linear_fp8(const uint16_t* w, const uint8_t* codes, const float* scales, int N, int K,
                           int transpose, uint8_t* packed, float* packed_scales, hipStream_t stream) {
  const dim3 grid(K / 128, (N + 127) / 128);
#define MOE_PACK(Q, T)                                                                          \
  hipLaunchKernelGGL((pack_linear_kernel<Q, T>), grid, dim3(256), 0, stream, w, codes, scales, N, K, \
                     packed, packed_scales)
  if (w) {
    if (transpose) MOE_PACK(true, true); else MOE_PACK(true, false);
  } else {
    if (transpose) MOE_PACK(false, true); else MOE_PACK(false, false);
  }
#undef MOE_PACK
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

size_t linear_fp8_workspace_bytes(int64_t M, int N, int K) {
  (void)M, (void)N, (void)K;
  return 0;
}

int launch_linear_fp8(const uint8_t* x, const float* xs, int64_t sstride, int64_t M, int N, int K,
                      const uint8_t* wq, const float* wsc, void* y, int f32, void* workspace,
                      hipStream_t stream) {
  (void)workspace;
  const int nkb = K / 128;
  const int n_ct = (N + 15) / 16;
#define MOE_ROWS(MT, NW, PF)                                                                       \
  do {                                                                                             \
    const int64_t my = (M + 16 * MT - 1) / (16 * MT);                                              \
    if (my > 65535) return MOE_ERR_UNSUPPORTED;                                                    \
    if (f32)                                                                                       \
      hipLaunchKernelGGL((linear_rows_kernel<MT, NW, PF, true>), dim3(n_ct, (unsigned)my), dim3(NW * kWave), \
                         0, stream, x, xs, sstride, M, wq, wsc, N, nkb, y);                        \
    else                                                                                           \
      hipLaunchKernelGGL((linear_rows_kernel<MT, NW, PF, false>), dim3(n_ct, (unsigned)my), dim3(NW * kWave), \
                         0, stream, x, xs, sstride, M, wq, wsc, N, nkb, y);                        \
  } while (0)
  if (M <= 16) MOE_ROWS(1, 4, 4);
  else if (M <= 32) MOE_ROWS(2, 4, 4);
  else MOE_ROWS(4, 4, 2);
#undef MOE_ROWS
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
