// Root-mean-square norm of the residual stream with the residual's addition
// in front and FP8 codes behind, and its gradient.
//
// Forward, per row of H channels (float32 between the two roundings):
//   h = bf16(x + residual)                       (x itself without a residual)
//   r = 1 / sqrt(sum(h^2) / H + eps),  p = h w,  v = p r
//   y = bf16(v);  per 128 channels s = amax |v| / 448, code = e4m3(v / s)
// h is rounded before it is normed because that rounded value is what the
// stream keeps: the gradient, which starts from the stored h, is then exactly
// the forward's.  The codes come from the unrounded row,
// as 448 p / amax |p|: r falls out of the quotient, which is rounded once.
//
// Gradient, with hat = h r and g = dy w:
//   dh = r (g - hat sum(g hat) / H) (+ the stream's own gradient),
//   dw = sum over the rows of dy hat.
//
// Both are bound by memory: every tensor is read or written once, a row stays
// in registers between the reduction and its use.  One row belongs to kWaves
// waves (1, 4 or 16 by H, four 16-byte vectors a thread at most), so that the
// loads of a whole row are in flight at once and no loop runs over it.
#include <algorithm>
#include <type_traits>

#include "reduce.h"

namespace moe {

// A row's sum over its kWaves waves; `buf` is theirs, used by one call at a time.
template <int kWaves>
__device__ __forceinline__ float row_sum(float v, float* buf, int wave) {
  v = wave_sum_f32(v);
  if (kWaves == 1) return v;
  if ((threadIdx.x & 63) == 0) buf[wave] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) s += buf[i];
  return s;
}

// The group of rows of workgroup `bid`: workgroups go round the 8 XCDs, and runs of
// 32 groups stay on one, so that the scales of neighbouring rows, which share a
// line, meet in one L2.
__device__ __forceinline__ unsigned row_group(unsigned bid, unsigned groups) {
  constexpr unsigned kRun = 32, kXcds = 8;
  if (bid >= groups / (kRun * kXcds) * (kRun * kXcds)) return bid;
  const unsigned xcd = bid % kXcds, at = bid / kXcds;
  return (at / kRun * kXcds + xcd) * kRun + at % kRun;
}

// Rows pass the caches by, read and written: each is touched once, and what reads
// them next comes after all of them (16384 x 2048: 59.5 us with ordinary accesses,
// 57.5 and 56.4 with the reads or the writes past the caches).
typedef uint32_t vec4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 load_row(const uint4* p) {
  const vec4_t v = __builtin_nontemporal_load(reinterpret_cast<const vec4_t*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ void store_row(uint4* p, const uint4& v) {
  __builtin_nontemporal_store(vec4_t{v.x, v.y, v.z, v.w}, reinterpret_cast<vec4_t*>(p));
}

template <bool kF32>
__device__ __forceinline__ void load_gain(const void* w, int vec, float* out) {
  if (kF32) {
    const float4* p = static_cast<const float4*>(w) + 2 * vec;
    const float4 a = p[0], b = p[1];
    out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
    out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
  } else {
    unpack8(static_cast<const uint4*>(w)[vec], out);
  }
}

__device__ __forceinline__ uint4 to_bf16x8(const float* v) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[2 * j], v[2 * j + 1]}, b2));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Codes of 448 h w / (the block's largest h w) for a float32 gain, whose products have
// 32 bits.  p (the rounded products) times 448 / top is off by 4 roundings, 2^-22; where
// both ends of twice that give the same codes, those are the nearest to the unrounded
// quotient.  Else (0.6 % of the waves) it is rounded to odd in float32, from where the
// rounding to nearest goes the same way: the residuals of the quotient, before and after
// its correction, are put together from exact parts, and the second is 0 where the
// quotient lies half way between two codes, else its sign shows the side.
__device__ __forceinline__ uint2 codes_f32(const float (&p)[8], const uint4& h, const void* weight, int c, float top) {
  const float inv = 448.0f / top;
  float u[8], o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = p[j] * (inv * (1.0f - 0x1p-21f)), o[j] = p[j] * (inv * (1.0f + 0x1p-21f));
  uint2 q = e4m3x8(u);
  const uint2 over = e4m3x8(o);
  if (__any(q.x != over.x || q.y != over.y)) {
    float lo[8], w[8], top_lo = -__builtin_inff();
    unpack8(h, lo);
    load_gain<true>(weight, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {       // h w = p + lo; top_lo of the products that share the largest p
      lo[j] = __builtin_fmaf(lo[j], w[j], -p[j]);
      top_lo = fabsf(p[j]) == top ? fmaxf(top_lo, __builtin_copysignf(1.0f, p[j]) * lo[j]) : top_lo;
    }
    top_lo = row16_top_f32(top_lo);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v0 = p[j] * inv, a = 448.0f * p[j];
      const float rest = __builtin_fmaf(448.0f, lo[j], __builtin_fmaf(448.0f, p[j], -a));
      const float left0 = __builtin_fmaf(-v0, top, a) + __builtin_fmaf(-v0, top_lo, rest);
      const float v = __builtin_fmaf(left0, 1.0f / top, v0);
      const float left = __builtin_fmaf(-v, top, a) + __builtin_fmaf(-v, top_lo, rest);
      const uint32_t bits = __float_as_uint(v);
      const int step = ((int)(__float_as_uint(left) ^ bits) >> 31) | 1;     // away from 0 or towards it
      u[j] = __uint_as_float(left != 0.0f && !(bits & 1) ? bits + step : bits);
    }
    q = e4m3x8(u);
  }
  return q;
}

// A workgroup of 4 waves (16 for the longest rows) holds 4 / kWaves rows.  4096 x 7168
// with the residual, bf16 rows and codes 48 us, 5.6 TB/s; 16384 x 4096 without the
// bf16 rows 76 us, 6.2 TB/s (a copy of 1 GiB: 5.85).
// x, residual and h may be one buffer: a thread stores what it has read.
template <int kWaves, int kVecs, bool kWF32>
__global__ void __launch_bounds__(kWaves == 16 ? 1024 : 256) rmsnorm_kernel(
    const uint16_t* x, const uint16_t* residual, const void* __restrict__ weight, int64_t T, int H,
    float eps, uint16_t* h_out, uint16_t* y, uint8_t* __restrict__ codes,
    float* __restrict__ scales, int64_t sstride, float* __restrict__ rstd) {
  constexpr int kRows = kWaves == 1 ? 4 : 1;
  constexpr int kThreads = kWaves * kWave;
  __shared__ float part[kWaves];
  const int wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)row_group(blockIdx.x, gridDim.x) * kRows + (kWaves == 1 ? wave : 0);
  if (t >= T) return;
  const int tid = kWaves == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int nvec = H / 8;
  const uint4* xr = reinterpret_cast<const uint4*>(x) + t * nvec;
  uint4 hv[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = tid + i * kThreads;
    hv[i] = c < nvec ? load_row(xr + c) : make_uint4(0, 0, 0, 0);
  }
  if (residual) {
    const uint4* rr = reinterpret_cast<const uint4*>(residual) + t * nvec;
    uint4 rv[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = tid + i * kThreads;
      rv[i] = c < nvec ? load_row(rr + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float a[8], b[8];
      unpack8(hv[i], a);
      unpack8(rv[i], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
      hv[i] = to_bf16x8(a);
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float f[8];
    unpack8(hv[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(f[j], f[j], sum);
  }
  sum = row_sum<kWaves>(sum, part, wave);
  const float r = 1.0f / sqrtf(sum / (float)H + eps);
  if (rstd && tid == 0) rstd[t] = r;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = tid + i * kThreads;
    if (c >= nvec) break;               // (all 16 lanes of a block together: nvec % 16 == 0)
    if (h_out) store_row(reinterpret_cast<uint4*>(h_out) + t * nvec + c, hv[i]);
    float p[8], w[8];
    unpack8(hv[i], p);
    load_gain<kWF32>(weight, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] *= w[j];
    if (y) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p[j] * r;
      store_row(reinterpret_cast<uint4*>(y) + t * nvec + c, to_bf16x8(v));
    }
    if (codes) {
      // |p| compared as integers: the order of the magnitudes, a NaN above all,
      // so that a block with a NaN gets a NaN scale instead of losing it
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(p[j]) & 0x7fffffffu);
      const float top = __uint_as_float(row16_max_u32(m));
      const float s = top * r / 448.0f;
      uint2 q = make_uint2(0, 0);
      if (!(s <= 0.0f)) {
        const bool plain = top >= 0x1p-90f && top <= 0x1p110f;
        if (kWF32 && plain) {
          q = codes_f32(p, hv[i], weight, c, top);
        } else {
          const float inv = 448.0f / top, inv_top = inv * (1.0f / 448.0f);
          if (plain) {
            // 448 p / top from the quotient's reciprocal, put right by its residual: the
            // nearest float32.  p has 16 bits and 448 p / top, where it is not half way
            // between two codes, is 2^-21 away from there: the code is the nearest too.
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float u = p[j] * inv;
              p[j] = __builtin_fmaf(-__builtin_fmaf(u, top, -448.0f * p[j]), inv_top, u);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = p[j] / top * 448.0f;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] = __builtin_amdgcn_fmed3f(p[j], -448.0f, 448.0f);
          q = e4m3x8(p);
        }
        if (!(s < __builtin_inff())) q = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      }
      reinterpret_cast<uint2*>(codes)[t * nvec + c] = q;
      if ((c & 15) == 0) scales[(int64_t)(c / 16) * sstride + t] = s;
    }
  }
}

// The thread's vectors of a gain as they lie in memory: it uses them for every row, twice.
// (With 16 waves of four vectors there are no registers for them: read again each time.)
template <int kWaves, int kVecs, bool kWF32>
struct Gain {
  static constexpr bool kHeld = kWaves < 16 || kVecs < 4;
  static constexpr int kUnits = kWF32 ? 2 : 1;
  const uint4* p;
  uint4 v[kHeld ? kVecs : 1][kUnits];
  __device__ __forceinline__ Gain(const void* weight, int tid, int nvec)
      : p(static_cast<const uint4*>(weight) + (int64_t)tid * kUnits) {
    if (!kHeld) return;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        v[kHeld ? i : 0][u] = tid + i * kWaves * kWave < nvec ? p[i * kWaves * kWave * kUnits + u]
                                                              : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(int i, float (&w)[8]) const {
    uint4 u[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) u[k] = kHeld ? v[kHeld ? i : 0][k] : p[i * kWaves * kWave * kUnits + k];
    if (kWF32) {
      const uint4 &a = u[0], &b = u[kUnits - 1];
      w[0] = __uint_as_float(a.x), w[1] = __uint_as_float(a.y), w[2] = __uint_as_float(a.z);
      w[3] = __uint_as_float(a.w), w[4] = __uint_as_float(b.x), w[5] = __uint_as_float(b.y);
      w[6] = __uint_as_float(b.z), w[7] = __uint_as_float(b.w);
    } else {
      unpack8(u[0], w);
    }
  }
};

// The thread's vectors of a row of dy, h and d_residual.
template <int kWaves, int kVecs>
struct BackwardRow {
  uint4 dy[kVecs], h[kVecs], dres[kVecs];
  __device__ __forceinline__ void load(const uint16_t* dy_, const uint16_t* h_, const uint16_t* d_residual, int64_t t,
                                       bool real, int nvec, int tid) {
    const uint4* a = reinterpret_cast<const uint4*>(dy_) + t * nvec;
    const uint4* b = reinterpret_cast<const uint4*>(h_) + t * nvec;
    const uint4* d = reinterpret_cast<const uint4*>(d_residual) + t * nvec;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = tid + i * kWaves * kWave;
      const bool in = real && c < nvec;
      dy[i] = in ? load_row(a + c) : zero;
      h[i] = in ? load_row(b + c) : zero;
      dres[i] = in && d_residual ? load_row(d + c) : zero;
    }
  }
};

// A row's part in dx, and with kDw in the thread's sums of dw: what both forms of the
// gradient do with it.
template <int kWaves, int kVecs, bool kWF32, bool kDw>
__device__ __forceinline__ void backward_row(const BackwardRow<kWaves, kVecs>& row, float r,
                                             const Gain<kWaves, kVecs, kWF32>& gain, int64_t t, int nvec, int tid,
                                             int wave, bool d_residual, uint16_t* dx, float* part,
                                             float (&dw)[kVecs][8]) {
  constexpr int kThreads = kWaves * kWave;
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = tid + i * kThreads;
    if (c >= nvec) break;
    float g[8], f[8], w[8];
    unpack8(row.dy[i], g);
    unpack8(row.h[i], f);
    gain.get(i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float hat = f[j] * r;
      if (kDw) dw[i][j] = __builtin_fmaf(g[j], hat, dw[i][j]);
      dot = __builtin_fmaf(g[j] * w[j], hat, dot);
    }
  }
  dot = row_sum<kWaves>(dot, part, wave) / (float)(nvec * 8);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = tid + i * kThreads;
    if (c >= nvec) break;
    float g[8], f[8], w[8], e[8];
    unpack8(row.dy[i], g);
    unpack8(row.h[i], f);
    unpack8(row.dres[i], e);
    gain.get(i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = r * __builtin_fmaf(-dot, f[j] * r, g[j] * w[j]);
      g[j] = d_residual ? v + e[j] : v;
    }
    store_row(reinterpret_cast<uint4*>(dx) + t * nvec + c, to_bf16x8(g));
  }
}

// Many rows: one workgroup walks the rows blockIdx.x, blockIdx.x + gridDim.x, .. (in
// groups of kRows) and keeps its share of dw in registers; `partial` [gridDim.x, H]
// takes the shares, which norm_dw_kernel adds up in order.  kAhead: the next row is
// loaded before this one is worked on.  16384 x 4096 85 + 5 us.
template <int kWaves, int kVecs, bool kWF32, bool kAhead>
__global__ void __launch_bounds__(kWaves == 16 ? 1024 : 256) rmsnorm_backward_kernel(
    const uint16_t* dy, const uint16_t* __restrict__ h, const float* __restrict__ rstd,
    const void* __restrict__ weight, int64_t T, int H, const uint16_t* d_residual, uint16_t* dx,
    float* __restrict__ partial) {
  constexpr int kRows = kWaves == 1 ? 4 : 1;
  constexpr int kThreads = kWaves * kWave;
  __shared__ float part[2][kWaves];
  __shared__ float4 join[kWaves == 1 ? 3 : 1][kWaves == 1 ? 2 * kWave : 1];
  const int wave = threadIdx.x >> 6;
  const int tid = kWaves == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int nvec = H / 8;
  float dw[kVecs][8];
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  const Gain<kWaves, kVecs, kWF32> gain(weight, tid, nvec);
  int flip = 0;                         // the next row's sums go to the other buffer: one barrier a row
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t t = (int64_t)blockIdx.x * kRows + (kWaves == 1 ? wave : 0);
  BackwardRow<kWaves, kVecs> row, next;
  float r = 0.0f, next_r = 0.0f;
  auto load = [&](BackwardRow<kWaves, kVecs>& to, float& to_r, int64_t at) __attribute__((always_inline)) {
    to.load(dy, h, d_residual, at, at < T, nvec, tid);
    to_r = rstd[min(at, T - 1)];
  };
  if (kAhead) load(row, r, t);
  for (; t < T; t += step, flip ^= 1) {
    if (kAhead) load(next, next_r, t + step);
    else load(row, r, t);
    backward_row<kWaves, kVecs, kWF32, true>(row, r, gain, t, nvec, tid, wave, d_residual != nullptr, dx, part[flip],
                                             dw);
    if (kAhead) row = next, r = next_r;
  }
  float* out = partial + (int64_t)blockIdx.x * H;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = tid + i * kThreads;
    float4 lo = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
    float4 hi = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    if (kWaves == 1) {                  // the four rows' waves meet in LDS, in order
      if (wave > 0) join[wave - 1][tid] = lo, join[wave - 1][kWave + tid] = hi;
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int v = 0; v < 3; ++v) {
          const float4 p = join[v][tid], q = join[v][kWave + tid];
          lo.x += p.x, lo.y += p.y, lo.z += p.z, lo.w += p.w;
          hi.x += q.x, hi.y += q.y, hi.z += q.z, hi.w += q.w;
        }
      }
      __syncthreads();
    }
    if (c < nvec && (kWaves != 1 || wave == 0)) {
      reinterpret_cast<float4*>(out)[2 * c] = lo;
      reinterpret_cast<float4*>(out)[2 * c + 1] = hi;
    }
  }
}

// Few rows, in one launch: the first `row_blocks` workgroups write dx, the others dw,
// 64 channels each over all rows: they read dy and h again, from the caches, and
// need no row's sum (r is given).  dx must not be dy here.
template <int kWaves, int kVecs, bool kWF32>
__global__ void __launch_bounds__(kWaves == 16 ? 1024 : 256) rmsnorm_backward_few_kernel(
    const uint16_t* dy, const uint16_t* __restrict__ h, const float* __restrict__ rstd,
    const void* __restrict__ weight, int T, int H, const uint16_t* d_residual, uint16_t* dx,
    float* __restrict__ d_weight, int row_blocks) {
  constexpr int kRows = kWaves == 1 ? 4 : 1;
  constexpr int kSlices = (kWaves == 16 ? 1024 : 256) / 8;
  __shared__ float part[kWaves];
  __shared__ float sums[kSlices][64];
  const int nvec = H / 8;
  if ((int)blockIdx.x < row_blocks) {
    const int wave = threadIdx.x >> 6;
    const int t = blockIdx.x * kRows + (kWaves == 1 ? wave : 0);
    if (t >= T) return;
    const int tid = kWaves == 1 ? threadIdx.x & 63 : threadIdx.x;
    float none[kVecs][8];
    BackwardRow<kWaves, kVecs> row;
    row.load(dy, h, d_residual, t, true, nvec, tid);
    backward_row<kWaves, kVecs, kWF32, false>(row, rstd[t], Gain<kWaves, kVecs, kWF32>(weight, tid, nvec), t, nvec,
                                              tid, wave, d_residual != nullptr, dx, part, none);
    return;
  }
  const int col = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int c = ((int)blockIdx.x - row_blocks) * 8 + col;
  const uint4* dyc = reinterpret_cast<const uint4*>(dy) + c;
  const uint4* hc = reinterpret_cast<const uint4*>(h) + c;
  float dw[8] = {};
#pragma unroll 4
  for (int t = slice; t < T; t += kSlices) {
    float g[8], f[8];
    unpack8(dyc[(int64_t)t * nvec], g);
    unpack8(hc[(int64_t)t * nvec], f);
    const float r = rstd[t];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = __builtin_fmaf(g[j], f[j] * r, dw[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[slice][8 * col + j] = dw[j];
  __syncthreads();
  if (threadIdx.x >= 64) return;
  float s = 0.0f;
#pragma unroll 8
  for (int i = 0; i < kSlices; ++i) s += sums[i][threadIdx.x];
  d_weight[((int)blockIdx.x - row_blocks) * 64 + threadIdx.x] = s;
}

// dw[c] = sum over the n shares, four channels a thread, 32 threads along the
// shares (each every 32nd, ascending), of whose sums those of a wave meet in pairs,
// then the four waves' in order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* __restrict__ partial, int n, int H,
                                                      float* __restrict__ dw) {
  __shared__ float4 sums[4][8];
  const int col = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int c = blockIdx.x * 8 + col;   // of H / 4
  float4 s = make_float4(0, 0, 0, 0);
  const float4* p = reinterpret_cast<const float4*>(partial) + c;
#pragma unroll 8
  for (int i = slice; i < n; i += 32) {
    const float4 v = p[(int64_t)i * (H / 4)];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
#pragma unroll
  for (int off = 8; off < 64; off *= 2) {
    s.x += __shfl_xor(s.x, off, kWave), s.y += __shfl_xor(s.y, off, kWave);
    s.z += __shfl_xor(s.z, off, kWave), s.w += __shfl_xor(s.w, off, kWave);
  }
  if ((slice & 7) == 0) sums[slice >> 3][col] = s;
  __syncthreads();
  if (slice) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    const float4 v = sums[i][col];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  reinterpret_cast<float4*>(dw)[c] = s;
}

static int norm_waves(int H) { return H <= 2048 ? 1 : H <= 8192 ? 4 : 16; }

// Calls f with the row's form as types: waves and vectors a thread.
template <typename F>
static void norm_form(int H, F f) {
  const int waves = norm_waves(H), vecs = (H / 8 + waves * kWave - 1) / (waves * kWave);
  using std::integral_constant;
  if (waves == 1) {
    if (vecs == 1) f(integral_constant<int, 1>(), integral_constant<int, 1>());
    else if (vecs == 2) f(integral_constant<int, 1>(), integral_constant<int, 2>());
    else f(integral_constant<int, 1>(), integral_constant<int, 4>());
  } else if (waves == 4) {
    if (vecs <= 2) f(integral_constant<int, 4>(), integral_constant<int, 2>());
    else f(integral_constant<int, 4>(), integral_constant<int, 4>());
  } else {
    if (vecs <= 2) f(integral_constant<int, 16>(), integral_constant<int, 2>());
    else f(integral_constant<int, 16>(), integral_constant<int, 4>());
  }
}

int launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const void* weight, int wf32,
                   int64_t T, int H, float eps, uint16_t* h, uint16_t* y, uint8_t* codes,
                   float* scales, int64_t sstride, float* rstd, hipStream_t stream) {
  norm_form(H, [&](auto waves, auto vecs) {
    constexpr int W = decltype(waves)::value, V = decltype(vecs)::value;
    const dim3 grid((unsigned)(W == 1 ? (T + 3) / 4 : T)), block(W == 16 ? 1024 : 256);
    if (wf32)
      hipLaunchKernelGGL((rmsnorm_kernel<W, V, true>), grid, block, 0, stream, x, residual, weight, T, H, eps, h, y,
                         codes, scales, sstride, rstd);
    else
      hipLaunchKernelGGL((rmsnorm_kernel<W, V, false>), grid, block, 0, stream, x, residual, weight, T, H, eps, h, y,
                         codes, scales, sstride, rstd);
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// Workgroups of the gradient at most.  Each leaves H floats of dw behind, so no more than
// keep the memory busy, and the CUs evenly: 256, 384, 512, 640 and 768 take 55.8, 49.3,
// 48.2, 53.4, 50.9 us for 4096 x 7168, 108, 92, 95, 105, 101 for 16384 x 4096, 57, 53, 51.5,
// 56, 52.7 for 16384 x 2048.
static int64_t norm_shares(int64_t T, int H) {
  const int waves = norm_waves(H);
  const int64_t rows = waves == 1 ? (T + 3) / 4 : T;
  const int64_t most = waves == 16 ? 256 : 512;
  return rows < most ? rows : most;
}

// With the next row ahead 256 are enough, us against 512 without: 16384 x 4096 89 and 95,
// 4096 x 7168 47.2 and 48.6, 16384 x 2048 49.8 and 51.8, 8192 x 1024 18.1 and 19.1; without
// d_residual 16384 x 2048 40.9 and 41.2, but 16384 x 4096 78 and 72, 8192 x 6144 68 and 59;
// 16384 x 768 25.1 and 24.5, 20000 x 512 34 and 20.5; 16 waves no difference.
constexpr int kAheadShares = 256;
static bool norm_ahead(int H, bool d_residual) {
  const int waves = norm_waves(H);
  return H >= 1024 && (waves == 1 || (waves == 4 && d_residual));
}

// One launch for few rows; one launch against two, us: 333 x 2048 4.5 and 9.2, 1024 x
// 512 5.6 and 6.3, 1024 x 2048 6.9 and 9.5, 1024 x 7168 19 and 27, 1024 x 16384 39
// and 36, 2048 x 512 8.6 and 7.4, 2048 x 4096 27 and 24.
bool norm_one_launch(int64_t T, const uint16_t* dy, const uint16_t* dx) {
  return T > 0 && T <= MOE_NORM_FEW_ROWS && dx != dy;
}

size_t rmsnorm_backward_workspace_bytes(int64_t T, int H) {
  return (size_t)norm_shares(T, H) * H * sizeof(float);
}

int launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const float* rstd,
                            const void* weight, int wf32, int64_t T, int H,
                            const uint16_t* d_residual, uint16_t* dx, float* dw, void* workspace,
                            hipStream_t stream) {
  if (norm_one_launch(T, dy, dx)) {
    norm_form(H, [&](auto waves, auto vecs) {
      constexpr int W = decltype(waves)::value, V = decltype(vecs)::value;
      const int rows = (int)(W == 1 ? (T + 3) / 4 : T);
      const dim3 grid(rows + H / 64), block(W == 16 ? 1024 : 256);
      if (wf32)
        hipLaunchKernelGGL((rmsnorm_backward_few_kernel<W, V, true>), grid, block, 0, stream, dy, h, rstd, weight,
                           (int)T, H, d_residual, dx, dw, rows);
      else
        hipLaunchKernelGGL((rmsnorm_backward_few_kernel<W, V, false>), grid, block, 0, stream, dy, h, rstd, weight,
                           (int)T, H, d_residual, dx, dw, rows);
    });
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
  }
  const bool ahead = norm_ahead(H, d_residual);
  const int most = (int)norm_shares(T, H), shares = ahead ? std::min(most, kAheadShares) : most;
  float* partial = static_cast<float*>(workspace);
  auto launch = [&](auto waves, auto vecs, auto next) {
    constexpr int W = decltype(waves)::value, V = decltype(vecs)::value;
    constexpr bool A = decltype(next)::value;
    const dim3 grid(shares), block(W == 16 ? 1024 : 256);
    if (wf32)
      hipLaunchKernelGGL((rmsnorm_backward_kernel<W, V, true, A>), grid, block, 0, stream, dy, h, rstd, weight, T, H,
                         d_residual, dx, partial);
    else
      hipLaunchKernelGGL((rmsnorm_backward_kernel<W, V, false, A>), grid, block, 0, stream, dy, h, rstd, weight, T, H,
                         d_residual, dx, partial);
  };
  if (shares)
    norm_form(H, [&](auto waves, auto vecs) {
      if constexpr (decltype(waves)::value < 16 && decltype(vecs)::value > 1) {
        if (ahead) return launch(waves, vecs, std::true_type());
      }
      launch(waves, vecs, std::false_type());
    });
  hipLaunchKernelGGL(norm_dw_kernel, dim3(H / 32), dim3(256), 0, stream, partial, shares, H, dw);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
