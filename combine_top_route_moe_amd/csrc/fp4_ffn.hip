// The grouped SwiGLU FFN on 4-bit expert weights (MXFP4: E2M1 codes, one
// power-of-two scale per 32 weights of a row; NVFP4: one E4M3 scale per 16
// under a float32 scale per expert), and the packing of such weights.
//
//   gate/up:  a[r, j] = silu(x[r] . w13[e, j]) * (x[r] . w13[e, I + j])
//   down:     y[r, n] = bf16( row_scale[r] * (a[r] . w2[e, n]) )
//
// Two forms.  Short segments take the few-row kernels (decode.hip), bound by
// the weight bytes.  Long ones take the tile kernel here: a workgroup of 4
// waves covers 128 rows of a segment and 4 column tiles of 64 weight rows.
// A wave streams its own tile's codes straight into registers (1 KB loads,
// one 16-row fragment of a 128-wide K-block each) and converts them to bf16
// MFMA operands there, once per 128 rows: 16 conversions against 32 MFMAs per
// 32-wide K-step for MXFP4.  The 128 activation rows are shared by the waves
// through LDS, filled by direct-to-LDS DMA one K-block (128 columns) ahead,
// in MFMA fragment order, so every LDS read is one conflict-free 1 KB.
// Measured, MXFP4, gate/up + down: 32768 skewed rows of 64 experts (H = 4096, I =
// 1536) 1115 us, 1.11 PFLOP/s (traced 800 + 408), the rate that a large library
// product in bf16 reaches (1.12 to 1.15; 757 + 392 us on the fastest card seen);
// 4096 rows of 64 experts (H = 2048, I = 1024), half a tile each, 39 + 25, where
// the wait at each K-block is not covered by the other workgroup on the CU.
#include <algorithm>

#include "weight_block.h"

namespace moe {

constexpr int kTileWaves = 4;
constexpr int kTileSub = kBM / 16;   // 16-row subtiles of a tile

// ---- packing ------------------------------------------------------------------
// The E2M1 code of r, |r| <= 6: nearest, halfway values to the even code.
__device__ __forceinline__ uint32_t e2m1_code(float r) {
  const float a = fabsf(r);
  const uint32_t c = a <= 0.25f   ? 0u
                     : a < 0.75f  ? 1u
                     : a <= 1.25f ? 2u
                     : a < 1.75f  ? 3u
                     : a <= 2.5f  ? 4u
                     : a < 3.5f   ? 5u
                     : a <= 5.0f  ? 6u
                                  : 7u;
  return c | (__float_as_uint(r) >> 31 << 3);
}

// One wave per fragment (16 rows x 128 columns): lane l reads its 32 weights
// (row l % 16, columns 32 p + 8 (l / 16) .. +8), the group maxima come from
// the lanes of the same row (four for MXFP4's 32 columns, two for NVFP4's
// 16), and the lane's 16 bytes of codes are stored in lane order.
template <int FMT>
__global__ void __launch_bounds__(256) pack_weights_fp4_kernel(
    const uint16_t* __restrict__ W, const float* __restrict__ tensor_scale,
    u32x4_t* __restrict__ Q, uint32_t* __restrict__ S, int64_t n_frag, int N, int Kdim,
    int gate_up) {
  const int lane = threadIdx.x & 63;
  const int64_t frag = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (frag >= n_frag) return;
  const int n_ct = N / 64, nkb = Kdim / 128;
  const int f = (int)(frag & 3);
  const int64_t t = frag >> 2;
  const int kb = (int)(t % nkb);
  const int ct = (int)(t / nkb % n_ct);
  const int64_t g = t / n_ct / nkb;
  const int row0 = !gate_up ? 64 * ct + 16 * f : f < 2 ? 32 * ct + 16 * f : N / 2 + 32 * ct + 16 * (f - 2);
  const uint16_t* src = W + (g * N + row0 + (lane & 15)) * Kdim + kb * 128 + 8 * (lane >> 4);
  const float tg = FMT == MOE_W_NVFP4 ? tensor_scale[g] : 0.0f;
  uint32_t code[4], scales = 0u;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint4 raw = *reinterpret_cast<const uint4*>(src + 32 * p);
    float v[8];
    unpack8(raw, v);
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
    m = fmaxf(m, __shfl_xor(m, 16, kWave));
    code[p] = 0u;
    if constexpr (FMT == MOE_W_MXFP4) {
      m = fmaxf(m, __shfl_xor(m, 32, kWave));
      if (m > 0.0f) {
        int e;
        frexpf(m, &e);   // m = f 2^e, f in [0.5, 1): floor(log2 m) = e - 1
        const int xexp = min(max(e - 1 - 2, -127), 127);
        scales |= (uint32_t)(xexp + 127) << (8 * p);
        const float inv = ldexpf(1.0f, -xexp);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          code[p] |= e2m1_code(fminf(fmaxf(v[j] * inv, -6.0f), 6.0f)) << (4 * j);
      }
    } else {
      float q = m / (6.0f * tg);   // IEEE; 0 / 0 (an all-zero tensor) -> 0
      if (q != q) q = 0.0f;
      q = fminf(q, 448.0f);
      const uint32_t b = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false) & 0xffu;
      scales |= b << (8 * p);
      const float s = __builtin_amdgcn_cvt_f32_fp8((int)b, 0) * tg;
      if (s > 0.0f) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          code[p] |= e2m1_code(fminf(fmaxf(v[j] / s, -6.0f), 6.0f)) << (4 * j);
      }
    }
  }
  Q[frag * 64 + lane] = u32x4_t{code[0], code[1], code[2], code[3]};
  if constexpr (FMT == MOE_W_MXFP4) {
    if (lane < 16) S[(t * 16 + lane) * 4 + f] = scales;
  } else {
    if (!(lane & 16)) S[((t * 2 + (lane >> 5)) * 16 + (lane & 15)) * 4 + f] = scales;
  }
}

int launch_pack_weights_fp4(const uint16_t* w13, const uint16_t* w2, int G, int H, int I, int mode,
                            const float* g13, const float* g2, uint8_t* w13q, uint8_t* w13s,
                            uint8_t* w2q, uint8_t* w2s, hipStream_t stream) {
  auto one = [&](const uint16_t* w, const float* tg, uint8_t* q, uint8_t* s, int N, int Kdim,
                 int gate_up) -> int {
    const int64_t n_frag = (int64_t)G * (N / 16) * (Kdim / 128);
    const int64_t blocks = (n_frag + 3) / 4;
    if (blocks >= kMaxGrid) return MOE_ERR_UNSUPPORTED;
    auto* kern = mode == MOE_FQ_MXFP4 ? pack_weights_fp4_kernel<MOE_W_MXFP4>
                                      : pack_weights_fp4_kernel<MOE_W_NVFP4>;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), 0, stream, w, tg,
                       reinterpret_cast<u32x4_t*>(q), reinterpret_cast<uint32_t*>(s), n_frag, N,
                       Kdim, gate_up);
    return MOE_OK;
  };
  int st = MOE_OK;
  if (w13) st = one(w13, g13, w13q, w13s, 2 * I, H, 1);
  if (st == MOE_OK && w2) st = one(w2, g2, w2q, w2s, H, I, 0);
  if (st != MOE_OK) return st;
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// ---- the tile kernel ------------------------------------------------------------
// One 128-row tile x one 64-row column tile per wave.  NT: the expert's rows
// fit one tile, so its weights are read once and stream past the caches.
template <bool GATE_UP, int FMT, bool NT>
__device__ __forceinline__ void fp4_tile_body(u32x4_t (*As)[kTileSub][4][kWave],
                                              const WStream<FMT, 4, GATE_UP>& ws, const uint16_t* a_base,
                                              const uint32_t* a_voff, int64_t a_sub_stride,
                                              int a_kb_stride, int w, int lane, int nkb,
                                              int nlive, f32x4_t (*acc)[4]) {
  // the wave fills subtiles 2 w and 2 w + 1 of the K-block, 1 KB per K-step
  auto fill = [&](int kb, int buf) {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * w + h >= nlive) break;   // never read past the segment's end
#pragma unroll
      for (int p = 0; p < 4; ++p)
        dma16(a_base + (int64_t)(2 * w + h) * a_sub_stride + (int64_t)kb * a_kb_stride,
              a_voff[h] + (uint32_t)p * (GATE_UP ? 64u : 1024u), &As[buf][2 * w + h][p][0]);
    }
    asm volatile("" ::: "memory");
  };
  typename WStream<FMT, 4, GATE_UP>::Tile cur, nxt;
  fill(0, 0);
  ws.template load<NT>(nxt, 0);
  for (int kb = 0; kb < nkb; ++kb) {
    const int buf = kb & 1;
    // everything in flight is block kb's: its DMA has landed in LDS after
    // this wait and the barrier, and its codes are in the registers
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    lds_barrier();
    cur = nxt;
    if (kb + 1 < nkb) {
      // the other buffer was last read for block kb - 1, which every wave
      // has finished
      fill(kb + 1, buf ^ 1);
      ws.template load<NT>(nxt, kb + 1);
      asm volatile("" ::: "memory");
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      bf16x8_t bfr[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) bfr[f] = cur.operand(f, p);
      u32x4_t a[kTileSub];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = As[buf][i][p][lane];
      if (nlive > 4) {
#pragma unroll
        for (int i = 4; i < 8; ++i) a[i] = As[buf][i][p][lane];
      }
#pragma unroll
      for (int i = 0; i < kTileSub; ++i) {
        if (i >= nlive) break;
        const bf16x8_t af = __builtin_bit_cast(bf16x8_t, a[i]);
#pragma unroll
        for (int f = 0; f < 4; ++f)
          acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, bfr[f], acc[i][f], 0, 0, 0);
      }
    }
  }
}

// Row tiles of all groups, as decode_tile counts them (every lane active).
__device__ __forceinline__ long long total_row_tiles(const int32_t* __restrict__ counts, int G,
                                                     int64_t capacity) {
  long long n = 0;
  for (int e = threadIdx.x & 63; e < G; e += kWave)
    n += (min((int64_t)max(counts[e], 0), capacity) + kBM - 1) / kBM;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off, kWave);
  return n;
}

template <bool GATE_UP, int FMT>
__global__ void __launch_bounds__(kTileWaves * kWave, 2) fp4_tile_kernel(
    const uint16_t* __restrict__ A, WMat W, const int32_t* __restrict__ cu_seqlens,
    const int32_t* __restrict__ counts, int G, int Kdim, int Nw /* weight rows per group */,
    int Nout, const float* __restrict__ row_scale, uint16_t* __restrict__ Out, int64_t capacity,
    int32_t* __restrict__ dev_error) {
  __shared__ __attribute__((aligned(16))) u32x4_t As[2][kTileSub][4][kWave];
  __shared__ __attribute__((aligned(16))) uint16_t Epi[kTileWaves][16 * 72];

  const int n_ct = Nw / 64, n_cb = (n_ct + kTileWaves - 1) / kTileWaves;
  const int pid = xcd_remap(blockIdx.x);
  int g, mt, cb;
  int64_t mt_before;
  if (!decode_tile(pid, counts, G, n_cb, capacity, g, mt, cb, &mt_before)) return;
  // the intermediate's m-tile must lie in the workspace (ceil(capacity/128)
  // + G m-tiles): overlapping segments could place it past the end, or past the
  // grid, whose last workgroup has no tile of disjoint segments
  const int64_t most = (capacity + kBM - 1) / kBM + G;
  if (pid == (int)gridDim.x - 1 && total_row_tiles(counts, G, capacity) > most &&
      (threadIdx.x & 63) == 0)
    raise_error(dev_error, MOE_DEVERR_ROW_RANGE);
  if (mt_before + mt >= most) {
    if ((threadIdx.x & 63) == 0) raise_error(dev_error, MOE_DEVERR_ROW_RANGE);
    return;
  }
  g = __builtin_amdgcn_readfirstlane(g);
  mt = __builtin_amdgcn_readfirstlane(mt);
  cb = __builtin_amdgcn_readfirstlane(cb);
  const int64_t mt_glob = __builtin_amdgcn_readfirstlane((int)mt_before) + mt;
  const int seg0 = cu_seqlens[g];
  const int nrows = counts[g];
  if ((int64_t)seg0 + nrows > capacity || seg0 < 0) {
    if ((threadIdx.x & 63) == 0) raise_error(dev_error, MOE_DEVERR_ROW_RANGE);
    return;
  }
  const int valid = min(kBM, nrows - mt * kBM);
  if (valid <= 0) return;
  const int64_t row_base = (int64_t)seg0 + mt * kBM;
  const int nlive = (valid + 15) >> 4;   // subtiles holding real rows
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // spare waves of the last column block stream a real tile and store nothing
  const bool ct_ok = cb * kTileWaves + w < n_ct;
  const int ct = ct_ok ? cb * kTileWaves + w : n_ct - 1;
  const int nkb = Kdim / 128;

  WStream<FMT, 4, GATE_UP> ws;
  ws.init(W, g, ct, 0, n_ct, nkb, 0, 0, lane);
  // gate/up reads the rows themselves (rows past the end re-read the last);
  // down the gate/up kernel's output, in fragment order per m-tile: block
  // (subtile, K-step) of 64 lanes x 8 values
  const uint16_t* a_base = GATE_UP ? A + row_base * Kdim
                                   : A + mt_glob * kTileSub * (int64_t)(Kdim / 32) * (kWave * 8);
  uint32_t a_voff[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = min((2 * w + h) * 16 + (lane & 15), valid - 1);
    a_voff[h] = GATE_UP ? (uint32_t)(r * Kdim + 8 * (lane >> 4)) * 2u : (uint32_t)lane * 16u;
  }
  const int64_t a_sub_stride = GATE_UP ? 0 : (int64_t)(Kdim / 32) * (kWave * 8);
  const int a_kb_stride = GATE_UP ? 128 : 4 * kWave * 8;

  f32x4_t acc[kTileSub][4];
#pragma unroll
  for (int i = 0; i < kTileSub; ++i)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[i][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (nrows <= kBM)
    fp4_tile_body<GATE_UP, FMT, true>(As, ws, a_base, a_voff, a_sub_stride, a_kb_stride, w, lane,
                                      nkb, nlive, acc);
  else
    fp4_tile_body<GATE_UP, FMT, false>(As, ws, a_base, a_voff, a_sub_stride, a_kb_stride, w, lane,
                                       nkb, nlive, acc);
  if (!ct_ok) return;

  // epilogue: lane holds D[4*(lane/16) + q][lane%16] of every 16x16 tile.
  // Each subtile goes through the wave's LDS staging area (rows padded so the
  // 2-byte writes are conflict-free) and out as 16-byte vectors; rows past
  // the segment end are neither staged nor stored.
  constexpr int kCol = GATE_UP ? 32 : 64;   // the wave's output columns
  constexpr int kEpiStride = kCol + 8;
  uint16_t* epi = Epi[w];
#pragma unroll
  for (int i = 0; i < kTileSub; ++i) {
    if (i >= nlive) break;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int rr = 4 * (lane >> 4) + q;
      if (i * 16 + rr >= valid) continue;
      if (GATE_UP) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
          epi[rr * kEpiStride + f * 16 + (lane & 15)] =
              (uint16_t)f32_to_bf16(silu_f(acc[i][f][q]) * acc[i][f + 2][q]);
      } else {
        const float sc = row_scale ? row_scale[row_base + i * 16 + rr] : 1.0f;
#pragma unroll
        for (int f = 0; f < 4; ++f)
          epi[rr * kEpiStride + f * 16 + (lane & 15)] = (uint16_t)f32_to_bf16(sc * acc[i][f][q]);
      }
    }
    // the staging area is the wave's own: its LDS operations run in order,
    // and the fences keep the compiler from moving them across each other
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    if (GATE_UP) {
      // fragment order of the down product: K-step ct, lane row + 16 c8
      const int row = lane & 15;
      uint16_t* blk = Out + ((mt_glob * kTileSub + i) * (int64_t)(Nout / 32) + ct) * (kWave * 8);
      if (i * 16 + row < valid)
        reinterpret_cast<u32x4_t*>(blk)[lane] =
            *reinterpret_cast<const u32x4_t*>(&epi[row * kEpiStride + 8 * (lane >> 4)]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int piece = lane + h * kWave, row = piece >> 3, c8 = piece & 7;
        if (i * 16 + row < valid)
          reinterpret_cast<u32x4_t*>(Out + (row_base + i * 16 + row) * Nout + ct * 64)[c8] =
              *reinterpret_cast<const u32x4_t*>(&epi[row * kEpiStride + 8 * c8]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  }
}

size_t few_ffn_workspace_bytes(int64_t capacity, int I);
int launch_few_ffn(const uint16_t*, const int32_t*, const int32_t*, int, int, int,
                   const moe_ffn_weights*, const float*, uint16_t*, int64_t, int, void*, int32_t*,
                   hipStream_t);

// Few-row or tile kernels, by what the host knows.  Both read each weight once
// while a group has few rows.  The few-row kernels split the reduction over
// waves, so a few groups fill the GPU, but they read the weights again for
// every 16 rows (on average every 12 or so).  The tile kernel reads them once
// per 128 rows, but a workgroup walks the whole reduction by itself, at about
// 0.9 us a 128-wide block of either stage however few there are (the time in
// which 42 KB are streamed for each column of H and I) and more than twice that
// with a tile's 128; further rows are other workgroups'.  Where both stream at
// the memory's rate, sharing the rows through LDS pays from 8 rows a group.
// Measured, both stages, few / tile in us, MXFP4: H = 4096, I = 1536, 4 groups of
// 32 rows 27 / 50, of 96 57 / 86; 16 groups of 16 rows 47 / 53, of 24 77 / 57; 32
// groups of 4 rows 61 / 63, of 16 85 / 69; H = 2048, I = 768, 128 groups of 4
// rows 70 / 73, of 8 76 / 72, of 32 170 / 93; H = 1024, I = 512, 8 groups of 200
// rows 28 / 41; H = 512, I = 256, 64 groups of 32 rows 16 / 16, of 64 24 / 21.
// NVFP4, H = 4096, I = 1536, 16 groups of 16 rows 51 / 58, of 24 85 / 69; 32
// groups of 4 rows 76 / 90, of 24 162 / 104.
constexpr double kWalkBytes = 42e3;   // a column's, see above
static bool few_rows(int64_t capacity, int G, int H, int I) {
  const int64_t active = std::min<int64_t>(G, capacity);
  if (capacity < 8 * active) return true;
  const double bytes = 1.6 * H * I;   // an expert's weights
  const double walk = 1.0 + std::min<double>(kBM, (double)capacity / active) / 96.0;
  const double tile = std::max(active * bytes, kWalkBytes * ((double)H + I) * walk);
  return std::max<double>(active, capacity / 12.0) * bytes < tile;
}

// Both forms', the few-row one's up to the capacities it is taken for: a buffer
// for the largest batch does for every smaller one.  As a tile's walk grows with
// its rows, the rule can give tiles from 8 rows a group on, the few-row kernels
// again from about 10 and tiles from about 12 (where the weights take 1.08 to 1.13
// times the shortest walk: 26 groups, H = 4096, I = 1536; at 268 to 312 rows, few /
// tile in us, MXFP4 59 to 62 / 54, NVFP4 64 to 66 / 74); the sizes in between
// hold the tiles of the smaller ones, too.
size_t grouped_ffn_fp4_workspace_bytes(int64_t capacity, int G, int H, int I) {
  if (capacity == 0) return 0;
  const double walk = kWalkBytes * ((double)H + I) * (1.0 + kBM / 96.0) / (1.6 * H * I);
  const int64_t most = (int64_t)std::max(8.0 * G, 12.0 * std::max((double)G, walk)) + 1;
  const size_t few = few_ffn_workspace_bytes(std::min(capacity, most), I);
  const int64_t eight = std::min<int64_t>(capacity, 8LL * G);   // where tiles are first taken
  if (few_rows(capacity, G, H, I) && few_rows(eight, G, H, I)) return few;
  const int64_t rows = ((capacity + kBM - 1) / kBM + G) * kBM;
  return std::max(few, (((size_t)rows * I * 2) + 255) & ~(size_t)255);
}

template <int FMT>
static int launch_tiles(const uint16_t* x, const int32_t* cu, const int32_t* counts, int G, int H,
                        int I, const moe_ffn_weights* wt, const float* row_scale, uint16_t* y,
                        int64_t capacity, int flags, uint16_t* act, int32_t* dev_error,
                        hipStream_t stream) {
  const int64_t m_tiles = (capacity + kBM - 1) / kBM + G;
  const int64_t unit = (int64_t)kNumXcd * kXcdChunk;
  auto grid = [&](int n_ct) {
    return (m_tiles * ((n_ct + kTileWaves - 1) / kTileWaves) + unit - 1) / unit * unit;
  };
  const int64_t gu = grid(I / 32), dn = grid(H / 64);
  if (gu >= kMaxGrid || dn >= kMaxGrid) return MOE_ERR_UNSUPPORTED;
  if (flags & MOE_FFN_GATE_UP)
    hipLaunchKernelGGL((fp4_tile_kernel<true, FMT>), dim3((unsigned)gu), dim3(kTileWaves * kWave),
                       0, stream, x, (WMat{wt->w13, wt->w13_scales, wt->w13_tensor_scale}), cu,
                       counts, G, H, 2 * I, I, nullptr, act, capacity, dev_error);
  if (flags & MOE_FFN_DOWN)
    hipLaunchKernelGGL((fp4_tile_kernel<false, FMT>), dim3((unsigned)dn), dim3(kTileWaves * kWave),
                       0, stream, act, (WMat{wt->w2, wt->w2_scales, wt->w2_tensor_scale}), cu,
                       counts, G, I, H, H, row_scale, y, capacity, dev_error);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int launch_grouped_ffn_fp4(const uint16_t* x, const int32_t* cu, const int32_t* counts, int G,
                           int H, int I, const moe_ffn_weights* wt, const float* row_scale,
                           uint16_t* y, int64_t capacity, int flags, void* workspace,
                           int32_t* dev_error, hipStream_t stream) {
  if (few_rows(capacity, G, H, I))
    return launch_few_ffn(x, cu, counts, G, H, I, wt, row_scale, y, capacity, flags, workspace,
                          dev_error, stream);
  uint16_t* act = static_cast<uint16_t*>(workspace);
  if (wt->format == MOE_W_MXFP4)
    return launch_tiles<MOE_W_MXFP4>(x, cu, counts, G, H, I, wt, row_scale, y, capacity, flags,
                                     act, dev_error, stream);
  return launch_tiles<MOE_W_NVFP4>(x, cu, counts, G, H, I, wt, row_scale, y, capacity, flags, act,
                                   dev_error, stream);
}

}  // namespace moe
