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
#include <algorithm>
#include <cmath>

#include "gemm_common.h"
#include "reduce.h"

namespace moe {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t operand(const u32x4_t& lo, const u32x4_t& hi) {
  return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ f32x4_t mfma_codes(const i32x8_t& a, const i32x8_t& b) {
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
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
      *reinterpret_cast<u32x2_t*>(p) = u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    } else {
      for (int q = 0; q < 4; ++q)
        if (q < some) p[q] = (uint16_t)f32_to_bf16(v[q]);
    }
  }
}

// A wave's outputs: rows m0 + 16 j + lane % 16 of y, columns n0 + 16 i + 4 (lane / 16)
// .. +4.  In bf16 two neighbouring i's trade places between lanes 16 apart, so that
// each lane stores 16 bytes and 64 of a row lie together.
template <bool F32, int kIN, int kIM>
__device__ __forceinline__ void store_tile(void* y, const f32x4_t (&acc)[kIN][kIM], int64_t m0, int n0, int64_t M,
                                           int N, int lane) {
  const int g = lane >> 4;
  if (!F32 && kIN % 2 == 0 && (N & 7) == 0) {
#pragma unroll
    for (int j = 0; j < kIM; ++j) {
      const int64_t m = m0 + 16 * j + (lane & 15);
#pragma unroll
      for (int i = 0; i < kIN; i += 2) {
        const f32x4_t &p = acc[i][j], &q = acc[i + 1][j];
        const auto lo = __builtin_amdgcn_permlane16_swap(bf16_pair(p[0], p[1]), bf16_pair(q[0], q[1]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(bf16_pair(p[2], p[3]), bf16_pair(q[2], q[3]), false, false);
        const int n = n0 + 16 * (i + (g & 1)) + 8 * (g >> 1);
        if (m < M && n < N)
          *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(y) + m * N + n) = u32x4_t{lo[0], hi[0], lo[1], hi[1]};
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kIM; ++j) {
    const int64_t m = m0 + 16 * j + (lane & 15);
    if (m >= M) continue;
#pragma unroll
    for (int i = 0; i < kIN; ++i) {
      const int n = n0 + 16 * i + 4 * g;
      if (n < N) store4<F32>(y, m * N + n, acc[i][j], N - n, (N & 3) == 0);
    }
  }
}

// ---------------------------------------------------------------------------
// Up to 16 rows: a workgroup owns 16 rows of W; its waves take the blocks of K in
// turn, kAhead of a wave's at a time on their way from memory straight into the
// operands' registers (W's past the caches' order: each is read once), and add up
// through LDS, in order.  Bound by W's bytes (16 x 7168 x 7168 13.9 us, 3.7 TB/s; the
// rows of x come out of the L2s as often again), and where these are few by
// a load's way through the memory (1 x 7168 x 2048 5.1 us with its launch).
template <int kNW, int kAhead, bool F32>
__global__ void __launch_bounds__(kNW * kWave) linear_rows_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t sstride, int M,
    const uint8_t* __restrict__ wq, const float* __restrict__ wsc, int N, int nkb, void* __restrict__ y) {
  __shared__ f32x4_t sums[kNW][kWave];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ct = blockIdx.x;
  const int m = min(lane & 15, M - 1);           // rows past the end re-read the last
  const uint8_t* xr = x + (int64_t)m * nkb * 128 + 16 * (lane >> 4);
  const u32x4_t* wr = reinterpret_cast<const u32x4_t*>(wq) + (int64_t)ct * nkb * 128 + lane;
  const float* sw = wsc + (int64_t)(ct / 8) * nkb;

  u32x4_t wv[kAhead][2], xv[kAhead][2];
  float sx[kAhead], s[kAhead];
  auto fill = [&](int slot, int b) {
    if (b >= nkb) return;
    const u32x4_t* p = wr + (int64_t)b * 128;
    const u32x4_t* q = reinterpret_cast<const u32x4_t*>(xr + (int64_t)b * 128);
    wv[slot][0] = __builtin_nontemporal_load(p);
    wv[slot][1] = __builtin_nontemporal_load(p + kWave);
    xv[slot][0] = q[0];
    xv[slot][1] = q[4];
    sx[slot] = xs[b * sstride + m];
    s[slot] = sw[b];
  };
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < kAhead; ++u) fill(u, w + kNW * u);
  for (int b0 = w; b0 < nkb; b0 += kNW * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int b = b0 + kNW * u;
      if (b >= nkb) break;
      const f32x4_t t = mfma_codes(operand(wv[u][0], wv[u][1]), operand(xv[u][0], xv[u][1]));
      const float c = sx[u] * s[u];
      fill(u, b + kNW * kAhead);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = __builtin_fmaf(t[q], c, acc[q]);
    }
  }
  sums[w][lane] = acc;
  __syncthreads();
  const int n = ct * 16 + 4 * (lane >> 4);
  if (w > 0 || (lane & 15) >= M || n >= N) return;
#pragma unroll
  for (int i = 1; i < kNW; ++i) {
    const f32x4_t v = sums[i][lane];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] += v[q];
  }
  store4<F32>(y, (int64_t)m * N + n, acc, N - n, (N & 3) == 0);
}

// ---------------------------------------------------------------------------
// Tiles: a workgroup of (BM / WM) x (BN / WN) waves owns BM rows of x and BN rows
// of W, a wave WM x WN of them.  Blocks of K pass through LDS, in a few stages:
// W's 16 x 128 operands as they are packed; x's as 16 rows of 128 bytes, the
// 16-byte units of row r in the order u ^ (r % 8).  Eight lanes of a load then
// take one whole line of memory (16 rows x 64 bytes a load, the operand's own
// order, made the 4096 x 4096 x 7168 product 145 us instead of 134), and the
// 16 rows that are read back together still lie in different banks.
template <int BM, int BN>
struct LinearStage {
  u32x4_t w[BN / 16][2 * kWave];
  u32x4_t x[BM / 16][2 * kWave];
  float sx[BM < 64 ? 64 : BM];
};

// What brings a block of K into a stage: pieces of 1 KB, half operands, W's first,
// piece w + kNW n by wave w; the scales of x's rows by the first waves.  Rows past
// the end of a matrix repeat its last ones.
template <int BM, int BN, int kNW>
struct LinearLoads {
  using Stage = LinearStage<BM, BN>;
  static constexpr int kPiecesW = BN / 8 / kNW, kPieces = (BN / 8 + BM / 8) / kNW;
  static_assert(BN / 8 % kNW == 0 && BM / 8 % kNW == 0 && BM / 64 <= kNW, "the pieces go round");
  const uint8_t* wbase[kPiecesW];
  const uint8_t* xbase;
  const float* sbase;
  int64_t sstride;
  uint32_t rows8;             // bytes of 8 rows of x
  uint32_t xlane, xlast;      // this lane's offset in 8 rows, and in the last row
  uint32_t slane, wlane, lds;
  int w;

  __device__ __forceinline__ LinearLoads(Stage* stages, const uint8_t* x, const float* xs, int64_t sstride_,
                                         int64_t M, const uint8_t* wq, int N, int nkb, int64_t m0, int ct0, int w_,
                                         int lane) {
    w = w_, sstride = sstride_, lds = lds_addr(stages);
    const int n_ct = (N + 15) / 16;
    const uint32_t K = (uint32_t)nkb * 128;
#pragma unroll
    for (int n = 0; n < kPiecesW; ++n) {
      const int p = w + kNW * n;
      wbase[n] = wq + ((int64_t)min(ct0 + p / 2, n_ct - 1) * nkb * 2 + (p & 1)) * 1024;
    }
    const uint32_t unit = 16 * ((lane & 7) ^ (lane >> 3));
    const uint32_t last = (uint32_t)min((int64_t)BM - 1, M - 1 - m0);
    xbase = x + m0 * K;
    rows8 = 8 * K;
    xlane = (lane >> 3) * K + unit;
    xlast = last * K + unit;
    sbase = xs + m0;
    slane = 4 * min((uint32_t)(64 * w + lane), last);
    wlane = 16 * lane;
  }
  __device__ __forceinline__ void piece(int n, int b, int stage) const {
    const int p = w + kNW * n;
    const uint32_t at = lds + stage * (uint32_t)sizeof(Stage) + p * 1024;
    if (n < kPiecesW)
      dma16_at(wbase[n < kPiecesW ? n : 0] + (int64_t)b * 2048, wlane, at);
    else
      dma16_at(xbase + (int64_t)b * 128, min(xlane + (p - BN / 8) * rows8, xlast), at);
  }
  __device__ __forceinline__ void scales(int b, int stage) const {
    if (w < (BM < 64 ? 1 : BM / 64))
      dma4_at(sbase + b * sstride, slane,
              lds + stage * (uint32_t)sizeof(Stage) + (BN / 8 + BM / 8) * 1024 + w * 256);
  }
  __device__ __forceinline__ void all(int b, int stage) const {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int n = 0; n < kPieces; ++n) piece(n, b, stage);
    scales(b, stage);
    asm volatile("" ::: "memory");
  }
};

// Workgroup ids go round the 8 XCDs; each XCD takes one run of consecutive tiles,
// and a run walks down columns of up to 8 tiles of x before the next column of
// W, so that what an XCD works on at a time is near a square and shares its L2.
__device__ __forceinline__ void linear_tile(int pid, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n;
  const int xcd = pid % kNumXcd, q = total / kNumXcd, r = total % kNumXcd;
  const int at = xcd * q + min(xcd, r) + pid / kNumXcd;
  constexpr int kGroup = 8;
  const int group = at / (kGroup * tiles_n), first = group * kGroup;
  const int rows = min(kGroup, tiles_m - first), in = at - group * kGroup * tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

// s_waitcnt for what a wave has to do with LDS: its own loads into it (vmcnt 0), and
// what it has read of it (lgkmcnt 0); `&`: both.
constexpr int kWaitLoads = 0x0f70, kWaitReads = 0xc07f;

// One tile: the next blocks are fetched while this one is multiplied, one barrier a
// block.  Bound by what a CU gets out of its L2 (58 to 73 GB/s) for the small tiles,
// by the matrix cores for the large: 128 x 128 reaches 1.9 PFLOP/s on 2048 x 4096 x
// 7168, 62 us.
// SPLIT: part blockIdx.y of gridDim.y of K; y is then float32 [part][M][N].
// MINW waves a SIMD leave a wave at most 256 registers: with more the compiler puts
// the products into accumulation registers and moves each back.
template <int BM, int BN, int WM, int WN, int kStages, int MINW, bool F32, bool SPLIT>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * kWave, MINW) linear_tile_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t sstride, int64_t M,
    const uint8_t* __restrict__ wq, const float* __restrict__ wsc, int N, int nkb, int tiles_m, int tiles_n,
    void* __restrict__ y) {
  constexpr int kWavesM = BM / WM, kNW = kWavesM * (BN / WN);
  constexpr int kIN = WN / 16, kIM = WM / 16;
  __shared__ LinearStage<BM, BN> stages[kStages];
  int tm, tn;
  linear_tile(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (w % kWavesM) * kIM, wn = (w / kWavesM) * kIN;   // in units of 16
  const int64_t m0 = (int64_t)tm * BM;
  const int ct0 = tn * (BN / 16);
  const int b0 = SPLIT ? (int)((int64_t)nkb * blockIdx.y / gridDim.y) : 0;
  const int b1 = SPLIT ? (int)((int64_t)nkb * (blockIdx.y + 1) / gridDim.y) : nkb;
  const LinearLoads<BM, BN, kNW> loads(stages, x, xs, sstride, M, wq, N, nkb, m0, ct0, w, lane);
  const float* sw = wsc + (int64_t)min((ct0 + wn) / 8, (N - 1) / 128) * nkb;
  const int xlo = (lane & 15) * 8 + ((lane >> 4) ^ (lane & 7)), xhi = xlo ^ 4;

  f32x4_t acc[kIN][kIM];
#pragma unroll
  for (int i = 0; i < kIN; ++i)
#pragma unroll
    for (int j = 0; j < kIM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // kStages - 1 blocks are on their way; past the end the last one again, so that a
  // wave's loads can be counted
#pragma unroll
  for (int n = 0; n < kStages - 1; ++n) loads.all(min(b0 + n, b1 - 1), n);
  int stage = 0;
  for (int b = b0; b < b1; ++b) {
    // this stage has landed (but for kStages - 2 blocks' loads) and the one before it
    // has been read, by this wave and, after the barrier, by all
    __builtin_amdgcn_s_waitcnt(vmcnt_imm((kStages - 2) * decltype(loads)::kPieces) & kWaitReads);
    lds_barrier();
    loads.all(min(b + kStages - 1, b1 - 1), stage == 0 ? kStages - 1 : stage - 1);
    const LinearStage<BM, BN>& st = stages[stage];
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const float scale = sw[b];
    i32x8_t a[kIN];
#pragma unroll
    for (int i = 0; i < kIN; ++i) a[i] = operand(st.w[wn + i][lane], st.w[wn + i][kWave + lane]);
#pragma unroll
    for (int j = 0; j < kIM; ++j) {
      const i32x8_t v = operand(st.x[wm + j][xlo], st.x[wm + j][xhi]);
      const float c = st.sx[(wm + j) * 16 + (lane & 15)] * scale;
#pragma unroll
      for (int i = 0; i < kIN; ++i) {
        const f32x4_t t = mfma_codes(a[i], v);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(t[q], c, acc[i][j][q]);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(kWaitLoads);      // no load into LDS may outlive the workgroup
  if (SPLIT) y = static_cast<float*>(y) + (int64_t)blockIdx.y * M * N;
  store_tile<F32, kIN, kIM>(y, acc, m0 + wm * 16, (ct0 + wn) * 16, M, N, lane);
}

// Large products: 256 x 256, eight waves of 128 x 64, of which the two of a SIMD
// take turns: one reads a whole block's operands from LDS into registers while
// the other multiplies.  Phase 2 b: the first four waves read block b, the others
// multiply block b - 1; phase 2 b + 1: the other way round; a barrier between
// phases.  A stage is free once both have read it, after phase 2 b + 1: block b
// + 2's loads go out in phase 2 b + 2 (by the first waves while they read, by the
// others one by one between the matrix instructions) and are waited for at the
// end of phase 2 b + 3.  8192^3 447 us (480 with all waves in step, as the other
// tiles are), 4096 x 4096 x 7168 94 to 105: 2.3 to 2.55 PFLOP/s, the matrix cores busy
// 71 % of the time at the clock that the power limit leaves.
constexpr int kBig = 256;
template <bool F32>
__global__ void __launch_bounds__(512, 2) linear_big_kernel(
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t sstride, int64_t M,
    const uint8_t* __restrict__ wq, const float* __restrict__ wsc, int N, int nkb, int tiles_m, int tiles_n,
    void* __restrict__ y) {
  constexpr int kIN = 4, kIM = 8, kNW = 8;
  // A product's multiply-adds follow its matrix instruction by kBehind others: its
  // result takes that long (1: 592 us for 8192^3, 2: 477, 3: 451, 4: 455).
  constexpr int kBehind = 3;
  __shared__ LinearStage<kBig, kBig> stages[2];
  int tm, tn;
  linear_tile(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (w % 2) * kIM, wn = (w / 2) * kIN;
  const int64_t m0 = (int64_t)tm * kBig;
  const int ct0 = tn * (kBig / 16);
  const LinearLoads<kBig, kBig, kNW> loads(stages, x, xs, sstride, M, wq, N, nkb, m0, ct0, w, lane);
  constexpr int kPieces = LinearLoads<kBig, kBig, kNW>::kPieces;
  const float* sw = wsc + (int64_t)min((ct0 + wn) / 8, (N - 1) / 128) * nkb;
  const int xlo = (lane & 15) * 8 + ((lane >> 4) ^ (lane & 7)), xhi = xlo ^ 4;

  f32x4_t acc[kIN][kIM];
#pragma unroll
  for (int i = 0; i < kIN; ++i)
#pragma unroll
    for (int j = 0; j < kIM; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  i32x8_t a[kIN], v[kIM];
  float c[kIM], scale = sw[0];
  auto read = [&](int b) __attribute__((always_inline)) {
    const LinearStage<kBig, kBig>& st = stages[b & 1];
#pragma unroll
    for (int i = 0; i < kIN; ++i) a[i] = operand(st.w[wn + i][lane], st.w[wn + i][kWave + lane]);
#pragma unroll
    for (int j = 0; j < kIM; ++j) v[j] = operand(st.x[wm + j][xlo], st.x[wm + j][xhi]);
#pragma unroll
    for (int j = 0; j < kIM; ++j) c[j] = st.sx[(wm + j) * 16 + (lane & 15)] * scale;
    scale = sw[min(b + 1, nkb - 1)];
  };
  auto scaled = [&](int n, const f32x4_t& t) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      acc[n % kIN][n / kIN][q] = __builtin_fmaf(t[q], c[n / kIN], acc[n % kIN][n / kIN][q]);
  };
  auto multiply = [&](int b, bool load) __attribute__((always_inline)) {
    constexpr int kAll = kIN * kIM;
    f32x4_t t[kBehind + 1];
    const int next = min(b + 2, nkb - 1);      // (past the end: the last block again)
    if (load) loads.scales(next, b & 1);
#pragma unroll
    for (int n = 0; n < kAll; ++n) {
      if (load && n % (kAll / kPieces) == 0) loads.piece(n / (kAll / kPieces), next, b & 1);
      t[n % (kBehind + 1)] = mfma_codes(a[n % kIN], v[n / kIN]);
      if (n >= kBehind) scaled(n - kBehind, t[(n - kBehind) % (kBehind + 1)]);
      __builtin_amdgcn_sched_barrier(0);       // the order as it stands here
    }
#pragma unroll
    for (int n = kAll - kBehind; n < kAll; ++n) scaled(n, t[n % (kBehind + 1)]);
  };

  loads.all(0, 0);
  __builtin_amdgcn_s_waitcnt(kWaitLoads);
  lds_barrier();
  if (w < kNW / 2) {
    for (int b = 0; b < nkb; ++b) {
      read(b);
      loads.all(min(b + 1, nkb - 1), (b + 1) & 1);
      __builtin_amdgcn_s_waitcnt(kWaitReads);
      lds_barrier();
      __builtin_amdgcn_s_setprio(1);
      multiply(b, false);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_s_waitcnt(kWaitLoads);
      lds_barrier();
    }
    lds_barrier();
  } else {
    loads.all(min(1, nkb - 1), 1);
    lds_barrier();
    for (int b = 0; b < nkb; ++b) {
      read(b);
      __builtin_amdgcn_s_waitcnt(kWaitLoads & kWaitReads);
      lds_barrier();
      __builtin_amdgcn_s_setprio(1);
      multiply(b, true);
      __builtin_amdgcn_s_setprio(0);
      lds_barrier();
    }
    __builtin_amdgcn_s_waitcnt(kWaitLoads);    // no load into LDS may outlive the workgroup
  }
  store_tile<F32, kIN, kIM>(y, acc, m0 + wm * 16, (ct0 + wn) * 16, M, N, lane);
}

// y = the sum of the parts, in order, four outputs a thread, all parts' loads on
// their way before the first addition.
template <int kParts, bool F32>
__global__ void __launch_bounds__(256) linear_join_kernel(const float* __restrict__ parts, int64_t total,
                                                          void* __restrict__ y) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= total) return;
  const int some = (int)min((int64_t)4, total - at);
  const bool wide = (total & 3) == 0;
  f32x4_t u[kParts];
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    const float* q = parts + p * total + at;
    if (wide) {
      u[p] = *reinterpret_cast<const f32x4_t*>(q);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) u[p][k] = q[min(k, some - 1)];
    }
  }
#pragma unroll
  for (int p = 1; p < kParts; ++p)
#pragma unroll
    for (int k = 0; k < 4; ++k) u[0][k] += u[p][k];
  store4<F32>(y, at, u[0], some, wide);
}

// ---------------------------------------------------------------------------
// Packing: one workgroup per 128 x 128 tile of W [N, K], through LDS, so that
// the transposed order costs no more than the plain one.
template <bool QUANT, bool TRANS>
__global__ void __launch_bounds__(256) pack_linear_kernel(
    const uint16_t* __restrict__ wide, const uint8_t* __restrict__ codes, const float* __restrict__ scales,
    int N, int K, uint8_t* __restrict__ packed, float* __restrict__ packed_scales) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[128][144];
  __shared__ uint32_t top[4];
  const int nb = blockIdx.y, kb = blockIdx.x, n_nb = gridDim.y, n_kb = gridDim.x;
  const int64_t row0 = (int64_t)nb * 128;
  float s;
  if (QUANT) {
    uint4 v[8];
    uint32_t m = 0;                     // |w| as integers: the order of the magnitudes, a NaN above all
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = threadIdx.x + 256 * i, r = c >> 4;
      v[i] = row0 + r < N ? reinterpret_cast<const uint4*>(wide + (row0 + r) * K + kb * 128)[c & 15]
                          : make_uint4(0, 0, 0, 0);
      float f[8];
      unpack8(v[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, kWave));
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(top[0], top[1]), max(top[2], top[3]));
    const bool finite = m < 0x7f800000u;         // else no scale: the tile is NaN, not some finite number
    s = finite ? __uint_as_float(m) / 448.0f : __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = threadIdx.x + 256 * i;
      float f[8];
      unpack8(v[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = s > 0.0f ? fminf(fmaxf(f[j] / s, -448.0f), 448.0f) : 0.0f;
      *reinterpret_cast<uint2*>(&tile[c >> 4][8 * (c & 15)]) =
          finite ? e4m3x8(f) : make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
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

// ---------------------------------------------------------------------------
// Which kernel.  Up to 16 rows: linear_rows_kernel (64 x 64 tiles, the next best
// there: 7.9 us against 5.1 for one row of 7168 x 2048, 18 against 7 for 13 of 576
// x 7168).  Else the tile, and the number of parts of K, with the shortest
// estimated time: kStart for launch and fill, then per block of K the longer of
// what one workgroup takes (its loads' way through the memory) and what a CU takes
// for all of its tiles, measured:
//                         us a block, one tile   us a block and tile, many
//   64 x 64                     0.28                   0.225
//   64 x 128                    0.40                   0.345
//   128 x 128                   0.72                   0.55
//   256 x 256                   1.15                   1.65
// and for parts the join's launch and its bytes.  A CU holds one 256 x 256 workgroup,
// so that every round of them fills (and drains) for itself, kFill, and a block of the
// last takes from the first figure, with a few CUs at work, to the second, with all of
// them at the clock that the power limit leaves.  Over 230 products of 17 to 8192
// rows, N from 64 to 8192 and K from 256 to 8192 the form it takes is 1.8 % slower
// in the geometric mean than the fastest.  Both sides of a border, us (N = 4096, K = 7168):
// 64 rows in 64 x 64 tiles 18.2, in 2 parts 13.8, in 4 11.5, in 8 13.4; 512 rows in
// 64 x 64 26, 64 x 128 28, 128 x 128 39; 1024 rows 50, 41, 43; 2048 rows 99, 79, 63,
// 256 x 256 83; 2304 rows 108, 95, 92, 80; 4096 rows 200, 159, 126, 100; 5120 rows 240,
// 191, 162, 167.
struct LinearForm {
  int tile, parts;              // of kTiles; parts of K
};

struct LinearTile {
  int m, n, threads;
  double one, many;
  bool alone;                   // one workgroup a CU
};
constexpr LinearTile kTiles[4] = {{64, 64, 256, 0.28, 0.225, false}, {64, 128, 512, 0.40, 0.345, false},
                                  {128, 128, 256, 0.72, 0.55, false}, {256, 256, 512, 1.15, 1.65, true}};
constexpr double kThreadsMost = 0xffffffffu;       // of a launch
constexpr int kPartsMost = 8;                      // 2, 4 or 8 (linear_join_kernel)
constexpr int64_t kPartBytes = 32 << 20;           // all parts together: more costs more than it gives

static LinearForm linear_form(int64_t M, int N, int nkb) {
  constexpr double kCUs = 256, kStart = 3.0, kFill = 6.0, kJoin = 3.3, kJoinBytesPerUs = 5e6;
  LinearForm best = {3, 1};
  double least = 1e300;
  for (int i = 0; i < 4; ++i) {
    const double tiles = (double)((M + kTiles[i].m - 1) / kTiles[i].m) * ((N + kTiles[i].n - 1) / kTiles[i].n);
    for (int parts = 1; parts <= (i < 3 ? kPartsMost : 1) && parts <= nkb; parts *= 2) {
      const int64_t bytes = (int64_t)parts * M * N * 4;
      if ((parts > 1 && bytes > kPartBytes) || tiles * parts * kTiles[i].threads > kThreadsMost) break;
      const double rounds = std::ceil(tiles * parts / kCUs);
      const double one = kTiles[i].one, many = kTiles[i].many, last = tiles * parts / kCUs - (rounds - 1);
      const double block = kTiles[i].alone ? (rounds - 1) * many + one + last * (many - one)
                                           : std::max(one, rounds * many);
      double us = (kTiles[i].alone ? kFill * rounds : kStart) + (double)nkb / parts * block;
      if (parts > 1) us += kJoin + 2.0 * bytes / kJoinBytesPerUs;
      if (us < least) least = us, best = {i, parts};
    }
  }
  return best;
}

// Parts of K of a product, and its workgroups' tile: {rows, columns}.
int linear_fp8_parts(int64_t M, int N, int K, int32_t* tile) {
  const bool few = M <= MOE_LINEAR_FEW_ROWS;
  const LinearForm form = few ? LinearForm{0, 1} : linear_form(M, N, K / 128);
  if (tile) {
    tile[0] = few ? MOE_LINEAR_FEW_ROWS : kTiles[form.tile].m;
    tile[1] = few ? 16 : kTiles[form.tile].n;
  }
  return form.parts;
}

// Enough for every smaller M too.
size_t linear_fp8_workspace_bytes(int64_t M, int N, int K) {
  if (M <= MOE_LINEAR_FEW_ROWS || K == 128) return 0;
  return (size_t)std::min(kPartBytes, (int64_t)kPartsMost * 4 * M * N);
}

struct LinearCall {
  const uint8_t* x;
  const float* xs;
  int64_t sstride, M;
  const uint8_t* wq;
  const float* wsc;
  int N, nkb;
  void* y;
  void* parts;
  hipStream_t stream;
};

template <bool F32>
static void launch_linear_rows(const LinearCall& c) {
  // 8 waves, 4 blocks of each on their way; of (2, 4), (4, 4), (8, 2), (8, 4), (16, 1), (16, 4)
  // within 5 % of the best from 1 x 512 x 1024 to 16 x 7168 x 7168
  hipLaunchKernelGGL((linear_rows_kernel<8, 4, F32>), dim3((c.N + 15) / 16), dim3(8 * kWave), 0, c.stream, c.x, c.xs,
                     c.sstride, (int)c.M, c.wq, c.wsc, c.N, c.nkb, c.y);
}

template <int BM, int BN, int WM, int WN, int kStages, int MINW, bool F32>
static int launch_linear_tiles(const LinearCall& c, int parts) {
  const int64_t tm = (c.M + BM - 1) / BM, tn = (c.N + BN - 1) / BN;
  constexpr int kThreads = (BM / WM) * (BN / WN) * kWave;
  if (tm * tn * kThreads * parts > 0xffffffffLL) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(tm * tn), parts);
  if (parts > 1) {
    hipLaunchKernelGGL((linear_tile_kernel<BM, BN, WM, WN, kStages, MINW, true, true>), grid, dim3(kThreads), 0,
                       c.stream, c.x, c.xs, c.sstride, c.M, c.wq, c.wsc, c.N, c.nkb, (int)tm, (int)tn, c.parts);
    const int64_t total = c.M * c.N;
    const dim3 blocks((unsigned)((total + 1023) / 1024));
    const float* from = static_cast<const float*>(c.parts);
    if (parts == 2)
      hipLaunchKernelGGL((linear_join_kernel<2, F32>), blocks, dim3(256), 0, c.stream, from, total, c.y);
    else if (parts == 4)
      hipLaunchKernelGGL((linear_join_kernel<4, F32>), blocks, dim3(256), 0, c.stream, from, total, c.y);
    else
      hipLaunchKernelGGL((linear_join_kernel<8, F32>), blocks, dim3(256), 0, c.stream, from, total, c.y);
  } else {
    hipLaunchKernelGGL((linear_tile_kernel<BM, BN, WM, WN, kStages, MINW, F32, false>), grid, dim3(kThreads), 0,
                       c.stream, c.x, c.xs, c.sstride, c.M, c.wq, c.wsc, c.N, c.nkb, (int)tm, (int)tn, c.y);
  }
  return MOE_OK;
}

template <bool F32>
static int launch_linear_big(const LinearCall& c) {
  const int64_t tm = (c.M + kBig - 1) / kBig, tn = (c.N + kBig - 1) / kBig;
  if (tm * tn * 512 > 0xffffffffLL) return MOE_ERR_UNSUPPORTED;
  hipLaunchKernelGGL(linear_big_kernel<F32>, dim3((unsigned)(tm * tn)), dim3(512), 0, c.stream, c.x, c.xs, c.sstride,
                     c.M, c.wq, c.wsc, c.N, c.nkb, (int)tm, (int)tn, c.y);
  return MOE_OK;
}

template <bool F32>
static int launch_linear(const LinearCall& c) {
  if (c.M <= MOE_LINEAR_FEW_ROWS) {
    launch_linear_rows<F32>(c);
    return MOE_OK;
  }
  const LinearForm form = linear_form(c.M, c.N, c.nkb);
  switch (form.tile) {
    case 0: return launch_linear_tiles<64, 64, 32, 32, 4, 2, F32>(c, form.parts);
    case 1: return launch_linear_tiles<64, 128, 32, 32, 3, 4, F32>(c, form.parts);
    case 2: return launch_linear_tiles<128, 128, 64, 64, 2, 2, F32>(c, form.parts);
    default: return launch_linear_big<F32>(c);
  }
}

int launch_linear_fp8(const uint8_t* x, const float* xs, int64_t sstride, int64_t M, int N, int K,
                      const uint8_t* wq, const float* wsc, void* y, int f32, void* workspace,
                      hipStream_t stream) {
  const LinearCall call = {x, xs, sstride, M, wq, wsc, N, K / 128, y, workspace, stream};
  const int st = f32 ? launch_linear<true>(call) : launch_linear<false>(call);
  if (st != MOE_OK) return st;
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
