// The whole MoE layer for a few tokens (moe_decode), and the few-row form of
// the grouped FFN on 4-bit weights.
//
// For token t with chosen experts e_k and weights w_k:
//   h = W13[e_k] x_t,  a = silu(h[:I]) * h[I:],
//   out_t = bf16( sum_k w_k W2[e_k] a  +  the shared expert's row )
// With few tokens every product is a matrix times a handful of columns: the
// time is that of reading the chosen experts' weights once.  So nothing is
// permuted or written that a later launch would read back but `a`:
//   plan      (one workgroup) routes every token and lists, per expert that
//             any token chose, its tokens in runs of at most 16 ("entries");
//   gate_up   a workgroup owns 16 gate rows and the 16 matching up rows of
//             one entry's expert; its waves split H and add up through LDS;
//   down      a workgroup owns 16 output columns of every token; its waves
//             split the concatenated (entry, I) axis, each keeps all tokens'
//             float32 sums in registers, and the waves add up through LDS in
//             order: the combine needs no second pass and no atomics.
// The products run on the matrix cores with the weights as the A operand (16
// weight rows) and the tokens as the B operand's 16 columns, so columns are
// independent: a token sees its own experts only, whatever values the others
// hold.  `a` is kept as two bf16 numbers (high and low part, 16 significant
// bits) and multiplied in two MFMAs, so no intermediate is rounded to bf16;
// sums are float32 throughout.
#include <algorithm>

#include "route_common.h"
#include "weight_block.h"

namespace moe {

constexpr int kMaxTokens = 64;    // one bit of an expert's token mask each
constexpr int kCols = 16;         // tokens (or rows) of an entry
constexpr int kPlanThreads = 1024;
constexpr int kFewWaves = 4;      // waves of a gate/up (or row-wise down) workgroup
constexpr int kDownWaves = 8;     // waves of a down + combine workgroup

// A run of at most 16 tokens of one local expert.
struct PlanEntry {
  int32_t e;       // local expert
  int32_t base;    // first compact row of the run
  int32_t cnt;     // rows of the run
  int32_t sub;     // rows of the expert before the run
  uint64_t mask;   // the expert's tokens
};

// The workspace: plan, then the intermediate rows (routed, then shared).
struct DecodeLayout {
  size_t entries, row_tok, row_w, a_hi, a_lo, s_hi, s_lo, total;
  int64_t max_entries;
};
static size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
static DecodeLayout decode_layout(int T, int I, int K, int El, int sI) {
  DecodeLayout L;
  const int64_t rows = (int64_t)T * K;
  L.max_entries = std::min<int64_t>(El, rows) + rows / kCols;
  size_t o = 256;   // the entry count
  auto put = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  L.entries = put((size_t)L.max_entries * sizeof(PlanEntry));
  L.row_tok = put((size_t)rows * 4);
  L.row_w = put((size_t)rows * 4);
  L.a_hi = put((size_t)rows * I * 2);
  L.a_lo = put((size_t)rows * I * 2);
  L.s_hi = put((size_t)T * sI * 2);
  L.s_lo = put((size_t)T * sI * 2);
  L.total = o;
  return L;
}

size_t decode_workspace_bytes(int T, int I, int K, int El, int sI) {
  return decode_layout(T, I, K, El, sI).total;
}

// ---- plan -------------------------------------------------------------------
// One workgroup.  EPL 0: the routes are given (topk_idx, topk_w are inputs),
// else experts per lane of the top-k selection.
template <int EPL>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ row_valid, int T, int E, int K,
    int renorm, int expert_begin, int El, int32_t* __restrict__ topk_idx,
    float* __restrict__ topk_w, int32_t* __restrict__ n_entries, PlanEntry* __restrict__ entries,
    int32_t* __restrict__ row_tok, float* __restrict__ row_w, int32_t* __restrict__ dev_error) {
  __shared__ uint32_t mask[1024][2];
  __shared__ int sel_e[kMaxTokens * 32];
  __shared__ float sel_w[kMaxTokens * 32];
  __shared__ int base_of[1024];
  __shared__ int wave_sum[kPlanThreads / kWave];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  mask[tid][0] = 0u;
  mask[tid][1] = 0u;
  __syncthreads();
  for (int t = wv; t < T; t += kPlanThreads / kWave) {
    const bool real = !row_valid || row_valid[t];
    int e = -1;
    float w = 0.0f;
    if constexpr (EPL > 0) {
      if (real) route_row<EPL>(logits + (int64_t)t * E, E, K, renorm, lane, e, w);
      if (!real) {
        e = -1;
        w = 0.0f;
      }
      if (lane < K) {
        topk_idx[(int64_t)t * K + lane] = e;
        topk_w[(int64_t)t * K + lane] = w;
      }
    } else if (lane < K && real) {
      e = topk_idx[(int64_t)t * K + lane];
      w = topk_w[(int64_t)t * K + lane];
      if (e >= E) raise_error(dev_error, MOE_DEVERR_EXPERT_RANGE);
    }
    if (lane < K) {
      const bool here = e >= expert_begin && e < E && e - expert_begin < El;
      const int le = here ? e - expert_begin : -1;
      sel_e[t * K + lane] = le;
      sel_w[t * K + lane] = w;
      if (here) atomicOr(&mask[le][t >> 5], 1u << (t & 31));
    }
  }
  __syncthreads();
  // entries and compact rows before each expert: one scan of (entries, rows)
  // packed in one word (both totals stay below 2^15)
  const uint64_t m = (uint64_t)mask[tid][1] << 32 | mask[tid][0];
  const int c = __popcll(m), ne = (c + kCols - 1) / kCols;
  int incl = ne << 16 | c;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(incl, off, kWave);
    if (lane >= off) incl += y;
  }
  if (lane == 63) wave_sum[wv] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kPlanThreads / kWave; ++i) {
    if (i < wv) before += wave_sum[i];
    total += wave_sum[i];
  }
  const int excl = before + incl - (ne << 16 | c);
  const int ent0 = excl >> 16, base = excl & 0xffff;
  base_of[tid] = base;
  for (int v = 0; v < ne; ++v)
    entries[ent0 + v] = PlanEntry{tid, base + v * kCols, min(kCols, c - v * kCols), v * kCols, m};
  if (tid == 0) *n_entries = total >> 16;
  __syncthreads();
  // each (token, expert) pair's compact row; a token that names one expert in
  // several slots has one row there, with the slots' weights added
  for (int i = tid; i < T * K; i += kPlanThreads) {
    const int e = sel_e[i];
    if (e < 0) continue;
    const int t = i / K;
    float w = 0.0f;
    bool first = true;
    for (int j = t * K; j < (t + 1) * K; ++j)
      if (sel_e[j] == e) {
        first = first && j >= i;
        w += sel_w[j];
      }
    if (!first) continue;
    const uint64_t em = (uint64_t)mask[e][1] << 32 | mask[e][0];
    const int pos = base_of[e] + __popcll(em & ((1ull << t) - 1));
    row_tok[pos] = t;
    row_w[pos] = w;
  }
}

// ---- the streamed product ---------------------------------------------------
// acc[f] += W_f[16 rows, blocks kb0, kb0 + step, ..] * B^T for NF weight
// fragments and one 16-column B given as NB bf16 addends (b[i] is the lane's
// column at its first element).  D blocks are in flight per wave; the loop
// that refills is free of branches, so that each wait covers one block only.
template <int FMT, int NF, int NB, int D>
__device__ __forceinline__ void few_stream(const WStream<FMT>* ws, const uint16_t* const* b,
                                           int kb0, int step, int nkb, f32x4_t* acc) {
  struct Buf {
    typename WStream<FMT>::Block w[NF];
    u32x4_t x[NB][4];
  } buf[D];
  const int n = kb0 < nkb ? (nkb - kb0 + step - 1) / step : 0;
  if (n == 0) return;
  auto load = [&](Buf& t, int i) {
    const int kb = kb0 + i * step;
#pragma unroll
    for (int f = 0; f < NF; ++f) ws[f].load(t.w[f], kb);
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int p = 0; p < 4; ++p)
        t.x[a][p] = *reinterpret_cast<const u32x4_t*>(b[a] + kb * 128 + p * 32);
  };
  auto use = [&](const Buf& t) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const bf16x8_t wf = t.w[f].operand(p);
#pragma unroll
        for (int a = 0; a < NB; ++a)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              wf, __builtin_bit_cast(bf16x8_t, t.x[a][p]), acc[f], 0, 0, 0);
      }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(buf[d], min(d, n - 1));
  int i = 0;
  for (; i + 2 * D <= n; i += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      use(buf[d]);
      load(buf[d], i + d + D);
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (i + d < n) {
      use(buf[d]);
      if (i + d + D < n) load(buf[d], i + d + D);
    }
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (i + D + d < n) use(buf[d]);
}

// Blocks in flight per wave, by the block's registers (two fragments of bf16
// weights are 32 registers a block, of 4-bit ones 10).
template <int FMT>
constexpr int few_depth() {
  return FMT == MOE_W_BF16 ? 2 : FMT == MOE_W_FP8 ? 2 : 3;
}

// v as the sum of two bf16 numbers, high part first
__device__ __forceinline__ void split_bf16(float v, uint32_t& hi, uint32_t& lo) {
  hi = f32_to_bf16(v);
  lo = f32_to_bf16(v - bf16_to_f32(hi));
}

// One workgroup's gate/up tile: rows 16 rt .. of the gate half and of the up
// half of expert g, for the cnt <= 16 rows whose x this lane's column is
// xcol (columns past cnt repeat the last one and are not stored).  a rows
// go to hi / lo + column * I.
template <int FMT, int NW>
__device__ __forceinline__ void few_gate_up(const WMat& W, int g, int rt, int H, int I,
                                            const uint16_t* xcol, int cnt, uint16_t* hi,
                                            uint16_t* lo, f32x4_t (*red)[2][kWave]) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = H / 128, ct = rt >> 1, f = rt & 1;
  WStream<FMT> ws[2];
  ws[0].init(W, g, ct, f, I / 32, nkb, 16 * rt, lane);
  ws[1].init(W, g, ct, f + 2, I / 32, nkb, I + 16 * rt, lane);
  f32x4_t acc[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
  const uint16_t* b[1] = {xcol + 8 * (lane >> 4)};
  few_stream<FMT, 2, 1, few_depth<FMT>()>(ws, b, w, NW, nkb, acc);
  red[w][0][lane] = acc[0];
  red[w][1][lane] = acc[1];
  __syncthreads();
  if (w != 0) return;
  f32x4_t gt = red[0][0][lane], up = red[0][1][lane];
#pragma unroll
  for (int i = 1; i < NW; ++i) {
    gt += red[i][0][lane];
    up += red[i][1][lane];
  }
  // lane holds rows 4 (l / 16) .. +4 of the tile for column l % 16
  const int col = lane & 15;
  if (col >= cnt) return;
  uint32_t h[4], l[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) split_bf16(silu_f(gt[q]) * up[q], h[q], l[q]);
  const int64_t o = (int64_t)col * I + rt * 16 + 4 * (lane >> 4);
  *reinterpret_cast<uint2*>(hi + o) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  *reinterpret_cast<uint2*>(lo + o) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// ---- moe_decode: gate/up ------------------------------------------------------
// Blocks [0, shared_blocks): the shared expert's tiles, 16 tokens a run; then
// (entry, tile), the entries past the plan's leaving at once.
template <int FMT, int NW>
__global__ void __launch_bounds__(NW * kWave, 4) decode_gate_up_kernel(
    const uint16_t* __restrict__ x, int T, int H, int I, WMat routed, WMat shared, int sI,
    int shared_blocks, const int32_t* __restrict__ n_entries,
    const PlanEntry* __restrict__ entries, const int32_t* __restrict__ row_tok,
    uint16_t* __restrict__ a_hi, uint16_t* __restrict__ a_lo, uint16_t* __restrict__ s_hi,
    uint16_t* __restrict__ s_lo) {
  __shared__ f32x4_t red[NW][2][kWave];
  const int col = threadIdx.x & 15;
  int b = blockIdx.x;
  if (b < shared_blocks) {
    const int nt = sI / 16, v = b / nt;
    const int t0 = v * kCols, cnt = min(kCols, T - t0);
    const uint16_t* xc = x + (int64_t)(t0 + min(col, cnt - 1)) * H;
    few_gate_up<FMT, NW>(shared, 0, b - v * nt, H, sI, xc, cnt, s_hi + (int64_t)t0 * sI,
                         s_lo + (int64_t)t0 * sI, red);
    return;
  }
  b -= shared_blocks;
  const int nt = I / 16, j = b / nt;
  if (j >= *n_entries) return;
  const int base = entries[j].base, cnt = entries[j].cnt;
  const uint16_t* xc = x + (int64_t)row_tok[base + min(col, cnt - 1)] * H;
  few_gate_up<FMT, NW>(routed, entries[j].e, b - j * nt, H, I, xc, cnt, a_hi + (int64_t)base * I,
                       a_lo + (int64_t)base * I, red);
}

// ---- moe_decode: down + combine -----------------------------------------------
// A workgroup owns output columns 16 rt .. +16 of all T tokens.  The blocks
// of 128 intermediate columns of all entries (the shared expert's runs last)
// form one axis, which the waves split evenly; a wave keeps every token's sum
// over its stretch in registers: per entry an accumulator over compact rows,
// which at the end of the entry is weighted and moved to the tokens' lanes.
// TS: token subtiles of 16.
template <int FMT, int TS, int NW>
__global__ void __launch_bounds__(NW * kWave, 2) decode_down_kernel(
    int T, int H, int I, WMat routed, WMat shared, int sI, int shared_runs,
    const int32_t* __restrict__ n_entries, const PlanEntry* __restrict__ entries,
    const float* __restrict__ row_w, const uint16_t* __restrict__ a_hi,
    const uint16_t* __restrict__ a_lo, const uint16_t* __restrict__ s_hi,
    const uint16_t* __restrict__ s_lo, uint16_t* __restrict__ out) {
  constexpr int D = 2;
  __shared__ f32x4_t red[NW][TS][kWave];
  const int lane = threadIdx.x & 63, col = lane & 15, q8 = 8 * (lane >> 4);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rt = blockIdx.x, ct = rt >> 2, f = rt & 3, n_ct = H / 64;
  const int nb = I / 128, nbs = sI / 128;
  const int n = *n_entries;
  const int nr = n * nb, total = nr + shared_runs * nbs;
  const int b0 = (int)((int64_t)total * w / NW), b1 = (int)((int64_t)total * (w + 1) / NW);
  f32x4_t tok[TS];
#pragma unroll
  for (int s = 0; s < TS; ++s) tok[s] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  struct Buf {
    typename WStream<FMT>::Block w;
    u32x4_t hi[4], lo[4];
    float rw;
  } buf[D];
  // a position on the axis: entry (or shared run) and block within it
  struct Cursor {
    int j, kb;
  };
  auto at = [&](int b) -> Cursor {
    if (b < nr) return {b / nb, b % nb};
    const int r = b - nr;
    return {n + r / max(nbs, 1), r % max(nbs, 1)};
  };
  auto next = [&](Cursor& c) {
    ++c.kb;
    if (c.kb == (c.j < n ? nb : nbs)) {
      c.kb = 0;
      ++c.j;
    }
  };
  auto load = [&](Buf& t, const Cursor& c) {
    const int j = __builtin_amdgcn_readfirstlane(c.j), kb = __builtin_amdgcn_readfirstlane(c.kb);
    const bool sh = j >= n;
    const int jj = sh ? 0 : j;   // n may be 0
    const int t0 = (j - n) * kCols;
    const int base = sh ? t0 : entries[jj].base;
    const int cnt = sh ? min(kCols, T - t0) : entries[jj].cnt;
    const int g = sh ? 0 : entries[jj].e;
    const int Ic = sh ? sI : I;
    const WMat m = sh ? shared : routed;
    WStream<FMT> ws;
    ws.init(m, g, ct, f, n_ct, Ic / 128, 16 * rt, lane);
    ws.load(t.w, kb);
    const int row = base + min(col, cnt - 1);
    const int64_t o = (int64_t)row * Ic + q8 + kb * 128;
    const uint16_t* ph = (sh ? s_hi : a_hi) + o;
    const uint16_t* pl = (sh ? s_lo : a_lo) + o;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      t.hi[p] = *reinterpret_cast<const u32x4_t*>(ph + p * 32);
      t.lo[p] = *reinterpret_cast<const u32x4_t*>(pl + p * 32);
    }
    const float rw = row_w[sh ? 0 : row];   // the load itself unconditional: no branch here
    t.rw = sh ? 1.0f : rw;
  };
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  Cursor cu = at(b0), cl = cu;
  auto use = [&](const Buf& t, bool last) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const bf16x8_t wf = t.w.operand(p);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8_t, t.hi[p]), acc,
                                                    0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8_t, t.lo[p]), acc,
                                                    0, 0, 0);
    }
    const int j = __builtin_amdgcn_readfirstlane(cu.j);
    next(cu);
    if (last || cu.kb == 0) {   // the entry (or the wave's part of it) is done
      const bool sh = j >= n;
      const int jj = sh ? 0 : j;
      const int sub = sh ? (j - n) * kCols : entries[jj].sub;
      const uint64_t mask = sh ? ~0ull : entries[jj].mask;
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] *= t.rw;
#pragma unroll
      for (int s = 0; s < TS; ++s) {
        const int tk = 16 * s + col;   // this lane's token
        const int i = __popcll(mask & ((1ull << tk) - 1)) - sub;
        const bool mine = ((mask >> tk) & 1) && i >= 0 && i < kCols;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v = __shfl(acc[q], (lane & 48) | (i & 15), kWave);
          tok[s][q] += mine ? v : 0.0f;
        }
      }
      acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  };
  const int cntb = b1 - b0;
  if (cntb > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(buf[d], cl);
      if (d + 1 < cntb) next(cl);   // past the end: the last block again
    }
    int i = 0;
    for (; i + 2 * D <= cntb; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        use(buf[d], false);
        load(buf[d], cl);
        if (i + d + D + 1 < cntb) next(cl);
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (i + d < cntb) {
        use(buf[d], i + d + 1 == cntb);
        if (i + d + D < cntb) {
          load(buf[d], cl);
          if (i + d + D + 1 < cntb) next(cl);
        }
      }
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (i + D + d < cntb) use(buf[d], i + D + d + 1 == cntb);
  }
#pragma unroll
  for (int s = 0; s < TS; ++s) red[w][s][lane] = tok[s];
  __syncthreads();
  if (w >= TS) return;
  f32x4_t v = red[0][w][lane];
#pragma unroll
  for (int i = 1; i < NW; ++i) v += red[i][w][lane];
  const int t = 16 * w + col;
  if (t >= T) return;
  *reinterpret_cast<uint2*>(out + (int64_t)t * H + rt * 16 + 4 * (lane >> 4)) =
      make_uint2(f32_to_bf16(v[0]) | f32_to_bf16(v[1]) << 16,
                 f32_to_bf16(v[2]) | f32_to_bf16(v[3]) << 16);
}

template <int FMT>
static void launch_decode_ffn(const uint16_t* x, int T, int H, int I, int K, const WMat* r13,
                              const WMat* r2, const WMat* s13, const WMat* s2, int sI,
                              const DecodeLayout& L, char* ws, uint16_t* out, hipStream_t stream) {
  const int32_t* n_entries = reinterpret_cast<const int32_t*>(ws);
  const PlanEntry* entries = reinterpret_cast<const PlanEntry*>(ws + L.entries);
  const int32_t* row_tok = reinterpret_cast<const int32_t*>(ws + L.row_tok);
  const float* row_w = reinterpret_cast<const float*>(ws + L.row_w);
  uint16_t* a_hi = reinterpret_cast<uint16_t*>(ws + L.a_hi);
  uint16_t* a_lo = reinterpret_cast<uint16_t*>(ws + L.a_lo);
  uint16_t* s_hi = reinterpret_cast<uint16_t*>(ws + L.s_hi);
  uint16_t* s_lo = reinterpret_cast<uint16_t*>(ws + L.s_lo);
  const int runs = sI ? (T + kCols - 1) / kCols : 0;
  const int shared_blocks = runs * (sI / 16);
  const unsigned blocks = (unsigned)(shared_blocks + L.max_entries * (I / 16));
  hipLaunchKernelGGL((decode_gate_up_kernel<FMT, kFewWaves>), dim3(blocks),
                     dim3(kFewWaves * kWave), 0, stream, x, T, H, I, *r13, *s13, sI, shared_blocks,
                     n_entries, entries, row_tok, a_hi, a_lo, s_hi, s_lo);
#define MOE_DECODE_DOWN(TS)                                                                    \
  hipLaunchKernelGGL((decode_down_kernel<FMT, TS, kDownWaves>), dim3((unsigned)(H / 16)),        \
                     dim3(kDownWaves * kWave), 0, stream, T, H, I, *r2, *s2, sI, runs, n_entries, \
                     entries, row_w, a_hi, a_lo, s_hi, s_lo, out)
  if (T <= 16) MOE_DECODE_DOWN(1);
  else if (T <= 32) MOE_DECODE_DOWN(2);
  else MOE_DECODE_DOWN(4);
#undef MOE_DECODE_DOWN
}

int launch_decode(const float* logits, const uint8_t* row_valid, const uint16_t* x, int T, int H,
                  int I, int E, int K, int expert_begin, int El, int renorm, int32_t* topk_idx,
                  float* topk_w, const moe_ffn_weights* routed, const moe_ffn_weights* shared,
                  int sI, uint16_t* out, void* workspace, int32_t* dev_error, hipStream_t stream) {
  const DecodeLayout L = decode_layout(T, I, K, El, sI);
  if ((int64_t)L.max_entries * (I / 16) + (int64_t)(T + kCols - 1) / kCols * (sI / 16) > 0x7fffffff)
    return MOE_ERR_UNSUPPORTED;
  char* ws = static_cast<char*>(workspace);
  const int epl = (E + kWave - 1) / kWave;
#define MOE_PLAN(N)                                                                             \
  hipLaunchKernelGGL(plan_kernel<N>, dim3(1), dim3(kPlanThreads), 0, stream, logits, row_valid, T, \
                     E, K, renorm, expert_begin, El, topk_idx, topk_w,                          \
                     reinterpret_cast<int32_t*>(ws), reinterpret_cast<PlanEntry*>(ws + L.entries), \
                     reinterpret_cast<int32_t*>(ws + L.row_tok),                                \
                     reinterpret_cast<float*>(ws + L.row_w), dev_error)
  if (!logits) MOE_PLAN(0);
  else if (epl <= 1) MOE_PLAN(1);
  else if (epl <= 2) MOE_PLAN(2);
  else if (epl <= 4) MOE_PLAN(4);
  else if (epl <= 8) MOE_PLAN(8);
  else MOE_PLAN(16);
#undef MOE_PLAN
  const WMat r13{routed->w13, routed->w13_scales, routed->w13_tensor_scale};
  const WMat r2{routed->w2, routed->w2_scales, routed->w2_tensor_scale};
  WMat s13{}, s2{};
  if (shared) {
    s13 = WMat{shared->w13, shared->w13_scales, shared->w13_tensor_scale};
    s2 = WMat{shared->w2, shared->w2_scales, shared->w2_tensor_scale};
  }
  switch (routed->format) {
    case MOE_W_BF16:
      launch_decode_ffn<MOE_W_BF16>(x, T, H, I, K, &r13, &r2, &s13, &s2, sI, L, ws, out, stream);
      break;
    case MOE_W_FP8:
      launch_decode_ffn<MOE_W_FP8>(x, T, H, I, K, &r13, &r2, &s13, &s2, sI, L, ws, out, stream);
      break;
    case MOE_W_MXFP4:
      launch_decode_ffn<MOE_W_MXFP4>(x, T, H, I, K, &r13, &r2, &s13, &s2, sI, L, ws, out, stream);
      break;
    default:
      launch_decode_ffn<MOE_W_NVFP4>(x, T, H, I, K, &r13, &r2, &s13, &s2, sI, L, ws, out, stream);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// ---- the grouped FFN on 4-bit weights, few rows ---------------------------------
// Entry j of the segments: the j-th run of at most 16 rows, over the groups in
// order; a run's place follows from a scan of the counts by every wave (its
// answer the same in every lane).  A segment that leaves [0, capacity) has no
// runs and raises ROW_RANGE.  Returns false past the last run; `total` is the
// number of runs then.
struct RowRun {
  int g, row0, cnt;
};
__device__ __forceinline__ bool find_run(int j, const int32_t* __restrict__ cu_seqlens,
                                         const int32_t* __restrict__ counts, int G,
                                         int64_t capacity, int32_t* dev_error, RowRun& r,
                                         long long& total) {
  const int lane = threadIdx.x & 63;
  long long carry = 0;
  for (int base = 0; base < G; base += kWave) {
    const int e = base + lane;
    int c = 0, s0 = 0;
    if (e < G) {
      c = max(counts[e], 0);
      s0 = cu_seqlens[e];
      if (c > 0 && (s0 < 0 || (int64_t)s0 + c > capacity)) {
        raise_error(dev_error, MOE_DEVERR_ROW_RANGE);
        c = 0;
      }
    }
    const long long runs = ((long long)c + kCols - 1) / kCols;
    long long incl = runs;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const long long y = __shfl_up(incl, off, kWave);
      if (lane >= off) incl += y;
    }
    incl += carry;
    const uint64_t hit = __ballot(j >= incl - runs && j < incl);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      const int v = j - (int)__shfl(incl - runs, src, kWave);
      r.g = __builtin_amdgcn_readfirstlane(base + src);
      r.row0 = __builtin_amdgcn_readfirstlane(__shfl(s0, src, kWave) + v * kCols);
      r.cnt = __builtin_amdgcn_readfirstlane(min(kCols, __shfl(c, src, kWave) - v * kCols));
      return true;
    }
    carry = __shfl(incl, 63, kWave);
  }
  total = carry;
  return false;
}

template <int FMT, int NW>
__global__ void __launch_bounds__(NW * kWave, 4) few_gate_up_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ cu_seqlens,
    const int32_t* __restrict__ counts, int G, int H, int I, WMat W, int64_t capacity,
    uint16_t* __restrict__ a_hi, uint16_t* __restrict__ a_lo, int32_t* __restrict__ dev_error) {
  __shared__ f32x4_t red[NW][2][kWave];
  const int nt = I / 16, j = blockIdx.x / nt;
  RowRun r;
  long long total;
  if (!find_run(j, cu_seqlens, counts, G, capacity, dev_error, r, total)) return;
  const int col = threadIdx.x & 15;
  const uint16_t* xc = x + (int64_t)(r.row0 + min(col, r.cnt - 1)) * H;
  few_gate_up<FMT, NW>(W, r.g, blockIdx.x - j * nt, H, I, xc, r.cnt, a_hi + (int64_t)r.row0 * I,
                       a_lo + (int64_t)r.row0 * I, red);
}

// One workgroup: 16 output columns of one run; its waves split I.
template <int FMT, int NW>
__global__ void __launch_bounds__(NW * kWave, 4) few_down_kernel(
    const uint16_t* __restrict__ a_hi, const uint16_t* __restrict__ a_lo,
    const int32_t* __restrict__ cu_seqlens, const int32_t* __restrict__ counts, int G, int H,
    int I, WMat W, const float* __restrict__ row_scale, uint16_t* __restrict__ y,
    int64_t capacity, int64_t max_runs, int32_t* __restrict__ dev_error) {
  __shared__ f32x4_t red[NW][kWave];
  const int lane = threadIdx.x & 63, col = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nt = H / 16, j = blockIdx.x / nt, rt = blockIdx.x - j * nt;
  RowRun r;
  long long total;
  if (blockIdx.x == 0 && w == 0) {
    // overlapping segments can hold more runs than the grid: said, not dropped silently
    if ((find_run(0x7fffffff, cu_seqlens, counts, G, capacity, dev_error, r, total) ||
         total > max_runs) && lane == 0)
      raise_error(dev_error, MOE_DEVERR_ROW_RANGE);
  }
  if (!find_run(j, cu_seqlens, counts, G, capacity, dev_error, r, total)) return;
  const int64_t row = r.row0 + min(col, r.cnt - 1);
  WStream<FMT> ws[1];
  ws[0].init(W, r.g, rt >> 2, rt & 3, H / 64, I / 128, 16 * rt, lane);
  const int64_t o = row * I + 8 * (lane >> 4);
  const uint16_t* b[2] = {a_hi + o, a_lo + o};
  f32x4_t acc[1] = {f32x4_t{0.f, 0.f, 0.f, 0.f}};
  few_stream<FMT, 1, 2, 2>(ws, b, w, NW, I / 128, acc);
  red[w][lane] = acc[0];
  __syncthreads();
  if (w != 0) return;
  f32x4_t v = red[0][lane];
#pragma unroll
  for (int i = 1; i < NW; ++i) v += red[i][lane];
  if (col >= r.cnt) return;
  const float sc = row_scale ? row_scale[row] : 1.0f;
  *reinterpret_cast<uint2*>(y + row * H + rt * 16 + 4 * (lane >> 4)) =
      make_uint2(f32_to_bf16(sc * v[0]) | f32_to_bf16(sc * v[1]) << 16,
                 f32_to_bf16(sc * v[2]) | f32_to_bf16(sc * v[3]) << 16);
}

// Runs that disjoint segments of `capacity` rows over G groups can hold.
static int64_t max_row_runs(int64_t capacity, int G) {
  return std::min<int64_t>(G, capacity) + capacity / kCols;
}

template <int FMT>
static int launch_few_fmt(const uint16_t* x, const int32_t* cu, const int32_t* counts, int G,
                          int H, int I, const WMat& w13, const WMat& w2, const float* row_scale,
                          uint16_t* y, int64_t capacity, int flags, uint16_t* hi, uint16_t* lo,
                          int32_t* dev_error, hipStream_t stream) {
  const int64_t runs = max_row_runs(capacity, G);
  const int64_t gu = runs * (I / 16), dn = runs * (H / 16);
  if (gu > 0x7fffffff || dn > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  if (flags & MOE_FFN_GATE_UP)
    hipLaunchKernelGGL((few_gate_up_kernel<FMT, kFewWaves>), dim3((unsigned)gu),
                       dim3(kFewWaves * kWave), 0, stream, x, cu, counts, G, H, I, w13, capacity,
                       hi, lo, dev_error);
  if (flags & MOE_FFN_DOWN)
    hipLaunchKernelGGL((few_down_kernel<FMT, kFewWaves>), dim3((unsigned)dn),
                       dim3(kFewWaves * kWave), 0, stream, hi, lo, cu, counts, G, H, I, w2,
                       row_scale, y, capacity, runs, dev_error);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// The intermediate: capacity rows of I, high and low parts.
size_t few_ffn_workspace_bytes(int64_t capacity, int I) {
  return 2 * align256((size_t)capacity * I * 2);
}

int launch_few_ffn(const uint16_t* x, const int32_t* cu, const int32_t* counts, int G, int H,
                   int I, const moe_ffn_weights* wt, const float* row_scale, uint16_t* y,
                   int64_t capacity, int flags, void* workspace, int32_t* dev_error,
                   hipStream_t stream) {
  uint16_t* hi = static_cast<uint16_t*>(workspace);
  uint16_t* lo = hi + align256((size_t)capacity * I * 2) / 2;
  const WMat w13{wt->w13, wt->w13_scales, wt->w13_tensor_scale};
  const WMat w2{wt->w2, wt->w2_scales, wt->w2_tensor_scale};
  if (wt->format == MOE_W_MXFP4)
    return launch_few_fmt<MOE_W_MXFP4>(x, cu, counts, G, H, I, w13, w2, row_scale, y, capacity,
                                       flags, hi, lo, dev_error, stream);
  return launch_few_fmt<MOE_W_NVFP4>(x, cu, counts, G, H, I, w13, w2, row_scale, y, capacity,
                                     flags, hi, lo, dev_error, stream);
}

}  // namespace moe
