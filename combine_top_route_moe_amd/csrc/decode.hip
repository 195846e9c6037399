// The whole MoE layer for a few tokens (moe_decode), and the few-row form of
// the grouped FFN on 4-bit weights.
//
// For token t with chosen experts e_k and weights w_k:
//   h = W13[e_k] x_t,  a = silu(h[:I]) * h[I:],
//   out_t = bf16( sum_k w_k W2[e_k] a  +  the shared expert's row )
// With few tokens every product is a matrix times a handful of columns: the
// time is that of reading the chosen experts' weights once.  So no row is
// permuted or copied; the launches are
//   plan      (one workgroup) routes every token and lists, per expert that
//             any token chose, its tokens in runs of at most 16 ("entries");
//             for very few tokens gate_up does this itself;
//   gate_up   a workgroup owns a tile of gate rows and the matching up rows of
//             one entry's expert; its waves split H and add up through LDS;
//   down      a workgroup owns a tile of output columns of one entry, its waves
//             split I; the rows go out unrounded, in float32;
//   combine   weights and adds each token's rows in slot order, the shared
//             expert's last, and rounds once (small layers: within down).
// (Down and combine in one launch were tried two ways for all sizes.  A
// workgroup per 16 columns of all entries has too few workgroups to keep the
// memory busy: 1.6 TB/s at 13 tokens, 64 experts, H = 2048.  Splitting those
// and adding the parts in the last workgroup to arrive needs a device-wide
// release in each: writing back the L2s took 150 us at one token.)
// The products run on the matrix cores with the weights as the A operand (16
// weight rows) and the tokens as the B operand's 16 columns, so columns are
// independent: a token sees its own experts only, whatever values the others
// hold.  `a` is kept as two bf16 numbers (high and low part, 16 significant
// bits) and multiplied in two MFMAs, so no intermediate is rounded to bf16;
// sums are float32 throughout.
#include <algorithm>
#include <type_traits>

#include "route_common.h"
#include "weight_block.h"

namespace moe {

constexpr int kMaxTokens = 64;    // one bit of an expert's token mask each
constexpr int kCols = 16;         // tokens (or rows) of an entry
constexpr int kPlanThreads = 1024;
constexpr int kFusedTokens = 8;   // up to here gate/up routes by itself (and T * K <= 64, E <= 256)

// A run of at most 16 tokens of one local expert.
struct PlanEntry {
  int32_t e;       // local expert
  int32_t base;    // first compact row of the run
  int32_t cnt;     // rows of the run
};

// The workspace: plan, intermediate rows (routed, then shared), float32 rows.
struct DecodeLayout {
  size_t entries, row_tok, row_of, row_w, a, s_a, rows, s_rows, total;
  int64_t max_entries;
};
static size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
static DecodeLayout decode_layout(int T, int H, int I, int K, int El, int sI) {
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
  L.row_of = put((size_t)rows * 4);
  L.row_w = put((size_t)rows * 4);
  L.a = put((size_t)rows * I * 4);
  L.s_a = put((size_t)T * sI * 4);
  L.rows = put((size_t)rows * H * 4);
  L.s_rows = put(sI ? (size_t)T * H * 4 : 0);
  L.total = o;
  return L;
}

size_t decode_workspace_bytes(int T, int H, int I, int K, int El, int sI) {
  return decode_layout(T, H, I, K, El, sI).total;
}

// ---- top-k selection ----------------------------------------------------------
// A logit as a signed integer in the same order (NaN as -inf, -0 as +0), and
// back; every real logit lies above the integer minimum, which stands for "no
// expert".
__device__ __forceinline__ int order_key(float x) {
  const int b = __float_as_int(rank_value(x) + 0.0f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_value(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}
constexpr int kNoKey = (int)0x80000000;

// Wave-wide integer maximum, uniform: register moves within 16 lanes, then
// the four rows' maxima in scalar registers.
__device__ __forceinline__ int wave_max_i32(int v) {
  v = max(v, row16_dpp<0xB1>(v));
  v = max(v, row16_dpp<0x4E>(v));
  v = max(v, row16_dpp<0x141>(v));
  v = max(v, row16_dpp<0x140>(v));
  return max(max(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
             max(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}

// Keys of one token's logits, experts lane, lane + 64, .. (EPL a lane).
template <int EPL>
__device__ __forceinline__ void load_keys(const float* __restrict__ row, int E, int lane,
                                          int* key) {
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int x = lane + j * kWave;
    key[j] = x < E ? order_key(row[x]) : kNoKey;
  }
}

// One token's K best experts by one wave (every lane active), the same choice
// and order as moe_route's: lane k < K gets slot k's expert in sel_e and its
// logit in sel_v.  Each lane first sorts its keys, so that a round compares
// one head per lane: the wave maximum, the lanes that hold it (one, but for
// ties), and the winner drops its head.  Sorting pays while a lane holds few
// experts.
template <int EPL>
__device__ __forceinline__ void select_topk(const int* key, int K, int lane, int& sel_e,
                                            float& sel_v) {
  int h[EPL], e[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    h[j] = key[j];
    e[j] = lane + j * kWave;
  }
#pragma unroll
  for (int i = 1; i < EPL; ++i)               // stable: equal keys keep the lower index first
#pragma unroll
    for (int j = EPL - 1; j >= i; --j) {
      const bool sw = h[j] > h[j - 1];
      const int a = h[j - 1], b = e[j - 1];
      h[j - 1] = sw ? h[j] : a;
      e[j - 1] = sw ? e[j] : b;
      h[j] = sw ? a : h[j];
      e[j] = sw ? b : e[j];
    }
  int best = kNoKey;
  sel_e = -1;
  for (int k = 0; k < K; ++k) {
    const int mv = wave_max_i32(h[0]);
    uint64_t at = __ballot(h[0] == mv);
    int win = __builtin_amdgcn_readlane(e[0], __ffsll((unsigned long long)at) - 1);
    for (at &= at - 1; at; at &= at - 1)      // ties: the lowest index
      win = min(win, __builtin_amdgcn_readlane(e[0], __ffsll((unsigned long long)at) - 1));
    sel_e = lane == k ? win : sel_e;
    best = lane == k ? mv : best;
    const bool mine = (win & 63) == lane;
#pragma unroll
    for (int j = 0; j + 1 < EPL; ++j) {
      h[j] = mine ? h[j + 1] : h[j];
      e[j] = mine ? e[j + 1] : e[j];
    }
    h[EPL - 1] = mine ? kNoKey : h[EPL - 1];
  }
  sel_v = key_value(best);
}

// Four tokens at once, 16 lanes each, for E <= 64 and K <= 16: lane i of a
// token's row of lanes holds experts i, i + 16, .. and gets slot i.  Maximum
// and lowest index come by register moves within the row, nothing passes
// through scalar registers: 64 tokens of 64 experts, top-8, take the plan 6 us
// instead of the 11 of a wave per token.
__device__ __forceinline__ int row16_max(int v) {
  v = max(v, row16_dpp<0xB1>(v));
  v = max(v, row16_dpp<0x4E>(v));
  v = max(v, row16_dpp<0x141>(v));
  return max(v, row16_dpp<0x140>(v));
}
__device__ __forceinline__ int row16_min(int v) {
  v = min(v, row16_dpp<0xB1>(v));
  v = min(v, row16_dpp<0x4E>(v));
  v = min(v, row16_dpp<0x141>(v));
  return min(v, row16_dpp<0x140>(v));
}
__device__ __forceinline__ void select_topk_row16(const float* __restrict__ row, int E, int K,
                                                  int i, int& sel_e, float& sel_v) {
  int h[4], e[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    e[j] = i + 16 * j;
    h[j] = e[j] < E ? order_key(row[e[j]]) : kNoKey;
  }
#pragma unroll
  for (int p = 1; p < 4; ++p)                 // stable: equal keys keep the lower index first
#pragma unroll
    for (int j = 3; j >= p; --j) {
      const bool sw = h[j] > h[j - 1];
      const int a = h[j - 1], b = e[j - 1];
      h[j - 1] = sw ? h[j] : a;
      e[j - 1] = sw ? e[j] : b;
      h[j] = sw ? a : h[j];
      e[j] = sw ? b : e[j];
    }
  int best = kNoKey;
  sel_e = -1;
  for (int k = 0; k < K; ++k) {
    const int mv = row16_max(h[0]);
    const int win = row16_min(h[0] == mv ? e[0] : 0x7fffffff);
    sel_e = i == k ? win : sel_e;
    best = i == k ? mv : best;
    const bool mine = e[0] == win && h[0] == mv;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      h[j] = mine ? h[j + 1] : h[j];
      e[j] = mine ? e[j + 1] : e[j];
    }
    h[3] = mine ? kNoKey : h[3];
  }
  sel_v = key_value(best);
}

// The selected experts' weights (lane k < K: slot k's), as moe_route's.
template <int EPL>
__device__ __forceinline__ float topk_weight(const int* key, int E, int K, int renorm, int lane,
                                             float sel_v) {
  const float lmax = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sel_v), 0));
  double num = 0.0;
  if (lane < K) num = weight_term(sel_v, lmax);
  double den = 0.0;
  if (renorm) {
    den = sum_lanes_below(num, K);
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane + j * kWave < E) den += weight_term(key_value(key[j]), lmax);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) den += __shfl_xor(den, off, kWave);
  }
  return (float)(num / den);
}

// ---- plan -------------------------------------------------------------------
// One workgroup.  EPL 0: the routes are given (topk_idx, topk_w are inputs),
// else experts per lane of the selection by a wave per token.  The weights'
// exponentials (double, as moe_route's) are taken by one thread per slot, not
// by a few lanes of each token's wave.  All latency: 5 us from 13 to 64 tokens of
// 64 experts, top-8, and 5 on given routes.  Routing more tokens than there are
// waves here is left to route_few_kernel, over many CUs, unless 16 lanes can
// do one.
struct DecodePlan {
  int32_t* n_entries;
  PlanEntry* entries;
  int32_t* row_tok;   // token of a compact row
  int32_t* row_of;    // compact row of a slot, -1: no local expert
  float* row_w;       // weight of a compact row (written by gate/up's plan only)
};

template <int EPL>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ row_valid, int T, int E, int K,
    int renorm, int expert_begin, int El, int32_t* __restrict__ topk_idx,
    float* __restrict__ topk_w, DecodePlan plan, int32_t* __restrict__ dev_error) {
  constexpr int kSlots = EPL > 0 ? kMaxTokens * 32 : 1;
  __shared__ uint32_t mask[1024][2];
  __shared__ int sel_e[kMaxTokens * 32];
  __shared__ float sel_v[kSlots];
  __shared__ double term[kSlots];
  __shared__ int base_of[1024];
  __shared__ int wave_sum[kPlanThreads / kWave];
  constexpr int kWaves = kPlanThreads / kWave;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  mask[tid][0] = 0u;
  mask[tid][1] = 0u;
  __syncthreads();
  // slot k of token t goes to expert e (-1: none), its logit being v
  auto note = [&](int t, int k, int e, float v) {
    const int slot = t * K + k;
    const bool here = e >= expert_begin && e < E && e - expert_begin < El;
    // -2: no expert at all (a masked token's weight is 0)
    sel_e[slot] = here ? e - expert_begin : e < 0 ? -2 : -1;
    if (here) atomicOr(&mask[e - expert_begin][t >> 5], 1u << (t & 31));
    if constexpr (EPL > 0) {
      sel_v[slot] = v;
      topk_idx[slot] = e;
    }
  };
  if constexpr (EPL == 0) {
    for (int i = tid; i < T * K; i += kPlanThreads) {
      const int t = i / K;
      const int e = !row_valid || row_valid[t] ? topk_idx[i] : -1;
      if (e >= E) raise_error(dev_error, MOE_DEVERR_EXPERT_RANGE);
      note(t, i - t * K, e, 0.0f);
    }
  } else if (EPL == 1 && K <= 16 && renorm) {
    const int t = tid >> 4, i = tid & 15;
    if (4 * wv < T) {                       // the whole wave or none of it
      int e;
      float v;
      select_topk_row16(logits + (int64_t)min(t, T - 1) * E, E, K, i, e, v);
      if (t < T && i < K) note(t, i, !row_valid || row_valid[t] ? e : -1, v);
    }
  } else {
    for (int t = wv; t < T; t += kWaves) {
      int key[EPL > 0 ? EPL : 1], e = -1;
      float v = 0.0f;
      if (!row_valid || row_valid[t]) {
        load_keys<EPL>(logits + (int64_t)t * E, E, lane, key);
        select_topk<EPL>(key, K, lane, e, v);
        if (!renorm) {
          const float w = topk_weight<EPL>(key, E, K, renorm, lane, v);
          if (lane < K) topk_w[t * K + lane] = w;
        }
      }
      if (lane < K) note(t, lane, e, v);
    }
  }
  __syncthreads();
  if constexpr (EPL > 0) {
    for (int i = tid; i < T * K; i += kPlanThreads)
      term[i] = weight_term(sel_v[i], sel_v[i / K * K]);
  }
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
  for (int i = 0; i < kWaves; ++i) {
    if (i < wv) before += wave_sum[i];
    total += wave_sum[i];
  }
  const int excl = before + incl - (ne << 16 | c);
  const int ent0 = excl >> 16, base = excl & 0xffff;
  base_of[tid] = base;
  for (int v = 0; v < ne; ++v)
    plan.entries[ent0 + v] = PlanEntry{tid, base + v * kCols, min(kCols, c - v * kCols)};
  if (tid == 0) *plan.n_entries = total >> 16;
  __syncthreads();
  // each slot's compact row: a (token, expert) pair has one, also where the
  // token names the expert in several slots
  for (int i = tid; i < T * K; i += kPlanThreads) {
    const int e = sel_e[i], t = i / K;
    if constexpr (EPL > 0) {
      if (renorm) {
        double den = 0.0;
        for (int j = t * K; j < (t + 1) * K; ++j) den += term[j];   // slot order
        topk_w[i] = e == -2 ? 0.0f : (float)(term[i] / den);
      } else if (e == -2) {
        topk_w[i] = 0.0f;
      }
    }
    int pos = -1;
    if (e >= 0) {
      const uint64_t em = (uint64_t)mask[e][1] << 32 | mask[e][0];
      pos = base_of[e] + __popcll(em & ((1ull << t) - 1));
      plan.row_tok[pos] = t;
    }
    plan.row_of[i] = pos;
  }
}

// Routes alone, a wave per token over as many CUs, for a plan on given routes.
template <int EPL>
__global__ void __launch_bounds__(kWave) route_few_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ row_valid, int E, int K,
    int renorm, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  const int t = blockIdx.x, lane = threadIdx.x;
  int key[EPL], e = -1;
  float v = 0.0f, w = 0.0f;
  if (!row_valid || row_valid[t]) {
    load_keys<EPL>(logits + (int64_t)t * E, E, lane, key);
    select_topk<EPL>(key, K, lane, e, v);
    w = topk_weight<EPL>(key, E, K, renorm, lane, v);
  }
  if (lane < K) {
    topk_idx[t * K + lane] = e;
    topk_w[t * K + lane] = w;
  }
}

// ---- the streamed product ---------------------------------------------------
// acc[i] += W_i[16 rows, blocks kb0, kb0 + step, ..] * (sum over a of B_a)^T for
// NF weight fragments of one column tile and NB 16-column operands out of the
// buffer b (boff[a]: the byte offset of the lane's column's first element).
// A wave has one block in flight, into registers that the block before leaves
// free as its MFMAs go; the waves of the other workgroups on the CU cover the
// wait.  (Two in flight, with fewer waves: MXFP4 4 to 8 % longer at 8 tokens and
// as long at one; NVFP4 52 us for 333 rows of ragged experts instead of 49; bf16
// and FP8 within 2 %.)
template <int FMT, int NF, int NB, bool GU>
__device__ __forceinline__ void few_stream(const WStream<FMT, NF, GU>& ws, buffer_t b,
                                           const uint32_t* boff, int kb0, int step, int nkb,
                                           f32x4_t* acc) {
  typename WStream<FMT, NF, GU>::Tile w;
  u32x4_t x[NB][4];
  auto load = [&](int kb) {
    ws.load(w, kb);
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
      for (int p = 0; p < 4; ++p) x[a][p] = load_b128<false>(b, boff[a] + p * 64, kb * 256);
  };
  auto use = [&]() {
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const bf16x8_t wf = w.operand(f, p);
#pragma unroll
        for (int a = 0; a < NB; ++a)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              wf, __builtin_bit_cast(bf16x8_t, x[a][p]), acc[f], 0, 0, 0);
      }
  };
  if (kb0 >= nkb) return;
  load(kb0);
  for (int kb = kb0 + step; kb < nkb; kb += step) {
    use();
    load(kb);
  }
  use();
}

// The shape of a few-row product, by format: NF fragments a wave (gate/up: half
// gate, half up), kWaves waves to a SIMD (what the registers of that allow).  A
// whole 64-row column tile reads each row of x, or of a, for four fragments;
// bf16 (4 KB a fragment and block) and FP8 can take two (NARROW), the 4-bit
// formats' blocks are whole tiles.
template <int FMT, bool NARROW = false>
struct FewShape {
  static constexpr int NF = NARROW ? 2 : 4;
  static constexpr int kWaves = FMT >= MOE_W_MXFP4 || NARROW ? 5 : 4;
};
// FP8 is narrow while the launch has so few workgroups that all run at once,
// three to a CU: one token, 8 of 64 experts, H = 2048, I = 1024 19 us instead of
// 22; with more, reading x twice as often costs more: 40 tokens, H = 7168, I =
// 2048 554 us instead of 459.  bf16 goes by the rows that share an expert and
// their length, wide / narrow: 64 experts, top-8, H = 7168, I = 2048 and a shared
// one, 64 tokens 886 / 1010 us, 32 840 / 889, 8 581 / 605 (and one, by another
// run, 134 / 130); 8 experts, top-2, H = 4096, I = 8192, 64 tokens 375 / 434; 64
// experts, top-8, H = 2048, I = 1024, 64 tokens 149 / 152, 32 145 / 136.
template <int FMT>
static bool narrow_tiles(int64_t workgroups, int64_t slots, int E, int reduction) {
  return FMT == MOE_W_FP8 ? workgroups <= 3 * 256 : slots * reduction < 12288LL * E;
}

// Waves of a workgroup, which split the reduction: 4, or 8 where the launch has
// at most a workgroup for each CU and a wave of 4 would walk two blocks or more.
// MXFP4, the grouped FFN's two stages, 4 / 8 waves in us: H = 7168, I = 2048, 1
// row 21 / 16; H = 2048, I = 1024, 4 experts of a row 11.5 / 10.6, 8 (256
// workgroups) 12.8 / 11.8, 16 15.6 / 16.1; H = 512, I = 256 7.8 / 8.1; one token
// of 64 experts, top-2, H = 7168, I = 2048, 24.7 / 20.0 (FP8 29.5 / 25.1, bf16 35.4
// / 35.5: its waves have twice the tiles and keep four).
template <int FMT>
static bool eight_waves(int64_t workgroups, int reduction) {
  return FMT != MOE_W_BF16 && workgroups <= 256 && reduction >= 8 * 128;
}
using Four = std::integral_constant<int, 4>;
using Eight = std::integral_constant<int, 8>;

// v as the sum of two bf16 numbers, high part first (an infinity or NaN, also
// one that v rounds to, alone)
__device__ __forceinline__ void split_bf16(float v, uint32_t& hi, uint32_t& lo) {
  hi = f32_to_bf16(v);
  lo = (hi & 0x7f80u) == 0x7f80u ? 0u : f32_to_bf16(v - bf16_to_f32(hi));
}

// One workgroup's gate/up tile: 8 NF intermediate columns, nt of expert g, for
// the cnt <= 16 rows whose x this lane's column is at byte xoff of x (columns
// past cnt repeat the last one and are not stored).  a rows go to a + column *
// 2 I, the I high parts before the I low ones.
template <int FMT, int NW, typename Shape>
__device__ __forceinline__ void few_gate_up(const WMat& W, int g, int nt, int H, int I,
                                            buffer_t x, uint32_t xoff, int cnt,
                                            uint16_t* a,
                                            f32x4_t (*red)[Shape::NF][kWave]) {
  constexpr int NF = Shape::NF, NH = NF / 2;   // NH gate and NH up fragments
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = H / 128, ct = nt * NH / 2, f0 = nt * NH % 2;
  WStream<FMT, NF, true> ws;
  ws.init(W, g, ct, f0, I / 32, nkb, 32 * ct, I + 32 * ct, lane);
  f32x4_t acc[NF];
#pragma unroll
  for (int i = 0; i < NF; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint32_t off[1] = {xoff + 16 * (lane >> 4)};
  few_stream<FMT, NF, 1, true>(ws, x, off, w, NW, nkb, acc);
#pragma unroll
  for (int i = 0; i < NF; ++i) red[w][i][lane] = acc[i];
  __syncthreads();
  if (w >= NH) return;
  f32x4_t gt = red[0][w][lane], up = red[0][NH + w][lane];
#pragma unroll
  for (int i = 1; i < NW; ++i) {
    gt += red[i][w][lane];
    up += red[i][NH + w][lane];
  }
  // lane holds rows 4 (l / 16) .. +4 of the fragment for column l % 16
  const int col = lane & 15;
  if (col >= cnt) return;
  uint32_t h[4], l[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) split_bf16(silu_f(gt[q]) * up[q], h[q], l[q]);
  uint16_t* o = a + (int64_t)col * 2 * I + 32 * ct + 16 * (f0 + w) + 4 * (lane >> 4);
  *reinterpret_cast<uint2*>(o) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  *reinterpret_cast<uint2*>(o + I) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// ---- the plan of a few routed tokens, by every wave on its own ------------------
// Lane i stands for slot i = t K + k < 64 and knows its local expert (-1: none).
// Entries are the experts in the order of their first slots.
struct SmallPlan {
  uint64_t same;      // slots of this lane's expert
  uint64_t leaders;   // first slots of the experts
  int base;           // for a leader: compact rows of the experts before its own
};
__device__ __forceinline__ SmallPlan small_plan(int e, int n_slots, int T, int lane) {
  SmallPlan p;
  p.same = 1ull << lane;
  if (T > 1) {
    for (int s = 0; s < n_slots; ++s) {
      const uint64_t b = __ballot(e == __builtin_amdgcn_readlane(e, s));
      if (lane == s) p.same = b;
    }
  }
  const bool leader = e >= 0 && !(p.same & ((1ull << lane) - 1));
  p.leaders = __ballot(leader);
  const int c = leader ? __popcll(p.same) : 0;
  int incl = c;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(incl, off, kWave);
    if (lane >= off) incl += y;
  }
  p.base = incl - c;
  return p;
}

// ---- moe_decode: gate/up ------------------------------------------------------
// Blocks [0, shared_blocks): the shared expert's tiles, 16 tokens a run; then
// (entry, tile), the entries past the plan's leaving at once.  EPL > 0: no plan
// was made; every workgroup routes the (few) tokens itself, and one more at the
// end of the grid writes the plan for the down kernel.  That saves a launch,
// 5 us, and costs each workgroup about 1.
// Bound by the memory: at one token of 256 experts, top-8 and a shared one (H =
// 7168, I = 2048) 83 us in bf16, 6.4 TB/s, 29 in MXFP4, where a plain read of as
// many bytes takes 24; 13 tokens of 64 experts in FP8 (H = 2048, I = 1024) 42,
// a plain read 33.  NVFP4 by its conversion: 24 tokens of 128 experts, top-8 (H =
// 4096, I = 1536) 136 us, 5.2 TB/s, the vector units busy 87 % of the time.
template <int FMT, int NW, bool NARROW, int EPL>
__global__ void __launch_bounds__(NW * kWave, (FewShape<FMT, NARROW>::kWaves)) decode_gate_up_kernel(
    const uint16_t* __restrict__ x, int T, int H, int I, WMat routed, WMat shared, int sI,
    int shared_blocks, DecodePlan plan, uint16_t* __restrict__ a, uint16_t* __restrict__ s_a,
    const float* __restrict__ logits,
    const uint8_t* __restrict__ row_valid, int E, int K, int renorm, int expert_begin, int El,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  using Shape = FewShape<FMT, NARROW>;
  constexpr int kTile = 8 * Shape::NF;   // intermediate columns of a workgroup
  __shared__ f32x4_t red[NW][Shape::NF][kWave];
  __shared__ int sel[64];
  __shared__ float sel_w[64];
  const int lane = threadIdx.x & 63, col = lane & 15;
  const buffer_t xbuf = uniform_buffer(x, (int64_t)T * H * 2);
  int b = blockIdx.x;
  const bool sh = b < shared_blocks;
  if (!sh) b -= shared_blocks;
  const int Ic = sh ? sI : I;
  const int nt = Ic / kTile, j = b / nt;
  int g, base, cnt, tok = 0;
  if (sh) {
    g = 0;
    base = j * kCols;
    cnt = min(kCols, T - base);
    tok = base + min(col, cnt - 1);
  } else
  if constexpr (EPL > 0) {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool writer = blockIdx.x == gridDim.x - 1;
    for (int t = w; t < T; t += NW) {
      int e = -1;
      int v[EPL];
      float sv = 0.0f, wt = 0.0f;
      if (!row_valid || row_valid[t]) {
        load_keys<EPL>(logits + (int64_t)t * E, E, lane, v);
        select_topk<EPL>(v, K, lane, e, sv);
        if (writer) wt = topk_weight<EPL>(v, E, K, renorm, lane, sv);
      }
      if (lane < K) {
        if (writer) {
          topk_idx[t * K + lane] = e;
          topk_w[t * K + lane] = wt;
          sel_w[t * K + lane] = wt;
        }
        sel[t * K + lane] = e >= expert_begin && e - expert_begin < El ? e - expert_begin : -1;
      }
    }
    __syncthreads();
    const int e = lane < T * K ? sel[lane] : -1;
    const SmallPlan p = small_plan(e, T * K, T, lane);
    const int n = __popcll(p.leaders);
    if (writer) {
      if (w != 0) return;
      if (lane == 0) *plan.n_entries = n;
      const int lead = __ffsll((unsigned long long)p.same) - 1;
      const int pos = __shfl(p.base, lead, kWave) + __popcll(p.same & ((1ull << lane) - 1));
      if (lane < T * K) plan.row_of[lane] = e >= 0 ? pos : -1;
      if (e >= 0) {
        plan.row_tok[pos] = lane / K;
        plan.row_w[pos] = sel_w[lane];
        if (lead == lane)
          plan.entries[__popcll(p.leaders & ((1ull << lane) - 1))] =
              PlanEntry{e, p.base, (int)__popcll(p.same)};
      }
      return;
    }
    if (j >= n) return;
    const bool it = ((p.leaders >> lane) & 1) && __popcll(p.leaders & ((1ull << lane) - 1)) == j;
    const int src = __ffsll((unsigned long long)__ballot(it)) - 1;
    g = __builtin_amdgcn_readlane(e, src);
    base = __builtin_amdgcn_readlane(p.base, src);
    uint64_t m = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(p.same >> 32), src) << 32 |
                 (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)p.same, src);
    cnt = __popcll(m);
    for (int c = 0; m; m &= m - 1, ++c)   // columns past the last repeat it
      if (col >= c) tok = (__ffsll((unsigned long long)m) - 1) / K;
  } else {
    if (j >= *plan.n_entries) return;
    g = plan.entries[j].e;
    base = plan.entries[j].base;
    cnt = plan.entries[j].cnt;
    tok = plan.row_tok[base + min(col, cnt - 1)];
  }
  few_gate_up<FMT, NW, Shape>(sh ? shared : routed, g, b - j * nt, H, Ic, xbuf,
                          (uint32_t)tok * H * 2u, cnt, (sh ? s_a : a) + (int64_t)base * 2 * Ic,
                          red);
}

// ---- down ---------------------------------------------------------------------
// One workgroup's down tile: 16 NF output columns of the cnt <= 16 rows of a
// (each I high parts, then I low ones), for expert g; store(first of four
// columns, row, their sums) for every row.  The high and the low part of up to
// 8 rows share one B operand, columns c and c + 8, and are added at the end:
// one MFMA and one read of a for both.  9 to 16 rows take two operands, into
// the same sums.
template <int FMT, int NF, int NW, int NB>
__device__ __forceinline__ void few_down_rows(const WStream<FMT, NF, false>& ws, buffer_t a,
                                              const uint32_t* off, int nkb,
                                              f32x4_t (*red)[NF][kWave]) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  f32x4_t acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  few_stream<FMT, NF, NB, false>(ws, a, off, w, NW, nkb, acc);
#pragma unroll
  for (int f = 0; f < NF; ++f) red[w][f][lane] = acc[f];
}

template <int FMT, int NW, typename Shape, typename Store>
__device__ __forceinline__ void few_down(const WMat& W, int g, int tile, int H, int I,
                                         const uint16_t* rows, int cnt,
                                         f32x4_t (*red)[Shape::NF][kWave], Store store) {
  constexpr int NF = Shape::NF;
  const int lane = threadIdx.x & 63, col = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  WStream<FMT, NF, false> ws;
  ws.init(W, g, tile * NF / 4, tile * NF % 4, H / 64, I / 128, 16 * NF * tile, 0, lane);
  const buffer_t a = uniform_buffer(rows, (int64_t)cnt * I * 4);
  const bool one = cnt <= 8;
  uint32_t off[2];
  off[0] = (uint32_t)(min(one ? col & 7 : col, cnt - 1) * 2 * I + (one && col & 8 ? I : 0) +
                      8 * (lane >> 4)) * 2u;
  off[1] = off[0] + 2u * I;
  if (one)
    few_down_rows<FMT, NF, NW, 1>(ws, a, off, I / 128, red);
  else
    few_down_rows<FMT, NF, NW, 2>(ws, a, off, I / 128, red);
  __syncthreads();
  for (int f = w; f < NF; f += NW) {
    f32x4_t v = red[0][f][lane];
#pragma unroll
    for (int k = 1; k < NW; ++k) v += red[k][f][lane];
    if (one) {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += __shfl_xor(v[q], 8, kWave);
    }
    if (col < cnt && (col < 8 || !one)) store(16 * (tile * NF + f) + 4 * (lane >> 4), col, v);
  }
}

// moe_decode: the rows go out in float32, unweighted; blocks as in gate/up.
// Bound as gate/up is, at half its bytes: 40 us (6.6 TB/s), 13.5, 20 and 73 for
// the sizes named there.
template <int FMT, int NW, bool NARROW>
__global__ void __launch_bounds__(NW * kWave, (FewShape<FMT, NARROW>::kWaves)) decode_down_kernel(
    int T, int H, int I, WMat routed, WMat shared, int sI, int shared_blocks, DecodePlan plan,
    const uint16_t* __restrict__ a, const uint16_t* __restrict__ s_a, float* __restrict__ rows,
    float* __restrict__ s_rows) {
  using Shape = FewShape<FMT, NARROW>;
  __shared__ f32x4_t red[NW][Shape::NF][kWave];
  const int nt = H / (16 * Shape::NF);
  int b = blockIdx.x;
  const bool sh = b < shared_blocks;
  if (!sh) b -= shared_blocks;
  const int j = b / nt;
  if (!sh && j >= *plan.n_entries) return;
  const int g = sh ? 0 : plan.entries[j].e;
  const int base = sh ? j * kCols : plan.entries[j].base;
  const int cnt = sh ? min(kCols, T - base) : plan.entries[j].cnt;
  const int Ic = sh ? sI : I;
  float* r = (sh ? s_rows : rows) + (int64_t)base * H;
  few_down<FMT, NW, Shape>(sh ? shared : routed, g, b - j * nt, H, Ic,
                    (sh ? s_a : a) + (int64_t)base * 2 * Ic, cnt, red,
                    [&](int c, int row, f32x4_t v) {
                      *reinterpret_cast<f32x4_t*>(r + (int64_t)row * H + c) = v;
                    });
}

// ---- moe_decode: down + combine of a small layer ----------------------------------
// After gate/up's own plan, where the down weights are so few that launches are
// what counts: a workgroup of 16 waves owns 16 NF output columns of all the (at
// most 8) tokens.  The blocks of 128 intermediate columns of all entries (the
// shared expert's last) form one axis, which the waves split evenly; a wave
// accumulates an entry's rows, high parts in columns 0 .. 7 and low ones in
// 8 .. 15 as in few_down, and at its end weights them and adds them to the
// tokens' lanes; the waves' sums are added through LDS in order and rounded.
// It saves a launch and has few workgroups: one token, 16 experts, top-2, H =
// 1024, I = 512, bf16, the layer takes 9.3 us instead of 10.2; 64 experts,
// top-8, H = 2048, I = 1024 29 instead of 25.  Like few_stream, one block in
// flight a wave.
constexpr int64_t kSmallDown = 1 << 20;   // down weights of a call's slots, up to here
template <int FMT>
struct FewDownShape {
  static constexpr int NF = FMT == MOE_W_BF16 || FMT == MOE_W_FP8 ? 2 : 4;
};
template <int FMT>
__global__ void __launch_bounds__(16 * kWave) decode_down_combine_kernel(
    int T, int H, int I, WMat routed, WMat shared, int sI, DecodePlan plan,
    const uint16_t* __restrict__ a, const uint16_t* __restrict__ s_a, uint16_t* __restrict__ out) {
  constexpr int NF = FewDownShape<FMT>::NF, NW = 16;
  __shared__ f32x4_t red[NW][NF][kWave];
  const int lane = threadIdx.x & 63, col = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ct = blockIdx.x * NF / 4, f0 = blockIdx.x * NF % 4, n_ct = H / 64;
  const int nb = I / 128, n = *plan.n_entries, nr = n * nb, total = nr + sI / 128;
  const int b0 = total * w / NW, b1 = total * (w + 1) / NW;
  f32x4_t tok[NF], acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) tok[f] = acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  typename WStream<FMT, NF, false>::Tile wt;
  u32x4_t x[4];
  auto load = [&](int b) {
    const bool sh = b >= nr;
    const int j = sh ? 0 : b / nb;
    const int kb = sh ? b - nr : b - j * nb;
    const PlanEntry en = plan.entries[j];   // (unused past the plan: the shared expert)
    const int cnt = sh ? T : en.cnt;
    const int64_t base = sh ? 0 : en.base;
    const int Ic = sh ? sI : I;
    WStream<FMT, NF, false> ws;
    ws.init(sh ? shared : routed, sh ? 0 : en.e, ct, f0, n_ct, Ic / 128, 64 * ct, 0, lane);
    ws.load(wt, kb);
    const buffer_t r = uniform_buffer((sh ? s_a : a) + base * 2 * Ic, (int64_t)cnt * Ic * 4);
    const uint32_t off =
        (uint32_t)(min(col & 7, cnt - 1) * 2 * Ic + (col & 8 ? Ic : 0) + 8 * (lane >> 4)) * 2u;
#pragma unroll
    for (int p = 0; p < 4; ++p) x[p] = load_b128<false>(r, off + p * 64, kb * 256);
  };
  auto use = [&](int b) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int f = 0; f < NF; ++f)
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            wt.operand(f, p), __builtin_bit_cast(bf16x8_t, x[p]), acc[f], 0, 0, 0);
    const bool sh = b >= nr;
    const int j = sh ? 0 : b / nb;
    if (b + 1 != b1 && b + 1 != (sh ? total : (j + 1) * nb)) return;
    // the entry (or the wave's part of it) is done: row i is column i, its low
    // part column i + 8
    const int cnt = sh ? T : plan.entries[j].cnt, base = sh ? 0 : plan.entries[j].base;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[f][q] += __shfl_xor(acc[f][q], 8, kWave);
    for (int i = 0; i < cnt; ++i) {
      const int t_ = sh ? i : plan.row_tok[base + i];
      const float rw = sh ? 1.0f : plan.row_w[base + i];
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v = __shfl(acc[f][q], (lane & 48) | i, kWave);
          tok[f][q] += col == t_ ? rw * v : 0.0f;
        }
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  };
  if (b1 > b0) {
    load(b0);
    for (int b = b0; b + 1 < b1; ++b) {
      use(b);
      load(b + 1);
    }
    use(b1 - 1);
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) red[w][f][lane] = tok[f];
  __syncthreads();
  if (w >= NF || col >= T) return;
  f32x4_t v = red[0][w][lane];
#pragma unroll
  for (int i = 1; i < NW; ++i) v += red[i][w][lane];
  *reinterpret_cast<uint2*>(out + (int64_t)col * H + 16 * (blockIdx.x * NF + w) + 4 * (lane >> 4)) =
      make_uint2(f32_to_bf16(v[0]) | f32_to_bf16(v[1]) << 16,
                 f32_to_bf16(v[2]) | f32_to_bf16(v[3]) << 16);
}

// ---- moe_decode: combine --------------------------------------------------------
// out[t] = bf16( sum over the slots in order of w * row, then the shared row ):
// one thread per 4 columns of a token, 64-thread workgroups.  Two dependent
// loads and the launch: 4 to 5 us from 1 to 64 tokens.
__global__ void __launch_bounds__(64) decode_combine_kernel(
    int T, int H, int K, const int32_t* __restrict__ row_of, const float* __restrict__ topk_w,
    const float* __restrict__ rows, const float* __restrict__ s_rows, uint16_t* __restrict__ out) {
  const int t = blockIdx.y, c = (blockIdx.x * 64 + threadIdx.x) * 4;
  if (c >= H) return;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  // 8 slots' rows in flight together; slots without a row read row 0 and drop it
  for (int k0 = 0; k0 < K; k0 += 8) {
    int r[8];
    float w[8];
    f32x4_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = t * K + min(k0 + i, K - 1);
      r[i] = k0 + i < K ? row_of[at] : -1;
      r[i] = r[i] < T * K ? r[i] : -1;   // never past the rows, whatever the plan holds
      w[i] = topk_w[at];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = *reinterpret_cast<const f32x4_t*>(rows + (int64_t)max(r[i], 0) * H + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r[i] < 0) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] += w[i] * v[i][q];
    }
  }
  if (s_rows) acc += *reinterpret_cast<const f32x4_t*>(s_rows + (int64_t)t * H + c);
  *reinterpret_cast<uint2*>(out + (int64_t)t * H + c) =
      make_uint2(f32_to_bf16(acc[0]) | f32_to_bf16(acc[1]) << 16,
                 f32_to_bf16(acc[2]) | f32_to_bf16(acc[3]) << 16);
}

// What launch_decode hands on, with the workspace laid out.
struct DecodeArgs {
  const float* logits;
  const uint8_t* row_valid;
  const uint16_t* x;
  int T, H, I, E, K, expert_begin, El, renorm, sI;
  int32_t* topk_idx;
  float* topk_w;
  WMat r13, r2, s13, s2;
  uint16_t* out;
  DecodeLayout L;
  char* ws;
};

static DecodePlan plan_of(const DecodeArgs& d) {
  return {reinterpret_cast<int32_t*>(d.ws), reinterpret_cast<PlanEntry*>(d.ws + d.L.entries),
          reinterpret_cast<int32_t*>(d.ws + d.L.row_tok),
          reinterpret_cast<int32_t*>(d.ws + d.L.row_of),
          reinterpret_cast<float*>(d.ws + d.L.row_w)};
}

template <int FMT>
static void launch_decode_ffn(const DecodeArgs& d, bool fused, hipStream_t stream) {
  const DecodeLayout& L = d.L;
  const DecodePlan plan = plan_of(d);
  uint16_t* a = reinterpret_cast<uint16_t*>(d.ws + L.a);
  uint16_t* s_a = reinterpret_cast<uint16_t*>(d.ws + L.s_a);
  float* rows = reinterpret_cast<float*>(d.ws + L.rows);
  float* s_rows = d.sI ? reinterpret_cast<float*>(d.ws + L.s_rows) : nullptr;
  const int runs = d.sI ? (d.T + kCols - 1) / kCols : 0;
  auto gate = [&](auto narrow, auto epl, auto nw) {
    constexpr bool NARROW = decltype(narrow)::value;
    constexpr int EPL = decltype(epl)::value, NW = decltype(nw)::value;
    constexpr int kTile = 8 * FewShape<FMT, NARROW>::NF;
    const int sb = runs * (d.sI / kTile);
    hipLaunchKernelGGL((decode_gate_up_kernel<FMT, NW, NARROW, EPL>),
                       dim3((unsigned)(sb + L.max_entries * (d.I / kTile) + (EPL ? 1 : 0))),
                       dim3(NW * kWave), 0, stream, d.x, d.T, d.H, d.I, d.r13, d.s13, d.sI, sb,
                       plan, a, s_a, d.logits, d.row_valid, d.E, d.K, d.renorm, d.expert_begin,
                       d.El, d.topk_idx, d.topk_w);
  };
  auto gate_shape = [&](auto narrow, auto nw) {
    if (!fused) gate(narrow, std::integral_constant<int, 0>{}, nw);
    else if (d.E <= 64) gate(narrow, std::integral_constant<int, 1>{}, nw);
    else gate(narrow, std::integral_constant<int, 4>{}, nw);
  };
  auto down = [&](auto narrow, auto nw) {
    constexpr bool NARROW = decltype(narrow)::value;
    constexpr int NW = decltype(nw)::value;
    const int nt = d.H / (16 * FewShape<FMT, NARROW>::NF);
    hipLaunchKernelGGL((decode_down_kernel<FMT, NW, NARROW>),
                       dim3((unsigned)((runs + L.max_entries) * nt)), dim3(NW * kWave), 0, stream,
                       d.T, d.H, d.I, d.r2, d.s2, d.sI, runs * nt, plan, a, s_a, rows, s_rows);
  };
  // workgroups of the two stages at NF = 4
  const int64_t wg_gate = runs * (d.sI / 32) + L.max_entries * (d.I / 32);
  const int64_t wg_down = (runs + L.max_entries) * (d.H / 64);
  constexpr std::bool_constant<FMT == MOE_W_BF16 || FMT == MOE_W_FP8> kNarrow{};   // (false: one shape)
  constexpr int kHalf = kNarrow ? 2 : 1;   // NF = 2 wherever few
  const int64_t slots = (int64_t)d.T * d.K;
  using Most = std::conditional_t<FMT == MOE_W_BF16, Four, Eight>;
  if (eight_waves<FMT>(kHalf * wg_gate, d.H)) gate_shape(kNarrow, Most{});
  else if (narrow_tiles<FMT>(wg_gate, slots, d.E, d.H)) gate_shape(kNarrow, Four{});
  else gate_shape(std::false_type{}, Four{});
  if (fused && ((int64_t)d.T * d.K * d.I + d.sI) * d.H <= kSmallDown) {
    hipLaunchKernelGGL((decode_down_combine_kernel<FMT>),
                       dim3((unsigned)(d.H / (16 * FewDownShape<FMT>::NF))), dim3(16 * kWave), 0,
                       stream, d.T, d.H, d.I, d.r2, d.s2, d.sI, plan, a, s_a, d.out);
    return;
  }
  if (eight_waves<FMT>(kHalf * wg_down, std::max(d.I, d.sI))) down(kNarrow, Most{});
  else if (narrow_tiles<FMT>(wg_down, slots, d.E, d.I)) down(kNarrow, Four{});
  else down(std::false_type{}, Four{});
  hipLaunchKernelGGL(decode_combine_kernel, dim3((unsigned)((d.H + 255) / 256), (unsigned)d.T),
                     dim3(64), 0, stream, d.T, d.H, d.K, plan.row_of, d.topk_w, rows, s_rows, d.out);
}

int launch_route(const float*, const uint8_t*, int, int, int, int, int32_t*, float*, hipStream_t);

int launch_decode(const float* logits, const uint8_t* row_valid, const uint16_t* x, int T, int H,
                  int I, int E, int K, int expert_begin, int El, int renorm, int32_t* topk_idx,
                  float* topk_w, const moe_ffn_weights* routed, const moe_ffn_weights* shared,
                  int sI, uint16_t* out, void* workspace, int32_t* dev_error, hipStream_t stream) {
  DecodeArgs d{logits, row_valid, x, T, H, I, E, K, expert_begin, El, renorm, sI, topk_idx, topk_w,
               {routed->w13, routed->w13_scales, routed->w13_tensor_scale},
               {routed->w2, routed->w2_scales, routed->w2_tensor_scale}, {}, {}, out,
               decode_layout(T, H, I, K, El, sI), static_cast<char*>(workspace)};
  if (shared) {
    d.s13 = WMat{shared->w13, shared->w13_scales, shared->w13_tensor_scale};
    d.s2 = WMat{shared->w2, shared->w2_scales, shared->w2_tensor_scale};
  }
  const int64_t most = d.L.max_entries + (T + kCols - 1) / kCols;
  if (most * std::max(std::max(I, sI) / 16, H / 32) >= kMaxGrid) return MOE_ERR_UNSUPPORTED;
  const bool fused = logits && T <= kFusedTokens && T * K <= 64 && E <= 256;
#define MOE_PLAN(N)                                                                             \
  hipLaunchKernelGGL(plan_kernel<N>, dim3(1), dim3(kPlanThreads), 0, stream, logits, row_valid, T, \
                     E, K, renorm, expert_begin, El, topk_idx, topk_w, plan_of(d), dev_error)
#define MOE_ROUTE_FEW(N)                                                                       \
  hipLaunchKernelGGL(route_few_kernel<N>, dim3((unsigned)T), dim3(kWave), 0, stream, logits,    \
                     row_valid, E, K, renorm, topk_idx, topk_w)
  if (!fused) {
    // one workgroup routes as it plans while it has a wave per token, or 16
    // lanes (at 64 tokens, top-8: 64 experts 5 us; 256 experts 16 us, in two
    // launches 8 us)
    const bool in_plan = logits && (T <= kPlanThreads / kWave ? E <= 256 : E <= 64 && K <= 16 && renorm);
    if (!logits) MOE_PLAN(0);
    else if (in_plan && E <= 64) MOE_PLAN(1);
    else if (in_plan) MOE_PLAN(4);
    else {
      if (E <= 64) MOE_ROUTE_FEW(1);
      else if (E <= 256) MOE_ROUTE_FEW(4);
      else {
        const int st = launch_route(logits, row_valid, T, E, K, renorm, topk_idx, topk_w, stream);
        if (st != MOE_OK) return st;
      }
      MOE_PLAN(0);
    }
  }
#undef MOE_PLAN
#undef MOE_ROUTE_FEW
  switch (routed->format) {
    case MOE_W_BF16: launch_decode_ffn<MOE_W_BF16>(d, fused, stream); break;
    case MOE_W_FP8: launch_decode_ffn<MOE_W_FP8>(d, fused, stream); break;
    case MOE_W_MXFP4: launch_decode_ffn<MOE_W_MXFP4>(d, fused, stream); break;
    default: launch_decode_ffn<MOE_W_NVFP4>(d, fused, stream);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// ---- the grouped FFN on 4-bit weights, few rows ---------------------------------
// Entry j of the segments: the j-th run of at most 16 rows, over the groups in
// order; a run's place follows from a scan of the counts by every wave (its
// answer the same in every lane).  A segment that leaves [0, capacity) has no
// runs and raises ROW_RANGE.  333 ragged rows of 64 experts (H = 2048, I = 1024),
// NVFP4, take 28 + 19 us, bound by the conversion (the vector units busy 83 and
// 71 % of the time), 59 runs of 51 experts reading 135 MB past the L2 for
// gate/up's 120; one row of one expert, MXFP4, 6 + 5, the launches.  Returns
// false past the last run; `total` is the number of runs then.
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
__global__ void __launch_bounds__(NW * kWave, FewShape<FMT>::kWaves) few_gate_up_kernel(
    const uint16_t* __restrict__ x, const int32_t* __restrict__ cu_seqlens,
    const int32_t* __restrict__ counts, int G, int H, int I, WMat W, int64_t capacity,
    uint16_t* __restrict__ a, int32_t* __restrict__ dev_error) {
  __shared__ f32x4_t red[NW][FewShape<FMT>::NF][kWave];
  const int nt = I / (8 * FewShape<FMT>::NF), j = blockIdx.x / nt;
  RowRun r;
  long long total;
  if (!find_run(j, cu_seqlens, counts, G, capacity, dev_error, r, total)) return;
  const int col = threadIdx.x & 15;
  few_gate_up<FMT, NW, FewShape<FMT>>(W, r.g, blockIdx.x - j * nt, H, I,
                       uniform_buffer(x + (int64_t)r.row0 * H, (int64_t)r.cnt * H * 2),
                       (uint32_t)min(col, r.cnt - 1) * H * 2u, r.cnt,
                       a + (int64_t)r.row0 * 2 * I, red);
}

template <int FMT, int NW>
__global__ void __launch_bounds__(NW * kWave, FewShape<FMT>::kWaves) few_down_kernel(
    const uint16_t* __restrict__ a, const int32_t* __restrict__ cu_seqlens,
    const int32_t* __restrict__ counts, int G, int H, int I, WMat W,
    const float* __restrict__ row_scale, uint16_t* __restrict__ y,
    int64_t capacity, int64_t max_runs, int32_t* __restrict__ dev_error) {
  __shared__ f32x4_t red[NW][FewShape<FMT>::NF][kWave];
  const int nt = H / (16 * FewShape<FMT>::NF), j = blockIdx.x / nt;
  RowRun r;
  long long total;
  if (blockIdx.x == 0 && threadIdx.x < kWave) {
    // overlapping segments can hold more runs than the grid: said, not dropped silently
    if ((find_run(0x7fffffff, cu_seqlens, counts, G, capacity, dev_error, r, total) ||
         total > max_runs) && threadIdx.x == 0)
      raise_error(dev_error, MOE_DEVERR_ROW_RANGE);
  }
  if (!find_run(j, cu_seqlens, counts, G, capacity, dev_error, r, total)) return;
  few_down<FMT, NW, FewShape<FMT>>(W, r.g, blockIdx.x - j * nt, H, I, a + (int64_t)r.row0 * 2 * I, r.cnt,
                    red, [&](int c, int i, f32x4_t v) {
                      const int64_t row = r.row0 + i;
                      const float sc = row_scale ? row_scale[row] : 1.0f;
                      *reinterpret_cast<uint2*>(y + row * H + c) =
                          make_uint2(f32_to_bf16(sc * v[0]) | f32_to_bf16(sc * v[1]) << 16,
                                     f32_to_bf16(sc * v[2]) | f32_to_bf16(sc * v[3]) << 16);
                    });
}

// Runs that disjoint segments of `capacity` rows over G groups can hold.
static int64_t max_row_runs(int64_t capacity, int G) {
  return std::min<int64_t>(G, capacity) + capacity / kCols;
}

template <int FMT>
static int launch_few_fmt(const uint16_t* x, const int32_t* cu, const int32_t* counts, int G,
                          int H, int I, const WMat& w13, const WMat& w2, const float* row_scale,
                          uint16_t* y, int64_t capacity, int flags, uint16_t* a,
                          int32_t* dev_error, hipStream_t stream) {
  const int64_t runs = max_row_runs(capacity, G);
  const int64_t gu = runs * (I / (8 * FewShape<FMT>::NF)), dn = runs * (H / (16 * FewShape<FMT>::NF));
  if (gu >= kMaxGrid || dn >= kMaxGrid) return MOE_ERR_UNSUPPORTED;
  auto gate = [&](auto nw) {
    constexpr int NW = decltype(nw)::value;
    hipLaunchKernelGGL((few_gate_up_kernel<FMT, NW>), dim3((unsigned)gu), dim3(NW * kWave), 0,
                       stream, x, cu, counts, G, H, I, w13, capacity, a, dev_error);
  };
  auto down = [&](auto nw) {
    constexpr int NW = decltype(nw)::value;
    hipLaunchKernelGGL((few_down_kernel<FMT, NW>), dim3((unsigned)dn), dim3(NW * kWave), 0, stream,
                       a, cu, counts, G, H, I, w2, row_scale, y, capacity, runs, dev_error);
  };
  if (flags & MOE_FFN_GATE_UP) {
    if (eight_waves<FMT>(gu, H)) gate(Eight{});
    else gate(Four{});
  }
  if (flags & MOE_FFN_DOWN) {
    if (eight_waves<FMT>(dn, I)) down(Eight{});
    else down(Four{});
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// The intermediate: capacity rows of I high and I low parts.
size_t few_ffn_workspace_bytes(int64_t capacity, int I) {
  return align256((size_t)capacity * I * 4);
}

int launch_few_ffn(const uint16_t* x, const int32_t* cu, const int32_t* counts, int G, int H,
                   int I, const moe_ffn_weights* wt, const float* row_scale, uint16_t* y,
                   int64_t capacity, int flags, void* workspace, int32_t* dev_error,
                   hipStream_t stream) {
  uint16_t* a = static_cast<uint16_t*>(workspace);
  const WMat w13{wt->w13, wt->w13_scales, wt->w13_tensor_scale};
  const WMat w2{wt->w2, wt->w2_scales, wt->w2_tensor_scale};
  if (wt->format == MOE_W_MXFP4)
    return launch_few_fmt<MOE_W_MXFP4>(x, cu, counts, G, H, I, w13, w2, row_scale, y, capacity,
                                       flags, a, dev_error, stream);
  return launch_few_fmt<MOE_W_NVFP4>(x, cu, counts, G, H, I, w13, w2, row_scale, y, capacity,
                                     flags, a, dev_error, stream);
}

}  // namespace moe
