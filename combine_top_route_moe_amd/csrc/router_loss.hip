// The router's losses and its gradient.
//
// Over the n tokens that are real, p_t = softmax(logits_t):
//   counts_e = slots that name expert e,   f_e = counts_e / (n K),
//   P_e = sum_t p_te / n,   balance = E sum_e f_e P_e,   z = sum_t lse_t^2 / n
// and with the upstream gradients d0 of balance, d1 of z and dw_tk of the
// routing weights w_tk,
//   d logit_te = d0/n p_te (b_e - sum_j p_tj b_j) + 2 d1/n lse_t p_te
//              + sum_{k: id_tk = e} w_tk dw_tk - (w_tk | p_te) sum_k w_tk dw_tk,
// b_e = E f_e - 1: the 1 leaves the difference as it is (the p_t sum to one) and
// takes away what would cancel in it.  The last factor is w_tk where the
// weights were renormalised over the chosen experts, p_te (for every expert)
// where they were not.
//
// One wave per token, expert lane + 64 j in register j: a token's logits are
// read once, maximum, sum and products stay in registers.  Bound on few tokens by the
// launch, else by a token's own chain of reductions and by vector instructions: 16384
// tokens of 128 experts take 6.8 + 5.6 us for the losses (vector units 51 % busy, waves
// waiting 64 % of their time; then one workgroup's join) and 10.4 for the gradient (76 %
// busy); their bytes alone would take 1.3 and 3.2.  Counts are
// integers and every float sum has a fixed order, so equal calls give equal bits.
#include <algorithm>

#include "reduce.h"

namespace moe {

constexpr int kLossWaves = 16;          // waves of a loss workgroup
constexpr int kLossMaxGroups = 256;     // workgroups of the first launch at most,
constexpr int kLossMaxShares = 32768;   // and their shares of experts: one workgroup joins them

// exp, log and reciprocal in float32 by the hardware's own: exp(x) = 2^(x log2 e) to
// (1.23 |x| + 2) 2^-24 relative: the product's rounding |x|, that of log2 e 0.224 |x|, the
// hardware's step 2 (and what the rounding of x = l - l_max has left).  A token costs
// some 40 instructions less than with the library's.  With the product's residual put
// back the kernels take 1 to 5 % longer, and the losses are no closer to 64 bits.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ float fast_log(float x) { return __builtin_amdgcn_logf(x) * 0.693147181f; }

// A token's probabilities from its logits (v: -inf where there is no expert);
// returns logsumexp.  As in the routing, a NaN counts as -inf and a logit equal
// to the largest counts exp(0) even where both are infinite.
template <int EPL>
__device__ __forceinline__ float softmax(float (&v)[EPL], int E, int lane) {
  float top = v[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) top = fmaxf(top, v[j]);
  top = wave_top_f32(top);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    v[j] = lane + 64 * j >= E ? 0.0f : v[j] == top ? 1.0f : fast_exp(v[j] - top);
    sum += v[j];
  }
  sum = wave_sum_f32(sum);
  const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
  for (int j = 0; j < EPL; ++j) v[j] *= inv;
  return top + fast_log(sum);
}

template <int EPL>
__device__ __forceinline__ void load_logits(const float* __restrict__ row, int E, int lane, float (&v)[EPL]) {
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 64 * j;
    const float x = e < E ? row[e] : -__builtin_inff();
    v[j] = x != x ? -__builtin_inff() : x;
  }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// Tokens that a wave loads before it works on the first.
template <int EPL>
constexpr int kTokensAhead = EPL <= 2 ? 4 : EPL <= 8 ? 2 : 1;

// Shares of one workgroup, in the workspace: [groups] float64 of sum lse^2, then
// [groups] x {E floats of sum p, E int32 counts}, then [groups] int32 of n.
struct LossShares {
  double* z;
  float* probs;
  int32_t* counts;
  int32_t* tokens;
};
__device__ __forceinline__ LossShares loss_shares(void* ws, int groups, int E) {
  LossShares s;
  s.z = static_cast<double*>(ws);
  s.probs = reinterpret_cast<float*>(s.z + groups);
  s.counts = reinterpret_cast<int32_t*>(s.probs + (size_t)groups * E);
  s.tokens = s.counts + (size_t)groups * E;
  return s;
}

struct LossOut {
  float* loss;
  int32_t* counts;
  float* probs;
  int32_t* tokens;
};

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// dot = sum_e (sum p)_e counts_e
__device__ __forceinline__ void write_losses(const LossOut& out, double dot, double z, int n, int E, int K) {
  const double inv = n > 0 ? 1.0 / n : 0.0;
  out.loss[0] = (float)(dot * inv * inv * E / K);
  out.loss[1] = (float)(z * inv);
  out.tokens[0] = n;
}

// ONE: the only workgroup, which writes the outputs; else it leaves its share.
template <int EPL, bool ONE>
__global__ void __launch_bounds__(kLossWaves * kWave) balance_share_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ row_valid,
    const int32_t* __restrict__ topk_idx, int T, int E, int K, void* ws, LossOut out,
    int32_t* __restrict__ dev_error) {
  __shared__ float meet[kLossWaves / 2][EPL * kWave];
  __shared__ int32_t hist[EPL * kWave];
  __shared__ double zs[kLossWaves];
  __shared__ int32_t ns[kLossWaves];
  constexpr int kTok = kTokensAhead<EPL>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < EPL * kWave; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  float acc[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) acc[j] = 0.0f;
  double z = 0.0;
  int n = 0;
  // wave w of all takes tokens w, w + waves, ..
  const int64_t waves = (int64_t)gridDim.x * kLossWaves;
  for (int64_t t0 = (int64_t)blockIdx.x * kLossWaves + wave; t0 < T; t0 += waves * kTok) {
    float v[kTok][EPL];
    int id[kTok];
    bool real[kTok];
#pragma unroll
    for (int u = 0; u < kTok; ++u) {
      const int64_t t = min(t0 + u * waves, (int64_t)T - 1);
      real[u] = t0 + u * waves < T && (!row_valid || row_valid[t]);
      load_logits<EPL>(logits + t * E, E, lane, v[u]);
      id[u] = real[u] && lane < K ? topk_idx[t * K + lane] : -1;
    }
    // (no branch on what is real: the tokens' chains of operations run side by side)
#pragma unroll
    for (int u = 0; u < kTok; ++u) {
      const float lse = softmax<EPL>(v[u], E, lane);
      n += real[u];
      z += real[u] && finite(lse) ? (double)lse * lse : 0.0;
#pragma unroll
      for (int j = 0; j < EPL; ++j) acc[j] += real[u] ? v[u][j] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kTok; ++u) {
      if (id[u] >= E) raise_error(dev_error, MOE_DEVERR_EXPERT_RANGE);
      else if (id[u] >= 0) atomicAdd(&hist[id[u]], 1);
    }
  }
  if (lane == 0) zs[wave] = z, ns[wave] = n;
  // the waves' sums meet in halves: 8 + 8, 4 + 4, ..
#pragma unroll
  for (int half = kLossWaves / 2; half > 0; half /= 2) {
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int j = 0; j < EPL; ++j) meet[wave - half][lane + 64 * j] = acc[j];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int j = 0; j < EPL; ++j) acc[j] += meet[wave][lane + 64 * j];
    __syncthreads();
  }
  if (wave > 0) return;
  for (int i = 1; i < kLossWaves; ++i) z += zs[i], n += ns[i];
  const LossShares s = loss_shares(ws, gridDim.x, E);
  double dot = 0.0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 64 * j;
    if (e >= E) break;
    if (ONE) {
      out.counts[e] = hist[e];
      out.probs[e] = n > 0 ? acc[j] / (float)n : 0.0f;
      dot += (double)acc[j] * hist[e];
    } else {
      s.counts[(size_t)blockIdx.x * E + e] = hist[e];
      s.probs[(size_t)blockIdx.x * E + e] = acc[j];
    }
  }
  if (ONE) dot = wave_sum_f64(dot);
  if (lane > 0) return;
  if (ONE) {
    write_losses(out, dot, z, n, E, K);
  } else {
    s.z[blockIdx.x] = z;
    s.tokens[blockIdx.x] = n;
  }
}

// The shares' sums, by one workgroup: 1024 / kE threads an expert (kE the power of
// two above E), each every so many shares, their sums in order.
__global__ void __launch_bounds__(1024) balance_join_kernel(void* ws, int groups, int E, int log_kE, int K,
                                                            LossOut out) {
  __shared__ double ps[1024];
  __shared__ int32_t cs[1024];
  __shared__ double zs[16];
  __shared__ int32_t n_all;
  const LossShares s = loss_shares(ws, groups, E);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int kE = 1 << log_kE, e = tid & (kE - 1), slice = tid >> log_kE, slices = 1024 >> log_kE;
  double p = 0.0;
  int c = 0;
  if (e < E) {
#pragma unroll 8
    for (int g = slice; g < groups; g += slices) p += s.probs[(size_t)g * E + e], c += s.counts[(size_t)g * E + e];
  }
  ps[tid] = p;
  cs[tid] = c;
  double z = 0.0;
  if (wave == 0) {
    int n = 0;
    for (int g = lane; g < groups; g += kWave) z += s.z[g], n += s.tokens[g];
    z = wave_sum_f64(z);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off, kWave);
    if (lane == 0) n_all = n;
  }
  __syncthreads();
  const int n = n_all;
  double dot = 0.0;
  if (slice == 0 && e < E) {
    for (int i = 1; i < slices; ++i) p += ps[i * kE + e], c += cs[i * kE + e];
    out.counts[e] = c;
    out.probs[e] = n > 0 ? (float)(p / n) : 0.0f;
    dot = p * c;
  }
  dot = wave_sum_f64(dot);
  if (lane == 0) zs[wave] = dot;
  __syncthreads();
  if (tid > 0) return;
  for (int i = 1; i < 16; ++i) dot += zs[i];
  write_losses(out, dot, z, n, E, K);
}

// Few tokens in one launch: the second costs more than the longer walk.
static int loss_groups(int T, int E) {
  if (T <= MOE_LOSS_FEW_TOKENS) return T > 0;
  return std::min({(T - 1) / kLossWaves + 1, kLossMaxGroups, std::max(32, kLossMaxShares / E)});
}

size_t balance_loss_workspace_bytes(int T, int E) {
  const int groups = loss_groups(T, E);
  return groups > 1 ? (size_t)groups * (8 + 8 * (size_t)E + 4) : 0;
}

int launch_balance_loss(const float* logits, const uint8_t* row_valid, const int32_t* topk_idx, int T,
                        int E, int K, float* loss, int32_t* counts, float* probs, int32_t* tokens,
                        void* ws, int32_t* dev_error, hipStream_t stream) {
  const int groups = std::max(1, loss_groups(T, E)), epl = (E + kWave - 1) / kWave;
  const LossOut out = {loss, counts, probs, tokens};
#define MOE_LOSS(N)                                                                                       \
  if (groups == 1)                                                                                        \
    hipLaunchKernelGGL((balance_share_kernel<N, true>), dim3(1), dim3(kLossWaves * kWave), 0, stream,     \
                       logits, row_valid, topk_idx, T, E, K, ws, out, dev_error);                         \
  else                                                                                                    \
    hipLaunchKernelGGL((balance_share_kernel<N, false>), dim3(groups), dim3(kLossWaves * kWave), 0, stream, \
                       logits, row_valid, topk_idx, T, E, K, ws, out, dev_error)
  if (epl <= 1) {
    MOE_LOSS(1);
  } else if (epl <= 2) {
    MOE_LOSS(2);
  } else if (epl <= 4) {
    MOE_LOSS(4);
  } else if (epl <= 8) {
    MOE_LOSS(8);
  } else {
    MOE_LOSS(16);
  }
#undef MOE_LOSS
  if (groups > 1) {
    int log_kE = 0;
    while (1 << log_kE < E) ++log_kE;
    hipLaunchKernelGGL(balance_join_kernel, dim3(1), dim3(1024), 0, stream, ws, groups, E, log_kE, K, out);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// RENORM: the weights were renormalised over the chosen experts.  The logits are
// read where a softmax over all experts is needed: for the losses, or for
// weights that are such probabilities.
template <int EPL, bool RENORM>
__global__ void __launch_bounds__(256) route_backward_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ row_valid,
    const int32_t* __restrict__ topk_idx, const float* __restrict__ topk_w,
    const float* __restrict__ d_topk_w, int T, int E, int K, const float* __restrict__ d_loss,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ num_tokens,
    float* __restrict__ d_logits, int32_t* __restrict__ dev_error) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float b[EPL], d0 = 0.0f, d1 = 0.0f;
  if (d_loss) {
    const int n = max(num_tokens[0], 1);
    const float slots = (float)E / ((float)n * (float)K);
    d0 = d_loss[0] / (float)n;
    d1 = 2.0f * d_loss[1] / (float)n;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 64 * j;
      b[j] = e < E ? __builtin_fmaf((float)counts[e], slots, -1.0f) : 0.0f;
    }
  }
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < T; t += (int64_t)gridDim.x * 4) {
    float* out = d_logits + t * E;
    if (row_valid && !row_valid[t]) {
      for (int e = lane; e < E; e += kWave) out[e] = 0.0f;
      continue;
    }
    // lane k < K: slot k's expert (-1: none), weight and weight's gradient
    int id = -1;
    float w = 0.0f, wd = 0.0f, dot = 0.0f;
    if (d_topk_w) {
      if (lane < K) {
        id = topk_idx[t * K + lane];
        if (id >= E) raise_error(dev_error, MOE_DEVERR_EXPERT_RANGE);
        if (id >= E || id < 0) id = -1;
        else w = topk_w[t * K + lane], wd = w * d_topk_w[t * K + lane];
      }
      dot = wave_sum_f32(wd);
      if (RENORM) wd -= w * dot;
    }
    float g[EPL];
    if (d_loss || (!RENORM && d_topk_w)) {
      load_logits<EPL>(logits + t * E, E, lane, g);
      const float lse = softmax<EPL>(g, E, lane);
      const bool ok = d_loss && finite(lse);
      float mean = 0.0f;
      if (ok) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) mean = __builtin_fmaf(g[j], b[j], mean);
        mean = wave_sum_f32(mean);
      }
      const float all = (ok ? d1 * lse : 0.0f) - (RENORM ? 0.0f : dot);
#pragma unroll
      for (int j = 0; j < EPL; ++j) g[j] *= ok ? __builtin_fmaf(d0, b[j] - mean, all) : all;
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) g[j] = 0.0f;
    }
    if (d_topk_w) {
      for (int k = 0; k < K; ++k) {
        const int e = __builtin_amdgcn_readlane(id, k);
        const float add = lane_f32(wd, k);
        if ((e & 63) == lane && e >= 0) {
#pragma unroll
          for (int j = 0; j < EPL; ++j)
            if (e >> 6 == j) g[j] += add;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane + 64 * j < E) out[lane + 64 * j] = g[j];
  }
}

int launch_route_backward(const float* logits, const uint8_t* row_valid, const int32_t* topk_idx,
                          const float* topk_w, const float* d_topk_w, int T, int E, int K, int renorm,
                          const float* d_loss, const int32_t* counts, const int32_t* num_tokens,
                          float* d_logits, int32_t* dev_error, hipStream_t stream) {
  const int epl = (E + kWave - 1) / kWave;
  const int blocks = (int)((T + 3LL) / 4 < 2048 ? (T + 3LL) / 4 : 2048);
#define MOE_RB(N)                                                                                   \
  if (epl <= N) {                                                                                   \
    if (renorm)                                                                                     \
      hipLaunchKernelGGL((route_backward_kernel<N, true>), dim3(blocks), dim3(256), 0, stream, logits, \
                         row_valid, topk_idx, topk_w, d_topk_w, T, E, K, d_loss, counts, num_tokens, \
                         d_logits, dev_error);                                                      \
    else                                                                                            \
      hipLaunchKernelGGL((route_backward_kernel<N, false>), dim3(blocks), dim3(256), 0, stream, logits, \
                         row_valid, topk_idx, topk_w, d_topk_w, T, E, K, d_loss, counts, num_tokens, \
                         d_logits, dev_error);                                                      \
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;                                  \
  }
  MOE_RB(1)
  MOE_RB(2)
  MOE_RB(4)
  MOE_RB(8)
  MOE_RB(16)
#undef MOE_RB
  return MOE_ERR_UNSUPPORTED;
}

}  // namespace moe
