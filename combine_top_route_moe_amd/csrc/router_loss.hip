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
// read once, maximum, sum and products stay in registers.  Memory bound on
// many tokens (4 E bytes read, in the gradient 4 E more written), launch bound
// on few.  Counts are integers and every float sum has a fixed order, so equal
// calls give equal bits.
#include "reduce.h"

namespace moe {

constexpr int kLossWaves = 16;          // waves of a loss workgroup
constexpr int kLossMaxGroups = 128;     // workgroups of the first launch at most

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
    v[j] = lane + 64 * j >= E ? 0.0f : v[j] == top ? 1.0f : expf(v[j] - top);
    sum += v[j];
  }
  sum = wave_sum_f32(sum);
  const float inv = 1.0f / sum;
#pragma unroll
  for (int j = 0; j < EPL; ++j) v[j] *= inv;
  return top + logf(sum);
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

// Shares of one workgroup, in the workspace: [groups] x {E floats of sum p, E
// int32 counts}, then [groups] float64 of sum lse^2, then [groups] int32 of n.
struct LossShares {
  float* probs;
  int32_t* counts;
  double* z;
  int32_t* tokens;
};
__host__ __device__ inline LossShares loss_shares(void* ws, int groups, int E) {
  LossShares s;
  s.z = static_cast<double*>(ws);
  s.probs = reinterpret_cast<float*>(s.z + groups);
  s.counts = reinterpret_cast<int32_t*>(s.probs + (size_t)groups * E);
  s.tokens = s.counts + (size_t)groups * E;
  return s;
}

// What the shares come to: the outputs, by one workgroup.
__device__ __forceinline__ void write_losses(const LossShares& s, int groups, int E, int K,
                                             float* __restrict__ loss, int32_t* __restrict__ counts,
                                             float* __restrict__ probs, int32_t* __restrict__ tokens,
                                             double* sums) {
  int n = 0;
  double z = 0.0;
  for (int g = 0; g < groups; ++g) n += s.tokens[g], z += s.z[g];
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double dot = 0.0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    double p = 0.0;
    int c = 0;
    for (int g = 0; g < groups; ++g) p += s.probs[(size_t)g * E + e], c += s.counts[(size_t)g * E + e];
    p *= inv;
    counts[e] = c;
    probs[e] = (float)p;
    dot += p * c;
  }
  sums[threadIdx.x] = dot;
  __syncthreads();
  for (int half = blockDim.x / 2; half > 0; half /= 2) {
    if ((int)threadIdx.x < half) sums[threadIdx.x] += sums[threadIdx.x + half];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    loss[0] = (float)(sums[0] * inv * E / K);
    loss[1] = (float)(z * inv);
    tokens[0] = n;
  }
}

template <int EPL>
__global__ void __launch_bounds__(kLossWaves * kWave) balance_share_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ row_valid,
    const int32_t* __restrict__ topk_idx, int T, int E, int K, void* ws, int32_t* __restrict__ dev_error) {
  __shared__ float meet[kLossWaves / 2][EPL * kWave];
  __shared__ int32_t hist[EPL * kWave];
  __shared__ double zs[kLossWaves];
  __shared__ int32_t ns[kLossWaves];
  const LossShares out = loss_shares(ws, gridDim.x, E);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < EPL * kWave; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  float acc[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) acc[j] = 0.0f;
  double z = 0.0;
  int n = 0;
  for (int64_t t = (int64_t)blockIdx.x * kLossWaves + wave; t < T; t += (int64_t)gridDim.x * kLossWaves) {
    if (row_valid && !row_valid[t]) continue;
    float v[EPL];
    load_logits<EPL>(logits + t * E, E, lane, v);
    if (lane < K) {
      const int id = topk_idx[t * K + lane];
      if (id >= E) raise_error(dev_error, MOE_DEVERR_EXPERT_RANGE);
      else if (id >= 0) atomicAdd(&hist[id], 1);
    }
    const float lse = softmax<EPL>(v, E, lane);
    ++n;
    if (finite(lse)) z += (double)lse * lse;
#pragma unroll
    for (int j = 0; j < EPL; ++j) acc[j] += v[j];
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
  if (wave == 0) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 64 * j;
      if (e < E) out.probs[(size_t)blockIdx.x * E + e] = acc[j], out.counts[(size_t)blockIdx.x * E + e] = hist[e];
    }
    if (lane == 0) {
      for (int i = 1; i < kLossWaves; ++i) z += zs[i], n += ns[i];
      out.z[blockIdx.x] = z;
      out.tokens[blockIdx.x] = n;
    }
  }
}

__global__ void __launch_bounds__(1024) balance_join_kernel(void* ws, int groups, int E, int K,
                                                            float* __restrict__ loss,
                                                            int32_t* __restrict__ counts,
                                                            float* __restrict__ probs,
                                                            int32_t* __restrict__ tokens) {
  __shared__ double sums[1024];
  write_losses(loss_shares(ws, groups, E), groups, E, K, loss, counts, probs, tokens, sums);
}

static int loss_groups(int T) {
  const int groups = (T + kLossWaves - 1) / kLossWaves;
  return groups < kLossMaxGroups ? groups : kLossMaxGroups;
}

size_t balance_loss_workspace_bytes(int T, int E) {
  return (size_t)loss_groups(T) * (8 + 8 * (size_t)E + 4);
}

int launch_balance_loss(const float* logits, const uint8_t* row_valid, const int32_t* topk_idx, int T,
                        int E, int K, float* loss, int32_t* counts, float* probs, int32_t* tokens,
                        void* ws, int32_t* dev_error, hipStream_t stream) {
  const int groups = loss_groups(T), epl = (E + kWave - 1) / kWave;
#define MOE_LOSS(N)                                                                              \
  hipLaunchKernelGGL(balance_share_kernel<N>, dim3(groups), dim3(kLossWaves * kWave), 0, stream, \
                     logits, row_valid, topk_idx, T, E, K, ws, dev_error)
  if (groups == 0) {
  } else if (epl <= 1) {
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
  hipLaunchKernelGGL(balance_join_kernel, dim3(1), dim3(1024), 0, stream, ws, groups, E, K, loss, counts,
                     probs, tokens);
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
