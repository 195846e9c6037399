// Expert weights that exist as codes and scales already (a checkpoint in FP8,
// MXFP4 or NVFP4) into the order the kernels stream: bytes are moved, none is
// decoded or changed, so the products read exactly the stored values.
// Quantizing the dequantized weights again would not do: an FP8 tile whose
// scale is another float32 than amax / 448 rounds to other codes, and so does an
// NVFP4 block whose largest code is not 6.
//
// One wave per fragment (16 weight rows x 128 columns); lane l moves row l % 16,
// columns 32 p + 8 (l / 16) .. +8 for p = 0..3.  Reads are 4 or 8 bytes a lane,
// writes whole lines; at load time once, bound by the memory.
#include <algorithm>

#include "weight_block.h"

namespace moe {

template <int FMT>
__global__ void __launch_bounds__(256) pack_codes_kernel(
    const uint8_t* __restrict__ W, const uint8_t* __restrict__ Sin, uint8_t* __restrict__ Q,
    uint8_t* __restrict__ Sout, int64_t n_frag, int N, int Kdim, int gate_up) {
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
  const int64_t row = g * N + row0 + (lane & 15);
  const int col = kb * 128 + 8 * (lane >> 4);
  if constexpr (FMT == MOE_W_FP8) {
    // the tile scales have one order in both forms and stay where they are
    u32x2_t* out = reinterpret_cast<u32x2_t*>(Q);
#pragma unroll
    for (int p = 0; p < 4; ++p)
      out[((g * (Kdim / 32) + 4 * kb + p) * n_ct + ct) * 256 + f * 64 + lane] =
          *reinterpret_cast<const u32x2_t*>(W + row * Kdim + col + 32 * p);
  } else {
    u32x4_t c;
#pragma unroll
    for (int p = 0; p < 4; ++p)
      c[p] = *reinterpret_cast<const uint32_t*>(W + (row * Kdim + col + 32 * p) / 2);
    reinterpret_cast<u32x4_t*>(Q)[frag * 64 + lane] = c;
    uint32_t* out = reinterpret_cast<uint32_t*>(Sout);
    if constexpr (FMT == MOE_W_MXFP4) {
      if (lane < 16)
        out[(t * 16 + lane) * 4 + f] =
            *reinterpret_cast<const uint32_t*>(Sin + row * (Kdim / 32) + 4 * kb);
    } else if (lane < 32) {
      // half h = lane / 16 takes every second of the row's 8 scales of the block
      const int h = lane >> 4;
      const u32x2_t s = *reinterpret_cast<const u32x2_t*>(Sin + row * (Kdim / 16) + 8 * kb);
      uint32_t b = 0u;
#pragma unroll
      for (int p = 0; p < 4; ++p) b |= (s[p >> 1] >> (16 * (p & 1) + 8 * h) & 0xffu) << (8 * p);
      out[((t * 2 + h) * 16 + (lane & 15)) * 4 + f] = b;
    }
  }
}

int launch_pack_codes(const moe_ffn_weights* rows, int G, int H, int I, uint8_t* w13q,
                      uint8_t* w13s, uint8_t* w2q, uint8_t* w2s, hipStream_t stream) {
  auto* kern = rows->format == MOE_W_FP8     ? pack_codes_kernel<MOE_W_FP8>
               : rows->format == MOE_W_MXFP4 ? pack_codes_kernel<MOE_W_MXFP4>
                                             : pack_codes_kernel<MOE_W_NVFP4>;
  const int64_t frag13 = rows->w13 ? (int64_t)G * (I / 8) * (H / 128) : 0;
  const int64_t frag2 = rows->w2 ? (int64_t)G * (H / 16) * (I / 128) : 0;
  // both are checked before either starts
  if (std::max(frag13, frag2) / 4 >= kMaxGrid) return MOE_ERR_UNSUPPORTED;
  auto one = [&](const void* w, const void* s, uint8_t* q, uint8_t* sq, int64_t n_frag, int N,
                 int Kdim, int gate_up) {
    hipLaunchKernelGGL(kern, dim3((unsigned)((n_frag + 3) / 4)), dim3(256), 0, stream,
                       static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(s), q, sq,
                       n_frag, N, Kdim, gate_up);
  };
  if (rows->w13) one(rows->w13, rows->w13_scales, w13q, w13s, frag13, 2 * I, H, 1);
  if (rows->w2) one(rows->w2, rows->w2_scales, w2q, w2s, frag2, H, I, 0);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe
