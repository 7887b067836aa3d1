// diff_out.cuh -- the end of a row of differential attention: what a warp does with the pair's two maps.
#pragma once

#include "diff.cuh"
#include "mma_ops.cuh"
#include "pkv_device.cuh"

namespace pkv {

// Four consecutive columns a lane of one output row, y0 and y1 the two maps' outputs (normalised, V's scale
// included): difference, norm over the warp's 128 columns, scale, store.  none: the row saw no key.
__device__ __forceinline__ void diff_store(const DiffParams& p, int row, int head, bool none, const float (&y0)[4],
                                           const float (&y1)[4], int lane) {
  const float lam = p.lambda[row * p.lambda_stride + head];
  float y[4], square = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = none ? 0.f : y0[i] - lam * y1[i];
    square = fmaf(y[i], y[i], square);
  }
  float by = p.out_scale;
  if (p.norm_weight != nullptr) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) square += shfl_xor(square, m);
    if (!none) by *= rsqrtf(square * (1.f / kDiffW) + p.eps);  // (eps may be 0: an empty row stays 0)
    const uint2 w = *reinterpret_cast<const uint2*>(p.norm_weight + 4 * lane);
    y[0] *= bf16_lo(w.x);
    y[1] *= bf16_hi(w.x);
    y[2] *= bf16_lo(w.y);
    y[3] *= bf16_hi(w.y);
  }
  const int64_t at = (static_cast<int64_t>(row) * p.heads + head) * kDiffW + 4 * lane;
  if (p.out_fp32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(y[0] * by, y[1] * by, y[2] * by, y[3] * by);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
        make_uint2(pack_bf16(y[0] * by, y[1] * by), pack_bf16(y[2] * by, y[3] * by));
}

}  // namespace pkv
