// merge_prefill.cu -- join the partial results of a context split across CTAs by the chunk
// attention: with M the largest reference of a row's records,
//   out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j,   lse = ln 2 (M + log2 sum ..).
// One warp per (token, head); records are taken in order, so the result does not depend on
// timing.  Bound by reading the records once, which the attention before it leaves in L2: 24 x 3 to 8
// tokens, 32 heads of 128, 3 splits (6 MB): 7.6 us by itself with cold caches, most of it the chain
// row -> sequence -> records; its launch alone runs under the attention's end.
#include <cuda_runtime.h>

#include <type_traits>

#include "mma_ops.cuh"
#include "pkv_device.cuh"
#include "prompt.cuh"

namespace pkv {

template <int D, bool FP8>
__global__ void __launch_bounds__(256) merge_prefill_kernel(const PrefillParams p) {
  constexpr int DPL = D / 32;
  using VecT = typename std::conditional<DPL == 4, float4, float2>::type;
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + warp;  // token * hq + head
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.hq;
  if (row >= rows) return;
  const int tok = static_cast<int>(row / p.hq), head = static_cast<int>(row - static_cast<int64_t>(tok) * p.hq);
  // the row's sequence: the last that starts at or before it.  A row of none, behind the last one or of
  // a bad range (which the attention skipped), is left as it was
  int b = 0, e = p.batch;
  while (e - b > 1) {
    const int mid = (b + e) >> 1;
    if (p.q_indptr[mid] <= tok) b = mid;
    else e = mid;
  }
  const int first = p.q_indptr[b], last = p.q_indptr[b + 1];
  bool written = tok >= first && tok < last && first >= 0 && last <= p.total_q;
  if (!written) {
    // offsets out of order (a bad range) lead the search astray: the warp looks through all ranges
    bool mine = false;
#pragma unroll 4
    for (int i = lane; i < p.batch; i += 32) {
      const int from = p.q_indptr[i], to = p.q_indptr[i + 1];
      mine |= from >= 0 && tok >= from && tok < to && to <= p.total_q;
    }
    written = __any_sync(kFull, mine);
  }
  if (!written) return;

  float M = -INFINITY;
  for (int j = lane; j < p.splits; j += 32) M = fmaxf(M, p.part_ml[j * rows + row].x);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) M = fmaxf(M, shfl_xor(M, m));
  float den = 0.f;
  float num[DPL];
#pragma unroll
  for (int i = 0; i < DPL; ++i) num[i] = 0.f;
#pragma unroll 4
  for (int j = 0; j < p.splits; ++j) {
    const float2 ml = p.part_ml[j * rows + row];
    if (ml.y == 0.f) continue;  // an empty record has no output part
    // (a record whose first scores held a NaN has reference -inf and a sum that is NaN)
    const float wgt = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
    const VecT v = __ldcs(reinterpret_cast<const VecT*>(p.part_acc + (j * rows + row) * D) + lane);
    den = fmaf(wgt, ml.y, den);
    num[0] = fmaf(wgt, v.x, num[0]);
    num[1] = fmaf(wgt, v.y, num[1]);
    if constexpr (DPL == 4) {
      num[2] = fmaf(wgt, v.z, num[2]);
      num[3] = fmaf(wgt, v.w, num[3]);
    }
  }
  float inv = 0.f;  // of a row without keys
  if (den > 0.f || den != den) {
    inv = 1.f / den;
    if constexpr (FP8) inv *= p.scales[p.hkv + head / p.group];
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * D + lane * DPL);
  if constexpr (DPL == 4)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16(num[0] * inv, num[1] * inv), pack_bf16(num[2] * inv, num[3] * inv));
  else
    *dst = pack_bf16(num[0] * inv, num[1] * inv);
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = den == 0.f ? -INFINITY
                            : (M - (FP8 ? kPrefillWeightBias : 0.f) + log2f(den)) * 0.69314718055994531f;
}

cudaError_t launch_merge_prefill(int d, const PrefillParams& p, bool fp8, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.hq;
  const int64_t ctas = (rows + 7) / 8;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (d == 64)
    return fp8 ? cudaLaunchKernelEx(&cfg, merge_prefill_kernel<64, true>, p)
               : cudaLaunchKernelEx(&cfg, merge_prefill_kernel<64, false>, p);
  return fp8 ? cudaLaunchKernelEx(&cfg, merge_prefill_kernel<128, true>, p)
             : cudaLaunchKernelEx(&cfg, merge_prefill_kernel<128, false>, p);
}

}  // namespace pkv
