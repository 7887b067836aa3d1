// diff_merge.cu -- join the partial results of differential attention's split contexts and shared prefixes, and
// end the rows: with M the largest reference of a row's records under a map,
//   y_m = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j,  then the difference, the norm and the store.
// One to eight warps per (row, output head), which take runs of slots, both maps each; records in order within a
// warp, warps in order, so the result does not depend on timing.  Bound by reading the records once, which the
// kernels before it leave in L2: 256 rows of 32 heads, two or three records a map (20 MB): 10 us by itself with cold
// caches, its launch under the end of the kernel before; one row of 32 heads, 13 records: 4 us, the chain row -> length
// -> records -> norm.
#include <cuda_runtime.h>

#include "diff.cuh"
#include "diff_out.cuh"

namespace pkv {

template <bool FP8, int W>
__global__ void __launch_bounds__(256) diff_merge_kernel(const DiffParams p) {
  constexpr int kBatch = 4;  // slots whose records a warp has in flight
  __shared__ float4 nums[8][2][32];
  __shared__ float2 mls[8][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % W;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (8 / W) + warp / W, step = static_cast<int64_t>(p.rows) * p.heads;
  pdl_wait();
  pdl_launch_dependents();
  bool mine = unit < step;
  const int row = mine ? static_cast<int>(unit / p.heads) : 0;
  const int head = static_cast<int>(unit - static_cast<int64_t>(row) * p.heads);
  int lo = 0, hi = 0;  // slots with records
  if (mine && p.q_indptr != nullptr) {
    // the row's sequence: the last that starts at or before it.  A row of none, behind the last one or of a bad
    // range (which was skipped), is left as it was
    int b = 0, e = p.batch;
    while (e - b > 1) {
      const int mid = (b + e) >> 1;
      if (p.q_indptr[mid] <= row) b = mid;
      else e = mid;
    }
    int first = p.q_indptr[b], last = p.q_indptr[b + 1];
    mine = first >= 0 && row >= first && row < last && last <= p.rows;
    if (!mine)  // offsets out of order lead the search astray: the warp looks through all ranges
      for (int b0 = 0; b0 < p.batch && !mine; b0 += 32) {
        const int i = min(b0 + lane, p.batch - 1);
        first = p.q_indptr[i];
        last = p.q_indptr[i + 1];
        mine = __any_sync(kFull, first >= 0 && row >= first && row < last && last <= p.rows);
      }
    hi = p.max_splits;
  } else if (mine) {
    const int len = max(0, min(p.context_lens[row], p.max_context_len));
    const int nblk = (len + kBlockSize - 1) / kBlockSize, nsplit = (nblk + p.split_blocks - 1) / p.split_blocks;
    const bool with_prefix = p.pre_slots > 0 && p.seq_prefix[row] >= 0;
    mine = nsplit > 1 || with_prefix;  // else the decode kernel ended it
    lo = with_prefix ? 0 : p.pre_slots;
    hi = p.pre_slots + nsplit;
  }
  if (!mine) hi = lo;
  // this warp's slots
  const int each = (hi - lo + W - 1) / W, from = lo + part * each, to = min(hi, from + each);
  float top[2] = {-INFINITY, -INFINITY}, den[2] = {};
  float num[2][4] = {};
  for (int j0 = from; j0 < to; j0 += kBatch) {
    float2 ml[kBatch][2];
    float4 v[kBatch][2];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int64_t rec = static_cast<int64_t>((j0 + u) * 2 + m) * step + unit;
        ml[u][m] = j0 + u < to ? __ldcg(p.part_ml + rec) : make_float2(-INFINITY, 0.f);
        v[u][m] = j0 + u < to ? __ldcg(reinterpret_cast<const float4*>(p.part_acc + rec * kDiffW) + lane) : float4{};
      }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float n = fmaxf(top[m], ml[u][m].x);
        if (ml[u][m].y == 0.f) {  // no output part: a record of no keys, or of none but scores of -inf (kDiffNothing)
          top[m] = n;
          continue;
        }
        // (a record whose first scores held a NaN has reference -inf and a sum that is NaN)
        const float a = top[m] == -INFINITY ? 0.f : fast_exp2(top[m] - n);
        const float f = ml[u][m].x == -INFINITY ? 1.f : fast_exp2(ml[u][m].x - n);
        top[m] = n;
        den[m] = fmaf(f, ml[u][m].y, den[m] * a);
        num[m][0] = fmaf(f, v[u][m].x, num[m][0] * a);
        num[m][1] = fmaf(f, v[u][m].y, num[m][1] * a);
        num[m][2] = fmaf(f, v[u][m].z, num[m][2] * a);
        num[m][3] = fmaf(f, v[u][m].w, num[m][3] * a);
      }
  }
  bool no_keys = top[0] == -INFINITY;  // (both maps see the same keys)
  if constexpr (W > 1) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      nums[warp][m][lane] = make_float4(num[m][0], num[m][1], num[m][2], num[m][3]);
      if (lane == 0) mls[warp][m] = make_float2(top[m], den[m]);
    }
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, mls[warp + w][m].x);
      no_keys = M == -INFINITY;
      den[m] = num[m][0] = num[m][1] = num[m][2] = num[m][3] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 ml = mls[warp + w][m];
        const float f = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - M);  // (-inf: nothing, or a sum that is NaN)
        const float4 v = nums[warp + w][m][lane];
        den[m] = fmaf(f, ml.y, den[m]);
        num[m][0] = fmaf(f, v.x, num[m][0]);
        num[m][1] = fmaf(f, v.y, num[m][1]);
        num[m][2] = fmaf(f, v.z, num[m][2]);
        num[m][3] = fmaf(f, v.w, num[m][3]);
      }
    }
  }
  if (!mine) return;
  const float vs = FP8 ? p.scales[2 * (p.pairs + head / p.group) + lane / 16] : 1.f;
  const bool none = den[0] == 0.f && den[1] == 0.f && no_keys;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float by = vs / den[m];
#pragma unroll
    for (int i = 0; i < 4; ++i) num[m][i] *= by;
  }
  diff_store(p, row, head, none, num[0], num[1], lane);
}

template <bool FP8, int W>
static cudaError_t launch(const DiffParams& p, cudaStream_t stream) {
  const int64_t ctas = (static_cast<int64_t>(p.rows) * p.heads * W + 7) / 8;
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
  return cudaLaunchKernelEx(&cfg, diff_merge_kernel<FP8, W>, p);
}

// Warps per row and head: few where there are few records, or rows enough to fill the SMs; more shorten the chain of a
// lone row.  Whole calls with 1 / 4 / 8, us: 64 rows of 32 heads, 2 slots 97.0 / 99.9 / 103; 256, 2 slots 70.4 / 85 / 102;
// 134, 5 slots 136 / 142 / 152; 9 rows of 8 heads, 8 slots 13.5 / 12.3 / 12.3; one of 32, 63 slots 28.6 / 15.4 / 13.9; one
// of 64, 170 slots 148 / 111 / 104.
cudaError_t launch_diff_merge(bool fp8, const DiffParams& p, cudaStream_t stream) {
  const int slots = p.pre_slots + p.max_splits;
  const bool many = static_cast<int64_t>(p.rows) * p.heads >= 2048;
  if (slots <= (many ? 8 : 4)) return fp8 ? launch<true, 1>(p, stream) : launch<false, 1>(p, stream);
  if (slots <= 16) return fp8 ? launch<true, 4>(p, stream) : launch<false, 4>(p, stream);
  return fp8 ? launch<true, 8>(p, stream) : launch<false, 8>(p, stream);
}

}  // namespace pkv
