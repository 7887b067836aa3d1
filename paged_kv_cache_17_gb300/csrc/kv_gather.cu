// kv_gather.cu -- read ranges of cached positions back out of the paged pool, dequantised,
// into ragged rows: the inverse of the append.
//
//   out[indptr[b] + i][h][:] = value(cache[table[b][n / 16]][n % 16][h][:]),  n = starts[b] + i
//
// with value the element itself (bf16) or code * scale of its head (E4M3: one fp32 product,
// rounded once more for bf16 output).  A position's row (every head) is contiguous in the pool
// and in the output, and so are the 16 rows of a block.
//
// Bound by memory: each row is read once and written once.  A CTA takes a run of rows of K or
// of V: it finds their sequences once (a search of indptr, sampled into shared memory; a pass over all of
// it when a row is not found), keeps the pool slot of each row there, and then moves 8 elements per thread
// at a time with four
// loads in flight.  Measured, 8 heads of 128: bf16, 64 ranges of 512 to 4096 tokens (1.19 GB moved),
// 175 us, the time of a plain copy of as many bytes; E4M3 to fp32, four of 32 to 70 thousand
// (1.73 GB), 262 us, 97 % of it; one range of 1000 tokens 3.7 us, launch and three dependent loads.
#include <cuda_runtime.h>

#include <algorithm>

#include "mma_ops.cuh"
#include "pkv_device.cuh"
#include "prompt.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 32;   // rows of a CTA
constexpr int kSamples = 256;  // entries of indptr kept in shared memory
constexpr int kUnroll = 4;

}  // namespace

template <bool FP8, bool F32>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const GatherParams p, int rows_per_cta) {
  __shared__ int sample[kSamples + 1];
  __shared__ int64_t slot_of[kMaxRows];  // pool slot; -1: reads as zeros; -2: not a row of any sequence
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_per_cta;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(rows_per_cta), p.num_rows - row0));
  const bool is_v = blockIdx.y != 0;

  // b with indptr[b] <= row < indptr[b + 1]: the last sampled entry <= row, then the rest
  const int step = (p.batch + kSamples - 1) / kSamples;
  const int ns = (p.batch + step - 1) / step;  // samples at 0, step, 2 step, ..
  for (int i = threadIdx.x; i < ns; i += kThreads) sample[i] = p.kv_indptr[i * step];
  __syncthreads();
  int b = 0;
  bool lost = false;  // this thread's row is of no range that the search finds
  const int64_t row = row0 + threadIdx.x;
  if (threadIdx.x < nrows) {
    int lo = 0, hi = ns;  // the answer's sample is in [lo, hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sample[mid] <= row) lo = mid;
      else hi = mid;
    }
    b = lo * step;
    int e = min(p.batch, b + step);
    while (e - b > 1) {
      const int mid = (b + e) >> 1;
      if (p.kv_indptr[mid] <= row) b = mid;
      else e = mid;
    }
    const int first = p.kv_indptr[b], last = p.kv_indptr[b + 1];
    lost = first < 0 || row < first || row >= last || last > p.num_rows;
  }
  // rows outside every range, or offsets out of order (a bad range), among which the search goes astray: all
  // ranges are looked through, and the good ones say which rows are theirs
  if (__syncthreads_or(lost)) {
    int* range_of = sample;  // (the samples are done with)
    if (threadIdx.x < nrows) range_of[threadIdx.x] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < p.batch; i += kThreads) {
      const int64_t first = p.kv_indptr[i], last = p.kv_indptr[i + 1];
      if (first < 0 || last > p.num_rows) continue;
      const int64_t end = min(last, row0 + nrows);
      for (int64_t r = max(first, row0); r < end; ++r) range_of[r - row0] = i;
    }
    __syncthreads();
    if (lost) b = range_of[threadIdx.x];
  }
  if (threadIdx.x < nrows) {
    int64_t slot = -2;
    if (b >= 0) {
      const int64_t n = (p.starts != nullptr ? static_cast<int64_t>(p.starts[b]) : 0) + (row - p.kv_indptr[b]);
      slot = -1;
      if (n < 0 || n >= static_cast<int64_t>(p.max_blocks) * kBlockSize) {
        set_flag(p.status, PKV_DEVFLAG_BAD_CONTEXT_LEN);
      } else {
        const int id = p.block_tables[static_cast<int64_t>(b) * p.max_blocks + n / kBlockSize];
        if (id >= 0 && id < p.num_blocks) slot = static_cast<int64_t>(id) * kBlockSize + n % kBlockSize;
        else set_flag(p.status, PKV_DEVFLAG_BAD_BLOCK_ID);
      }
    }
    slot_of[threadIdx.x] = slot;
  }
  if (blockIdx.x == 0 && is_v)
    for (int i = threadIdx.x; i < p.batch; i += kThreads) {
      const int first = p.kv_indptr[i], last = p.kv_indptr[i + 1];
      if (first < 0 || last < first || last > p.num_rows) set_flag(p.status, PKV_DEVFLAG_BAD_INDPTR);
    }
  __syncthreads();

  using In = typename std::conditional<FP8, uint2, uint4>::type;  // 8 elements
  const In* pool = reinterpret_cast<const In*>(is_v ? p.v_cache : p.k_cache);
  void* out = is_v ? p.v_out : p.k_out;
  const int pieces = p.hkv * (p.d / 8);  // 8-element pieces of a row
  const int items = nrows * pieces;
  for (int i0 = threadIdx.x; i0 < items; i0 += kThreads * kUnroll) {
    In w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      w[u] = In{};
      if (i < items) {
        const int r = i / pieces;
        const int64_t slot = slot_of[r];
        if (slot >= 0) w[u] = __ldcs(&pool[slot * pieces + (i - r * pieces)]);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= items) break;
      const int r = i / pieces, c = i - r * pieces;
      if (slot_of[r] == -2) continue;  // left as it was
      const int64_t at = (row0 + r) * pieces + c;
      if constexpr (!FP8 && !F32) {
        __stcs(&reinterpret_cast<uint4*>(out)[at], w[u]);
      } else {
        float x[8];
        if constexpr (FP8) {
          const float sc = p.scales[(is_v ? p.hkv : 0) + c / (p.d / 8)];
          const uint32_t h[4] = {e4m3_lo(w[u].x), e4m3_hi(w[u].x), e4m3_lo(w[u].y), e4m3_hi(w[u].y)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            x[2 * j] = f.x * sc;
            x[2 * j + 1] = f.y * sc;
          }
        } else {
          const uint32_t in[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf16_lo(in[j]);
            x[2 * j + 1] = bf16_hi(in[j]);
          }
        }
        if constexpr (F32) {
          float4* dst = reinterpret_cast<float4*>(out) + at * 2;
          __stcs(dst, make_float4(x[0], x[1], x[2], x[3]));
          __stcs(dst + 1, make_float4(x[4], x[5], x[6], x[7]));
        } else {
          __stcs(&reinterpret_cast<uint4*>(out)[at], make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                                 pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])));
        }
      }
    }
  }
}

cudaError_t launch_kv_gather(bool fp8, bool out_fp32, const GatherParams& p, int sm_count, cudaStream_t stream) {
  if (p.num_rows <= 0 || p.batch <= 0) return cudaSuccess;
  // rows per CTA: 16 (a block's worth), fewer when that leaves SMs without work
  int rows = 16;
  while (rows > 1 && 2 * ((p.num_rows + rows - 1) / rows) < 4LL * sm_count) rows /= 2;
  const int64_t ctas = (p.num_rows + rows - 1) / rows;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 2, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (fp8)
    return out_fp32 ? cudaLaunchKernelEx(&cfg, kv_gather_kernel<true, true>, p, rows)
                    : cudaLaunchKernelEx(&cfg, kv_gather_kernel<true, false>, p, rows);
  return out_fp32 ? cudaLaunchKernelEx(&cfg, kv_gather_kernel<false, true>, p, rows)
                  : cudaLaunchKernelEx(&cfg, kv_gather_kernel<false, false>, p, rows);
}

}  // namespace pkv
