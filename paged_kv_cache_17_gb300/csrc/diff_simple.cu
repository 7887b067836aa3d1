// diff_simple.cu -- differential attention, a warp per (row, output head), on the CUDA cores.
//
// Lane l holds elements 4 l .. 4 l + 3 of the pair's 128: lanes 0-15 the first map's half of q and K, lanes
// 16-31 the second's.  Each half warp sums its map's score and holds that map's running maximum and sum (log2
// units); every lane accumulates its four columns of the pair's value under both maps.
#include "diff.cuh"
#include "mma_ops.cuh"
#include "pkv_device.cuh"

namespace pkv {

template <bool FP8>
__device__ __forceinline__ void diff_row4(const void* base, int64_t at, float s, float (&x)[4]) {
  if constexpr (FP8) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(base) + at);
    const uint32_t h0 = e4m3_lo(w), h1 = e4m3_hi(w);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
    x[0] = a.x * s, x[1] = a.y * s, x[2] = b.x * s, x[3] = b.y * s;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
    x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  }
}

template <bool FP8>
__global__ void __launch_bounds__(256) diff_simple_kernel(const DiffParams p, const void* k_cache, const void* v_cache) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (unit >= static_cast<int64_t>(p.rows) * p.heads) return;
  const int row = static_cast<int>(unit / p.heads), head = static_cast<int>(unit % p.heads), pair = head / p.group;
  int seq = row, place = 0, n = 1;
  if (p.q_indptr != nullptr) {
    seq = -1;
    for (int b = lane; b < p.batch; b += 32) {
      const int first = p.q_indptr[b], last = p.q_indptr[b + 1];
      if (first < 0 || last < first || last > p.rows) set_flag(p.status, PKV_DEVFLAG_BAD_INDPTR);
      else if (row >= first && row < last) seq = b;
    }
    seq = __reduce_max_sync(kFull, seq);
    if (seq < 0) return;
    place = row - p.q_indptr[seq];
    n = p.q_indptr[seq + 1] - p.q_indptr[seq];
  }
  int ctx = p.context_lens[seq];
  if (ctx < 0 || ctx > p.max_context_len) {
    set_flag(p.status, PKV_DEVFLAG_BAD_CONTEXT_LEN);
    ctx = max(0, min(ctx, p.max_context_len));
  }
  const int prefix = p.seq_prefix != nullptr ? p.seq_prefix[seq] : -1;
  int lead = prefix >= 0 && prefix < p.num_prefixes ? max(0, min(p.prefix_lens[prefix], p.max_prefix_len)) : 0;
  const int own = p.causal ? max(0, min(ctx, ctx - n + place + 1)) : ctx;
  float qx[4];
  diff_row4<false>(p.q + row * p.q_stride, head * kDiffW + 4 * lane, 1.f, qx);
  const float ks = FP8 ? p.scales[2 * pair + lane / 16] : 1.f, vs = FP8 ? p.scales[2 * (p.pairs + pair) + lane / 16] : 1.f;
  float m = -INFINITY, l = 0.f, o[2][4] = {};
  for (int part = 0; part < 2; ++part) {
    const int32_t* table = part == 0 ? p.prefix_tables + static_cast<int64_t>(lead > 0 ? prefix : 0) * p.max_prefix_blocks
                                     : p.block_tables + static_cast<int64_t>(seq) * p.max_blocks;
    const int upto = part == 0 ? lead : own;
    for (int j = 0; j < upto; ++j) {
      const int id = table[j / kBlockSize];
      float kx[4] = {}, vx[4] = {};
      if (id >= 0 && id < p.num_blocks) {
        const int64_t at = ((static_cast<int64_t>(id) * kBlockSize + j % kBlockSize) * p.pairs + pair) * kDiffW + 4 * lane;
        diff_row4<FP8>(k_cache, at, ks, kx);
        diff_row4<FP8>(v_cache, at, vs, vx);
      } else if (lane == 0) {
        set_flag(p.status, PKV_DEVFLAG_BAD_BLOCK_ID);
      }
      float x = qx[0] * kx[0] + qx[1] * kx[1] + qx[2] * kx[2] + qx[3] * kx[3];
#pragma unroll
      for (int i = 8; i >= 1; i >>= 1) x += shfl_xor(x, i);
      x *= p.score_scale;
      const float top = fmaxf(m, x), alpha = top == -INFINITY ? 1.f : exp2f(m - top);
      const float w = top == -INFINITY ? 0.f * x : exp2f(x - top);
      m = top;
      l = l * alpha + w;
      const float other_alpha = shfl_xor(alpha, 16), other = shfl_xor(w, 16);
      const float a0 = lane < 16 ? alpha : other_alpha, a1 = lane < 16 ? other_alpha : alpha;
      const float w0 = lane < 16 ? w : other, w1 = lane < 16 ? other : w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[0][i] = o[0][i] * a0 + w0 * vx[i];
        o[1][i] = o[1][i] * a1 + w1 * vx[i];
      }
    }
  }
  const float other = shfl_xor(l, 16);
  const float l0 = lane < 16 ? l : other, l1 = lane < 16 ? other : l;
  const bool none = lead + own == 0;
  const float lam = p.lambda[row * p.lambda_stride + head];
  float y[4], square = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = none ? 0.f : o[0][i] / l0 - lam * (o[1][i] / l1);
    square += y[i] * y[i];
  }
  float by = p.out_scale;
  if (p.norm_weight != nullptr) {
#pragma unroll
    for (int i = 16; i >= 1; i >>= 1) square += shfl_xor(square, i);
    if (!none) by *= rsqrtf(square / kDiffW + p.eps);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= bf16_lo(p.norm_weight[4 * lane + i]);
  }
  const int64_t to = unit * kDiffW + 4 * lane;
  if (p.out_fp32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = make_float4(y[0] * by, y[1] * by, y[2] * by, y[3] * by);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + to) =
        make_uint2(pack_bf16(y[0] * by, y[1] * by), pack_bf16(y[2] * by, y[3] * by));
}

cudaError_t launch_diff_simple(bool fp8, const DiffParams& p, const void* k, const void* v, cudaStream_t stream) {
  const int64_t ctas = (static_cast<int64_t>(p.rows) * p.heads + 7) / 8;
  if (fp8) diff_simple_kernel<true><<<static_cast<unsigned>(ctas), 256, 0, stream>>>(p, k, v);
  else diff_simple_kernel<false><<<static_cast<unsigned>(ctas), 256, 0, stream>>>(p, k, v);
  return cudaGetLastError();
}

}  // namespace pkv
