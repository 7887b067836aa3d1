// qk_rope_append.cu -- a chunk's q, k and v from the projection to the attention and the
// pool in one pass: RMS norm of every q and k head, rotation by position, q written for the
// attention and k, v into the paged pool (bf16, or E4M3 quantised as written).
//
// Mathematics.  For a head row x of D elements at position n:
//   norm      y_i = x_i * w_i / sqrt(mean_j x_j^2 + eps)                 (skipped without w)
//   rotation  of the first R elements, pair p at angle a_p = n * f_p:
//             (y_a, y_b) -> scale * (y_a cos a_p - y_b sin a_p, y_b cos a_p + y_a sin a_p)
//             with (a, b) = (p, p + R/2) in the half layout, (2p, 2p + 1) interleaved.
// All of it in fp32, rounded once: to bf16, or divided by the head's scale to E4M3.  The angle
// alone is formed in fp64 (n * f_p / 2 pi turns, less the whole turns): at n = 2^20 an fp32
// product is off by up to 2^-4 rad, the fp64 one by less than 2^-30.  The R/2 sines and cosines
// of a token are computed once per CTA into shared memory and used by all its heads.
//
// Bound by memory: every element is read once and written once.  A thread owns 16 elements of
// a row as the two 16-byte pieces that the rotation pairs up, so no element crosses threads;
// the D/16 threads of a row sit side by side in a warp and add up the squares by shuffles.  A
// CTA takes one token, or as many as fill it when a token's heads are few, and issues its loads
// before the angles are ready.
#include <cuda_runtime.h>

#include <algorithm>

#include "mma_ops.cuh"
#include "pkv_device.cuh"
#include "prompt.cuh"

namespace pkv {

namespace {

constexpr int kMaxThreads = 512;
constexpr double kInvTwoPi = 0.15915494309189533577;

// eight fp32 values -> eight E4M3 codes, as e4m3_quant8 encodes bf16 ones
__device__ __forceinline__ uint2 e4m3_quant8_f32(const float (&x)[8], float sc) {
  uint32_t out[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[4 * j], sc), __fdiv_rn(x[4 * j + 1], sc)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[4 * j + 2], sc), __fdiv_rn(x[4 * j + 3], sc)), __NV_SATFINITE, __NV_E4M3);
    out[j] = (lo & 0xffffu) | (hi << 16);
  }
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = bf16_lo(in[j]);
    x[2 * j + 1] = bf16_hi(in[j]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

}  // namespace

template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(kMaxThreads) qk_rope_append_kernel(const RopeAppendParams p) {
  constexpr int S = D / 16;  // threads per row
  extern __shared__ float2 cs[];  // [token][R / 2] (cos, sin) * rope_scale
  pdl_wait();
  pdl_launch_dependents();
  const int half = p.rot / 2;
  const int rows = p.hq + 2 * p.hkv;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens_per_cta;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(p.tokens_per_cta), p.num_tokens - t0));
  const int items = ntok * rows * S;

  // the pieces of item i: row (token, head) and the two 16-byte pieces c0, c1 of the row
  const int s = threadIdx.x % S;
  int c0, c1;
  if (INTER || s >= p.rot / 16) {
    c0 = 2 * s;
    c1 = 2 * s + 1;
  } else {
    c0 = s;
    c1 = s + p.rot / 16;
  }
  const bool turns = s < p.rot / 16;  // this thread's elements are rotated
  auto load = [&](int i, int& tok, int& row, uint4& w0, uint4& w1) {
    const int rr = i / S;
    tok = rr / rows;
    row = rr - tok * rows;
    w0 = w1 = make_uint4(0u, 0u, 0u, 0u);
    if (i < items) {
      const int64_t t = t0 + tok;
      const uint16_t* src = row < p.hq            ? p.q + t * p.q_stride + row * D
                            : row < p.hq + p.hkv ? p.k + t * p.k_stride + (row - p.hq) * D
                                                 : p.v + t * p.v_stride + (row - p.hq - p.hkv) * D;
      w0 = reinterpret_cast<const uint4*>(src)[c0];
      w1 = reinterpret_cast<const uint4*>(src)[c1];
    }
  };
  int tok, row;
  uint4 w0, w1;
  load(threadIdx.x, tok, row, w0, w1);

  for (int i = threadIdx.x; i < ntok * half; i += blockDim.x) {
    const int tk = i / half;
    const double turn = static_cast<double>(p.positions[t0 + tk]) * (p.inv_freq[i - tk * half] * kInvTwoPi);
    const float r = 2.f * static_cast<float>(turn - rint(turn));  // half turns in [-1, 1]
    float sn, cn;
    sincospif(r, &sn, &cn);
    cs[i] = make_float2(cn * p.rope_scale, sn * p.rope_scale);
  }
  __syncthreads();

  // every warp runs the same number of rounds (the shuffles below need all its lanes)
  for (int base = 0; base < items; base += blockDim.x) {
    const int i = base + threadIdx.x;
    if (base > 0) load(i, tok, row, w0, w1);
    const bool is_v = row >= p.hq + p.hkv;
    const bool is_q = row < p.hq;
    float x[8], y[8];
    unpack8(w0, x);
    unpack8(w1, y);
    const uint16_t* wt = is_v ? nullptr : (is_q ? p.q_weight : p.k_weight);
    if (p.q_weight != nullptr || p.k_weight != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
      for (int m = 1; m < S; m <<= 1) ss += shfl_xor(ss, m);
      if (wt != nullptr) {
        const float inv = rsqrtf(fmaf(ss, 1.0f / D, p.eps));
        float a[8], b[8];
        unpack8(reinterpret_cast<const uint4*>(wt)[c0], a);
        unpack8(reinterpret_cast<const uint4*>(wt)[c1], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = x[e] * inv * a[e];
          y[e] = y[e] * inv * b[e];
        }
      }
    }
    if (i >= items) continue;
    if (turns && !is_v) {
      const float2* c = cs + tok * half + 8 * s;
      if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = c[e], g = c[4 + e];
          const float a0 = x[2 * e], b0 = x[2 * e + 1], a1 = y[2 * e], b1 = y[2 * e + 1];
          x[2 * e] = a0 * f.x - b0 * f.y;
          x[2 * e + 1] = b0 * f.x + a0 * f.y;
          y[2 * e] = a1 * g.x - b1 * g.y;
          y[2 * e + 1] = b1 * g.x + a1 * g.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = c[e];
          const float a0 = x[e], b0 = y[e];
          x[e] = a0 * f.x - b0 * f.y;
          y[e] = b0 * f.x + a0 * f.y;
        }
      }
    }
    const int64_t t = t0 + tok;
    if (is_q) {
      uint4* dst = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + row * D);
      dst[c0] = pack8(x);
      dst[c1] = pack8(y);
      continue;
    }
    const int64_t slot = p.slots[t];
    if (slot < 0) continue;  // padding token
    if (slot >= p.pool_slots) {
      set_flag(p.status, PKV_DEVFLAG_BAD_SLOT);
      continue;
    }
    const int h = row - p.hq - (is_v ? p.hkv : 0);
    const int64_t prow = (slot * p.hkv + h) * (D / 8);  // in 8-element pieces
    uint8_t* pool = is_v ? p.v_cache : p.k_cache;
    if constexpr (FP8) {
      const float sc = p.scales[(is_v ? p.hkv : 0) + h];
      reinterpret_cast<uint2*>(pool)[prow + c0] = e4m3_quant8_f32(x, sc);
      reinterpret_cast<uint2*>(pool)[prow + c1] = e4m3_quant8_f32(y, sc);
    } else {  // v is a bit copy
      reinterpret_cast<uint4*>(pool)[prow + c0] = is_v ? w0 : pack8(x);
      reinterpret_cast<uint4*>(pool)[prow + c1] = is_v ? w1 : pack8(y);
    }
  }
}

template <int D, bool FP8>
static cudaError_t launch_d(const RopeAppendParams& p, bool interleaved, const cudaLaunchConfig_t& cfg) {
  if (interleaved) return cudaLaunchKernelEx(&cfg, qk_rope_append_kernel<D, FP8, true>, p);
  return cudaLaunchKernelEx(&cfg, qk_rope_append_kernel<D, FP8, false>, p);
}

cudaError_t launch_qk_rope_append(int d, bool fp8, bool interleaved, const RopeAppendParams& p0, int sm_count,
                                  cudaStream_t stream) {
  RopeAppendParams p = p0;
  if (p.num_tokens <= 0) return cudaSuccess;
  const int per_token = (p.hq + 2 * p.hkv) * (d / 16);
  // tokens per CTA: as many as 512 threads hold, but no fewer CTAs than two per SM
  int64_t tpc = std::max(1, kMaxThreads / per_token);
  tpc = std::max<int64_t>(1, std::min(tpc, p.num_tokens / (2 * sm_count)));
  p.tokens_per_cta = static_cast<int>(tpc);
  const int64_t ctas = (p.num_tokens + tpc - 1) / tpc;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int64_t items = tpc * per_token;
  const int64_t rounds = (items + kMaxThreads - 1) / kMaxThreads;
  const int threads = static_cast<int>(((items + rounds - 1) / rounds + 31) / 32 * 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(tpc) * (p.rot / 2) * sizeof(float2);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (d == 64) return fp8 ? launch_d<64, true>(p, interleaved, cfg) : launch_d<64, false>(p, interleaved, cfg);
  return fp8 ? launch_d<128, true>(p, interleaved, cfg) : launch_d<128, false>(p, interleaved, cfg);
}

}  // namespace pkv
