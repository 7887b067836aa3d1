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
// alone needs more: at n = 2^20 an fp32 product is off by up to 2^-4 rad.  f_p / 2 pi is taken in
// fp64 as a fraction of 2^64ths of a turn, and n times that, modulo 2^64, is the part of the last turn, whole
// turns falling off: exact but for the fp64 value itself (2^-53 of the angle).  (The product in fp64
// kept a CTA waiting: GB300 has about two fp64 lanes per SM.)  The R/2 sines and cosines of a
// token are computed once per CTA into shared memory and used by all its heads.
//
// Bound by memory: every element is read once and written once.  A thread owns 16 elements of
// a row as the two 16-byte pieces that the rotation pairs up, so no element crosses threads; the
// D / 16 threads of a row sit side by side in a warp and add up the squares by shuffles.  The CTAs of
// at most 256 threads (the rows of one token, of several when they are few, or a part of them) stay
// and go through the tokens in rounds: the next round's pieces are on their way and its table of
// sines is made while this round's are worked on.  Measured for 8192 tokens of 32 + 8 + 8 heads of 128 into
// an E4M3 pool (184 MB) and 20,011 of 8 + 2 + 2 heads of 64, a quarter rotated, into bf16 (62 MB):
// 39 and 11.5 us one after another in a graph = 4.7 and 5.4 TB/s; a CTA per token 46 and 14, with the product of the angle in fp64 and
// every E4M3 code by a division 58 and 19; more CTAs per SM at 64 registers spill (64 and 18).  A warp per
// token, its rows in turns and its sines in registers, with no barrier: 51 and 17 (half of its life is
// the start: sines, then the first rows).
#include <cuda_runtime.h>

#include <algorithm>

#include "mma_ops.cuh"
#include "pkv_device.cuh"
#include "prompt.cuh"

namespace pkv {

namespace {

constexpr int kMaxThreads = 256;
constexpr int kThreadsPerSm = 768;  // at 80 registers a thread
constexpr double kInvTwoPi = 0.15915494309189533577;
constexpr double kTwo64 = 18446744073709551616.0;

// Eight fp32 values / scale as E4M3 codes, the quotients those of e4m3_quant8's divisions.  x * (1 / scale)
// is off by less than 2 units in the last place of fp32 and E4M3 keeps 4 bits, so the code is the
// same unless the product lies that near to a border of two codes, whose fp32 pattern ends in 19
// zeros; then (and in the rare other case) the division itself is taken.  With a power of two as the
// scale the product is exact.
__device__ __forceinline__ uint2 e4m3_codes(const float2 (&x)[4], float sc, float inv, bool exact) {
  float2 y[4];
  bool near = !(fabsf(inv) >= 1.17549435e-38f);  // a reciprocal below the normal range has lost bits
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[j] = fmul2(x[j], make_float2(inv, inv));
    near |= ((__float_as_uint(y[j].x) + 4u) & 0x7ffffu) < 9u;
    near |= ((__float_as_uint(y[j].y) + 4u) & 0x7ffffu) < 9u;
  }
  if (near && !exact) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = make_float2(__fdiv_rn(x[j].x, sc), __fdiv_rn(x[j].y, sc));
  }
  uint32_t out[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(y[2 * j], __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(y[2 * j + 1], __NV_SATFINITE, __NV_E4M3);
    out[j] = (lo & 0xffffu) | (hi << 16);
  }
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ void unpack8(uint4 w, float2 (&x)[4]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = make_float2(bf16_lo(in[j]), bf16_hi(in[j]));
}

__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  return make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y),
                    pack_bf16(x[3].x, x[3].y));
}

}  // namespace

// One row's 16 elements, from the pieces read to the pieces written.  Called by whole warps.
template <int D, bool FP8, bool INTER>
__device__ __forceinline__ void row_pieces(const RopeAppendParams& p, uint4 r0, uint4 r1, int64_t slot, int64_t t,
                                           bool live, const float* cs, int tok, int row, int h, int c0, int c1, int s,
                                           bool turns, bool is_q, bool is_v) {
  constexpr int S = D / 16;
  const int half = p.rot / 2;
  float2 x[4], y[4];
  unpack8(r0, x);
  unpack8(r1, y);
  if (p.q_weight != nullptr || p.k_weight != nullptr) {
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) sq = ffma2(x[e], x[e], ffma2(y[e], y[e], sq));
    float ss = sq.x + sq.y;
#pragma unroll
    for (int m = 1; m < S; m <<= 1) ss += shfl_xor(ss, m);
    const uint16_t* wt = is_v ? nullptr : (is_q ? p.q_weight : p.k_weight);
    if (wt != nullptr) {
      const float inv = rsqrtf(fmaf(ss, 1.0f / D, p.eps));
      const float2 inv2 = make_float2(inv, inv);
      float2 nw[4];
      unpack8(__ldg(reinterpret_cast<const uint4*>(wt) + c0), nw);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = fmul2(fmul2(x[e], inv2), nw[e]);
      unpack8(__ldg(reinterpret_cast<const uint4*>(wt) + c1), nw);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fmul2(fmul2(y[e], inv2), nw[e]);
    }
  }
  if (!live) return;
  if (turns && !is_v) {
    if constexpr (INTER) {
      const float4* c = reinterpret_cast<const float4*>(cs) + (tok * half + 8 * s) / 2;  // two pairs each
      auto turn = [](float2 v, float cn, float sn) {
        return ffma2(v, make_float2(cn, cn), fmul2(make_float2(v.y, v.x), make_float2(-sn, sn)));
      };
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 f = c[e], g = c[2 + e];
        x[2 * e] = turn(x[2 * e], f.x, f.y);
        x[2 * e + 1] = turn(x[2 * e + 1], f.z, f.w);
        y[2 * e] = turn(y[2 * e], g.x, g.y);
        y[2 * e + 1] = turn(y[2 * e + 1], g.z, g.w);
      }
    } else {
      const float4* cv = reinterpret_cast<const float4*>(cs + tok * p.rot + 8 * s);
      const float4* sv = reinterpret_cast<const float4*>(cs + tok * p.rot + half + 8 * s);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 c = cv[e], n = sv[e];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 c2 = k ? make_float2(c.z, c.w) : make_float2(c.x, c.y);
          const float2 s2 = k ? make_float2(n.z, n.w) : make_float2(n.x, n.y);
          const float2 a = x[2 * e + k], b = y[2 * e + k];
          x[2 * e + k] = ffma2(a, c2, fmul2(b, make_float2(-s2.x, -s2.y)));
          y[2 * e + k] = ffma2(b, c2, fmul2(a, s2));
        }
      }
    }
  }
  if (is_q) {
    uint4* dst = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + row * D);
    dst[c0] = pack8(x);
    dst[c1] = pack8(y);
    return;
  }
  if (slot < 0) return;  // padding token
  if (slot >= p.pool_slots) {
    set_flag(p.status, PKV_DEVFLAG_BAD_SLOT);
    return;
  }
  const int64_t prow = (slot * p.hkv + h) * (D / 8);  // in 8-element pieces
  uint8_t* pool = is_v ? p.v_cache : p.k_cache;
  if constexpr (FP8) {
    const float sc = p.scales[(is_v ? p.hkv : 0) + h];
    const float inv_sc = __fdiv_rn(1.f, sc);
    const bool exact = (__float_as_uint(sc) & 0x7fffffu) == 0u;  // a power of two: the product is the quotient
    reinterpret_cast<uint2*>(pool)[prow + c0] = e4m3_codes(x, sc, inv_sc, exact);
    reinterpret_cast<uint2*>(pool)[prow + c1] = e4m3_codes(y, sc, inv_sc, exact);
  } else {  // v is a bit copy
    reinterpret_cast<uint4*>(pool)[prow + c0] = is_v ? r0 : pack8(x);
    reinterpret_cast<uint4*>(pool)[prow + c1] = is_v ? r1 : pack8(y);
  }
}

template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(kMaxThreads, kThreadsPerSm / kMaxThreads)
    qk_rope_append_kernel(const RopeAppendParams p) {
  constexpr int S = D / 16;  // threads per row
  // two tables, of this round and the next.  Half layout: [token][cos of every pair, then sin];
  // interleaved: [token][pair] (cos, sin)
  extern __shared__ __align__(16) float tables[];
  pdl_wait();
  pdl_launch_dependents();
  const int half = p.rot / 2;

  // this thread: its token of a group, the row of the token and its pieces c0 and c1
  const int lane_row = static_cast<int>(threadIdx.x) / S;
  const int tok = lane_row / p.rows_per_cta;
  const int row = static_cast<int>(blockIdx.y) * p.rows_per_cta + lane_row - tok * p.rows_per_cta;
  const bool mine = tok < p.groups && row < p.hq + 2 * p.hkv;
  const int s = threadIdx.x % S;
  const bool turns = s < p.rot / 16;  // this thread's elements are rotated
  int c0, c1;
  if (INTER || !turns) {
    c0 = 2 * s;
    c1 = 2 * s + 1;
  } else {
    c0 = s;
    c1 = s + p.rot / 16;
  }
  const bool is_q = row < p.hq, is_v = row >= p.hq + p.hkv;
  const int h = is_q ? row : row - p.hq - (is_v ? p.hkv : 0);
  const uint16_t* src = (is_q ? p.q : is_v ? p.v : p.k) + h * D;
  const int64_t stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
  // the entry of the table that this thread makes (groups * half <= threads): its token, and
  // 2^64ths of a turn per position
  const bool makes = static_cast<int>(threadIdx.x) < p.groups * half;
  const int etok = makes ? static_cast<int>(threadIdx.x) / half : 0, pair = threadIdx.x - etok * half;
  unsigned long long step = 0;
  float amp = p.rope_scale;
  if (makes) {
    const double f = p.inv_freq[pair] * kInvTwoPi;
    // not finite: no angle (the integer below would be 0; by its bits, fp64 comparisons are slow here)
    if ((~__double2hiint(f) & 0x7ff00000) == 0) amp = __int_as_float(0x7fffffff);
    step = static_cast<unsigned long long>(static_cast<long long>((f - rint(f)) * kTwo64));
  }
  auto position = [&](int64_t t0) { return makes && t0 + etok < p.num_tokens ? p.positions[t0 + etok] : 0; };
  auto make = [&](float* table, int pos) {
    if (!makes) return;
    const long long part = static_cast<long long>(step * static_cast<unsigned long long>(static_cast<long long>(pos)));
    const float r = static_cast<float>(part) * 1.0842021724855044e-19f;  // 2^-63: half turns in [-1, 1]
    float sn, cn;
    sincospif(r, &sn, &cn);
    if constexpr (INTER) {
      reinterpret_cast<float2*>(table)[threadIdx.x] = make_float2(cn * amp, sn * amp);
    } else {
      table[etok * p.rot + pair] = cn * amp;
      table[etok * p.rot + half + pair] = sn * amp;
    }
  };
  uint4 n0 = make_uint4(0u, 0u, 0u, 0u), n1 = n0;
  int64_t nslot = -1;
  auto load = [&](int64_t t) {
    if (mine && t < p.num_tokens) {
      n0 = __ldcs(reinterpret_cast<const uint4*>(src + t * stride) + c0);
      n1 = __ldcs(reinterpret_cast<const uint4*>(src + t * stride) + c1);
      if (!is_q) nslot = p.slots[t];
    }
  };
  // rounds: group blockIdx.x, + gridDim.x, ..; the next round's pieces and table are on their way
  // while this one's are worked on
  const int64_t hop = static_cast<int64_t>(gridDim.x) * p.groups;
  int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.groups;
  load(t0 + tok);
  make(tables, position(t0));
  int npos = position(t0 + hop);
  __syncthreads();
  for (unsigned round = 0; t0 < p.num_tokens; t0 += hop, ++round) {
    const float* cs = tables + (round & 1) * p.groups * p.rot;
    const uint4 r0 = n0, r1 = n1;
    const int64_t slot = nslot, t = t0 + tok;
    const bool live = mine && t < p.num_tokens;
    if (t0 + hop < p.num_tokens) {
      load(t + hop);
      make(tables + (~round & 1) * p.groups * p.rot, npos);
      npos = position(t0 + 2 * hop);
    }
    row_pieces<D, FP8, INTER>(p, r0, r1, slot, t, live, cs, tok, row, h, c0, c1, s, turns, is_q, is_v);
    __syncthreads();
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
  const int rows = p.hq + 2 * p.hkv, per_row = d / 16;
  // CTAs of at most 256 threads: the rows of one token, of several side by side when they are few,
  // or a part of a token's rows (grid y)
  const int parts = (rows * per_row + kMaxThreads - 1) / kMaxThreads;
  p.rows_per_cta = (rows + parts - 1) / parts;
  const int threads_token = p.rows_per_cta * per_row;
  int64_t groups = std::min<int64_t>(kMaxThreads / threads_token, p.num_tokens);
  if (p.rot > 0) groups = std::min<int64_t>(groups, kMaxThreads / (p.rot / 2));  // the table's entries
  p.groups = static_cast<int>(std::max<int64_t>(1, groups));
  const int64_t all = (p.num_tokens + p.groups - 1) / p.groups;
  const int threads = (std::max(p.groups * threads_token, p.groups * p.rot / 2) + 31) / 32 * 32;
  const int64_t ctas = std::min<int64_t>(all, std::max(1, sm_count * (kThreadsPerSm / threads) / parts));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(parts), 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = 2 * static_cast<size_t>(p.groups) * p.rot * sizeof(float);
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
