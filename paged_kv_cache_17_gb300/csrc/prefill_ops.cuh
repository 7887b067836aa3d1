// prefill_ops.cuh -- building blocks of the chunk attention kernels on the fifth-generation tensor cores
// (prefill_tc.cu, diff_chunk.cu): MMAs issued by a whole warp with one lane electing, bounded waits, tensor-memory
// pieces, TMA of pool blocks, work taken over from CTAs that have not started, and the turn of rows for stores.
#pragma once

#include <cuda.h>

#include "mma_ops.cuh"
#include "pkv_device.cuh"
#include "prompt.cuh"
#include "tc_ops.cuh"

namespace pkv {
namespace {

// Shared-memory descriptors as two words (see tc_ops.cuh for the fields).  The high word is a
// constant of the operand; the low word is the address >> 4 plus the leading offset, so the
// K slices of an operand differ by an added constant.  The issuing warp computes them as a warp, so
// that they stay in uniform registers, and only the MMA itself is left to the elected lane: issued
// from a branch of one lane, each MMA took 70 cycles of moves between register files, more than it
// executes (64), and the step 4170 cycles for 2050 of products.
template <uint32_t kStride>
constexpr uint32_t kDesc128 = (kStride >> 4) | (1u << 14) | (2u << 29);  // groups of eight rows apart, 128-byte swizzle
constexpr uint32_t kDescK128 = kDesc128<1024>;
constexpr uint32_t kDescK64 = (512u >> 4) | (1u << 14) | (4u << 29);    // stride 512, 64-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}

// D[tmem] (+)= A[smem] B[smem]: 16-bit operands, or 8-bit ones (E4M3: formats 0 in the
// descriptor); D[tmem] (+)= A[tmem] B[smem], 16-bit operands.  Called by the whole warp; the lane
// with leader != 0 issues.
template <bool F8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t a_hi, uint32_t b_hi,
                                       uint32_t idesc, bool accumulate, uint32_t leader) {
  if constexpr (F8)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       bool accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader)
      : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// One arrival on bar once every tcgen05 operation the leader issued before has completed.
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}

// Wait for a phase; false when the CTA has aborted or after `tries` tries (2^23, tests set fewer; the hardware
// suspends each, for 3 to 10 us as measured, so half a minute or more, but promises no time, and works of 50 ms
// are waited for).  Shorter code than wait_or_abort, at 30 places: the roles together do not
// fit the SM's instruction cache, and the fetches beyond it were at 83 % of their peak rate.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, const volatile int* abort,
                                         int tries = kPrefillWaitTries) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int n = 0; n < tries && !*abort; ++n)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}
__device__ __forceinline__ void give_up(uint32_t* status, volatile int* abort) {
  set_flag(status, PKV_DEVFLAG_WAIT_TIMEOUT);
  *abort = 1;
}

// 16 consecutive columns of this thread's lane; the waits are inside.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 "
      "[%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
}

// the largest of three; a NaN among them is the result
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16 consecutive columns of this thread's lane; no wait (see tmem_wait_st).
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 "
      "[%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// two values as fp16 or bf16 pairs, the first in the low half
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return F16 ? pack_f16(a, b) : pack_bf16(a, b);
}

// four fp32 values as four E4M3 codes and what they leave over
__device__ __forceinline__ uint32_t e4m3x4_rest(float (&x)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t w = (lo & 0xffffu) | (hi << 16);
  const uint32_t h0 = e4m3_lo(w), h1 = e4m3_hi(w);
  const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  x[0] -= f0.x;
  x[1] -= f0.y;
  x[2] -= f1.x;
  x[3] -= f1.y;
  return w;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// One arrival by the lane with lead != 0, called by the whole warp: no branch, so the warp's lanes stay together for
// the tensor-memory accesses that follow
__device__ __forceinline__ void arrive_by(uint64_t* bar, bool lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead ? 1u : 0u)
      : "memory");
}

// Ask for the next CTA of the grid that has not started, to do its work here; the 16-byte
// answer lands in shared memory and completes on the barrier.
__device__ __forceinline__ void clc_ask(uint4* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}

// The answer: false when no CTA is left, else that CTA's grid index.
__device__ __forceinline__ bool clc_read(const uint4* answer, uint32_t& x, uint32_t& y) {
  uint32_t ok;
  [[maybe_unused]] uint32_t z;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 a, [%4];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %3, 1, 0, p;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, %2, _}, a;\n\t}"
      : "=r"(x), "=r"(y), "=r"(z), "=r"(ok)
      : "r"(smem_u32(answer))
      : "memory");
  return ok != 0;
}

// One box of a 3-D tensor into shared memory, issued by the leader of the calling warp
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2, uint32_t bar,
                                        uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "r"(leader)
      : "memory");
}

// One block's rows of a head, as two groups of eight rows x the 64-column halves
__device__ __forceinline__ void tma_block(uint32_t dst, const CUtensorMap* tm, int head, int group, uint32_t bar,
                                          uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%6, %6, %6, %2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(group), "r"(head), "r"(bar), "r"(leader), "r"(0)
      : "memory");
}

// 2^x by the hardware approximation, subnormal results flushed to zero
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A warp's 32 rows of 32-bit words, each row in its own thread, turned so that four lanes hold 16
// consecutive bytes each of one row and store 64 contiguous bytes together.  (Lanes storing their own
// rows touch 32 lines an instruction: 4100 cycles for a 256-row epilogue at D = 128.)  The turn goes
// through tensor memory: written a row a thread, 16 words at a time, read back with four lanes to a
// row's four columns.  No wait in put.
__device__ __forceinline__ void turn_put(uint32_t taddr, const uint32_t (&w)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 "
      "[%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(w[0]), "r"(w[4]), "r"(w[8]), "r"(w[12]), "r"(w[1]), "r"(w[5]), "r"(w[9]), "r"(w[13]), "r"(w[2]),
      "r"(w[6]), "r"(w[10]), "r"(w[14]), "r"(w[3]), "r"(w[7]), "r"(w[11]), "r"(w[15])
      : "memory");
}
// 32 words of rows lane / 4 and lane / 4 + 8 of the 16 from taddr's lane: v[8 c + 2 j + k], word
// 16 c + 4 (lane % 4) + j of row lane / 4 + 8 k
__device__ __forceinline__ void turn_get(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x128b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// A position in the ring and the parity of its round
template <int N>
struct Cursor {
  unsigned slot, phase;
  __device__ __forceinline__ void advance(unsigned k) {  // k < N
    slot += k;
    if (slot >= N) {
      slot -= N;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ void advance_by(unsigned k) {
    slot += k;
    phase ^= (slot / N) & 1;
    slot %= N;
  }
};

}  // namespace
}  // namespace pkv
