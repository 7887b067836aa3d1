// diff_chunk.cu -- differential attention of many rows over the same keys, on the fifth-generation tensor cores
// (tcgen05 MMAs accumulating in tensor memory): chunks of new tokens over the paged cache, and shared prefixes for
// all the sequences that have them.
//
// Mathematics.  For a row (token, output head) and the keys j < lim that it sees, under map m
//   o_m = sum_j 2^(x_j - r) V_j,  l_m = sum_j 2^(x_j - r),   x_j = scale log2(e) q_m . K_m,j,
// with a running reference r that moves only when a row's maximum passes it by more than 2^8, so that the
// accumulators are rescaled rarely; then  y = o_0 / l_0 - lam o_1 / l_1, its norm and the scale.  Statistics, both
// products, difference and norm are held in fp32.  Rounded to 16 bits are the weights alone, the A operand of the
// second product: bf16 for bf16 pools (half a step 2^-8), fp16 times 2^7 for E4M3 pools (2^-11; the factor keeps
// weights down to 2^-31 of the largest); in prefix passes as two such terms, hi + lo, but for E4M3 pools with a bf16
// output.  E4M3 pools: K enters as its codes, q as two E4M3 terms, hi + lo, after a power of two per row and map that
// takes its largest into [128, 256), exact for elements down to 2^-9 of the largest and off by at most 2^-17 of it
// below; V is expanded to fp16 (exact).
//
// Layout.  A work is 128 rows (128 / G tokens of the G heads of a pair) over one run of keys.  K's tile of 128 keys
// holds both maps' halves side by side, V's tile is the pair's value; each is loaded once for both maps.  The two
// softmax groups are the two maps of the same rows: while one map's softmax runs, the tensor cores work on the
// other's products.  So a row's two outputs lie in the same tensor-memory lane, and its end needs no more
// than two exchanges between two threads.
//
//   warps 0-3, 4-7  softmax of map 0 and 1: thread r owns row r (TMEM lane r): scores in, weights out over them as
//                   16-bit pairs, rare rescale of the output, epilogue (each group 64 columns of both outputs)
//   warps 8, 10     issue the MMAs of map 0 and 1, in turns: per step P V, then the next scores
//   warp 9          finds the work and passes it on; TMA of Q, K and V, a 16-token block at a time
//   warp 11         looks for bad ranges
//   warps 12-15     V: zero the rows past the context in the last tile, so that what a page holds there (NaN
//                   included) meets weight 0 as 0; E4M3: expand V to fp16
// A value of V that is not finite at a position some rows see and others do not would reach the latter as 0 * NaN;
// in the tiles where the mask cuts, such values are taken out of the tile, and added to the rows that see them in
// the epilogue.  A CTA stays: when its work is done it takes the next that no CTA has started (cluster launch
// control), so that Q, K, V and the first scores of the next work come in under the softmax and the epilogue of
// the last.
//
// Shared memory: Q (both halves; E4M3 hi and lo), a ring of K and V tiles in the order K0 K1 V0 K2 V1 .., E4M3 two
// fp16 V tiles.  TMEM (512 columns): scores, then weights, of map m at 128 m; outputs at 256 + 128 m.
//
// What bounds it.  A step of 128 keys is 1536 cycles of products for both maps and takes 2250 (2500 traced): the
// chain of a map, scores -> weights -> products, is 1250 cycles of softmax (220 to load the scores, 650 for the
// first 32 weights beside the maximum, 380 to the first half's arrival) and about 1000 from there to the next
// scores, and the other map covers as much of it as the turns allow.  Exponentials left out: 6 % less; softmax left
// out: 1.65 ms of 2.09, the measured cuBLAS rate.  4096 tokens over 32,768, 64 + 16 heads, bf16: 2.11 to 2.14 ms =
// 1.45 PFLOP/s, 76 % of the measured burst rate and 84 % of the sustained one (the power limit holds the clock at
// 1.9 GHz).  Nine prompts of 257 to 2048 tokens: 202 us = 0.96 PFLOP/s: 6.4 steps a work, and 6000 cycles of start,
// join, norm and store.  24 x 3 to 8 tokens over 1800 to 12,000, split: 136 us, 67 % of the copy rate: a step's
// chain takes as long for 32 rows as for 128.  E4M3, 4 x 700 to 1100 over 3000 to 9000, 128 + 16 heads: 0.90 ms =
// 1.2 PFLOP/s.  A prefix of 2048 tokens for 256 sequences: 42 us alone, 16 steps (29 us with one weight term).
//   Measured and left out: one issuing warp for both maps (2256 us against 2092 for the long chunk); half steps of 64
// keys in two score buffers a map, so that scores do not wait for weights (2363; products of 64 keys and every
// change between operand forms cost about 100 cycles a piece, 3060 when pieces of the two are interleaved); the
// weights of a step checked against the reference in two halves (2160); no turns (2430); a row's 64 columns of the
// output kept in registers through the epilogue (2250: spills in the softmax).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>

#include "diff.cuh"
#include "mma_ops.cuh"
#include "pkv_device.cuh"
#include "prefill_ops.cuh"
#include "prompt.cuh"
#include "tc_ops.cuh"

namespace pkv {

template <bool FP8>
struct DiffChunkCfg {
  static constexpr int kRows = 128, kKeys = 128;
  static constexpr int kStepBlocks = kKeys / kBlockSize;
  static constexpr int kHalf16 = 128 * 128;     // 64 columns of 128 16-bit rows
  static constexpr int kTile16 = 2 * kHalf16;   // a 16-bit tile of 128 rows
  static constexpr int kCodes = 128 * kDiffW;   // an E4M3 tile of 128 rows
  // bf16 K and V tiles: groups of eight keys, each group's halves side by side (one TMA box a block)
  static constexpr int kGroup = 2048;
  static constexpr int kQTile = FP8 ? 2 * kCodes : kTile16;
  static constexpr int kSlot = FP8 ? kCodes : kTile16;
  static constexpr int kSlots = FP8 ? 6 : 5;
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = kQTile;
  static constexpr int kOffExp = kOffRing + kSlots * kSlot;
  static constexpr int kOffBar = kOffExp + (FP8 ? 2 * kTile16 : 0);
  static constexpr int kBarBytes = 640;
  static constexpr int kOffJoin = kOffBar + kBarBytes;      // float[2][2][128]: factors, then squares
  static constexpr int kOffWeight = kOffJoin + 2048;        // float[128]: norm weights
  static constexpr int kOffPoison = kOffWeight + 512;       // int[kinds][128]
  static constexpr int kKinds = FP8 ? 1 : 3;                // NaN, +inf, -inf (E4M3 has no infinity)
  static constexpr int kBytes = 1008 + kOffPoison + kKinds * kDiffW * 4;  // 1008: alignment slack
  static constexpr int kColS = 0, kColO = 256, kTmemCols = 512;
  static constexpr int kIssuerWarp = 8, kProducerWarp = 9, kIssuer2Warp = 10, kRangeWarp = 11;
  static constexpr int kFixWarp0 = 12, kFixWarps = 4;
  static constexpr int kThreads = (kFixWarp0 + kFixWarps) * 32;
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;  // per thread
  static constexpr float kLazy = 8.f;
  static constexpr float kBias = FP8 ? kPrefillWeightBias : 0.f;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

namespace {

// barriers and small shared state, at kOffBar
struct DiffShared {
  uint64_t full[6], empty[6];  // ring: tile landed, tile consumed
  uint64_t s_full[2];          // scores of a step done (and every product issued before)
  uint64_t p_half[2];          // weights of a step's first 64 keys written, the output rescaled (an arrival per warp),
                               // and the other map's turn over
  uint64_t p_full[2];          // all weights of a step written (an arrival per warp)
  uint64_t o_full[2];          // every product of the map's work done
  uint64_t fixed[8];           // bf16: V tile of a cut step fixed; E4M3 (two in use): V tile expanded
  uint64_t exp_free[2];        // E4M3: expanded V tile consumed
  uint64_t v_sent[8];          // load of a V tile that warps 12-15 work on issued
  uint64_t q_full, q_empty;
  uint64_t work_full[2], work_empty[2];
  uint64_t clc;                // answer of the work query landed
  uint64_t drain[2];           // every MMA that an issuer has issued done
  alignas(16) uint4 clc_answer;
  int4 work[2][2];
  uint32_t tmem;
  int abort;
  int poisoned;  // 1 + number of the work whose V held values that are not finite
  uint16_t epilogues[8];  // of every softmax warp: works with steps that it is through with
};
static_assert(sizeof(DiffShared) <= DiffChunkCfg<true>::kBarBytes, "shared state");

// One CTA's worth of work, and what every role derives from it
struct DiffWork {
  int tok0;   // first token (row of q; prefix pass: place among the members)
  int ntok;   // its tokens
  int seq;    // sequence (prefix)
  int ctx;    // cached tokens
  int shift;  // causal: the work's token i sees keys < shift + i + 1
  int h, split;
};

struct DiffSteps {
  int k0, nstep;  // first 128-key step, steps
  int lim_min;    // keys that every row sees
  int first_cut;  // first step whose V needs care: some row does not see all of its keys
  __device__ __forceinline__ static int lim(const DiffWork& w, const DiffParams& p, int i) {
    return p.causal ? max(0, min(w.ctx, w.shift + i + 1)) : w.ctx;
  }
  __device__ __forceinline__ DiffSteps(const DiffWork& w, const DiffParams& p) {
    k0 = w.split * p.split_tiles;
    nstep = max(0, min((lim(w, p, w.ntok - 1) + 127) / 128, k0 + p.split_tiles) - k0);
    lim_min = lim(w, p, 0);
    first_cut = max(0, min(nstep, lim_min / 128 - k0));
  }
  // position of V of step j in the ring's order K0 K1 V0 K2 V1 ..
  __device__ __forceinline__ int v_item(int j) const { return min(2 * j + 2, 2 * nstep - 1); }
};

}  // namespace

template <bool FP8, DiffForm FORM>
__global__ void __launch_bounds__((DiffChunkCfg<FP8>::kThreads), 1)
    diff_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const DiffParams p) {
  using C = DiffChunkCfg<FP8>;
  constexpr int W = kDiffW;
  constexpr bool RECORDS = FORM != kDiffChunk, PREFIX = FORM == kDiffPrefix || FORM == kDiffPrefixFine;
  constexpr bool FINE = FORM == kDiffPrefixFine;  // weights in two terms
  // registers of a softmax thread (176: spills, the long chunk 2190 us against 2090; weights in two terms want 192:
  // prefix passes 2 to 4 % faster than with 184), and what that leaves of the launch's for another
  constexpr int kSoftRegs = FINE ? 192 : 184;
  constexpr int kAuxRegs = (C::kLaunchRegs * C::kThreads - kSoftRegs * 256) / (C::kThreads - 256) / 8 * 8;
  static_assert(kSoftRegs * 256 + kAuxRegs * (C::kThreads - 256) <= C::kLaunchRegs * C::kThreads, "register split");
  constexpr bool kQByThreads = FP8 || PREFIX;  // Q written by the softmax threads: converted, or gathered
  constexpr unsigned NS = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DiffShared& sh = *reinterpret_cast<DiffShared*>(smem + C::kOffBar);
  volatile int* abort = &sh.abort;
  volatile int* poisoned = &sh.poisoned;
  int* poison = reinterpret_cast<int*>(smem + C::kOffPoison);  // [kinds][128] first key with such a value

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group, log_g = 31 - __clz(G);  // a power of two
  const int cta_tok = C::kRows >> log_g;         // tokens of a work
  const int ranges_end = PREFIX ? p.num_members : p.rows;  // where the ranges of q_indptr end at most

  if (warp == 0) {
    __syncwarp();
    tmem_alloc(smem_u32(&sh.tmem), C::kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == C::kIssuerWarp * 32) {
    for (unsigned i = 0; i < 6; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 2);  // (both issuers; an expanded V tile's slot: twice by the warps that expand)
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&sh.fixed[i], 1);
      mbar_init(&sh.v_sent[i], 1);
      sh.epilogues[i] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_half[i], 5);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.exp_free[i], 2);
      mbar_init(&sh.work_full[i], 1);
      mbar_init(&sh.work_empty[i], 2 + C::kFixWarps + 8);  // one arrival per warp that reads it
    }
    mbar_init(&sh.q_full, kQByThreads ? 8 : 1);
    mbar_init(&sh.q_empty, 2);
    mbar_init(&sh.clc, 1);
    mbar_init(&sh.drain[0], 1);
    mbar_init(&sh.drain[1], 1);
    sh.abort = 0;
    sh.poisoned = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == C::kProducerWarp * 32) {
    if (!kQByThreads) tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  for (int i = threadIdx.x; i < C::kKinds * W; i += C::kThreads) poison[i] = 0x7fffffff;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);
  pdl_wait();  // nothing above touches global memory
  pdl_launch_dependents();

  const uint32_t q_base = smem_u32(smem + C::kOffQ);
  const uint32_t ring = smem_u32(smem + C::kOffRing);
  auto fail = [&]() { give_up(p.status, abort); };
  // the work number n (all roles see the same sequence); false: there is none left, or abort
  auto next_work = [&](unsigned n, DiffWork& w) -> bool {
    const bool ok = wait_for(&sh.work_full[n & 1], (n >> 1) & 1, abort, p.wait_tries);
    if (!__all_sync(kFull, ok)) {
      if (!*abort) fail();
      return false;
    }
    const int4 a = sh.work[n & 1][0], b = sh.work[n & 1][1];
    w = DiffWork{a.x, a.y, a.z, a.w, b.x, b.y, b.z};
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.work_empty[n & 1]);
    return w.seq >= 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAuxRegs));
    if (warp == C::kIssuerWarp || warp == C::kIssuer2Warp) {
      // ======================================================================== MMA issuers, one a map
      const int g = warp == C::kIssuerWarp ? 0 : 1;
      const uint32_t leader = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, wait_for(bar, parity, abort)); };
      auto same = [](uint32_t x) { return __shfl_sync(kFull, x, 0); };  // a value of the warp
      constexpr uint32_t kIdO = idesc_f16(C::kRows, W, !FP8, true);
      // scores: A = Q with its sign turned (bit 13) for a negative scale; E4M3 formats are 0
      const uint32_t id_s = idesc_f16(C::kRows, C::kKeys, !FP8, false) | (p.negate ? 1u << 13 : 0u);
      const uint32_t ring_lo = same(desc_lo(ring, 16)), ring_v_lo = same(desc_lo(ring, 1024));
      const uint32_t exp_v_lo = same(desc_lo(smem_u32(smem + C::kOffExp), C::kHalf16));
      // this map's half of Q's and K's columns
      const uint32_t q_lo = same(desc_lo(q_base, 16) + g * (FP8 ? 64 : C::kHalf16) / 16);
      const uint32_t k0_lo = same(ring_lo + g * (FP8 ? 64 : 1024) / 16);
      const uint32_t s_col = same(tmem + C::kColS + 128 * g), o_col = same(tmem + C::kColO + W * g);
      auto issue_s = [&](unsigned slot) {
        const uint32_t k_lo = same(k0_lo + slot * (C::kSlot / 16));
        if constexpr (FP8) {
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
              mma_ss<true>(s_col, q_lo + (part * C::kCodes + kk * 32) / 16, k_lo + kk * 2, kDescK128, kDescK128, id_s,
                           part > 0 || kk > 0, leader);
        } else {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss<false>(s_col, q_lo + kk * 2, k_lo + kk * 2, kDescK128, kDesc128<C::kGroup>, id_s, kk > 0, leader);
        }
        commit(&sh.s_full[g], leader);
      };
      // keys 64 half .. of a step
      auto issue_o = [&](int half, bool first, uint32_t v_lo) {
        constexpr uint32_t kVGroup = FP8 ? 1024 : C::kGroup;  // eight keys
#pragma unroll
        for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {
          mma_ts(o_col, s_col + 8 * kk, v_lo + kk * (2 * kVGroup / 16), kDesc128<kVGroup>, kIdO, !first || kk > 0, leader);
          if constexpr (FINE)
            mma_ts(o_col, s_col + 64 + 8 * kk, v_lo + kk * (2 * kVGroup / 16), kDesc128<kVGroup>, kIdO, true, leader);
        }
      };

      Cursor<C::kSlots> base{0, 0};  // ring position of the work's first tile
      unsigned steps_done = 0, cuts = 0, q_count = 0;
      bool ok = true;
      DiffWork w;
      for (unsigned n = 0; ok && next_work(n, w); ++n) {
        const DiffSteps st(w, p);
        const int nstep = st.nstep;
        if (nstep == 0) continue;
        Cursor<C::kSlots> kc = base, vc = base;
        vc.advance(nstep == 1 ? 1 : 2);
        auto wait_k = [&]() { return wait(&sh.full[kc.slot], kc.phase); };
        // V of step j is ready for the tensor cores
        auto wait_v = [&](int j) {
          if constexpr (FP8) {
            const unsigned v = steps_done + j;
            return wait(&sh.fixed[v & 1], (v >> 1) & 1);
          } else {
            if (j >= st.first_cut) {
              const unsigned c = cuts + j - st.first_cut;
              return wait(&sh.fixed[c & 7], (c >> 3) & 1);
            }
            return wait(&sh.full[vc.slot], vc.phase);
          }
        };
        // The maps take turns, so that one's products run under the other's softmax.  The fifth arrival on p_half is
        // the other issuer's, once its turn before is over: on map 0's for a work's first step when issuer 1 is
        // through with the work before, then after map 1's step before; on map 1's after map 0's same step.  So no
        // arrival comes before the phase it belongs to.
        if (g == 1 && leader) mbar_arrive(&sh.p_half[0]);
        ok = wait(&sh.q_full, q_count & 1);
        ++q_count;
        ok = ok && wait_k();
        if (!ok) break;
        tc_fence_after();
        issue_s(kc.slot);
        commit(&sh.empty[kc.slot], leader);
        if (nstep == 1) commit(&sh.q_empty, leader);
        for (int j = 0; j < nstep; ++j) {
          const bool more = j + 1 < nstep;
          const unsigned parity = (steps_done + j) & 1;
          ok = wait_v(j);
          if (more) kc.advance(j == 0 ? 1 : 2);
          if (!FP8 && more && ok) ok = wait_k();  // before the weights, where waiting costs nothing
          if (!ok) break;
          const uint32_t v_lo = same(FP8 ? exp_v_lo + ((steps_done + j) & 1) * (C::kTile16 / 16)
                                         : ring_v_lo + vc.slot * (C::kSlot / 16));
          ok = wait(&sh.p_half[g], parity);
          if (!ok) break;
          tc_fence_after();
          issue_o(0, j == 0, v_lo);
          ok = wait(&sh.p_full[g], parity);
          if (!ok) break;
          tc_fence_after();
          issue_o(1, false, v_lo);
          if (FP8 && more) {  // K may come later than the weights: V's expansion holds up the ring
            ok = wait_k();
            if (!ok) break;
            tc_fence_after();
          }
          // the next scores follow P V in the same columns, in issue order
          if (more) issue_s(kc.slot);
          else commit(&sh.o_full[g], leader);
          if ((g == 0 || more) && leader) mbar_arrive(&sh.p_half[g ^ 1]);
          commit(FP8 ? &sh.exp_free[(steps_done + j) & 1] : &sh.empty[vc.slot], leader);
          vc.advance(j + 2 == nstep ? 1 : 2);
          if (more) commit(&sh.empty[kc.slot], leader);
          if (j + 2 == nstep) commit(&sh.q_empty, leader);
        }
        base.advance_by(2 * nstep);
        steps_done += nstep;
        cuts += nstep - st.first_cut;
      }
      if (!ok && !*abort && lane == 0) fail();
      // nothing may run on the tensor cores when the CTA frees its tensor memory
      commit(&sh.drain[g], leader);
      mbar_wait(&sh.drain[g], 0);
      __syncwarp();
    } else if (warp == C::kProducerWarp) {
      // ======================================================================== work and TMA producer
      const uint32_t leader = elect_one();
      auto load = [&](const CUtensorMap* tm, unsigned item, int head, int row, int from) {
        const unsigned st = __shfl_sync(kFull, item % NS, 0);
        const uint32_t bar = smem_u32(&sh.full[st]), dst = ring + st * C::kSlot;
        if (leader) mbar_arrive_expect_tx(&sh.full[st], C::kSlot);
        __syncwarp();
#pragma unroll(FP8 ? 2 : C::kStepBlocks)
        for (int blk = 0; blk < C::kStepBlocks; ++blk) {
          const int r = __shfl_sync(kFull, row, from + blk);
          if constexpr (FP8) tma_box(dst + blk * kBlockSize * W, tm, 0, head, r, bar, leader);
          else tma_block(dst + blk * 2 * C::kGroup, tm, head, r >> 3, bar, leader);
        }
      };
      auto slot_free = [&](unsigned item) {
        const bool ok = item < NS || wait_for(&sh.empty[item % NS], ((item / NS) - 1) & 1, abort);
        return __all_sync(kFull, ok);
      };
      // the tokens of the work at (x, y) of the grid: tile slots count the sequences' tiles in order, each
      // sequence's longest (last) tile first.  seq < 0: a slot past the last tile
      auto find = [&](unsigned x, unsigned y) {
        DiffWork w{0, 0, -1, 0, 0, static_cast<int>(x % p.pairs), static_cast<int>(y)};
        const int slot = x / p.pairs;
        int before = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
          const int b = b0 + lane;
          int first = 0, n = 0, len = 0;
          if (b < p.batch) {
            first = p.q_indptr[b];
            const int last = p.q_indptr[b + 1];
            len = p.context_lens[b];
            n = last - first;
            if (first < 0 || last < first || last > ranges_end || (PREFIX && n > p.max_members)) {
              set_flag(p.status, PKV_DEVFLAG_BAD_INDPTR);
              n = 0;
            }
          }
          const int tiles = (n + cta_tok - 1) / cta_tok;
          int upto = tiles;
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) {
            const int v = __shfl_up_sync(kFull, upto, m);
            if (lane >= m) upto += v;
          }
          const unsigned hit = __ballot_sync(kFull, slot < before + upto);
          if (hit) {
            const int src = __ffs(hit) - 1;
            const int tile = __shfl_sync(kFull, before + upto - 1 - slot, src);  // tiles after this one
            first = __shfl_sync(kFull, first, src);
            n = __shfl_sync(kFull, n, src);
            w.seq = b0 + src;
            int ctx = __shfl_sync(kFull, len, src);
            const int cap = p.max_context_len;  // within the tables (checked on the host, in 64 bits)
            if (ctx < 0 || ctx > cap) {
              set_flag(p.status, PKV_DEVFLAG_BAD_CONTEXT_LEN);
              ctx = max(0, min(ctx, cap));
            }
            w.ctx = ctx;
            w.tok0 = first + tile * cta_tok;
            w.ntok = min(cta_tok, n - tile * cta_tok);
            w.shift = ctx - n + tile * cta_tok;
            break;
          }
          before += __shfl_sync(kFull, upto, 31);
        }
        return w;
      };

      unsigned n = 0, base = 0, steps_done = 0, cuts = 0, q_count = 0, asked = 0;
      uint32_t gx = blockIdx.x, gy = blockIdx.y;
      bool more = true, ok = true;
      while (more && ok) {
        const DiffWork w = find(gx, gy);
        if (lane == 0) clc_ask(&sh.clc_answer, &sh.clc);
        if (w.seq >= 0) {
          const DiffSteps st(w, p);
          const int nstep = st.nstep;
          const int32_t* table = p.block_tables + static_cast<int64_t>(w.seq) * p.max_blocks;
          const int nblk = (w.ctx + kBlockSize - 1) / kBlockSize;
          // ids of the blocks of four steps, one a lane, asked for four steps ahead of their use; a block past
          // the context, or with an id outside the pool, becomes a box entirely outside the tensor (zeros)
          auto ids_of = [&](int j) {
            const int at = (st.k0 + j) * C::kStepBlocks + lane;
            return j + lane / C::kStepBlocks < nstep && at < nblk ? __ldcg(table + at) : INT_MIN;
          };
          auto row_of = [&](int id) {
            if (id >= 0 && id < p.num_blocks) return id * kBlockSize;
            if (id != INT_MIN) set_flag(p.status, PKV_DEVFLAG_BAD_BLOCK_ID);
            return -kBlockSize;
          };
          const int ids0 = ids_of(0);
          int ids1 = ids_of(4);
          ok = n < 2 || wait_for(&sh.work_empty[n & 1], ((n >> 1) - 1) & 1, abort);
          ok = __all_sync(kFull, ok);
          if (ok) {
            if (p.test_post_delay_cycles > 0) spin_cycles(p.test_post_delay_cycles);
            if (lane == 0) {
              sh.work[n & 1][0] = make_int4(w.tok0, w.ntok, w.seq, w.ctx);
              sh.work[n & 1][1] = make_int4(w.shift, w.h, w.split, 0);
              mbar_arrive(&sh.work_full[n & 1]);
            }
            ++n;
          }
          if (ok && nstep > 0) {
            if constexpr (!kQByThreads) {
              // Q's tile is free once the last scores of the work before are done
              if (q_count > 0) ok = wait_for(&sh.q_empty, (q_count - 1) & 1, abort);
              ok = __all_sync(kFull, ok);
              if (ok && leader) {
                mbar_arrive_expect_tx(&sh.q_full, C::kQTile);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  tma_load_3d(smem + C::kOffQ + c * C::kHalf16, &tm_q, c * 64, w.h * G, w.tok0, &sh.q_full);
              }
              if (ok) ++q_count;
            }
            int rows_k = row_of(ids0), rows_v = rows_k;
            // tiles in the ring's order: K of step 0, then K of step j + 1 and V of step j in turns
            unsigned issued = base;
            int j = 0;
            bool is_v = false;
#pragma unroll 1
            for (int i = 0; i < 2 * nstep && ok; ++i) {
              ok = slot_free(base + i);
              if (!ok) break;
              const int step = is_v || i == 0 ? j : j + 1;
              if (!is_v && i > 0 && (step & 3) == 0) {
                rows_k = row_of(ids1);
                ids1 = ids_of(step + 4);
              }
              if (is_v && (step & 3) == 0) rows_v = rows_k;
              load(is_v ? &tm_v : &tm_k, base + i, w.h, is_v ? rows_v : rows_k, (step & 3) * C::kStepBlocks);
              issued = base + i + 1;
              if (is_v) {
                if (lane == 0 && (FP8 || j >= st.first_cut))
                  mbar_arrive(&sh.v_sent[(FP8 ? steps_done + j : cuts + j - st.first_cut) & 7]);
                ++j;
                is_v = j + 1 >= nstep;
              } else {
                is_v = i > 0 || nstep == 1;
              }
            }
            base = ok ? base + 2 * nstep : issued;
            steps_done += nstep;
            cuts += nstep - st.first_cut;
          }
        }
        // the next work: the answer is always taken, so that none is in flight at the end
        const bool told = mbar_wait(&sh.clc, asked & 1);
        ++asked;
        ok = __all_sync(kFull, told) && ok;
        more = told && clc_read(&sh.clc_answer, gx, gy);
        fence_proxy_async_smem();  // read before the next answer is written
        __syncwarp();
      }
      // no work left: tell the other roles
      if (ok) {
        ok = n < 2 || wait_for(&sh.work_empty[n & 1], ((n >> 1) - 1) & 1, abort);
        if (ok && lane == 0) {
          sh.work[n & 1][0] = make_int4(0, 0, -1, 0);
          sh.work[n & 1][1] = make_int4(0, 0, 0, 0);
          mbar_arrive(&sh.work_full[n & 1]);
        }
      }
      if (lane == 0) {
        if (!ok && !*abort) fail();
        // nothing may be in flight when the CTA exits: the last tiles issued have landed
        for (unsigned i = base > NS ? base - NS : 0; i < base; ++i)
          if (!mbar_wait(&sh.full[i % NS], (i / NS) & 1)) break;
        if (!kQByThreads && q_count > 0) mbar_wait(&sh.q_full, (q_count - 1) & 1);
      }
      __syncwarp();
    } else if (warp == C::kRangeWarp) {
      // bad ranges (whoever finds work stops at the sequence it belongs to); in every CTA that starts: any CTA's
      // start may be cancelled, the first one's too
      for (int b = lane; b < p.batch; b += 32) {
        const int first = p.q_indptr[b], last = p.q_indptr[b + 1];
        if (first < 0 || last < first || last > ranges_end || (PREFIX && last - first > p.max_members))
          set_flag(p.status, PKV_DEVFLAG_BAD_INDPTR);
      }
    } else if (warp >= C::kFixWarp0) {
      // ======================================================================== V: cut tiles, expansion
      constexpr int kFix = C::kFixWarps * 32;
      const int ft = threadIdx.x - C::kFixWarp0 * 32;
      unsigned number = 0;
      auto note = [&](int kind, int dim, int key) {
        atomicMin(&poison[kind * W + dim], key);
        *poisoned = static_cast<int>(number) + 1;
      };
      constexpr int kChunks = W / 8;  // 8-element pieces of a row
      constexpr int kStep = kFix / kChunks;
      const int c = ft % kChunks, r0 = ft / kChunks;
      unsigned base = 0, steps_done = 0, cuts = 0, with_steps = 0;
      bool ok = true;
      DiffWork w;
      for (unsigned n = 0; ok; ++n) {
        // the warps leave together
        const bool none = !next_work(n, w);
        __syncwarp();
        if (named_sync_or(1, kFix, none)) break;
        number = n;
        const DiffSteps st(w, p);
        const int nstep = st.nstep;
        if (nstep == 0) continue;
        // before values that are not finite are listed: the works before are through their epilogues, and what
        // they left in the list is cleared
        bool cleared = false;
        auto clear = [&]() {
          cleared = true;
          // (a thread looks at one warp: sums over warps, some of them ahead, would not do)
          const volatile uint16_t* through = &sh.epilogues[ft & 7];
          const long long start = clock64();
          while (ok && static_cast<int16_t>(*through - with_steps) < 0) {
            if (*abort) ok = false;
            if (clock64() - start > kWaitLimitCycles) {
              ok = false;
              fail();
            }
          }
          __syncwarp();
          named_sync(3, kFix);
          for (int i = ft; i < C::kKinds * W; i += kFix) poison[i] = 0x7fffffff;
          __syncwarp();
          named_sync(3, kFix);
        };
        for (int j = FP8 ? 0 : st.first_cut; j < nstep; ++j) {
          const bool cut = j >= st.first_cut;
          const unsigned item = base + st.v_item(j);
          // the parity of `full` means this load only once it is issued (the slot's loads before it are not waited
          // for here); v_sent itself is never a phase ahead: eight V tiles on, the ring has come round
          const unsigned sent = FP8 ? steps_done + j : cuts + j - st.first_cut;
          if (ok) ok = wait_for(&sh.v_sent[sent & 7], (sent >> 3) & 1, abort);
          if (ok) ok = wait_for(&sh.full[item % NS], (item / NS) & 1, abort);
          if constexpr (FP8)
            if (ok && sent >= 2) ok = wait_for(&sh.exp_free[sent & 1], ((sent >> 1) - 1) & 1, abort);
          if (!ok && !*abort) fail();
          const int key0 = (st.k0 + j) * C::kKeys;
          // rows below seen: every row's; from end on: no row's
          const int seen = st.lim_min - key0, end = w.ctx - key0;
          uint8_t* src = smem + C::kOffRing + (item % NS) * C::kSlot;
          auto odd8 = [](uint32_t x) { return (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u; };   // E4M3 NaN
          auto odd16 = [](uint32_t x) { return (((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0u; };  // bf16
          const uint32_t ex = smem_u32(smem + C::kOffExp + (sent & 1) * C::kTile16) + (c >> 3) * C::kHalf16;
          auto at16 = [&](int row) {
            return reinterpret_cast<uint4*>(src + (row >> 3) * C::kGroup + (c >> 3) * 1024 + (row & 7) * 128 +
                                            (((c & 7) ^ (row & 7)) << 4));
          };
          auto expand = [&](int row, uint2 v) {
            st_shared_v4(ex + (row >> 3) * 1024 + (row & 7) * 128 + (((c & 7) ^ (row & 7)) << 4), e4m3_lo(v.x),
                         e4m3_hi(v.x), e4m3_lo(v.y), e4m3_hi(v.y));
          };
          // E4M3: expand the tile, four pieces in registers at a time; rows no row sees become zeros.  bf16: only
          // the rows that not every row sees.  odd: one of those that some row sees is not finite.
          constexpr int kBatch = 4;
          bool odd = false;
          if (ok) {
            if constexpr (FP8) {
              static_assert(C::kKeys % (kBatch * kStep) == 0, "whole batches");
#pragma unroll 1
              for (int b0 = r0; b0 < C::kKeys; b0 += kBatch * kStep) {
                uint2 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                  v[i] = *reinterpret_cast<const uint2*>(src + (b0 + i * kStep) * W + c * 8);
                if (cut) {
#pragma unroll
                  for (int i = 0; i < kBatch; ++i) {
                    const int row = b0 + i * kStep;
                    if (row >= end) v[i] = make_uint2(0u, 0u);
                    else if (row >= seen) odd |= odd8(v[i].x) || odd8(v[i].y);
                  }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) expand(b0 + i * kStep, v[i]);
              }
            } else {
#pragma unroll 1
              for (int b0 = max(0, seen) + r0; b0 < min(end, C::kKeys); b0 += kBatch * kStep) {
                uint4 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                  const int row = b0 + i * kStep;
                  v[i] = row < min(end, C::kKeys) ? *at16(row) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) odd |= odd16(v[i].x) || odd16(v[i].y) || odd16(v[i].z) || odd16(v[i].w);
              }
              for (int row = max(0, end) + r0; row < C::kKeys; row += kStep) *at16(row) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          __syncwarp();  // (rows are dealt by lane; the barriers are for whole warps)
          if (cut && named_sync_or(3, kFix, odd)) {  // rare: list them and take them out of the tile
            if (!cleared) clear();
            for (int row = max(0, seen) + r0; ok && row < min(end, C::kKeys); row += kStep) {
              if constexpr (FP8) {
                uint2 v = *reinterpret_cast<const uint2*>(src + row * W + c * 8);
                if (!odd8(v.x) && !odd8(v.y)) continue;
                uint32_t* word = reinterpret_cast<uint32_t*>(&v);
                for (int e = 0; e < 8; ++e)
                  if (((word[e >> 2] >> (8 * (e & 3))) & 0x7fu) == 0x7fu) {  // the only code that is not finite
                    note(0, c * 8 + e, key0 + row);
                    word[e >> 2] &= ~(0xffu << (8 * (e & 3)));
                  }
                expand(row, v);
              } else {
                uint4 v = *at16(row);
                uint32_t* word = reinterpret_cast<uint32_t*>(&v);
                for (int e = 0; e < 8; ++e) {
                  const uint32_t x = (word[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                  if ((x & 0x7f80u) == 0x7f80u) {
                    note((x & 0x7fu) ? 0 : (x & 0x8000u) ? 2 : 1, c * 8 + e, key0 + row);
                    word[e >> 1] &= (e & 1) ? 0x0000ffffu : 0xffff0000u;
                  }
                }
                *at16(row) = v;
              }
            }
          }
          fence_proxy_async_smem();  // the tile is read by the tensor cores
          __syncwarp();
          if (named_sync_or(1, kFix, *abort != 0)) {
            ok = false;
            break;
          }
          if (ft == 0) {
            if constexpr (FP8) {
              mbar_arrive_n(&sh.empty[item % NS], 2);  // what both issuers would arrive
              mbar_arrive(&sh.fixed[sent & 1]);
            } else {
              mbar_arrive(&sh.fixed[sent & 7]);
            }
          }
        }
        ++with_steps;
        base += 2 * nstep;
        steps_done += nstep;
        cuts += nstep - st.first_cut;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ======================================================================== softmax
    const int g = warp >> 2;           // the map
    const int r = threadIdx.x & 127;   // row of the tile, TMEM lane
    const int my_i = r >> log_g;       // token within the work
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t scol = tmem + lane_base + C::kColS + 128 * g;
    const uint32_t ocol = tmem + lane_base + C::kColO;  // map 0's output
    const uint32_t mine = ocol + W * g;
    float* join = reinterpret_cast<float*>(smem + C::kOffJoin);  // [factors, squares][group][row]
    float* norm_w = reinterpret_cast<float*>(smem + C::kOffWeight);
    if constexpr (!RECORDS) {
      if (g == 0) norm_w[r] = p.norm_weight != nullptr ? bf16_lo(p.norm_weight[r]) : 1.f;
      __syncwarp();
      named_sync(2, 256);
    }
    unsigned c_s = 0, c_o = 0;  // steps and works with steps so far
    bool dead = false;
    DiffWork w;
    for (unsigned n = 0; !dead; ++n) {
      // the groups meet at barriers below, so all eight warps take the work or none does (one that gave up just
      // before the work was passed on would leave the others waiting for it there)
      bool none = !next_work(n, w);
      if constexpr (!RECORDS) {
        __syncwarp();
        none = named_sync_or(2, 256, none);
      }
      if (none) break;
      const DiffSteps st(w, p);
      const int nstep = st.nstep;
      const int head = w.h * G + (r & (G - 1));
      bool rv = my_i < w.ntok;
      int row = w.tok0 + my_i;  // of q and the output
      if constexpr (PREFIX) {
        row = rv ? p.member_seqs[row] : 0;
        if (row < 0 || row >= p.rows) {
          set_flag(p.status, PKV_DEVFLAG_BAD_INDPTR);
          rv = false;
          row = 0;
        }
      }
      const int64_t unit = static_cast<int64_t>(row) * p.heads + head;
      const int64_t rec = static_cast<int64_t>(w.split * 2 + g) * p.rows * p.heads + unit;
      if (nstep == 0) {  // rows that see nothing (of this split)
        if (rv) {
          if constexpr (RECORDS) {
            p.part_ml[rec] = make_float2(-INFINITY, 0.f);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + unit * W + kDiffD * g);
#pragma unroll
            for (int c = 0; c < kDiffD / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        continue;
      }
      float sscale = p.score_size;
      // lambda, asked for long before its use
      float sign = 1.f;
      if (!RECORDS && g == 1 && rv) sign = -__ldg(p.lambda + row * p.lambda_stride + head);

      if constexpr (kQByThreads) {
        // this map's half of the row of Q; the tile is free: the map's last scores of the work before are done
        const uint4* qr = reinterpret_cast<const uint4*>(p.q + row * p.q_stride + static_cast<int64_t>(head) * W +
                                                         kDiffD * g);
        uint4 x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = rv ? qr[c] : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (FP8) {
          // as hi and lo codes, times 2^e that takes the half row's largest into [128, 256)
          float top = 0.f;
          bool odd = false;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t e[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              top = fmaxf(top, fmaxf(fabsf(bf16_lo(e[k])), fabsf(bf16_hi(e[k]))));
              odd |= ((((e[k] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0u);
            }
          }
          int ex = 0;
          if (top > 0.f && !odd) ex = 7 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
          ex = min(ex, 126);  // rows below 2^-119: their codes lose what lies under 2^-135
          const float k_scale = p.scales[2 * w.h + g];
          const float size = __uint_as_float(static_cast<uint32_t>(max(ex, -126) + 127) << 23);
          const float up = k_scale < 0.f ? -size : size;  // the scores' factor below stays positive
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 16 codes: one 16-byte piece of the row
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a = u4_word(x[2 * c + k / 2], 2 * (k & 1)), b = u4_word(x[2 * c + k / 2], 2 * (k & 1) + 1);
              float v[4] = {bf16_lo(a) * up, bf16_hi(a) * up, bf16_lo(b) * up, bf16_hi(b) * up};
              hi[k] = e4m3x4_rest(v);
              lo[k] = e4m3x4_rest(v);
            }
            const uint32_t at = q_base + r * 128 + (((4 * g + c) ^ (r & 7)) << 4);
            st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(at + C::kCodes, lo[0], lo[1], lo[2], lo[3]);
          }
          // the row's scores come out times 2^ex; a row with a NaN or an infinity has no value, unless it sees no
          // key: its scores are all masked, whatever they are
          // (a zero scale: a factor that leaves every score at 0 while masked ones stay -inf)
          sscale = (odd || k_scale != k_scale) && DiffSteps::lim(w, p, my_i) > 0
                       ? __int_as_float(0x7fffffff)
                       : fmaxf(sscale * fabsf(k_scale) / size, 1e-37f);
        } else {
          const uint32_t at = q_base + g * C::kHalf16 + r * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) st_shared_v4(at + ((c ^ (r & 7)) << 4), x[c].x, x[c].y, x[c].z, x[c].w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full);
      }

      const int my_lim = DiffSteps::lim(w, p, my_i);
      // keys below every lim of the warp's rows need no mask (rows that do not exist do not count)
      const int warp_lim = __reduce_min_sync(kFull, rv ? my_lim : 0x7fffffff);
      const bool idle = !__any_sync(kFull, rv);  // no row of the warp exists: its products go nowhere
      float m_used = -INFINITY, l = 0.f;
      for (int t = 0; t < nstep; ++t) {
        const int key0 = (st.k0 + t) * C::kKeys;
        const bool ok = wait_for(&sh.s_full[g], (c_s + t) & 1, abort, p.wait_tries);
        if (!__all_sync(kFull, ok)) {  // tensor-memory loads are warp-collective: leave as a warp
          if (!*abort) fail();
          dead = true;
          break;
        }
        tc_fence_after();
        if (!idle) {
          // keys that a row does not see: -inf over their scores, in the columns (a loop of 32: this is for a
          // work's last steps, and straight code for 128 is slow to fetch)
          if (key0 + C::kKeys > warp_lim) {
            const int left = my_lim - key0;
#pragma unroll 1
            for (int c = max(0, warp_lim - key0) & ~31; c < C::kKeys; c += 32) {
              float x[32];
              tmem_ld32(scol + c, x);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= left - c) x[i] = -INFINITY;
              tmem_st32(scol + c, x);
            }
          }
          float s[128];
          // (one load of 128 columns wants more registers than 512 threads start with)
          tmem_ld64(scol, *reinterpret_cast<float(*)[64]>(s));
          tmem_ld64(scol + 64, *reinterpret_cast<float(*)[64]>(s + 64));
          // 32 weights from their scores, as 16-bit pairs into the columns of the scores
          float2 sum[2] = {};
          uint32_t pw[16], pl[FINE ? 16 : 1];
          auto weights = [&](int q, float negm) {
            const float2 sc2 = make_float2(sscale, sscale), nm2 = make_float2(negm, negm);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 x = ffma2(make_float2(s[32 * q + 2 * i], s[32 * q + 2 * i + 1]), sc2, nm2);
              x.x = exp2_ftz(x.x);
              x.y = exp2_ftz(x.y);
              sum[i & 1] = fadd2(sum[i & 1], x);
              if constexpr (FINE) split16<FP8>(x.x, x.y, pw[i], pl[i]);
              else pw[i] = pack16<FP8>(x.x, x.y);
            }
          };
          auto put = [&](int q) {
            tmem_st16u(scol + 16 * q, pw);
            if constexpr (FINE) tmem_st16u(scol + 64 + 16 * q, pl);
          };
          // a row that has seen nothing yet keeps reference 0: its weights are 2^-inf = 0
          auto minus_m = [&]() { return (m_used == -INFINITY ? 0.f : -m_used) + C::kBias; };
          // the first weights by the reference as it stands, while the maximum is being found; it moves rarely,
          // and they are then taken again
          weights(0, minus_m());
          do {
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int i = 4; i < 124; i += 8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], s[i + 2 * k], s[i + 2 * k + 1]);
            }
            const float top =
                max3(max3(mx[0], mx[1], mx[2]), mx[3], max3(max3(s[124], s[125], s[125]), s[126], s[127])) * sscale;
            if (!(top < INFINITY)) l = __int_as_float(0x7fffffff);  // a NaN or an infinity among the scores
            const bool grow = top > m_used + C::kLazy;
            if (!__any_sync(kFull, grow)) break;
            float alpha = 1.f;
            if (grow) {
              alpha = fast_exp2(m_used - top);  // 0 while the row has seen nothing
              l *= alpha;
              m_used = top;
            }
            __syncwarp();
            if (t > 0) {  // P V of the previous step was issued before these scores: it is done
#pragma unroll 1
              for (int ch = 0; ch < W / 16; ++ch) {
                float o[16];
                tmem_ld16(mine + 16 * ch, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= alpha;
                tmem_st16(mine + 16 * ch, o);
              }
            }
            sum[0] = sum[1] = make_float2(0.f, 0.f);
            weights(0, minus_m());
          } while (false);
          const float negm = minus_m();
          put(0);
          weights(1, negm);
          put(1);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          arrive_by(&sh.p_half[g], lane == 0);
          weights(2, negm);
          put(2);
          weights(3, negm);
          put(3);
          sum[0] = fadd2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
          tmem_wait_st();
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_half[g]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[g]);
      }
      c_s += nstep;

      // ---- epilogue: the map's record, or the output row
      if (!dead) {
        const bool ok = wait_for(&sh.o_full[g], c_o & 1, abort);
        if (!__all_sync(kFull, ok)) {
          if (!*abort) fail();
          dead = true;
        }
        ++c_o;
        tc_fence_after();
      }
      // rare: values of V that were taken out of the cut tiles are added to the outputs of the rows that see them
      auto add_odd = [&](int map, int dim0, int dim1) {
        if (*poisoned != static_cast<int>(n) + 1) return;
#pragma unroll 1
        for (int dim = dim0; dim < dim1; ++dim) {
          const bool nan = poison[dim] < my_lim, up = !FP8 && poison[(C::kKinds - 2) * W + dim] < my_lim,
                     down = !FP8 && poison[(C::kKinds - 1) * W + dim] < my_lim;
          const float add = nan || (up && down) ? __int_as_float(0x7fffffff) : up ? INFINITY : down ? -INFINITY : 0.f;
          if (!__any_sync(kFull, add != 0.f)) continue;
          uint32_t v;
          const uint32_t at = ocol + W * map + dim;
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                       : "=r"(v)
                       : "r"(at)
                       : "memory");
          v = __float_as_uint(__uint_as_float(v) + add);
          asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(at),
                       "r"(v)
                       : "memory");
        }
      };
      if constexpr (RECORDS) {
        if (!dead && !idle) {
          // (keys, but none of a score above -inf: kDiffNothing, not the -inf of a run without keys)
          const bool nothing = l == 0.f && my_lim > st.k0 * C::kKeys;
          if (rv) p.part_ml[rec] = make_float2(nothing ? kDiffNothing : m_used - C::kBias, l);
          __syncwarp();
          add_odd(g, 0, W);
          // turned, through the columns that are read, so that four lanes store 64 bytes of a row together (lanes
          // storing their own rows touch 32 lines an instruction)
#pragma unroll 1
          for (int col = 0; col < W; col += 32) {
            float o[32];
            tmem_ld32(mine + col, o);
            uint32_t words[16];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int i = 0; i < 16; ++i) words[i] = __float_as_uint(o[16 * c + i]);
              turn_put(mine + col + 16 * c, words);
            }
            tmem_wait_st();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t v[16];
              turn_get(mine + col + (static_cast<uint32_t>(16 * half) << 16), v);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int src = 16 * half + 8 * k + (lane >> 2);
                const int64_t to = __shfl_sync(kFull, rv ? rec : -1, src);
                if (to >= 0) {
                  uint4* dst = reinterpret_cast<uint4*>(p.part_acc + to * W + col) + (lane & 3);
                  dst[0] = make_uint4(v[k], v[2 + k], v[4 + k], v[6 + k]);
                  dst[4] = make_uint4(v[8 + k], v[10 + k], v[12 + k], v[14 + k]);
                }
                __syncwarp();
              }
            }
          }
        }
      } else {
        // this map's factor; then each group has both outputs' 64 columns of one value head
        // (a row without keys: 0; one of nothing but scores of -inf under this map: 0 / 0)
        const bool empty = !rv || my_lim <= 0;
        join[g * 128 + r] = empty ? 0.f : sign / l;
        tc_fence_before();
        __syncwarp();
        dead = named_sync_or(2, 256, dead);
        tc_fence_after();
        const int col0 = kDiffD * g;
        if (!dead && !idle) {
          add_odd(0, col0, col0 + kDiffD);
          add_odd(1, col0, col0 + kDiffD);
          float a0 = join[r], a1 = join[128 + r];
          if constexpr (FP8) {
            const float vs = p.scales[2 * (p.pairs + w.h) + g];
            a0 *= vs;
            a1 *= vs;
          }
          float2 square = make_float2(0.f, 0.f);
          const float2 f0 = make_float2(a0, a0), f1 = make_float2(a1, a1);
#pragma unroll 1
          for (int c = col0; c < col0 + kDiffD; c += 32) {  // the difference goes over this map's columns
            float y[32], o[32];
            tmem_ld32(ocol + c, y);
            tmem_ld32(ocol + W + c, o);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 d = ffma2(make_float2(y[i], y[i + 1]), f0, fmul2(make_float2(o[i], o[i + 1]), f1));
              square = ffma2(d, d, square);
              y[i] = d.x;
              y[i + 1] = d.y;
            }
            tmem_st32(mine + c, y);
          }
          join[256 + g * 128 + r] = square.x + square.y;
        }
        tc_fence_before();
        __syncwarp();
        named_sync(2, 256);  // the squares are there, and both groups are through with both outputs
        tc_fence_after();
        if (!dead && !idle) {
          float by = p.out_scale;
          if (p.norm_weight != nullptr) by *= rsqrtf((join[256 + r] + join[384 + r]) * (1.f / W) + p.eps);
          if (empty) by = 0.f;  // (eps may be 0)
          // rounded, turned (through columns of this map's that are read) and stored
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float y[32];
            tmem_ld32(mine + col0 + 32 * c, y);
            uint32_t words[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float4 nw = *reinterpret_cast<const float4*>(norm_w + col0 + 32 * c + 2 * i);
              words[i] = pack_bf16(y[2 * i] * by * nw.x, y[2 * i + 1] * by * nw.y);
              words[i + 1] = pack_bf16(y[2 * i + 2] * by * nw.z, y[2 * i + 3] * by * nw.w);
            }
            turn_put(mine + 16 * c, words);
          }
          tmem_wait_st();
          uint32_t v[2][16];
          turn_get(mine, v[0]);
          turn_get(mine + (16u << 16), v[1]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = (r & ~31) + 8 * k + (lane >> 2);
            const int i = rr >> log_g;
            const uint32_t* x = v[k >> 1] + (k & 1);
            const int64_t to = static_cast<int64_t>(w.tok0 + i) * p.heads + w.h * G + (rr & (G - 1));
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + to * W) + 8 * g + (lane & 3);
            if (i < w.ntok) {
              dst[0] = make_uint4(x[0], x[2], x[4], x[6]);
              dst[4] = make_uint4(x[8], x[10], x[12], x[14]);
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();  // (the list of values was read above; the output's stores need not have landed)
      if (lane == 0) ++*const_cast<volatile uint16_t*>(&sh.epilogues[warp]);
    }
  }

  // ======================================================================== teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <bool FP8, DiffForm FORM>
static cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p,
                          int tile_slots, int splits, cudaStream_t stream) {
  using C = DiffChunkCfg<FP8>;
  auto kern = diff_chunk_kernel<FP8, FORM>;
  static std::atomic<bool> configured[64] = {};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!configured[device].load(std::memory_order_acquire)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes)) != cudaSuccess)
      return e;
    configured[device].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tile_slots) * static_cast<unsigned>(p.pairs), static_cast<unsigned>(splits), 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p);
}

template <bool FP8>
static cudaError_t launch_form(DiffForm form, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const DiffParams& p, int tile_slots, int splits, cudaStream_t stream) {
  switch (form) {
    case kDiffChunk: return launch<FP8, kDiffChunk>(tq, tk, tv, p, tile_slots, splits, stream);
    case kDiffChunkSplit: return launch<FP8, kDiffChunkSplit>(tq, tk, tv, p, tile_slots, splits, stream);
    case kDiffPrefixFine: return launch<FP8, kDiffPrefixFine>(tq, tk, tv, p, tile_slots, splits, stream);
    case kDiffPrefix:
      if constexpr (FP8) return launch<FP8, kDiffPrefix>(tq, tk, tv, p, tile_slots, splits, stream);
      break;
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_diff_chunk(bool fp8, DiffForm form, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const DiffParams& p, int tile_slots, int splits,
                              cudaStream_t stream) {
  return fp8 ? launch_form<true>(form, tq, tk, tv, p, tile_slots, splits, stream)
             : launch_form<false>(form, tq, tk, tv, p, tile_slots, splits, stream);
}

}  // namespace pkv
