// prefill_tc.cu -- attention of a chunk of new tokens over the paged cache, on the
// fifth-generation tensor cores (tcgen05 MMAs accumulating in tensor memory).
//
// Mathematics.  For query row (token i of sequence b, head) and the keys j < lim, lim the
// context length or, when causal, the row's own position + 1:
//   out = sum_j 2^(x_j - m) V_j / sum_j 2^(x_j - m),   x_j = scale log2(e) q . K_j,
// with a running reference m: it moves only when a row's maximum passes it by more than 2^8,
// so the accumulators are rescaled rarely, and any m gives the same quotient.  Softmax
// statistics and both products are held in fp32.  Rounded to 16 bits are the weights alone
// (the A operand of the second product): bf16 for bf16 pools (half a step 2^-8), fp16 times
// 2^7 for E4M3 pools (2^-11; the factor keeps weights down to 2^-31 of the largest).
//   E4M3 pools: K enters as its codes; q enters as two E4M3 terms, hi + lo with lo the rest,
// after a power of two per row that takes its largest into [128, 256): a bf16 has 8 significant bits and
// each term 4, and E4M3's smallest step is 2^-9, so the pair is exact for elements down to 2^-9 of the
// row's largest and off by at most 2^-17 of the largest (half that step, of 128) below.  The
// two products add up in the same accumulators and cost what one 16-bit product does.  V is
// expanded to fp16 (exact) in shared memory.  The scales of K and V are applied in fp32.
//
// The query heads of a kv head are rows of one tile: row r is token r / G, head h G + r % G,
// so K and V are read once per group.  Two forms:
//   wide    256 rows: two tiles of 128 over the same keys; while one tile's softmax runs, the
//           tensor cores work on the other's products.
//   narrow  128 rows (few new tokens): one tile, whose 128-key steps are dealt alternately to
//           the two softmax groups, each with its own statistics and output; joined at the end.
//
//   warps 0-3, 4-7  softmax groups 0 and 1: thread r owns row r (TMEM lane r): scores in, weights
//                   out over them as 16-bit pairs, rare rescale of the output, epilogue
//   warps 8, 10     issue the MMAs, a warp per tile (narrow: warp 8 for both groups)
//   warp 9          finds the work and passes it on; TMA of Q, K and V, a 16-token block at a time
//   warp 11         looks for bad ranges
//   warps 12-15     V: zero the rows past the context in the last tile, so that what a page holds
//                   there (NaN included) meets weight 0 as 0; E4M3: expand V to fp16
// A value of V that is not finite at a position some rows see and others do not would reach
// the latter as 0 * NaN; in the tiles where the mask cuts, such values are taken out of the
// tile, and added to the rows that see them in the epilogue.
//
// A CTA stays: when its work (a tile or two of one kv head, or one of its context's splits) is
// done it takes the next that no CTA has started (cluster launch control), so that Q, K, V and
// the first scores of the next work come in under the softmax and the epilogue of the last.
//
// Shared memory: Q (both tiles, or E4M3 hi and lo), a ring of K and V tiles of 128 keys in the
// order K0 K1 V0 K2 V1 .., E4M3 two fp16 V tiles.  TMEM (512 columns): scores, then weights, of
// group w at 128 w; outputs at 256 + w D.
//
// What bounds it.  (Times with the caches flushed between calls; in brackets, calls one after another in
// a graph.)  A wide step is 2048 cycles of products at D = 128; the tensor cores are kept fed
// but for the part of the chain scores -> weights -> products that the other tile does not cover:
// 4096 tokens over 32,768, 32 + 8 heads, bf16: 1.30 ms (1.26) = 1.58 PFLOP/s, 85 % of the measured cuBLAS
// rate (1.08 ms with the softmax left out, when the whole took 1.29 in a graph).  The exponentials, 32 a cycle
// and SM, take half of a step; a polynomial on the FMA pipe for a share of them costs more than it saves, and
// two threads a row, 16 softmax warps, slow the other roles down more than they gain (1.46 ms).  Prompts of 257
// to 2048 tokens: 117 us (112), 59 % of the rate: a work is a handful of steps there, and its start, masked
// steps and epilogue weigh beside them.  24 x 3 to 8 tokens over 1800 to 12,000 (narrow, split in
// 3): 116 us (115) = 5.3 TB/s of K and V, 78 % of the measured copy.  E4M3, 4 x 700 to 1100 tokens over
// 3000 to 9000, 64 + 8 heads: 0.521 ms (0.500) = 1.39 PFLOP/s; V's expansion takes shared-memory
// bandwidth and issue slots from the products and the softmax.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>

#include "mma_ops.cuh"
#include "pkv_device.cuh"
#include "prefill_ops.cuh"
#include "prompt.cuh"
#include "tc_ops.cuh"

namespace pkv {

template <int D, bool FP8>
struct PrefillCfg {
  static constexpr int kRows = 128;  // rows of a tile: the MMA's M
  static constexpr int kKeys = 128;  // keys of a step
  static constexpr int kStepBlocks = kKeys / kBlockSize;
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf16 = 128 * 128;         // 64 columns of 128 16-bit rows
  static constexpr int kTile16 = kHalves * kHalf16;  // a 16-bit tile of 128 rows
  static constexpr int kCodes = 128 * D;             // an E4M3 tile of 128 rows
  // bf16 K and V tiles: groups of eight keys, each group's 64-column halves side by side, so that one
  // TMA box brings a block of the pool
  static constexpr int kGroup = kHalves * 1024;
  static constexpr int kQTile = FP8 ? 2 * kCodes : kTile16;
  static constexpr int kSlot = FP8 ? kCodes : kTile16;  // a K or V tile as loaded
  static constexpr int kSlots = D == 128 ? (FP8 ? 6 : 5) : 8;
  static constexpr int kExp = FP8 ? 2 : 0;  // expanded V tiles
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = kOffQ + 2 * kQTile;
  static constexpr int kOffExp = kOffRing + kSlots * kSlot;
  static constexpr int kOffBar = kOffExp + kExp * kTile16;
  static constexpr int kBarBytes = 528;
  static constexpr int kOffPoison = kOffBar + kBarBytes;  // int[kinds][D]
  static constexpr int kKinds = FP8 ? 1 : 3;               // NaN, +inf, -inf (E4M3 has no infinity)
  // 1008: alignment slack (the start of dynamic shared memory is 16-byte aligned)
  static constexpr int kBytes = 1008 + kOffPoison + kKinds * D * 4;
  static constexpr int kColS = 0, kColO = 256, kTmemCols = 512;
  static constexpr int kIssuerWarp = 8, kProducerWarp = 9, kIssuer2Warp = 10, kFixWarp0 = 12;
  static constexpr int kFixWarps = 4;
  static constexpr int kThreads = (kFixWarp0 + kFixWarps) * 32;
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;           // per thread
  static constexpr int kSoftRegs = 184;
  static constexpr int kAuxRegs = (kLaunchRegs * kThreads - kSoftRegs * 256) / (kThreads - 256) / 8 * 8;
  static_assert(kSoftRegs * 256 + kAuxRegs * (kThreads - 256) <= kLaunchRegs * kThreads, "register split");
  static constexpr float kLazy = 8.f;
  static constexpr float kBias = FP8 ? kPrefillWeightBias : 0.f;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// barriers and small shared state, at kOffBar
struct PrefillShared {
  uint64_t full[8], empty[8];  // ring: tile landed, tile consumed
  uint64_t s_full[2];          // scores of a step done (and every product issued before)
  uint64_t p_half[2];          // weights of a step's first 64 keys written, the output rescaled (an arrival
                               // per warp; wide: and the other tile's turn over)
  uint64_t p_full[2];          // all weights of a step written (an arrival per warp)
  uint64_t o_full[2];          // every product of the group's work done
  uint64_t fixed[8];           // bf16: V tile of a cut step fixed; E4M3 (two in use): V tile expanded
  uint64_t exp_free[2];        // E4M3: expanded V tile consumed
  uint64_t v_sent[8];          // load of a V tile that warps 12-15 work on issued
  uint64_t q_full[2], q_empty;  // E4M3 wide: a barrier per tile that has steps, else the first
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
static_assert(sizeof(PrefillShared) <= 528, "shared state");

namespace {

// One CTA's worth of work, and what every role derives from it
struct Work {
  int tok0;   // first query token (row of q)
  int ntok;   // its tokens
  int seq;    // sequence
  int ctx;    // cached tokens
  int shift;  // causal: the work's token i sees keys < shift + i + 1
  int h, split;
};

template <bool WIDE>
struct Steps {
  int k0, nstep, n_of[2];  // first 128-key step, steps, local steps of the groups
  int lim_min;             // keys that every row sees
  int first_cut;           // first step whose V needs care: some row does not see all of its keys
  __device__ __forceinline__ static int lim(const Work& w, const PrefillParams& p, int i) {
    return p.causal ? max(0, min(w.ctx, w.shift + i + 1)) : w.ctx;
  }
  __device__ __forceinline__ Steps(const Work& w, const PrefillParams& p, int tile_tok) {
    k0 = w.split * p.split_tiles;
    auto to = [&](int l) { return max(0, min((l + 127) / 128, k0 + p.split_tiles) - k0); };
    nstep = to(lim(w, p, w.ntok - 1));
    if constexpr (WIDE) {
      n_of[0] = to(lim(w, p, min(w.ntok, tile_tok) - 1));
      n_of[1] = w.ntok > tile_tok ? nstep : 0;
    } else {
      n_of[0] = (nstep + 1) / 2;
      n_of[1] = nstep / 2;
    }
    lim_min = lim(w, p, 0);
    first_cut = max(0, min(nstep, lim_min / 128 - k0));
  }
  // position of K and V of step j in the ring's order K0 K1 V0 K2 V1 ..
  __device__ __forceinline__ static int k_item(int j) { return j == 0 ? 0 : 2 * j - 1; }
  __device__ __forceinline__ int v_item(int j) const { return min(2 * j + 2, 2 * nstep - 1); }
};

}  // namespace

// The forms are kernels of their own for the instruction cache's sake: the lines of kWideLong (runs of more
// than kPrefillMaxRun steps) in every kernel took the E4M3 case above from 505 to 523 us and prompts from 118.6 to
// 120.8; without those that write records it is 500 and 117.6.
enum PrefillForm { kNarrow, kWide, kWideSplit, kWideLong };

template <int D, bool FP8, PrefillForm FORM>
__global__ void __launch_bounds__((PrefillCfg<D, FP8>::kThreads), 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PrefillParams p) {
  using C = PrefillCfg<D, FP8>;
  constexpr bool WIDE = FORM != kNarrow, LONG = FORM == kWideLong;
  constexpr unsigned NS = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PrefillShared& sh = *reinterpret_cast<PrefillShared*>(smem + C::kOffBar);
  volatile int* abort = &sh.abort;
  volatile int* poisoned = &sh.poisoned;
  int* poison = reinterpret_cast<int*>(smem + C::kOffPoison);  // [kinds][D] first key with such a value

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kIssuers = WIDE ? 2 : 1;
  const int G = p.group, log_g = 31 - __clz(G);  // a power of two
  const int tile_tok = C::kRows >> log_g;                   // tokens of a 128-row tile
  const int cta_tok = WIDE ? 2 * tile_tok : tile_tok;  // tokens of a work

  if (warp == 0) {
    __syncwarp();
    tmem_alloc(smem_u32(&sh.tmem), C::kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == C::kIssuerWarp * 32) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kIssuers);
      mbar_init(&sh.fixed[i], 1);
      mbar_init(&sh.v_sent[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_half[i], WIDE ? 5 : 4);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.exp_free[i], kIssuers);
      mbar_init(&sh.work_full[i], 1);
      mbar_init(&sh.work_empty[i], kIssuers + C::kFixWarps + 8);  // one arrival per warp that reads it
    }
    mbar_init(&sh.q_full[0], FP8 ? 4 : 1);
    mbar_init(&sh.q_full[1], 4);
    mbar_init(&sh.q_empty, kIssuers);
    mbar_init(&sh.clc, 1);
    mbar_init(&sh.drain[0], 1);
    mbar_init(&sh.drain[1], 1);
    sh.abort = 0;
    sh.poisoned = 0;
    for (int i = 0; i < 8; ++i) sh.epilogues[i] = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == C::kProducerWarp * 32) {
    if (!FP8) tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  for (int i = threadIdx.x; i < C::kKinds * D; i += C::kThreads) poison[i] = 0x7fffffff;
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
  auto next_work = [&](unsigned n, Work& w, unsigned lanes = kFull) -> bool {
    const bool ok = wait_for(&sh.work_full[n & 1], (n >> 1) & 1, abort, p.wait_tries);
    if (!__all_sync(lanes, ok)) {
      if (!*abort) fail();
      return false;
    }
    const int4 a = sh.work[n & 1][0], b = sh.work[n & 1][1];
    w = Work{a.x, a.y, a.z, a.w, b.x, b.y, b.z};
    __syncwarp(lanes);
    if (lane == 0) mbar_arrive(&sh.work_empty[n & 1]);
    return w.seq >= 0;
  };

  // the registers of the launch, dealt out anew: 184 to a softmax thread, 72 to another (208 and 48:
  // the other roles spill, 158 against 149 us for nine prompts of 257 to 2048 tokens)
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kAuxRegs));
    if (warp == C::kIssuerWarp || warp == C::kIssuer2Warp) {
      // ======================================================================== MMA issuers
      // wide: one warp per tile, each going through every step of K and V in order; narrow: one warp
      // for both groups
      if (warp == C::kIssuerWarp || WIDE) {
        const uint32_t leader = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, wait_for(bar, parity, abort)); };
        auto same = [](uint32_t x) { return __shfl_sync(kFull, x, 0); };  // a value of the warp
        constexpr uint32_t kIdO = idesc_f16(C::kRows, D, !FP8, true);
        // scores: A = Q with its sign turned (bit 13) for a negative scale; E4M3 formats are 0
        const uint32_t id_s = (FP8 ? idesc_f16(C::kRows, C::kKeys, false, false)
                                   : idesc_f16(C::kRows, C::kKeys, true, false)) |
                              (p.negate ? 1u << 13 : 0u);
        const uint32_t tm = same(tmem);
        const uint32_t ring_lo = same(desc_lo(ring, 16)), ring_v_lo = same(desc_lo(ring, 1024));
        const uint32_t exp_v_lo = same(desc_lo(smem_u32(smem + C::kOffExp), C::kHalf16));
        const uint32_t q0_lo = same(desc_lo(q_base, 16));
        auto issue_s = [&](int g, unsigned slot) {
          const uint32_t k_lo = same(ring_lo + slot * (C::kSlot / 16));
          const uint32_t q_lo = q0_lo + (WIDE ? g : 0) * (C::kQTile / 16);
          const uint32_t d = tm + C::kColS + 128 * g;
          if constexpr (FP8) {
            constexpr uint32_t hi = D == 128 ? kDescK128 : kDescK64;
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_ss<true>(d, q_lo + (part * C::kCodes + kk * 32) / 16, k_lo + kk * 2, hi, hi, id_s,
                             part > 0 || kk > 0, leader);
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              mma_ss<false>(d, q_lo + ((kk >> 2) * C::kHalf16 + (kk & 3) * 32) / 16,
                            k_lo + ((kk >> 2) * 1024 + (kk & 3) * 32) / 16, kDescK128, kDesc128<C::kGroup>, id_s, kk > 0,
                            leader);
            }
          }
          commit(&sh.s_full[g], leader);
        };
        // keys 64 half .. of a step
        auto issue_o = [&](int g, int half, bool first, uint32_t v_lo0) {
          const uint32_t pt = tm + C::kColS + 128 * g;
          const uint32_t v_lo = same(v_lo0);
          constexpr uint32_t kVGroup = FP8 ? 1024 : C::kGroup;  // eight keys
#pragma unroll
          for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
            mma_ts(tm + C::kColO + D * g, pt + 8 * kk, v_lo + kk * (2 * kVGroup / 16), kDesc128<kVGroup>, kIdO,
                   !first || kk > 0, leader);
        };

        Cursor<C::kSlots> base{0, 0};  // ring position of the work's first tile
        unsigned steps_done = 0, cuts = 0, q_count = 0;
        unsigned c_p[2] = {0, 0};  // steps of the groups so far
        bool ok = true;
        Work w;
        for (unsigned n = 0; ok && next_work(n, w); ++n) {
          const Steps<WIDE> st(w, p, tile_tok);
          const int nstep = st.nstep;
          if (nstep == 0) continue;
          Cursor<C::kSlots> kc = base, vc = base;
          vc.advance(nstep == 1 ? 1 : 2);
          auto next_k = [&](int j) { kc.advance(j == 0 ? 1 : 2); };               // from K of step j to the next
          auto next_v = [&](int j) { vc.advance(j + 2 == nstep ? 1 : 2); };       // from V of step j to the next
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
          auto v_lo = [&](int j) {
            return FP8 ? exp_v_lo + ((steps_done + j) & 1) * (C::kTile16 / 16) : ring_v_lo + vc.slot * (C::kSlot / 16);
          };
          auto free_v = [&](int j) { commit(FP8 ? &sh.exp_free[(steps_done + j) & 1] : &sh.empty[vc.slot], leader); };
          if (!(FP8 && WIDE)) {
            ok = wait(&sh.q_full[0], q_count & 1);
            ++q_count;
          }
          if constexpr (WIDE) {
            // The scores of step j + 1 follow P V of step j in the same columns, in issue order.  The
            // tiles take turns, so that one's products run under the other's softmax (left to themselves
            // they fall into step and wait for the tensor cores together: a tenth slower for 4096 tokens
            // over 32768, 32 heads).  The fifth arrival on p_half is the other issuer's, once its
            // turn before is over: on tile 0's for a work's first step when tile 1 is through with the work
            // before, then after tile 1's step before; on tile 1's after tile 0's same step, or, past
            // tile 0's last, issuer 1's own.  A tile 1 without steps watches tile 0's instead.  So no
            // arrival comes before the phase it belongs to: whoever arrives has seen the one before.
            // Steps past the tile's own are waited for all the same: a slot's phases are seen in order.
            const int g = warp == C::kIssuerWarp ? 0 : 1;
            const int mine = g == 0 ? st.n_of[0] : st.n_of[1], other = g == 0 ? st.n_of[1] : st.n_of[0];
            unsigned parity = (g == 0 ? c_p[0] : c_p[1]) & 1;
            if (ok && g == 1 && other > 0 && leader) mbar_arrive(&sh.p_half[0]);
            if (FP8 && mine > 0) {
              ok = ok && wait(&sh.q_full[g], q_count & 1);
              ++q_count;
            }
            ok = ok && wait_k();
            if (ok) {
              tc_fence_after();
              if (mine > 0) issue_s(g, kc.slot);
              commit(&sh.empty[kc.slot], leader);
              if (nstep == 1) commit(&sh.q_empty, leader);
            }
            for (int j = 0; j < nstep && ok; ++j) {
              const bool more = j + 1 < nstep;
              ok = wait_v(j);
              if (more) next_k(j);
              if (!FP8 && more && ok) ok = wait_k();  // before the weights, where waiting costs nothing
              if (!ok) break;
              if (j < mine) {
                if (g == 1 && j >= other && leader) mbar_arrive(&sh.p_half[1]);
                ok = wait(&sh.p_half[g], parity);
                if (!ok) break;
                tc_fence_after();
                issue_o(g, 0, LONG ? (j & (kPrefillMaxRun - 1)) == 0 : j == 0, v_lo(j));
                ok = wait(&sh.p_full[g], parity);
                if (!ok) break;
                parity ^= 1;
                tc_fence_after();
                issue_o(g, 1, false, v_lo(j));
                if (FP8 && j + 1 < mine) {  // K may come later than the weights: V's expansion holds up the ring
                  ok = wait_k();
                  if (!ok) break;
                  tc_fence_after();
                }
                if (j + 1 < mine) issue_s(g, kc.slot);
                else commit(&sh.o_full[g], leader);
                if ((g == 0 ? j < other : j + 1 < other) && leader) mbar_arrive(&sh.p_half[g ^ 1]);
              } else if (g == 1 && mine == 0 && j < other) {
                ok = wait(&sh.p_half[0], (c_p[0] + j) & 1);
                if (!ok) break;
                if (j + 1 < other && leader) mbar_arrive(&sh.p_half[0]);
              }
              free_v(j);
              next_v(j);
              if (FP8 && more && j + 1 >= mine) ok = wait_k();
              if (!ok) break;
              if (more) commit(&sh.empty[kc.slot], leader);
              if (j + 2 == nstep) commit(&sh.q_empty, leader);
            }
          } else {
            for (int j = 0; j < min(2, nstep) && ok; ++j) {
              if (j > 0) next_k(j - 1);
              ok = wait_k();
              if (!ok) break;
              tc_fence_after();
              issue_s(j, kc.slot);
              commit(&sh.empty[kc.slot], leader);
              if (j + 1 == nstep) commit(&sh.q_empty, leader);
            }
            for (int j = 0; j < nstep && ok; ++j) {
              const int g = j & 1, t = j >> 1;
              const unsigned parity = ((g == 0 ? c_p[0] : c_p[1]) + t) & 1;
              ok = wait(&sh.p_half[g], parity) && wait_v(j);
              if (!ok) break;
              tc_fence_after();
              issue_o(g, 0, t == 0, v_lo(j));
              ok = wait(&sh.p_full[g], parity);
              if (!ok) break;
              tc_fence_after();
              issue_o(g, 1, false, v_lo(j));
              free_v(j);
              next_v(j);
              if (j + 2 >= nstep) commit(&sh.o_full[g], leader);
              if (j + 2 < nstep) {
                next_k(j + 1);
                ok = wait_k();
                if (!ok) break;
                tc_fence_after();
                issue_s(g, kc.slot);
                commit(&sh.empty[kc.slot], leader);
                if (j + 3 == nstep) commit(&sh.q_empty, leader);
              }
            }
          }
          base.advance_by(2 * nstep);
          steps_done += nstep;
          cuts += nstep - st.first_cut;
          c_p[0] += st.n_of[0];
          c_p[1] += st.n_of[1];
        }
        if (!ok && !*abort && lane == 0) fail();
        // nothing may run on the tensor cores when the CTA frees its tensor memory
        commit(&sh.drain[warp == C::kIssuerWarp ? 0 : 1], leader);
        mbar_wait(&sh.drain[warp == C::kIssuerWarp ? 0 : 1], 0);
      }
      __syncwarp();
    } else if (warp == C::kProducerWarp) {
      // ======================================================================== work and TMA producer
      // the lanes know the pool rows of the blocks of four steps; the warp goes through the blocks as one
      // and the elected lane issues each box (16 lanes issuing their own took 100 cycles a box)
      const uint32_t leader = elect_one();
      auto load = [&](const CUtensorMap* tm, unsigned item, int head, int row, int from) {
        const unsigned st = __shfl_sync(kFull, item % NS, 0);
        const uint32_t bar = smem_u32(&sh.full[st]), dst = ring + st * C::kSlot;
        if (leader) mbar_arrive_expect_tx(&sh.full[st], C::kSlot);
        __syncwarp();
#pragma unroll(FP8 ? 2 : C::kStepBlocks)
        for (int blk = 0; blk < C::kStepBlocks; ++blk) {
          const int r = __shfl_sync(kFull, row, from + blk);
          if constexpr (FP8) {
            tma_box(dst + blk * kBlockSize * D, tm, 0, head, r, bar, leader);
          } else {
            tma_block(dst + blk * 2 * C::kGroup, tm, head, r >> 3, bar, leader);
          }
        }
      };
      auto slot_free = [&](unsigned item) {
        const bool ok = item < NS || wait_for(&sh.empty[item % NS], ((item / NS) - 1) & 1, abort);
        return __all_sync(kFull, ok);
      };
      // the tokens of the work at (x, y) of the grid: tile slots count the sequences' tiles in
      // order, each sequence's longest (last) tile first.  seq < 0: a slot past the last tile
      auto find = [&](unsigned x, unsigned y) {
        Work w{0, 0, -1, 0, 0, static_cast<int>(x % p.hkv), static_cast<int>(y)};
        const int slot = x / p.hkv;
        int before = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
          const int b = b0 + lane;
          int first = 0, n = 0, len = 0;
          if (b < p.batch) {
            first = p.q_indptr[b];
            const int last = p.q_indptr[b + 1];
            len = p.context_lens[b];
            n = last - first;
            if (first < 0 || last < first || last > p.total_q) {
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
        const Work w = find(gx, gy);
        if (lane == 0) clc_ask(&sh.clc_answer, &sh.clc);
        if (w.seq >= 0) {
          const Steps<WIDE> st(w, p, tile_tok);
          const int nstep = st.nstep;
          const int32_t* table = p.block_tables + static_cast<int64_t>(w.seq) * p.max_blocks;
          const int nblk = (w.ctx + kBlockSize - 1) / kBlockSize;
          // ids of the blocks of four steps, one a lane, asked for four steps ahead of their use (the first
          // ones before the work is passed on and Q asked for; a step at a time and two ahead, they
          // were late when the tables come from HBM: 117 against 114 us for the narrow case above, 521
          // against 505 for the E4M3 one): INT_MIN for a block past the context; the pool row: a block past the context, or with an id outside
          // the pool, becomes a box entirely outside the tensor, which reads zeros
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
            if constexpr (!FP8) {
              // Q's tiles are free once the last scores of the work before are done
              if (q_count > 0) ok = wait_for(&sh.q_empty, (q_count - 1) & 1, abort);
              ok = __all_sync(kFull, ok);
              if (ok && leader) {
                mbar_arrive_expect_tx(&sh.q_full[0], (WIDE ? 2 : 1) * C::kQTile);
#pragma unroll
                for (int t = 0; t < (WIDE ? 2 : 1); ++t)
#pragma unroll
                  for (int c = 0; c < C::kHalves; ++c)
                    tma_load_3d(smem + C::kOffQ + t * C::kQTile + c * C::kHalf16, &tm_q, c * 64, w.h * G,
                                w.tok0 + t * tile_tok, &sh.q_full[0]);
              }
            }
            if (ok) ++q_count;
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
        if (!FP8 && q_count > 0) mbar_wait(&sh.q_full[0], (q_count - 1) & 1);
      }
      __syncwarp();
    } else if (warp < C::kFixWarp0) {
      // the warp left over looks for bad ranges (whoever finds work stops at the sequence it belongs to); in
      // every CTA that starts: any CTA's start may be cancelled, the first one's too
      for (int b = lane; b < p.batch; b += 32) {
        const int first = p.q_indptr[b], last = p.q_indptr[b + 1];
        if (first < 0 || last < first || last > p.total_q) set_flag(p.status, PKV_DEVFLAG_BAD_INDPTR);
      }
    } else {
      // ======================================================================== V: cut tiles, expansion
      constexpr int kFix = C::kFixWarps * 32;
      const int ft = threadIdx.x - C::kFixWarp0 * 32;
      unsigned number = 0;
      auto note = [&](int kind, int dim, int key) {
        atomicMin(&poison[kind * D + dim], key);
        *poisoned = static_cast<int>(number) + 1;
      };
      constexpr int kChunks = D / 8;  // 8-element pieces of a row
      constexpr int kStep = kFix / kChunks;
      const int c = ft % kChunks, r0 = ft / kChunks;
      unsigned base = 0, steps_done = 0, cuts = 0, with_steps = 0;
      bool ok = true;
      Work w;
      for (unsigned n = 0; ok; ++n) {
        // the warps leave together
        const bool none = !next_work(n, w);
        __syncwarp();
        if (named_sync_or(1, kFix, none)) break;
        number = n;
        const Steps<WIDE> st(w, p, tile_tok);
        const int nstep = st.nstep;
        if (nstep == 0) continue;
        // before values that are not finite are listed: the works before are through their epilogues,
        // and what they left in the list is cleared
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
          for (int i = ft; i < C::kKinds * D; i += kFix) poison[i] = 0x7fffffff;
          __syncwarp();
          named_sync(3, kFix);
        };
        for (int j = FP8 ? 0 : st.first_cut; j < nstep; ++j) {
          const bool cut = j >= st.first_cut;
          const unsigned item = base + st.v_item(j);
          // the parity of `full` means this load only once it is issued (the slot's loads before it
          // are not waited for here); v_sent itself is never a phase ahead: eight V tiles on, the
          // ring has come round
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
          // E4M3: expand the tile, four pieces in registers at a time (one by one, a load and a store
          // each, a tile took 2600 cycles and the step waited for it); rows no row sees become zeros.
          // bf16: only the rows that not every row sees, four pieces at a time.  True if one of those
          // that some row sees is not finite.
          auto odd8 = [](uint32_t x) { return (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0u; };    // E4M3 NaN
          auto odd16 = [](uint32_t x) { return (((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0u; };   // bf16
          const uint32_t ex = smem_u32(smem + C::kOffExp + (sent & 1) * C::kTile16) + (c >> 3) * C::kHalf16;
          auto at16 = [&](int row) {
            return reinterpret_cast<uint4*>(src + (row >> 3) * C::kGroup + (c >> 3) * 1024 + (row & 7) * 128 +
                                            (((c & 7) ^ (row & 7)) << 4));
          };
          auto expand = [&](int row, uint2 v) {
            st_shared_v4(ex + (row >> 3) * 1024 + (row & 7) * 128 + (((c & 7) ^ (row & 7)) << 4), e4m3_lo(v.x),
                         e4m3_hi(v.x), e4m3_lo(v.y), e4m3_hi(v.y));
          };
          bool odd = false;
          if (ok) {
            if constexpr (FP8) {
              constexpr int kBatch = 4;
              static_assert(C::kKeys % (kBatch * kStep) == 0, "whole batches");
#pragma unroll 1
              for (int b0 = r0; b0 < C::kKeys; b0 += kBatch * kStep) {
                uint2 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                  v[i] = *reinterpret_cast<const uint2*>(src + (b0 + i * kStep) * D + c * 8);
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
              constexpr int kBatch = 4;
#pragma unroll 1
              for (int b0 = max(0, seen) + r0; b0 < min(end, C::kKeys); b0 += kBatch * kStep) {
                uint4 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                  const int row = b0 + i * kStep;
                  v[i] = row < min(end, C::kKeys) ? *at16(row) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                  odd |= odd16(v[i].x) || odd16(v[i].y) || odd16(v[i].z) || odd16(v[i].w);
                }
              }
              for (int row = max(0, end) + r0; row < C::kKeys; row += kStep) *at16(row) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          __syncwarp();  // (rows are dealt by lane; the barriers are for whole warps)
          if (cut && named_sync_or(3, kFix, odd)) {  // rare: list them and take them out of the tile
            if (!cleared) clear();
            for (int row = max(0, seen) + r0; ok && row < min(end, C::kKeys); row += kStep) {
              if constexpr (FP8) {
                uint2 v = *reinterpret_cast<const uint2*>(src + row * D + c * 8);
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
              mbar_arrive_n(&sh.empty[item % NS], kIssuers);  // what both issuers would arrive
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    // ======================================================================== softmax
    const int g = warp >> 2;               // accumulators: the tile (wide) or the parity of the steps (narrow)
    const int r = threadIdx.x & 127;       // row of the tile, TMEM lane
    const int my_i = (WIDE ? g * tile_tok : 0) + (r >> log_g);  // token within the work
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t scol = tmem + lane_base + C::kColS + 128 * g;
    const uint32_t ocol = tmem + lane_base + C::kColO;
    // narrow: (m, l) of both groups' rows and the rows' factors, where wide has its second Q tile
    float2* join_ml = reinterpret_cast<float2*>(smem + C::kOffQ + C::kQTile);
    float* join_scale = reinterpret_cast<float*>(join_ml + 256);
    unsigned c_s = 0, c_o = 0;  // steps and works of the group so far
    unsigned through = 0;       // works with steps that this warp is through with
    auto through_with = [&]() {
      ++through;
      if (lane == 0) *const_cast<volatile uint16_t*>(&sh.epilogues[warp]) = static_cast<uint16_t>(through);
    };
    bool dead = false;
    Work w;
    for (unsigned n = 0; !dead; ++n) {
      bool none = !next_work(n, w);
      // narrow: the groups meet at barriers below, so all eight warps take the work or none does (one that gave
      // up just before the work was passed on would leave the others waiting for it there)
      if constexpr (!WIDE) {
        __syncwarp();
        none = named_sync_or(2, 256, none);
      }
      if (none) break;
      const Steps<WIDE> st(w, p, tile_tok);
      const int nloc = st.n_of[g];
      const bool rv = my_i < w.ntok;
      const int hq = w.h * G + (r & (G - 1));
      const int64_t orow = static_cast<int64_t>(w.tok0 + my_i) * p.hq + hq;
      const int64_t rec = static_cast<int64_t>(w.split) * p.total_q * p.hq + orow;
      const bool split_out = FORM == kWideSplit || (FORM != kWide && p.splits > 1);
      if (WIDE ? nloc == 0 : st.nstep == 0) {  // rows that see nothing (of this split)
        if (rv && (WIDE || g == 0)) {
          if (split_out) {
            p.part_ml[rec] = make_float2(-INFINITY, 0.f);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse != nullptr) p.lse[orow] = -INFINITY;
          }
        }
        if (st.nstep > 0) through_with();
        continue;
      }
      float sscale = p.score_scale;

      if constexpr (FP8) {
        // this row of Q as hi and lo codes, times 2^e that takes its largest into [128, 256); the
        // tile is free: the group's last scores of the work before are done
        if (WIDE || g == 0) {
          const uint4* qr =
              reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(w.tok0 + my_i) * p.q_stride + hq * D);
          float top = 0.f;
          bool odd = false;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = rv ? qr[c] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              top = fmaxf(top, fmaxf(fabsf(bf16_lo(e[k])), fabsf(bf16_hi(e[k]))));
              odd |= ((((e[k] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0u);
            }
          }
          int ex = 0;
          if (top > 0.f && !odd) ex = 7 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
          ex = min(ex, 126);  // rows below 2^-119: their codes lose what lies under 2^-135
          const float k_scale = p.scales[w.h];
          const float size = __uint_as_float(static_cast<uint32_t>(max(ex, -126) + 127) << 23);
          const float up = k_scale < 0.f ? -size : size;  // the scores' factor below stays positive
          const uint32_t qt = q_base + (WIDE ? g : 0) * C::kQTile;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {  // 16 codes: one 16-byte piece of the row
            const uint4 v[2] = {rv ? qr[2 * c] : make_uint4(0u, 0u, 0u, 0u),
                                rv ? qr[2 * c + 1] : make_uint4(0u, 0u, 0u, 0u)};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a = u4_word(v[k / 2], 2 * (k & 1)), b = u4_word(v[k / 2], 2 * (k & 1) + 1);
              float x[4] = {bf16_lo(a) * up, bf16_hi(a) * up, bf16_lo(b) * up, bf16_hi(b) * up};
              hi[k] = e4m3x4_rest(x);
              lo[k] = e4m3x4_rest(x);
            }
            const uint32_t at = D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
            st_shared_v4(qt + at, hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(qt + C::kCodes + at, lo[0], lo[1], lo[2], lo[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.q_full[WIDE ? g : 0]);
          // the row's scores come out times 2^ex; a row with a NaN or an infinity has no value, unless it
          // sees no key: its scores are all masked, whatever they are
          // (a zero scale: a factor that leaves every score at 0 while masked ones stay -inf)
          sscale = (odd || k_scale != k_scale) && Steps<WIDE>::lim(w, p, my_i) > 0
                       ? __int_as_float(0x7fffffff)
                       : fmaxf(sscale * fabsf(k_scale) / size, 1e-37f);
        }
        if constexpr (!WIDE) {  // group 1 works on the same rows: it takes their factors over
          if (g == 0) join_scale[r] = sscale;
          __syncwarp();
          named_sync(2, 256);
          if (g == 1) sscale = join_scale[r];
        }
      }

      const int my_lim = Steps<WIDE>::lim(w, p, my_i);
      // keys below every lim of the warp's rows need no mask (rows that do not exist do not count)
      const int warp_lim = __reduce_min_sync(kFull, rv ? my_lim : 0x7fffffff);
      const bool idle = !__any_sync(kFull, rv);  // no row of the warp exists: its products go nowhere
      float m_used = -INFINITY, l = 0.f;
      // LONG: after every kPrefillMaxRun steps the output so far moves to the row's record, in rounded fp32
      // (the tensor cores' additions truncate), by reference m_moved; the next products start anew
      float m_moved = -INFINITY;
      bool moved = false;
      auto moved_by = [&]() { return m_moved == m_used ? 1.f : fast_exp2(m_moved - m_used); };
      auto add_moved = [&](float (&o)[32], int col, float by) {
        const float4* src = reinterpret_cast<const float4*>(p.part_acc + rec * D + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 v = src[i];
          o[4 * i] = fmaf(v.x, by, o[4 * i]);
          o[4 * i + 1] = fmaf(v.y, by, o[4 * i + 1]);
          o[4 * i + 2] = fmaf(v.z, by, o[4 * i + 2]);
          o[4 * i + 3] = fmaf(v.w, by, o[4 * i + 3]);
        }
      };
      for (int t = 0; t < nloc; ++t) {
        const int key0 = (st.k0 + (WIDE ? t : 2 * t + g)) * C::kKeys;
        const bool ok = wait_for(&sh.s_full[g], (c_s + t) & 1, abort, p.wait_tries);
        if (!__all_sync(kFull, ok)) {  // tensor-memory loads are warp-collective: leave as a warp
          if (!*abort) fail();
          dead = true;
          break;
        }
        tc_fence_after();
        if (!idle) {
          if (LONG && t > 0 && (t & (kPrefillMaxRun - 1)) == 0) {
            const float by = moved_by();
#pragma unroll 1
            for (int col = 0; col < D; col += 32) {
              float o[32];
              tmem_ld32(ocol + D * g + col, o);
              if (rv) {
                if (moved) add_moved(o, col, by);
                float4* dst = reinterpret_cast<float4*>(p.part_acc + rec * D + col);
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
              }
              __syncwarp();
            }
            moved = true;
            m_moved = m_used;
          }
          // keys that a row does not see: -inf over their scores, in the columns (a loop of 32: this is
          // for a work's last steps, and straight code for 128 is slow to fetch)
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
          auto weights = [&](int q, float negm, uint32_t (&pw)[16]) {
            const float2 sc2 = make_float2(sscale, sscale), nm2 = make_float2(negm, negm);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 x = ffma2(make_float2(s[32 * q + 2 * i], s[32 * q + 2 * i + 1]), sc2, nm2);
              x.x = exp2_ftz(x.x);
              x.y = exp2_ftz(x.y);
              sum[i & 1] = fadd2(sum[i & 1], x);
              pw[i] = pack16<FP8>(x.x, x.y);
            }
          };
          // a row that has seen nothing yet keeps reference 0: its weights are 2^-inf = 0
          auto minus_m = [&]() { return (m_used == -INFINITY ? 0.f : -m_used) + C::kBias; };
          // the first weights by the reference as it stands, while the maximum is being found; it
          // moves rarely, and they are then taken again
          uint32_t pw[16];
          weights(0, minus_m(), pw);
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
              for (int ch = 0; ch < D / 16; ++ch) {
                float o[16];
                tmem_ld16(ocol + D * g + 16 * ch, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= alpha;
                tmem_st16(ocol + D * g + 16 * ch, o);
              }
            }
            sum[0] = sum[1] = make_float2(0.f, 0.f);
            weights(0, minus_m(), pw);
          } while (false);
          const float negm = minus_m();
          tmem_st16u(scol, pw);
          weights(1, negm, pw);
          tmem_st16u(scol + 16, pw);
          weights(2, negm, pw);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          arrive_by(&sh.p_half[g], lane == 0);
          tmem_st16u(scol + 32, pw);
          weights(3, negm, pw);
          tmem_st16u(scol + 48, pw);
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
      c_s += nloc;

      // ---- epilogue: the output row, or its record
      if (!dead && nloc > 0) {
        const bool ok = wait_for(&sh.o_full[g], c_o & 1, abort);
        if (!__all_sync(kFull, ok)) {
          if (!*abort) fail();
          dead = true;
        }
        ++c_o;
        tc_fence_after();
      }
      // narrow: both groups' outputs are done and their statistics shared; each joins half of the
      // columns (the other group's output is in the same TMEM lanes)
      float a0 = 1.f, a1 = 0.f;
      if constexpr (!WIDE) {
        join_ml[g * 128 + r] = make_float2(m_used, l);
        tc_fence_before();
        __syncwarp();
        dead = named_sync_or(2, 256, dead);
        tc_fence_after();
        const float2 x0 = join_ml[r], x1 = join_ml[128 + r];
        const float top = fmaxf(x0.x, x1.x);
        a0 = x0.x == -INFINITY ? 0.f : fast_exp2(x0.x - top);
        a1 = x1.x == -INFINITY ? 0.f : fast_exp2(x1.x - top);
        if (x0.y != x0.y || x1.y != x1.y) a0 = a1 = __int_as_float(0x7fffffff);
        l = x0.y * a0 + x1.y * a1;
        m_used = top;
      }
      if (!dead && !idle) {
        float inv = 0.f;  // of a row without keys
        if (!split_out && (l > 0.f || l != l)) {
          inv = 1.f / l;
          if constexpr (FP8) inv *= p.scales[p.hkv + w.h];
        }
        if (rv && (WIDE || g == 0)) {
          if (split_out) p.part_ml[rec] = make_float2(m_used, l);
          else if (p.lse != nullptr)
            p.lse[orow] = l == 0.f ? -INFINITY : (m_used - C::kBias + log2f(l)) * 0.69314718055994531f;
        }
        // (the tensor-memory loads below are for whole warps, and rows that do not exist part from the others
        // between them)
        __syncwarp();
        if constexpr (WIDE) {
          if (!split_out) {
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {  // (the words go to columns already read)
              float o[32];
              tmem_ld32(ocol + D * g + 32 * ch, o);
              if constexpr (LONG) {
                if (moved && rv) add_moved(o, 32 * ch, moved_by());
                __syncwarp();
              }
              uint32_t words[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) words[i] = pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv);
              turn_put(ocol + D * g + 16 * ch, words);
            }
            tmem_wait_st();
#pragma unroll 1
            for (int it = 0; it < 2 * (D / 64); ++it) {
              const int half = it & 1, c = it >> 1;  // rows, 64 columns
              uint32_t v[16];
              turn_get(ocol + D * g + 32 * c + (static_cast<uint32_t>(16 * half) << 16), v);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int rr = (r & ~31) + 16 * half + 8 * k + (lane >> 2);
                const int i = g * tile_tok + (rr >> log_g);
                if (i >= w.ntok) continue;
                uint4* dst = reinterpret_cast<uint4*>(
                                 p.out + (static_cast<int64_t>(w.tok0 + i) * p.hq + w.h * G + (rr & (G - 1))) * D) +
                             8 * c + (lane & 3);
                dst[0] = make_uint4(v[k], v[2 + k], v[4 + k], v[6 + k]);
                dst[4] = make_uint4(v[8 + k], v[10 + k], v[12 + k], v[14 + k]);
              }
              __syncwarp();
            }
          }
        }
        constexpr int kMine = WIDE ? D : D / 2;  // columns of this group
        const int col0 = WIDE ? 0 : g * kMine;
#pragma unroll 1
        for (int ch = 0; (!WIDE || split_out) && ch < kMine / 32; ++ch) {
          const int col = col0 + 32 * ch;
          float o[32];
          if constexpr (WIDE) {
            tmem_ld32(ocol + D * g + col, o);
            if constexpr (LONG) {
              if (moved && rv) add_moved(o, col, moved_by());
            }
          } else {
            tmem_ld32(ocol + col, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= a0;
            if (st.n_of[1] > 0) {
              float o1[32];
              tmem_ld32(ocol + D + col, o1);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fmaf(o1[i], a1, o[i]);
            }
          }
          if (rv) {
            if (split_out) {
              float4* dst = reinterpret_cast<float4*>(p.part_acc + rec * D + col);
#pragma unroll
              for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + col);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                dst[i] = make_uint4(pack_bf16(o[8 * i] * inv, o[8 * i + 1] * inv),
                                    pack_bf16(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                    pack_bf16(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                    pack_bf16(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
            }
          }
          __syncwarp();
        }
        // rare: values of V taken out of the cut tiles are added to the rows that see them (the warp
        // stored them just now)
        __syncwarp();
        if (*poisoned == static_cast<int>(n) + 1 && rv) {
#pragma unroll 1
          for (int dim = col0; dim < col0 + kMine; ++dim) {
            const bool nan = poison[dim] < my_lim, up = !FP8 && poison[(C::kKinds - 2) * D + dim] < my_lim,
                       down = !FP8 && poison[(C::kKinds - 1) * D + dim] < my_lim;
            if (!nan && !up && !down) continue;
            const float x = nan || (up && down) ? __int_as_float(0x7fffffff) : up ? INFINITY : -INFINITY;
            if (split_out) {
              p.part_acc[rec * D + dim] += x;
            } else {
              __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(p.out) + orow * D + dim;
              *at = __float2bfloat16_rn(__bfloat162float(*at) + x);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if constexpr (!WIDE) dead = named_sync_or(2, 256, dead);  // both are through with both outputs
      __syncwarp();  // (the list of values was read above; the output's stores need not have landed)
      through_with();
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

template <int D, bool FP8, PrefillForm FORM>
static cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PrefillParams& p,
                          int tile_slots, cudaStream_t stream) {
  using C = PrefillCfg<D, FP8>;
  auto kern = prefill_tc_kernel<D, FP8, FORM>;
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
  cfg.gridDim = dim3(static_cast<unsigned>(tile_slots) * static_cast<unsigned>(p.hkv),
                     static_cast<unsigned>(p.splits), 1);
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

template <int D, bool FP8>
static cudaError_t launch_form(bool wide, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PrefillParams& p, int tile_slots, cudaStream_t stream) {
  if (!wide) return launch<D, FP8, kNarrow>(tq, tk, tv, p, tile_slots, stream);
  if (p.split_tiles > kPrefillMaxRun) return launch<D, FP8, kWideLong>(tq, tk, tv, p, tile_slots, stream);
  return p.splits > 1 ? launch<D, FP8, kWideSplit>(tq, tk, tv, p, tile_slots, stream)
                      : launch<D, FP8, kWide>(tq, tk, tv, p, tile_slots, stream);
}

cudaError_t launch_prefill(int d, bool fp8, bool wide, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, const PrefillParams& p, int tile_slots, cudaStream_t stream) {
  if (d == 64)
    return fp8 ? launch_form<64, true>(wide, tq, tk, tv, p, tile_slots, stream)
               : launch_form<64, false>(wide, tq, tk, tv, p, tile_slots, stream);
  return fp8 ? launch_form<128, true>(wide, tq, tk, tv, p, tile_slots, stream)
             : launch_form<128, false>(wide, tq, tk, tv, p, tile_slots, stream);
}

}  // namespace pkv
