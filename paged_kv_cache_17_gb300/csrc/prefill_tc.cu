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
// after a power of two per row: a bf16 has 8 significant bits and each term 4, so the pair is
// exact for elements down to 2^-10 of the row's largest and off by 2^-18 of that below.  The
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
//   warps 0-3, 4-7  softmax groups 0 and 1: thread r owns row r (TMEM lane r): scores in,
//                   weights out over them as 16-bit pairs, rare rescale of the output, epilogue
//   warp 8          lane 0 issues every MMA
//   warp 9          TMA: one 16-token block (and 64-column half) per lane and step
//   warps 10, 11    V: zero the rows past the context in the last tile, so that what a page
//                   holds there (NaN included) meets weight 0 as 0; E4M3: expand V to fp16
// A value of V that is not finite at a position some rows see and others do not would reach
// the latter as 0 * NaN; in the tiles where the mask cuts, such values are taken out of the
// tile, and added to the rows that see them in the epilogue.
//
// Shared memory: Q (both tiles, or E4M3 hi and lo), a ring of K and V tiles of 128 keys in the
// order K0 K1 V0 K2 V1 .., E4M3 two fp16 V tiles.  TMEM (512 columns): scores, then weights, of
// group w at 128 w; outputs at 256 + w D.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "mma_ops.cuh"
#include "pkv_device.cuh"
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
  static constexpr int kQTile = FP8 ? 2 * kCodes : kTile16;
  static constexpr int kSlot = FP8 ? kCodes : kTile16;  // a K or V tile as loaded
  static constexpr int kSlots = D == 128 ? (FP8 ? 6 : 5) : 8;
  static constexpr int kExp = FP8 ? 2 : 0;  // expanded V tiles
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = kOffQ + 2 * kQTile;
  static constexpr int kOffExp = kOffRing + kSlots * kSlot;
  static constexpr int kOffBar = kOffExp + kExp * kTile16;
  static constexpr int kBarBytes = 320;
  static constexpr int kOffPoison = kOffBar + kBarBytes;  // int[3][D]
  static constexpr int kBytes = 1024 + kOffPoison + 3 * D * 4;
  static constexpr int kColS = 0, kColO = 256, kTmemCols = 512;
  static constexpr int kThreads = 384;
  static constexpr int kIssuerWarp = 8, kProducerWarp = 9, kFixWarp0 = 10;
  static constexpr float kLazy = 8.f;
  static constexpr float kBias = FP8 ? kPrefillWeightBias : 0.f;
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert(kSlots * kSlot + kExp * kTile16 >= 128 * D * 4, "room for the join of two groups");
  static_assert((2 * kSlots + 18) * 8 + 12 <= kBarBytes, "barriers");
};

namespace {

// descriptor of an operand in shared memory with 128-byte (sw = 2) or 64-byte (sw = 4) swizzle
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint64_t sw) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (sw << 61);
}

// D[tmem] = A[smem] B[smem] (+ D) for 8-bit operands (E4M3: formats 0 in the descriptor)
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
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

// what a CTA works on
struct Work {
  int tok0;    // first query token (row of q) of the CTA
  int ntok;    // its tokens
  int seq;     // sequence
  int ctx;     // cached tokens
  int shift;   // causal: the CTA's token i sees keys < shift + i + 1
};

}  // namespace

template <int D, bool FP8, bool WIDE>
__global__ void __launch_bounds__(384, 1)
    prefill_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PrefillParams p) {
  using C = PrefillCfg<D, FP8>;
  constexpr int NS = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [NS] tile landed
  uint64_t* empty = full + NS;     // [NS] tile consumed
  uint64_t* s_full = empty + NS;   // [2] scores of a step done (and the products issued before)
  uint64_t* p_full = s_full + 2;   // [2] weights of a step written (one arrival per warp)
  uint64_t* o_full = p_full + 2;   // [2] every product of the group done
  uint64_t* fixed = o_full + 2;    // bf16: [4] V tile of a cut step fixed; E4M3: [2] V tile expanded
  uint64_t* exp_free = fixed + 4;  // E4M3: [2] expanded V tile consumed
  uint64_t* q_full = exp_free + 2;
  uint64_t* drain = q_full + 1;    // every MMA issued so far done (abort path)
  uint64_t* v_sent = drain + 1;    // [4] load of V of a step that warps 10, 11 work on issued
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_sent + 4);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* poisoned = abort + 1;
  int* poison = reinterpret_cast<int*>(smem + C::kOffPoison);  // [3][D] first key with NaN, +inf, -inf

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % p.hkv;
  const int slot = blockIdx.x / p.hkv;
  const int split = blockIdx.y;
  const int G = p.group;
  const int tile_tok = C::kRows / G;                   // tokens of a 128-row tile
  const int cta_tok = WIDE ? 2 * tile_tok : tile_tok;  // tokens of a CTA
  pdl_wait();
  pdl_launch_dependents();

  // ---- the CTA's tokens: tile slots count the sequences' tiles in order, each sequence's
  // longest (last) tile first; every warp finds them by itself
  Work w{0, 0, -1, 0, 0};
  {
    int before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      int first = 0, n = 0;
      if (b < p.batch) {
        first = p.q_indptr[b];
        const int last = p.q_indptr[b + 1];
        n = last - first;
        if (first < 0 || last < first || last > p.total_q) {
          if (warp == 0 && blockIdx.x == 0 && split == 0) set_flag(p.status, PKV_DEVFLAG_BAD_INDPTR);
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
        const int tile = __shfl_sync(kFull, before + upto - 1 - slot, src);  // tiles after this one: reversed order
        first = __shfl_sync(kFull, first, src);
        n = __shfl_sync(kFull, n, src);
        w.seq = b0 + src;
        int ctx = p.context_lens[w.seq];
        const int cap = min(p.max_context_len, p.max_blocks * kBlockSize);
        if (ctx < 0 || ctx > cap) {
          if (threadIdx.x == 0) set_flag(p.status, PKV_DEVFLAG_BAD_CONTEXT_LEN);
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
  }
  if (w.seq < 0) return;  // a slot past the last tile
  auto lim_of = [&](int i) { return p.causal ? max(0, min(w.ctx, w.shift + i + 1)) : w.ctx; };

  // ---- the steps (128-key tiles) of the split that each group takes part in
  const int k0 = split * p.split_tiles;
  auto steps_to = [&](int lim) { return max(0, min((lim + C::kKeys - 1) / C::kKeys, k0 + p.split_tiles) - k0); };
  const int nstep = steps_to(lim_of(w.ntok - 1));
  int n_of[2];  // local steps of the groups
  if constexpr (WIDE) {
    n_of[0] = steps_to(lim_of(min(w.ntok, tile_tok) - 1));
    n_of[1] = w.ntok > tile_tok ? nstep : 0;
  } else {
    n_of[0] = (nstep + 1) / 2;
    n_of[1] = nstep / 2;
  }
  const int lim_min = lim_of(0);
  // the first step whose V needs care: some row of the CTA does not see all of its keys
  const int first_cut = max(0, min(nstep, lim_min / C::kKeys - k0));

  const bool soft = warp < 8;
  const int group = WIDE ? (warp >> 2) & 1 : 0;  // which tile's rows a softmax thread owns
  const int r = threadIdx.x & 127;               // row of the tile, TMEM lane
  const int my_i = group * tile_tok + r / G;     // token within the CTA
  const bool rv = soft && my_i < w.ntok;
  const int hq = h * G + r % G;
  const int64_t orow = static_cast<int64_t>(w.tok0 + my_i) * p.hq + hq;
  const int64_t rec = static_cast<int64_t>(split) * p.total_q * p.hq + orow;

  if (nstep == 0) {  // nothing to see here: empty rows, or an empty record
    if (rv && (WIDE || warp < 4)) {
      if (p.splits > 1) {
        p.part_ml[rec] = make_float2(-INFINITY, 0.f);
      } else {
        uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse != nullptr) p.lse[orow] = -INFINITY;
      }
    }
    return;
  }

  if (warp == 0) {
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == C::kIssuerWarp * 32) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&exp_free[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&fixed[i], 1);
      mbar_init(&v_sent[i], 1);
    }
    mbar_init(q_full, FP8 ? (WIDE ? 8 : 4) : 1);
    mbar_init(drain, 1);
    *abort = 0;
    *poisoned = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 3 * D; i += C::kThreads) poison[i] = 0x7fffffff;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const uint32_t q_base = smem_u32(smem + C::kOffQ);
  const uint32_t ring = smem_u32(smem + C::kOffRing);
  auto fail = [&]() {
    set_flag(p.status, PKV_DEVFLAG_WAIT_TIMEOUT);
    *abort = 1;
  };
  // position of K and V of step j in the ring's order K0 K1 V0 K2 V1 ..
  auto k_item = [&](int j) { return j == 0 ? 0 : 2 * j - 1; };
  auto v_item = [&](int j) { return min(2 * j + 2, 2 * nstep - 1); };

  if (warp == C::kIssuerWarp) {
    // ======================================================================== MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdO = idesc_f16(C::kRows, D, !FP8, true);
      // scores: A = Q with its sign turned (bit 13) for a negative scale; E4M3 formats are 0
      const uint32_t id_s = (FP8 ? idesc_f16(C::kRows, C::kKeys, false, false)
                                 : idesc_f16(C::kRows, C::kKeys, true, false)) |
                            (p.negate ? 1u << 13 : 0u);
      auto issue_s = [&](int g, int item) {
        const uint32_t kt = ring + (item % NS) * C::kSlot;
        const uint32_t qt = q_base + (WIDE ? g : 0) * C::kQTile;
        const uint32_t d = tmem + C::kColS + 128 * g;
        if constexpr (FP8) {
          constexpr uint64_t sw = D == 128 ? 2 : 4;
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              mma_f8_ss(d, sdesc(qt + part * C::kCodes + kk * 32, 16, 8 * D, sw), sdesc(kt + kk * 32, 16, 8 * D, sw),
                        id_s, (part > 0 || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = (kk >> 2) * C::kHalf16 + (kk & 3) * 32;
            mma_f16_ss(d, sdesc_sw128(qt + at, 16, 1024), sdesc_sw128(kt + at, 16, 1024), id_s, kk > 0 ? 1u : 0u);
          }
        }
        tc_commit(&s_full[g]);
      };
      auto issue_o = [&](int g, int t, uint32_t vt) {
        const uint32_t pt = tmem + C::kColS + 128 * g;
#pragma unroll
        for (int kk = 0; kk < C::kKeys / 16; ++kk)
          mma_f16_ts(tmem + C::kColO + D * g, pt + 8 * kk, sdesc_sw128(vt + kk * 2048, C::kHalf16, 1024), kIdO,
                     (t > 0 || kk > 0) ? 1u : 0u);
      };
      auto wait_full = [&](int item) { return wait_or_abort(&full[item % NS], (item / NS) & 1, abort); };
      // V of step j is ready for the tensor cores
      auto wait_v = [&](int j) {
        if constexpr (FP8) return wait_or_abort(&fixed[j & 1], (j >> 1) & 1, abort);
        if (j >= first_cut) return wait_or_abort(&fixed[j - first_cut], 0, abort);
        return wait_full(v_item(j));
      };
      auto v_tile = [&](int j) {
        return FP8 ? smem_u32(smem + C::kOffExp + (j & 1) * C::kTile16) : ring + (v_item(j) % NS) * C::kSlot;
      };
      auto free_v = [&](int j) { tc_commit(FP8 ? &exp_free[j & 1] : &empty[v_item(j) % NS]); };

      bool ok = wait_or_abort(q_full, 0, abort);
      tc_fence_after();
      if constexpr (WIDE) {
        // step j of both tiles: S of step j + 1 follows P V of step j in the same columns, in
        // issue order
        if (ok) ok = wait_full(0);
        if (ok) {
          tc_fence_after();
          if (n_of[0] > 0) issue_s(0, 0);
          if (n_of[1] > 0) issue_s(1, 0);
          tc_commit(&empty[0]);
        }
        for (int j = 0; j < nstep && ok; ++j) {
          bool k_ready = false;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (ok && j < n_of[g]) {
              ok = wait_or_abort(&p_full[g], j & 1, abort) && wait_v(j);
              if (!ok) break;
              tc_fence_after();
              issue_o(g, j, v_tile(j));
              if (j + 1 == n_of[g]) tc_commit(&o_full[g]);
            }
            if (g == 1) free_v(j);
            if (ok && j + 1 < n_of[g]) {
              if (!k_ready) ok = wait_full(k_item(j + 1));
              if (!ok) break;
              k_ready = true;
              tc_fence_after();
              issue_s(g, k_item(j + 1));
            }
          }
          if (ok && j + 1 < nstep) tc_commit(&empty[k_item(j + 1) % NS]);
        }
      } else {
        for (int j = 0; j < min(2, nstep) && ok; ++j) {
          ok = wait_full(k_item(j));
          if (!ok) break;
          tc_fence_after();
          issue_s(j, k_item(j));
          tc_commit(&empty[k_item(j) % NS]);
        }
        for (int j = 0; j < nstep && ok; ++j) {
          const int g = j & 1, t = j >> 1;
          ok = wait_or_abort(&p_full[g], t & 1, abort) && wait_v(j);
          if (!ok) break;
          tc_fence_after();
          issue_o(g, t, v_tile(j));
          free_v(j);
          if (j + 2 >= nstep) tc_commit(&o_full[g]);
          if (j + 2 < nstep) {
            ok = wait_full(k_item(j + 2));
            if (!ok) break;
            tc_fence_after();
            issue_s(g, k_item(j + 2));
            tc_commit(&empty[k_item(j + 2) % NS]);
          }
        }
      }
      if (!ok && !*abort) fail();
      // nothing may run on the tensor cores when the CTA frees its tensor memory
      tc_commit(drain);
      mbar_wait(drain, 0);
    }
    __syncwarp();
  } else if (warp == C::kProducerWarp) {
    // ======================================================================== TMA producer
    const int32_t* table = p.block_tables + static_cast<int64_t>(w.seq) * p.max_blocks;
    const int nblk = (w.ctx + kBlockSize - 1) / kBlockSize;
    // bf16 at D = 128: lane 2 b + half takes half of block b; else lane b takes block b
    constexpr int kPer = FP8 ? 1 : C::kHalves;
    const bool loads = lane < C::kStepBlocks * kPer;
    const int blk = lane / kPer, hf = lane % kPer;
    // pool row of this lane's block in step j; a block past the context, or with an id outside
    // the pool, becomes a box entirely outside the tensor, which reads zeros
    auto row_of = [&](int j) {
      int row = -kBlockSize;
      const int at = (k0 + j) * C::kStepBlocks + blk;
      if (loads && j < nstep && at < nblk) {
        const int id = table[at];
        if (id >= 0 && id < p.num_blocks) row = id * kBlockSize;
        else set_flag(p.status, PKV_DEVFLAG_BAD_BLOCK_ID);
      }
      return row;
    };
    auto load = [&](const CUtensorMap* tm, int item, int row) {
      const int st = item % NS;
      if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kSlot);
      __syncwarp();
      if (loads) {
        uint8_t* dst = smem + C::kOffRing + st * C::kSlot;
        if constexpr (FP8) tma_load_3d(dst + blk * kBlockSize * D, tm, 0, h, row, &full[st]);
        else tma_load_3d(dst + hf * C::kHalf16 + blk * 2048, tm, hf * 64, h, row, &full[st]);
      }
    };
    auto slot_free = [&](int item) {
      const bool ok = item < NS || wait_or_abort(&empty[item % NS], ((item / NS) - 1) & 1, abort);
      return __all_sync(kFull, ok);
    };
    int cur = row_of(0), nxt = row_of(1), ahead = row_of(2);
    if constexpr (!FP8) {
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, (WIDE ? 2 : 1) * C::kQTile);
#pragma unroll
        for (int t = 0; t < (WIDE ? 2 : 1); ++t)
#pragma unroll
          for (int c = 0; c < C::kHalves; ++c)
            tma_load_3d(smem + C::kOffQ + t * C::kQTile + c * C::kHalf16, &tm_q, c * 64, h * G, w.tok0 + t * tile_tok,
                        q_full);
      }
    }
    load(&tm_k, 0, cur);
    int issued = 1;
    bool ok = true;
    for (int j = 0; j < nstep; ++j) {
      if (j + 1 < nstep) {
        if (!(ok = slot_free(k_item(j + 1)))) break;
        load(&tm_k, k_item(j + 1), nxt);
        issued = k_item(j + 1) + 1;
      }
      if (!(ok = slot_free(v_item(j)))) break;
      load(&tm_v, v_item(j), cur);
      issued = v_item(j) + 1;
      if (lane == 0 && (FP8 || j >= first_cut)) mbar_arrive(&v_sent[(FP8 ? j : j - first_cut) & 3]);
      cur = nxt;
      nxt = ahead;
      ahead = row_of(j + 3);
    }
    if (lane == 0) {
      if (!ok && !*abort) fail();
      // nothing may be in flight when the CTA exits: the last tiles issued have landed
      for (int i = max(0, issued - NS); i < issued; ++i)
        if (!mbar_wait(&full[i % NS], (i / NS) & 1)) break;
      if (!FP8) mbar_wait(q_full, 0);
    }
    __syncwarp();
  } else if (!soft) {
    // ======================================================================== V: cut tiles, expansion
    const int ft = threadIdx.x - C::kFixWarp0 * 32;  // 0 .. 63
    auto note = [&](int kind, int dim, int key) {
      atomicMin(&poison[kind * D + dim], key);
      *poisoned = 1;
    };
    const int j_first = FP8 ? 0 : first_cut;
    for (int j = j_first; j < nstep; ++j) {
      const int item = v_item(j);
      // the parity of `full` means this load only once it is issued (the slot's loads before it
      // are not waited for here); v_sent itself is at most one phase ahead: step j + 4 goes out
      // after V of step j, or of a later one, was consumed (bf16: at most 3 cut steps)
      const int sent = FP8 ? j : j - first_cut;
      bool ok = wait_or_abort(&v_sent[sent & 3], (sent >> 2) & 1, abort);
      if (ok) ok = wait_or_abort(&full[item % NS], (item / NS) & 1, abort);
      if constexpr (FP8)
        if (ok && j >= 2) ok = wait_or_abort(&exp_free[j & 1], ((j >> 1) - 1) & 1, abort);
      if (!ok && !*abort) fail();
      const int key0 = (k0 + j) * C::kKeys;
      const int seen = lim_min - key0, end = w.ctx - key0;  // rows below seen: every row's; from end on: no row's
      uint8_t* src = smem + C::kOffRing + (item % NS) * C::kSlot;
      if (ok) {
        if constexpr (FP8) {
          constexpr int kChunks = D / 8;  // 8-code pieces of a row
          constexpr int kStep = 64 / kChunks;
          const int c = ft % kChunks, r0 = ft / kChunks;
          const uint32_t ex = smem_u32(smem + C::kOffExp + (j & 1) * C::kTile16) + (c >> 3) * C::kHalf16;
#pragma unroll 4
          for (int row = r0; row < C::kKeys; row += kStep) {
            uint2 v = *reinterpret_cast<const uint2*>(src + row * D + c * 8);
            if (j >= first_cut && row >= seen) {
              if (row >= end) {
                v = make_uint2(0u, 0u);
              } else {
                uint8_t* b = reinterpret_cast<uint8_t*>(&v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if ((b[e] & 0x7f) == 0x7f) {  // NaN, the only E4M3 code that is not finite
                    note(0, c * 8 + e, key0 + row);
                    b[e] = 0;
                  }
              }
            }
            st_shared_v4(ex + (row >> 3) * 1024 + (row & 7) * 128 + (((c & 7) ^ (row & 7)) << 4), e4m3_lo(v.x),
                         e4m3_hi(v.x), e4m3_lo(v.y), e4m3_hi(v.y));
          }
        } else {
          constexpr int kChunks = D / 8;
          constexpr int kStep = 64 / kChunks;
          const int c = ft % kChunks;
#pragma unroll 2
          for (int row = max(0, seen) + ft / kChunks; row < C::kKeys; row += kStep) {
            uint4* at = reinterpret_cast<uint4*>(src + (c >> 3) * C::kHalf16 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
            if (row >= end) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
              uint4 v = *at;
              uint32_t* e = reinterpret_cast<uint32_t*>(&v);
              uint32_t odd = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) odd |= ((e[k] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
              if (odd) {  // exponent all ones somewhere
                for (int k = 0; k < 8; ++k) {
                  const uint32_t x = (e[k >> 1] >> (16 * (k & 1))) & 0xffffu;
                  if ((x & 0x7f80u) == 0x7f80u) {
                    note((x & 0x7fu) ? 0 : (x & 0x8000u) ? 2 : 1, c * 8 + k, key0 + row);
                    e[k >> 1] &= (k & 1) ? 0x0000ffffu : 0xffff0000u;
                  }
                }
                *at = v;
              }
            }
          }
        }
      }
      fence_proxy_async_smem();  // the tile is read by the tensor cores
      if (named_sync_or(1, 64, *abort != 0)) break;
      if (ft == 0) {
        if constexpr (FP8) {
          mbar_arrive(&empty[item % NS]);
          mbar_arrive(&fixed[j & 1]);
        } else {
          mbar_arrive(&fixed[j - first_cut]);
        }
      }
    }
  } else {
    // ======================================================================== softmax
    const int g = warp >> 2;  // accumulators: the tile (wide) or the parity of the steps (narrow)
    const int nloc = n_of[g];
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t scol = tmem + lane_base + C::kColS + 128 * g;
    const uint32_t ocol = tmem + lane_base + C::kColO + D * g;
    float sscale = p.score_scale;

    if constexpr (FP8) {
      // this row of Q as hi and lo codes, times 2^e that takes its largest into [128, 256)
      if (WIDE || g == 0) {
        const uint4* qr = reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(w.tok0 + my_i) * p.q_stride + hq * D);
        uint4 v[D / 8];
        float top = 0.f;
        bool odd = false;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          v[c] = rv ? qr[c] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t e[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            top = fmaxf(top, fmaxf(fabsf(bf16_lo(e[k])), fabsf(bf16_hi(e[k]))));
            odd |= ((((e[k] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0u);
          }
        }
        int ex = 0;
        if (top > 0.f && !odd) ex = 7 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
        ex = min(ex, 126);  // rows below 2^-119: their codes lose what lies under 2^-135
        const float up = __uint_as_float(static_cast<uint32_t>(max(ex, -126) + 127) << 23);
        const uint32_t qt = q_base + (WIDE ? g : 0) * C::kQTile;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {  // 16 codes: one 16-byte piece of the row
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a = u4_word(v[2 * c + k / 2], 2 * (k & 1)), b = u4_word(v[2 * c + k / 2], 2 * (k & 1) + 1);
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
        if (lane == 0) mbar_arrive(q_full);
        // the row's scores come out times 2^ex; a row with a NaN or an infinity has no value
        sscale = odd ? __int_as_float(0x7fffffff) : sscale * p.scales[h] / up;
      }
      if constexpr (!WIDE) {  // group 1 works on the same rows: it takes their factors over
        float* shared_scale = reinterpret_cast<float*>(smem + C::kOffQ + C::kQTile);  // no second Q tile here
        if (g == 0) shared_scale[r] = sscale;
        named_sync(2, 256);
        if (g == 1) sscale = shared_scale[r];
        named_sync(2, 256);
      }
    }

    const int my_lim = lim_of(my_i);
    // keys below every lim of the warp's rows need no mask (rows that do not exist do not count)
    const int warp_lim = __reduce_min_sync(kFull, rv ? my_lim : 0x7fffffff);
    const bool idle = !__any_sync(kFull, rv);  // no row of the warp exists: its products go nowhere
    float m_used = -INFINITY, l = 0.f;
    bool dead = false;
    for (int t = 0; t < nloc; ++t) {
      const int key0 = (k0 + (WIDE ? t : 2 * t + g)) * C::kKeys;
      bool ok = wait_or_abort(&s_full[g], t & 1, abort);
      if (!__all_sync(kFull, ok)) {  // tensor-memory loads are warp-collective: leave as a warp
        if (!*abort) fail();
        dead = true;
        break;
      }
      tc_fence_after();
      if (!idle) {
        float s[2][64];
        tmem_ld64(scol, s[0]);
        tmem_ld64(scol + 64, s[1]);
        if (key0 + C::kKeys > warp_lim) {
          const int left = my_lim - key0;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= left) s[i >> 6][i & 63] = -INFINITY;
        }
        float mx0 = s[0][0], mx1 = s[0][1];
#pragma unroll
        for (int i = 2; i < 128; i += 2) {
          mx0 = fmaxf(mx0, s[i >> 6][i & 63]);
          mx1 = fmaxf(mx1, s[i >> 6][(i & 63) + 1]);
        }
        const float mx = fmaxf(mx0, mx1) * sscale;
        const bool grow = mx > m_used + C::kLazy;
        float alpha = 1.f;
        if (grow) {
          alpha = fast_exp2(m_used - mx);  // 0 while the row has seen nothing
          l *= alpha;
          m_used = mx;
        }
        // a row that has seen nothing yet keeps reference 0: its weights are 2^-inf = 0
        const float negm = (m_used == -INFINITY ? 0.f : -m_used) + C::kBias;
        const float2 sc2 = make_float2(sscale, sscale), nm2 = make_float2(negm, negm);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pw[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float2 x = ffma2(make_float2(s[hf][2 * i], s[hf][2 * i + 1]), sc2, nm2);
            x.x = fast_exp2(x.x);
            x.y = fast_exp2(x.y);
            sum = fadd2(sum, x);
            pw[i] = pack16<FP8>(x.x, x.y);
          }
          tmem_st32u(scol + 32 * hf, pw);
        }
        l += sum.x + sum.y;
        // P V of the previous step was issued before these scores: it is done
        if (t > 0 && __any_sync(kFull, grow)) {
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            float o[32];
            tmem_ld32(ocol + 32 * ch, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            tmem_st32(ocol + 32 * ch, o);
          }
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[g]);
    }

    // ---- epilogue: the output row, or its record
    if (!dead && nloc > 0) {
      const bool ok = wait_or_abort(&o_full[g], 0, abort);
      if (!__all_sync(kFull, ok)) {
        if (!*abort) fail();
        dead = true;
      }
      tc_fence_after();
    }
    float* join = reinterpret_cast<float*>(smem + C::kOffRing);  // narrow: [D][128] of group 1
    float2* join_ml = reinterpret_cast<float2*>(smem + C::kOffQ + C::kQTile);  // narrow: [128]
    float a0 = 1.f, a1 = 0.f;
    if constexpr (!WIDE) {
      // every step of both groups is done before the ring is written over: group 1 finished
      // its own, and group 0's last products were waited for above
      dead = named_sync_or(2, 256, dead);
      if (g == 1 && !dead && nloc > 0) {
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          float o[32];
          tmem_ld32(ocol + 32 * ch, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) join[(32 * ch + i) * 128 + r] = o[i];
        }
        join_ml[r] = make_float2(m_used, l);
      }
      named_sync(2, 256);
      if (g == 0 && !dead && n_of[1] > 0) {
        const float2 o = join_ml[r];
        const float top = fmaxf(m_used, o.x);
        a0 = m_used == -INFINITY ? 0.f : fast_exp2(m_used - top);
        a1 = o.x == -INFINITY ? 0.f : fast_exp2(o.x - top);
        l = l * a0 + o.y * a1;
        m_used = top;
      }
    }
    if (!dead && nloc == 0 && WIDE) {  // a tile whose rows see nothing of this split
      if (rv) {
        if (p.splits > 1) {
          p.part_ml[rec] = make_float2(-INFINITY, 0.f);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse != nullptr) p.lse[orow] = -INFINITY;
        }
      }
    } else if (!dead && (WIDE || g == 0) && !idle) {
      const bool split_out = p.splits > 1;
      const bool bad = *poisoned != 0;
      float inv = 1.f;
      if (!split_out) {
        inv = l > 0.f || l != l ? 1.f / l : 0.f;
        if constexpr (FP8) inv *= p.scales[p.hkv + h];
        if (rv && p.lse != nullptr)
          p.lse[orow] = l == 0.f ? -INFINITY : (m_used - C::kBias + log2f(l)) * 0.69314718055994531f;
      } else if (rv) {
        p.part_ml[rec] = make_float2(m_used, l);
      }
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        float o[32];
        tmem_ld32(ocol + 32 * ch, o);
        if constexpr (!WIDE) {
          if (n_of[1] > 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = o[i] * a0 + join[(32 * ch + i) * 128 + r] * a1;
          }
        }
        if (bad) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int dim = 32 * ch + i;
            if (poison[dim] < my_lim) o[i] = __int_as_float(0x7fffffff);
            if (poison[D + dim] < my_lim) o[i] += INFINITY;
            if (poison[2 * D + dim] < my_lim) o[i] -= INFINITY;
          }
        }
        if (rv) {
          if (split_out) {
            float4* dst = reinterpret_cast<float4*>(p.part_acc + rec * D + 32 * ch);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + 32 * ch);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack_bf16(o[8 * i] * inv, o[8 * i + 1] * inv),
                                  pack_bf16(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                  pack_bf16(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                  pack_bf16(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
          }
        }
      }
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

template <int D, bool FP8, bool WIDE>
static cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PrefillParams& p,
                          int tile_slots, cudaStream_t stream) {
  using C = PrefillCfg<D, FP8>;
  auto kern = prefill_tc_kernel<D, FP8, WIDE>;
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

cudaError_t launch_prefill(int d, bool fp8, bool wide, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, const PrefillParams& p, int tile_slots, cudaStream_t stream) {
  if (d == 64) {
    if (fp8)
      return wide ? launch<64, true, true>(tq, tk, tv, p, tile_slots, stream)
                  : launch<64, true, false>(tq, tk, tv, p, tile_slots, stream);
    return wide ? launch<64, false, true>(tq, tk, tv, p, tile_slots, stream)
                : launch<64, false, false>(tq, tk, tv, p, tile_slots, stream);
  }
  if (fp8)
    return wide ? launch<128, true, true>(tq, tk, tv, p, tile_slots, stream)
                : launch<128, true, false>(tq, tk, tv, p, tile_slots, stream);
  return wide ? launch<128, false, true>(tq, tk, tv, p, tile_slots, stream)
              : launch<128, false, false>(tq, tk, tv, p, tile_slots, stream);
}

}  // namespace pkv
