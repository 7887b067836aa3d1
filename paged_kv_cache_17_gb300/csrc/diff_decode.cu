// diff_decode.cu -- differential attention of one token per sequence over the paged cache.
//
// Mathematics.  Per (sequence, pair of kv heads) and 16-token block, as two small products on the tensor cores
// (mma.sync m16n8k16, fp32 accumulation), with an online softmax per column between them, by a reference that moves
// when a score passes it by more than 2^8:
//   S^T [16 tokens x C] = K [16 x 128] . Q^T [128 x C],    O^T [128 x C] += V^T [128 x 16] . P^T [16 x C]
// A row of K holds the pair's two key heads side by side, a row of V is the pair's value.  The columns are (map,
// query head of the group): a column's query fills its map's half of the 128, the other half is zero, so one
// product gives the scores of both maps and the second one both outputs from one reading of V.  Groups of up to
// four heads make 8 columns, an MMA's N; a group of eight makes two tiles of 8, one map each, whose scores need
// only that map's half of K.  bf16 pools: the halves of K are summed apart, and a column takes its map's sum, because the
// zeros of the other half would make NaN of an infinite key there (E4M3 has no infinity, and a NaN key of either map
// is NaN in the output).  The weights enter as a 16-bit hi + lo pair: bf16, to 2^-16 of a weight; E4M3 pools, fp16
// times 2^7 (with a score 2^8 past the reference 2^15, and fp16 holds 2^16): to 2^-22, or, below that, 2^-32 of the
// column's largest weight.  (Without the factor that floor is 2^-25 of the reference, and keys that much behind, all
// of the output where the largest's value is 0 or the two maps cancel it, are lost.)
//   E4M3 pools: the codes go from the ring straight into the fragments, expanded to fp16 (exact); q is scaled per
// column by a power of two into fp16's range; K's scales (one per map) go into the scores' factor, V's into the
// output.
//
// Contexts are cut into runs of blocks, one CTA each: a producer warp that streams K and V by TMA, a block's pair
// as one box each, and two consumer warps that take the blocks in turn, each with its own statistics.  A sequence
// of one run ends here (difference, norm, store); others leave a record per map and the merge kernel ends them.
// Where few requests leave most SMs idle, a sequence's runs, at most eight, are a thread-block cluster instead: they
// read each other's states through distributed shared memory and end the rows themselves, without a second kernel.
//
// What bounds it.  Reading K and V once, for bf16 pools: 64 requests of 512 to 4096 tokens, 64 + 16 heads: 97 us = 6.2
// TB/s of all bytes, 91 % of the measured copy; 8 of 32 to 128 thousand, 128 + 16 heads: 374 us = 6.55 TB/s, 97 %
// (three consumer warps and a 48 KiB ring for two tiles; two and 32 KiB: 395).  E4M3, 33 of 1000 to 9001, 16 heads of
// their own: 68 us = 5.0 TB/s (71 with a maximum over the lanes for every block; 128 heads: 90, 100): some 360
// instructions a block from two warps a CTA, half of the issue slots, and a wave of uneven CTAs (an SM is busy 80 % of
// the time); two blocks at a time in a warp, or the next block's scores under this one's softmax, need more than the
// 96 registers that let six CTAs share an SM (79, 91), four warps a CTA the same; 80 registers for eight CTAs spill
// (81).  One request of 777 tokens: 7.2 us in a graph, launch and five dependent round trips.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "diff.cuh"
#include "diff_out.cuh"
#include "mma_ops.cuh"
#include "pkv_device.cuh"

namespace pkv {

template <int NT, bool FP8, bool CLUSTER>
struct DiffDecodeCfg {
  static constexpr int kWarps = CLUSTER ? 4 : NT == 2 ? 3 : 2;  // consumers
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kTile = kBlockSize * kDiffW * (FP8 ? 1 : 2);
  static constexpr int kStages = (CLUSTER ? 65536 : NT == 2 ? 49152 : 32768) / (2 * kTile);
  static constexpr int kRing = 2 * kStages * kTile;
  static constexpr int kCols = 8 * NT;
  static constexpr int kBytes = 1008 + kRing + 2 * kStages * 8;  // 1008: alignment slack
  static_assert(kStages % kWarps == 0, "each stage is always consumed by the same warp");
  static_assert(kWarps * kCols * (2 + kDiffW) * 4 <= kRing, "the warps' states fit in the ring");
};

// One box: the 16 rows of a block, both heads of the pair.  bf16: two groups of eight rows, each group's halves
// side by side, 128-byte swizzled; E4M3: rows of 128 codes, swizzled
template <bool FP8>
__device__ __forceinline__ void diff_box(void* dst, const CUtensorMap* tm, int pair, int row, uint64_t* bar) {
  if constexpr (FP8) {
    tma_load_3d(dst, tm, 0, pair, row, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%5, %5, %5, %2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(row >> 3), "r"(pair), "r"(smem_u32(bar)), "r"(0)
        : "memory");
  }
}

// 16-byte piece c (of 16) of row r in a bf16 tile
__device__ __forceinline__ uint32_t diff_at(uint32_t base, int r, int c) {
  return base + (r >> 3) * 2048 + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Every CTA of the cluster has come here; what it wrote to shared memory before is seen
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address in CTA `rank` of the cluster of what is at addr here
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_rank(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ float4 ld_rank4(uint32_t addr) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}

template <int NT, bool FP8, bool CLUSTER>
__global__ void __launch_bounds__((DiffDecodeCfg<NT, FP8, CLUSTER>::kThreads))
    diff_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const DiffParams p) {
  using C = DiffDecodeCfg<NT, FP8, CLUSTER>;
  constexpr int NW = C::kWarps, ST = C::kStages, KS = kDiffW / 16, MT = kDiffW / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* k_tiles = smem;
  uint8_t* v_tiles = smem + ST * C::kTile;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* empty = full + ST;

  const int pair = blockIdx.x, b = blockIdx.y, s = blockIdx.z, G = p.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;

  // Shared prefixes: this grid runs beside the prefix pass (nothing here reads its records), and is complete only
  // after it, because one CTA waits for it at its end.
  const bool beside = p.pre_slots > 0;
  if (!beside) pdl_wait();
  auto leave = [&]() {
    if constexpr (CLUSTER) cluster_sync();  // nobody reads this CTA's shared memory any more
    if (beside && (blockIdx.x | blockIdx.y | blockIdx.z) == 0) pdl_wait();
  };

  int len = p.context_lens[b];
  const int blk0 = s * p.split_blocks;
  const int32_t* table = p.block_tables + static_cast<int64_t>(b) * p.max_blocks + blk0;
  // the first 32 ids, asked for beside the length (valid entries of the row; past the context they are not used)
  int ids = warp == NW && blk0 + lane < p.max_blocks ? table[lane] : 0;
  // Q^T: column gid (of each tile), k-step kk: 16 of the 128 elements, the first map's for kk < 4.  E4M3: in
  // the order of the codes that a lane reads, 16 consecutive ones of each half.  (Asked for beside the length too, and
  // waited for by the warps that use it alone, so that K and V are asked for one round trip after the length is.)
  uint32_t qb[KS][2];
  if (warp < NW) {
    const int g = NT == 2 ? gid : gid & 3;
    const uint32_t* qr =
        reinterpret_cast<const uint32_t*>(p.q + b * p.q_stride + static_cast<int64_t>(pair * G + (g < G ? g : 0)) * kDiffW);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const bool live = g < G && (NT == 2 || (gid >> 2) == kk / 4);
      const int w0 = FP8 ? (kk / 4) * 32 + tig * 8 + (kk & 3) * 2 : kk * 8 + tig;
      qb[kk][0] = live ? qr[w0] : 0u;
      qb[kk][1] = live ? qr[w0 + (FP8 ? 1 : 4)] : 0u;
    }
  }
  if (len < 0 || len > p.max_context_len) {
    if (threadIdx.x == 0 && s == 0) set_flag(p.status, PKV_DEVFLAG_BAD_CONTEXT_LEN);
    len = max(0, min(len, p.max_context_len));
  }
  const int nblk = (len + kBlockSize - 1) / kBlockSize;
  const int nsplit = (nblk + p.split_blocks - 1) / p.split_blocks;
  const int prefix = beside ? p.seq_prefix[b] : -1;
  const bool with_prefix = prefix >= 0;
  const int head0 = pair * G;
  if (s >= nsplit) {
    if (s == 0 && !with_prefix) {  // no keys at all
      const float zero[4] = {};
      for (int g = warp; g < G; g += NW + 1) diff_store(p, b, head0 + g, true, zero, zero, lane);
    }
    if constexpr (CLUSTER) cluster_sync();
    leave();
    return;
  }
  const int nloc = min(nblk - blk0, p.split_blocks);

  if (threadIdx.x == NW * 32) tma_prefetch_desc(&tm_k), tma_prefetch_desc(&tm_v);
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    fence_mbar_init();
  }
  __syncthreads();

  int qexp[NT] = {};
  if (warp < NW) {
    if constexpr (FP8) {  // the column's largest goes to 2^13 .. 2^14
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float top = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
          if (NT == 1 || kk / 4 == t)
#pragma unroll
            for (int e = 0; e < 2; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(qb[kk][e])), fabsf(bf16_hi(qb[kk][e]))));
        top = fmaxf(top, shfl_xor(top, 1));
        top = fmaxf(top, shfl_xor(top, 2));
        qexp[t] = top > 0.f && top < INFINITY ? 13 - ilogbf(top) : 0;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
          if (NT == 1 || kk / 4 == t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              qb[kk][e] = pack_f16(ldexpf(bf16_lo(qb[kk][e]), qexp[t]), ldexpf(bf16_hi(qb[kk][e]), qexp[t]));
      }
    }
  }
  // factors of this thread's columns 2 tig and 2 tig + 1 of each tile
  float factor[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    factor[t][0] = factor[t][1] = p.score_scale;
    if constexpr (FP8) {
      const float ks = p.score_scale * p.scales[2 * pair + (NT == 2 ? t : tig >> 1)];
      factor[t][0] = ldexpf(ks, -__shfl_sync(kFull, qexp[t], 8 * tig));
      factor[t][1] = ldexpf(ks, -__shfl_sync(kFull, qexp[t], 8 * tig + 4));
    }
  }

  constexpr float kLazy = 8.f, kBias = FP8 ? 7.f : 0.f;  // weights are taken times 2^kBias: by a lower reference
  float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t][0] = m[t][1] = kDiffNothing;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[t][mt][0] = o[t][mt][1] = o[t][mt][2] = o[t][mt][3] = 0.f;
  }

  if (warp == NW) {
    // ================================================================ producer
    int issued = 0;
    bool ok = true;
    for (int base = 0; base < nloc && ok; base += 32) {
      const int next = base + 32 + lane < nloc ? table[base + 32 + lane] : 0;
      if (base + lane < nloc && (ids < 0 || ids >= p.num_blocks)) set_flag(p.status, PKV_DEVFLAG_BAD_BLOCK_ID);
      const int cnt = min(32, nloc - base);
      for (int k = 0; k < cnt && ok; ++k) {
        const int id = __shfl_sync(kFull, ids, k), it = base + k, st = it % ST;
        if (lane == 0) {
          if (it >= ST && !mbar_wait(&empty[st], ((it / ST) - 1) & 1)) {
            set_flag(p.status, PKV_DEVFLAG_WAIT_TIMEOUT);
            ok = false;
          } else {
            // an id outside the pool: a box entirely outside the tensor, which reads zeros
            const int row = id >= 0 && id < p.num_blocks ? id * kBlockSize : -kBlockSize;
            mbar_arrive_expect_tx(&full[st], 2 * C::kTile);
            diff_box<FP8>(k_tiles + st * C::kTile, &tm_k, pair, row, &full[st]);
            diff_box<FP8>(v_tiles + st * C::kTile, &tm_v, pair, row, &full[st]);
          }
        }
        ok = __shfl_sync(kFull, ok, 0);
        if (ok) issued = it + 1;
      }
      ids = next;
    }
    if (lane == 0)  // nothing may be in flight when the ring is used for something else
      for (int it = max(0, issued - ST); it < issued; ++it)
        if (!mbar_wait(&full[it % ST], (it / ST) & 1)) {
          set_flag(p.status, PKV_DEVFLAG_WAIT_TIMEOUT);
          break;
        }
    __syncwarp();
  } else {
    // ================================================================ consumers
    const int mi = lane >> 3;
    for (int it = warp; it < nloc; it += NW) {
      const int st = it % ST;
      if (!mbar_wait(&full[st], (it / ST) & 1)) {
        if (lane == 0) set_flag(p.status, PKV_DEVFLAG_WAIT_TIMEOUT);
        break;
      }
      __syncwarp();
      uint8_t *kt = k_tiles + st * C::kTile, *vt = v_tiles + st * C::kTile;
      const uint32_t kb = smem_u32(kt), vb = smem_u32(vt);
      const int valid = min(kBlockSize, len - (blk0 + it) * kBlockSize);  // >= 1
      if (valid < kBlockSize) {  // what a page holds past the context (NaN included) must not meet weight 0
        constexpr int kPieces = C::kTile / kBlockSize / 16;
        for (int i = lane; i < (kBlockSize - valid) * kPieces; i += 32) {
          const int r = valid + i / kPieces, c = i % kPieces;
          const uint32_t at = FP8 ? vb + e4m3_off<kDiffW>(r, c) : diff_at(vb, r, c);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0u) : "memory");
        }
        __syncwarp();
      }
      // ---- scores: rows = tokens gid, gid + 8; columns 2 tig, 2 tig + 1
      constexpr int kSums = FP8 ? NT : 2;  // of K's halves together, or each
      float sc[kSums][4] = {};
      uint32_t vr[4][4];  // E4M3: codes 16 gid .. + 15 of tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
      if constexpr (FP8) {
        uint4 kr[2][2];  // tokens gid, gid + 8; 16 codes of each half
        const int odd = gid & 1;  // (rows next to each other start with different halves: no bank conflicts)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 x = *reinterpret_cast<const uint4*>(kt + e4m3_off<kDiffW>(gid + 8 * r, odd * 4 + tig));
          const uint4 y = *reinterpret_cast<const uint4*>(kt + e4m3_off<kDiffW>(gid + 8 * r, (odd ^ 1) * 4 + tig));
          kr[r][0] = odd ? y : x;
          kr[r][1] = odd ? x : y;
        }
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          const uint32_t w0 = u4_word(kr[0][kk / 4], kk & 3), w1 = u4_word(kr[1][kk / 4], kk & 3);
          mma16<FP8>(sc[kSums == 2 ? kk / 4 : 0], e4m3_lo(w0), e4m3_lo(w1), e4m3_hi(w0), e4m3_hi(w1), qb[kk][0], qb[kk][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(vt + e4m3_off<kDiffW>(2 * tig + (i & 1) + 8 * (i >> 1), gid));
          vr[i][0] = v.x, vr[i][1] = v.y, vr[i][2] = v.z, vr[i][3] = v.w;
        }
        // both tiles are in registers: the slot goes back (generic reads, then the refill by the async proxy)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      } else {
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4(diff_at(kb, (lane & 7) + 8 * (mi & 1), 2 * kk + (mi >> 1)), a0, a1, a2, a3);
          mma16<FP8>(sc[kk / 4], a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
        }
        if constexpr (NT == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[0][e] = tig < 2 ? sc[0][e] : sc[1][e];
        }
      }
      uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sc[t][e] = gid + 8 * (e >> 1) < valid ? sc[t][e] * factor[t][e & 1] : -INFINITY;
        // ---- online softmax: the reference moves, to kBias below the block's maximum over the lanes of equal tig, when a
        // score passes that by more than 2^8 (any reference gives the same quotient): rarely, and only then the lanes
        // are asked
        const float b0 = fmaxf(sc[t][0], sc[t][2]), b1 = fmaxf(sc[t][1], sc[t][3]);
        if (__any_sync(kFull, b0 > m[t][0] + (kLazy + kBias) || b1 > m[t][1] + (kLazy + kBias))) {
          float n0 = b0, n1 = b1;
#pragma unroll
          for (int i = 4; i <= 16; i <<= 1) {
            n0 = fmaxf(n0, shfl_xor(n0, i));
            n1 = fmaxf(n1, shfl_xor(n1, i));
          }
          n0 = fmaxf(n0 - kBias, m[t][0]);
          n1 = fmaxf(n1 - kBias, m[t][1]);
          const float a0 = fast_exp2(m[t][0] - n0), a1 = fast_exp2(m[t][1] - n1);  // 0 at the start
          m[t][0] = n0;
          m[t][1] = n1;
          l[t][0] *= a0;
          l[t][1] *= a1;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            o[t][mt][0] *= a0;
            o[t][mt][1] *= a1;
            o[t][mt][2] *= a0;
            o[t][mt][3] *= a1;
          }
        }
        const float p0 = fast_exp2(sc[t][0] - m[t][0]), p1 = fast_exp2(sc[t][1] - m[t][1]);
        const float p2 = fast_exp2(sc[t][2] - m[t][0]), p3 = fast_exp2(sc[t][3] - m[t][1]);
        l[t][0] += p0 + p2;
        l[t][1] += p1 + p3;
        // ---- P^T as the B operand: (token, column pair) fragments turned to (column, token pair)
        uint32_t h01, l01, h23, l23;
        split16<FP8>(p0, p1, h01, l01);
        split16<FP8>(p2, p3, h23, l23);
        bh[t][0] = movm_t(h01);
        bh[t][1] = movm_t(h23);
        bl[t][0] = movm_t(l01);
        bl[t][1] = movm_t(l23);
      }
      if constexpr (FP8) {
        // word i of a token's codes: rows gid and gid + 8 of m-tiles 2 i and 2 i + 1 (dims 16 gid + 4 i ..)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x01 = __byte_perm(vr[0][i], vr[1][i], 0x5140), y01 = __byte_perm(vr[0][i], vr[1][i], 0x7362);
          const uint32_t x89 = __byte_perm(vr[2][i], vr[3][i], 0x5140), y89 = __byte_perm(vr[2][i], vr[3][i], 0x7362);
          const uint32_t e0 = e4m3_lo(x01), e1 = e4m3_hi(x01), e2 = e4m3_lo(x89), e3 = e4m3_hi(x89);
          const uint32_t f0 = e4m3_lo(y01), f1 = e4m3_hi(y01), f2 = e4m3_lo(y89), f3 = e4m3_hi(y89);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16<FP8>(o[t][2 * i], e0, e1, e2, e3, bh[t][0], bh[t][1]);
            mma16<FP8>(o[t][2 * i], e0, e1, e2, e3, bl[t][0], bl[t][1]);
            mma16<FP8>(o[t][2 * i + 1], f0, f1, f2, f3, bh[t][0], bh[t][1]);
            mma16<FP8>(o[t][2 * i + 1], f0, f1, f2, f3, bl[t][0], bl[t][1]);
          }
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t a0, a1, a2, a3;
          ldsm_x4_t(diff_at(vb, (lane & 7) + 8 * (mi >> 1), 2 * mt + (mi & 1)), a0, a1, a2, a3);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16<FP8>(o[t][mt], a0, a1, a2, a3, bh[t][0], bh[t][1]);
            mma16<FP8>(o[t][mt], a0, a1, a2, a3, bl[t][0], bl[t][1]);
          }
        }
        // read by ldmatrix (generic proxy), refilled by TMA (async proxy)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
    }
  }

  // ================================================================ the consumers' states together
  __syncthreads();  // every issued copy has landed and been read
  constexpr int NC = C::kCols;
  float* ms = reinterpret_cast<float*>(smem);  // [NW][NC] maximum
  float* ls = ms + NW * NC;                    // [NW][NC] sum
  float* os = ls + NW * NC;                    // [NW][NC][128] unnormalised output
  if (warp < NW) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[t][j];
#pragma unroll
        for (int i = 4; i <= 16; i <<= 1) sum += shfl_xor(sum, i);
        const int c = warp * NC + 8 * t + 2 * tig + j;
        if (gid == 0) {
          ms[c] = m[t][j];
          ls[c] = sum;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int d0 = FP8 ? 16 * gid + 2 * mt : 16 * mt + gid;
          os[c * kDiffW + d0] = o[t][mt][j];
          os[c * kDiffW + d0 + (FP8 ? 1 : 8)] = o[t][mt][2 + j];
        }
      }
  }
  __syncthreads();
  const bool ends = nsplit == 1 && !with_prefix;
  const float vs = FP8 ? p.scales[2 * (p.pairs + pair) + lane / 16] : 1.f;
  for (int g = warp; g < G; g += NW + 1) {
    float y[2][4];
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      const int c = NT == 2 ? 8 * map + g : 4 * map + g;
      float top = ms[c];
#pragma unroll
      for (int w = 1; w < NW; ++w) top = fmaxf(top, ms[w * NC + c]);
      float den = 0.f, num[4] = {};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        // (a warp without blocks has reference kDiffNothing and sum 0, one whose scores were all NaN kDiffNothing and NaN)
        const float f = fast_exp2(ms[w * NC + c] - top);
        const float4 x = *reinterpret_cast<const float4*>(os + (w * NC + c) * kDiffW + 4 * lane);
        den = fmaf(f, ls[w * NC + c], den);
        num[0] = fmaf(f, x.x, num[0]);
        num[1] = fmaf(f, x.y, num[1]);
        num[2] = fmaf(f, x.z, num[2]);
        num[3] = fmaf(f, x.w, num[3]);
      }
      if (ends) {
        const float by = vs / den;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[map][i] = num[i] * by;
      } else if constexpr (CLUSTER) {  // the run's state, in the place of the first warp's
        __syncwarp();
        *reinterpret_cast<float4*>(os + c * kDiffW + 4 * lane) = make_float4(num[0], num[1], num[2], num[3]);
        if (lane == 0) {
          ms[c] = top;
          ls[c] = den;
        }
      } else {
        const int64_t rec = (static_cast<int64_t>((p.pre_slots + s) * 2 + map) * p.rows + b) * p.heads + head0 + g;
        *reinterpret_cast<float4*>(p.part_acc + rec * kDiffW + 4 * lane) = make_float4(num[0], num[1], num[2], num[3]);
        if (lane == 0) p.part_ml[rec] = make_float2(top, den);
      }
    }
    if (ends) diff_store(p, b, head0 + g, false, y[0], y[1], lane);
  }
  if constexpr (CLUSTER) {
    cluster_sync();
    // head g of the group is ended by the cluster's CTA g mod nsplit; lane j holds run j's maximum and sum
    for (int g = s + warp * nsplit; !ends && g < G; g += (NW + 1) * nsplit) {
      float y[2][4];
      float4 x[2][kDiffCluster];
      float top[2], den[2];
#pragma unroll
      for (int map = 0; map < 2; ++map) {
        const int c = NT == 2 ? 8 * map + g : 4 * map + g, j = min(lane, nsplit - 1);
        top[map] = ld_rank(map_rank(smem_u32(ms + c), j));
        den[map] = ld_rank(map_rank(smem_u32(ls + c), j));
#pragma unroll
        for (int i = 0; i < kDiffCluster; ++i)
          if (i < nsplit) x[map][i] = ld_rank4(map_rank(smem_u32(os + c * kDiffW + 4 * lane), i));
      }
#pragma unroll
      for (int map = 0; map < 2; ++map) {
        const float own = top[map];
        float all = own, sum = lane < nsplit ? den[map] : 0.f;
#pragma unroll
        for (int k = 4; k >= 1; k >>= 1) all = fmaxf(all, shfl_xor(all, k));  // (lanes 0-7; the others repeat the last)
        all = __shfl_sync(kFull, all, 0);
        const float f = fast_exp2(own - all);
        sum *= f;
#pragma unroll
        for (int k = 4; k >= 1; k >>= 1) sum += shfl_xor(sum, k);
        sum = __shfl_sync(kFull, sum, 0);
        float num[4] = {};
#pragma unroll
        for (int i = 0; i < kDiffCluster; ++i) {
          const float w = __shfl_sync(kFull, f, i);
          if (i < nsplit) {
            num[0] = fmaf(w, x[map][i].x, num[0]);
            num[1] = fmaf(w, x[map][i].y, num[1]);
            num[2] = fmaf(w, x[map][i].z, num[2]);
            num[3] = fmaf(w, x[map][i].w, num[3]);
          }
        }
        const float by = vs / sum;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[map][k] = num[k] * by;
      }
      diff_store(p, b, head0 + g, false, y[0], y[1], lane);
    }
  }
  leave();
}

template <int NT, bool FP8, bool CLUSTER>
static cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p, cudaStream_t stream) {
  using C = DiffDecodeCfg<NT, FP8, CLUSTER>;
  auto kern = diff_decode_kernel<NT, FP8, CLUSTER>;
  static std::atomic<bool> configured[64] = {};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!configured[device].load(std::memory_order_acquire)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes)) != cudaSuccess) return e;
    configured[device].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.pairs), static_cast<unsigned>(p.batch), static_cast<unsigned>(p.max_splits));
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (CLUSTER) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = static_cast<unsigned>(p.max_splits);
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kern, tk, tv, p);
}

template <bool CLUSTER>
static cudaError_t launch_form(bool fp8, const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p,
                               cudaStream_t stream) {
  if (p.group <= 4) return fp8 ? launch<1, true, CLUSTER>(tk, tv, p, stream) : launch<1, false, CLUSTER>(tk, tv, p, stream);
  return fp8 ? launch<2, true, CLUSTER>(tk, tv, p, stream) : launch<2, false, CLUSTER>(tk, tv, p, stream);
}

cudaError_t launch_diff_decode(bool fp8, const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p,
                               cudaStream_t stream) {
  return p.cluster ? launch_form<true>(fp8, tk, tv, p, stream) : launch_form<false>(fp8, tk, tv, p, stream);
}

}  // namespace pkv
