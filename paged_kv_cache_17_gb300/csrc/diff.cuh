// diff.cuh -- parameters and launchers of differential attention over the paged cache (launched from
// pkv_api.cu): chunks of new tokens, one token per sequence, and one token per sequence over shared prefixes.
//
// Two kv heads 2n and 2n + 1 of 64 elements are side by side in a row of the pool, so the kernels see a pool of
// hkv / 2 heads of 128: its K row holds the keys of both maps, its V row is the pair's value.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {

constexpr int kDiffD = 64;            // elements of a head
constexpr int kDiffW = 2 * kDiffD;    // of a pair's value
constexpr int kDiffCluster = 8;       // the largest cluster that every launch may ask for
// The reference of keys that have no score above -inf: the lowest finite value, so that no difference of references
// or scores is inf - inf.  With the sum 0 beside it, such a row is 0 / 0; a row, or a run, without keys has -inf
constexpr float kDiffNothing = -3.402823466e38f;

struct DiffParams {
  const uint16_t* q;        // [rows][2 heads][64] bf16, rows q_stride apart
  int64_t q_stride;
  const int32_t* q_indptr;  // rows of the sequences, or NULL: row b is sequence b's
  const int32_t* block_tables;
  const int32_t* context_lens;
  const float* scales;      // E4M3: [2][2 pairs]
  const float* lambda;      // [heads] per row, lambda_stride apart
  int64_t lambda_stride;
  const uint16_t* norm_weight;  // [128] bf16, or NULL
  void* out;                // [rows][heads][128]
  uint32_t* status;
  const int32_t* seq_prefix;  // shared prefixes: >= 0 for the sequences that have one, or NULL
  // partial records, where a row's keys are split: of (slot, map, row, head) at index
  // ((slot * 2 + map) * rows + row) * heads + head; a shared prefix's slots first, then the row's own
  float2* part_ml;   // reference maximum (log2 units) and sum
  float* part_acc;   // [128], unnormalised, without V's scale
  int pre_slots;     // slots of a shared prefix (0: none)
  int split_blocks;  // 16-token blocks of one of a row's own slots
  int max_splits;    // own slots
  int cluster;       // one token: a sequence's runs (at most kDiffCluster) are a cluster and end its rows, no records
  int batch, rows;
  int heads, pairs, group;  // output heads, pairs of kv heads, heads / pairs
  int max_blocks, num_blocks, max_context_len;
  int causal, out_fp32;
  float score_scale;        // softmax_scale * log2(e)
  // chunks and prefix passes (diff_chunk.cu)
  const int32_t* member_seqs;  // prefix pass: rows of the members, q_indptr their ranges; max_members of one prefix
  int max_members, num_members;  // num_members: entries of member_seqs at most
  int split_tiles;          // 128-key steps of a slot
  int negate;               // softmax_scale is negative
  float score_size;         // |softmax_scale| * log2(e), positive
  int wait_tries;           // of a wait for work or scores: kPrefillWaitTries, or fewer (tests)
  long long test_post_delay_cycles;  // tests: the loading warp holds every work back so long
  float eps, out_scale;
};

// One token per sequence on mma.sync, and the merge of records that follows where there are any
cudaError_t launch_diff_decode(bool fp8, const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p,
                               cudaStream_t stream);
cudaError_t launch_diff_merge(bool fp8, const DiffParams& p, cudaStream_t stream);

// Chunks (rows ended, or records where contexts are split) and prefix passes (records) on tcgen05; prefix passes
// take their tables, lengths, ranges and sequences' count from p's q_indptr, block_tables, context_lens and batch
// (fine: with softmax weights in two 16-bit terms; else E4M3 pools only)
enum DiffForm { kDiffChunk, kDiffChunkSplit, kDiffPrefix, kDiffPrefixFine };
cudaError_t launch_diff_chunk(bool fp8, DiffForm form, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const DiffParams& p, int tile_slots, int splits,
                              cudaStream_t stream);

}  // namespace pkv
