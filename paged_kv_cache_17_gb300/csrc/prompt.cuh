// prompt.cuh -- parameters and launchers of the prompt side of the pool: norm + rotation +
// append, chunk attention over the pages, and reading pages back (qk_rope_append.cu,
// prefill_tc.cu, merge_prefill.cu, kv_gather.cu; launched from pkv_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {

struct RopeAppendParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* positions;
  const int64_t* slots;
  const uint16_t* q_weight;  // [D] bf16, or NULL: no norm
  const uint16_t* k_weight;
  const double* inv_freq;  // [rot / 2] radians per position
  uint16_t* q_out;
  int64_t q_out_stride;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const float* scales;
  uint32_t* status;
  int64_t num_tokens, pool_slots;
  int hq, hkv, rot;  // rot: elements of a head that are rotated (0: none)
  int rows_per_cta, groups;  // launch shape (launch_qk_rope_append)
  float eps, rope_scale;
};

cudaError_t launch_qk_rope_append(int d, bool fp8, bool interleaved, const RopeAppendParams& p, int sm_count,
                                  cudaStream_t stream);

struct GatherParams {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* scales;
  const int32_t* block_tables;
  const int32_t* kv_indptr;
  const int32_t* starts;  // NULL: every range starts at position 0
  void* k_out;
  void* v_out;
  uint32_t* status;
  int64_t num_rows, num_blocks;
  int batch, max_blocks, hkv, d;
};

cudaError_t launch_kv_gather(bool fp8, bool out_fp32, const GatherParams& p, int sm_count, cudaStream_t stream);

struct PrefillParams {
  const uint16_t* q;
  int64_t q_stride;  // elements between tokens
  const int32_t* q_indptr;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const float* scales;  // E4M3: [2][hkv]
  uint16_t* out;        // [total_q][hq][D] bf16
  float* lse;           // [total_q][hq], or NULL
  // partial records when the context is split (splits > 1): record of (split, token, head) at
  // index (split * total_q + token) * hq + head
  float2* part_ml;  // reference max (log2 units) and sum
  float* part_acc;  // [D], unnormalised
  uint32_t* status;
  int batch, total_q, hq, hkv, group;
  int max_blocks, num_blocks, max_context_len;
  int causal, negate;
  float score_scale;  // |softmax_scale| * log2(e), positive
  int splits;
  int split_tiles;  // 128-key tiles per split
  int wait_tries;   // of a wait for work or scores: kPrefillWaitTries, or fewer (tests)
  long long test_post_delay_cycles;  // tests: the loading warp holds every work back so long
};

// wide: 256 query rows per CTA (two tiles over the same keys); else 128 rows (one tile, its
// keys dealt alternately to the two softmax groups)
cudaError_t launch_prefill(int d, bool fp8, bool wide, const CUtensorMap& tq, const CUtensorMap& tk,
                           const CUtensorMap& tv, const PrefillParams& p, int tile_slots, cudaStream_t stream);
cudaError_t launch_merge_prefill(int d, const PrefillParams& p, bool fp8, cudaStream_t stream);

// Tries after which a wait of the attention gives up
constexpr int kPrefillWaitTries = 1 << 23;

// Weights are stored times 2^kWeightBias in E4M3 pools' fp16 products (see prefill_tc.cu).
constexpr float kPrefillWeightBias = 7.f;

// 128-key steps whose products go into one accumulator (see plan_prefill); a power of two
constexpr int kPrefillMaxRun = 512;

}  // namespace pkv
