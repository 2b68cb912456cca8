// serve.cuh -- structures of the causal attention over packed prompts
// (prompt.cu) and of the 8-bit cache (cache.cu), shared with the host code.
#pragma once
#include "internal.cuh"

namespace uly {

uint64_t prompt_violations(bool reset);
uint64_t cache_violations(bool reset);

// --------------------------------------------------------------- prompts --
// Causal attention over packed sequences on the shards (uly_sp_prompt_attention).
struct PromptParams {
  const uint8_t* q[kMaxRanks];
  const uint8_t* k[kMaxRanks];
  const uint8_t* v[kMaxRanks];
  uint8_t* out[kMaxRanks];
  float* lse[kMaxRanks];
  int32_t shard_begin[kMaxRanks + 1];  // global row of each shard's first row; [P]: all rows
  int32_t P, Hq, Hkv, G, n_seqs, lse_out;
  const int32_t* seq_starts;
  float scale_log2;
};

// ----------------------------------------------------------------- cache --
struct CacheParams {
  uint8_t* k_pages;  // e4m3 [n_pages][H][page_rows][D]
  uint8_t* v_pages;
  float* k_scale;    // [n_pages][H]
  float* v_scale;
  int32_t n_pages, page_rows, page_shift, H;
  const int32_t* starts;
  const int32_t* lens;
  const int32_t* table;
  int32_t n_seqs, table_width;
  int32_t n_rows;
};

struct AppendParams {
  CacheParams c;
  const uint8_t* x[2];       // k, v rows
  int64_t row_bytes[2];
  int32_t group;             // rows that a CTA looks after
};

struct CachedParams {
  CacheParams c;
  const uint8_t* q;
  int64_t q_row_bytes;
  int32_t Hq, G;
  float scale_log2;
  uint8_t* out;
  float* lse;
};

cudaError_t launch_prompt(const PromptParams& p, int D, cudaStream_t s);
cudaError_t launch_cache_append(const AppendParams& p, int D, cudaStream_t s);
cudaError_t launch_cache_attention(const CachedParams& p, int D, cudaStream_t s);

}  // namespace uly
