// serve.cuh -- structures of the causal attention over packed prompts
// (prompt.cu) and of the 8-bit cache (cache.cu), shared with the host code.
#pragma once
#include "internal.cuh"

namespace uly {

uint64_t prompt_violations(bool reset);
uint64_t cache_violations(bool reset);

// --------------------------------------------------------------- prompts --
// Causal attention over packed sequences on the shards (uly_sp_prompt_attention).

// Rows of one sequence in one shard, in global row order.
struct alignas(16) PromptRun {
  int32_t shard;
  int32_t row0;       // first row inside the shard
  int32_t len;        // at least 1
  int32_t first_run;  // the sequence's first run
};

// Query rows that a CTA takes at a time: one 128-row tile of two q heads, or
// (an odd number of q heads a kv head) two tiles of one head.
struct alignas(16) PromptUnit {
  int32_t run;
  int32_t tile;       // its (first) tile inside the run
  int32_t n_kv;       // 128-key tiles up to the diagonal of its (last) tile
  int32_t hp;         // direct: the item's place among the unit's
};

// Written by tables_kernel, in the caller's workspace.
struct PromptTables {
  int32_t* head;      // [0] units, [1] the next item that no CTA has taken
  PromptRun* runs;    // [n_seqs + P]
  int32_t* run_unit;  // [n_seqs + P + 1] units before the run
  int32_t* run_kv;    // [n_seqs + P] 128-key tiles of the sequence before the run
  PromptUnit* units;  // [max_units] those with most tiles first
  int32_t max_runs, max_units;
};

// How the rows are cut: all that the tables are made from.
struct PromptCut {
  PromptTables t;
  int32_t shard_begin[kMaxRanks + 1];  // global row of each shard's first row; [P]: all rows
  int32_t P, n_seqs;
  int32_t pair;       // two q heads of one kv head an item (else two tiles of one head)
  int32_t sort_shift; // a unit's place in the order goes by n_kv >> sort_shift
  int32_t grid;
  const int32_t* seq_starts;
};

struct PromptParams {
  CUtensorMap tq[kMaxRanks];
  CUtensorMap tk[kMaxRanks];
  CUtensorMap tv[kMaxRanks];
  PromptCut cut;
  uint8_t* out[kMaxRanks];
  float* lse[kMaxRanks];
  int32_t Hq, G, lse_out;
  int32_t n_hp;       // items of one unit: Hq / 2 or Hq
  int32_t direct;     // no tables: a CTA works its items, up to kDirectItems, out by itself
  float scale_log2;
  int32_t* status;
  uint64_t wait_ns;
  int32_t withhold_fill;  // test hook, as in AttnParams
};
constexpr int kSortBuckets = 2048;
constexpr int kDirectItems = 2;  // items that a CTA works out by itself, at most

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
  int32_t group;             // rows that a CTA looks after; 0: a warp a row (append_few_kernel)
};

// What a CTA of the attention over a cache worked on: part idx of n of a unit (n
// = 0: nothing).
struct alignas(16) CachedPart {
  int32_t n, idx;
  int32_t stride;  // CTAs from a part of the unit to its next
  int32_t live;    // rows of the unit that there are
  int64_t place;   // of its first row among all rows and heads of q
  int64_t row0;    // and among the sequence's
};
// Most parts of a unit: a lane of combine_kernel for each, which has sixteen warps
// where a unit or two are all (200 thousand tokens of one cache head: 22.0 -> 20.8
// us), eight where units are few, and four where its CTAs are many.
__host__ __device__ constexpr int max_unit_parts(int few) { return 128 << few; }
constexpr int kCachedPerSm[2] = {4, 3};    // CTAs an SM, with one and two 8-row tiles of queries

struct CachedParams {
  CacheParams c;
  int64_t* before;     // more than 128 sequences: [n_seqs + 2], see parts_kernel
  CachedPart* parts;   // [grid]
  float* sums;         // [grid][8 * row_tiles][D + 4]: O, M, m, l of parts of units
  int32_t grid;
  int32_t slots;       // CTAs that run at once
  int32_t few;         // 1: one unit at most for eight of those, 2: one for 256, 0: more
  int32_t whole;       // units in one part each
  int32_t row_tiles;   // 8-row tiles of queries a unit: 1 or 2
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
