// grad.cuh -- structures of the gradient kernels (attn_bwd.cu) and of the norm
// and rotation of q and k heads (norm_rope.cu), shared with the host code.
#pragma once
#include "internal.cuh"

namespace uly {

uint64_t bwd_violations(bool reset);
uint64_t norm_violations(bool reset);

// The gradient of the attention (attn_bwd.cu).  q tensors (q, o, do, dq) share
// their shape, as do k/v tensors (k, v, dk, dv).
struct BwdParams {
  // [p]: shard p (fused) or rank p's tensor.  Fused, replicated suffix: [p] ends
  // with the shard's image rows, and [kMaxRanks + p], of the whole shard, is for
  // the replicated rows, so that a tile at the end of the image rows is filled
  // with zeros there and not with copies that are not read.
  CUtensorMap tq[2 * kMaxRanks];
  CUtensorMap tk[2 * kMaxRanks];
  CUtensorMap tv[2 * kMaxRanks];
  CUtensorMap tdo[kMaxRanks];     // (replicated rows: tdo_hi, tdo_lo)
  CUtensorMap tdo_hi, tdo_lo;     // fused: replicated rows of do, summed over the shards, in two bf16 parts
  const uint8_t* o[kMaxRanks];
  const uint8_t* dout[kMaxRanks];
  const float* lse[kMaxRanks];
  uint8_t* dq[kMaxRanks];
  uint8_t* dk[kMaxRanks];
  uint8_t* dv[kMaxRanks];
  uint8_t *do_hi, *do_lo;         // [B][R][Hq][D] bf16 each
  // `first`: first 128-row tile, for q and kv alike; `src` < 0: map -1 - src +
  // the rank that owns the head; kseg's out_row0 / out_shard: where dk, dv rows go
  Seg qseg[kMaxSegs];
  Seg kseg[kMaxSegs];
  int32_t n_qseg, n_kseg, n_q_tiles, n_kv_tiles;
  int32_t fused, P, B, Hq, Hkv, Hq_l, Hkv_l, G;
  int32_t shard_len[kMaxRanks];   // image rows of each shard
  int64_t q_row_stride, kv_row_stride;                              // bytes
  int64_t q_batch_stride[kMaxRanks], kv_batch_stride[kMaxRanks];    // bytes
  int64_t lse_row_stride;                                           // floats
  int64_t lse_batch_stride[kMaxRanks];                              // floats
  float scale, scale_log2;
  const uint8_t* key_mask;        // admission as in TileParams
  const int32_t* key_ranges;
  int32_t n_ranges, Nk;
  uint4* tile_bits;               // tables as in AttnParams, the list in another order
  int32_t* active;
  uint4* active_bits;
  uint4* active_inv;
  int32_t* n_active;
  int32_t* n_full;                // [B]: the list's tiles whose keys are all admitted, listed from its front;
                                  // the others are listed from its back
  uint32_t n_kv_ctas;             // CTAs of dK and dV: n_kv_tiles * Hkv * B
  float* nl;                      // [B][Hq][n_q_tiles * 128]: -lse log2(e)
  float* dl;                      // [B][Hq][n_q_tiles * 128]: -delta (of do_hi)
  float* dl_lo;                   // [B][Hq][n_lo * 128]: -delta of do_lo
  int32_t n_lo;                   // tiles of the replicated run that do_lo adds (0: no replicated q rows, or one shard)
  int32_t rep_qseg;               // its index in qseg
  int32_t sms;                    // SMs of the device
  int32_t parts;                  // CTAs that share a tile's loop (a cluster): 1, 2 or 4
  int32_t masked_rows;
  int32_t withhold_fill;
  int32_t* status;
  uint64_t wait_ns;
};

// Norm and rotation of q and k heads, and the gradient (norm_rope.cu).  Tensor
// 0 is q, 1 is k.
struct NormParams {
  const uint8_t* x[2][kMaxRanks];
  const uint8_t* g[2][kMaxRanks];   // gradient of the output (backward)
  uint8_t* y[2][kMaxRanks];         // output, or the gradient of x
  const float* weight[2];           // [D] or null (ones)
  float* dweight[2];                // [D] or null
  const float* cos_table;           // [table_rows][D/2], per batch when the stride is not 0; null: no rotation
  const float* sin_table;
  int64_t table_batch_stride;       // floats
  int64_t table_rows;
  int64_t row_bytes[2];             // x: bytes from one row to the next (outputs and gradients are dense)
  int64_t rows_begin[2][kMaxRanks + 1];  // rows (batches included) of the shards before
  int64_t tensor_rows[2][kMaxRanks];     // rows (batches included) of a shard's tensor
  int32_t shard_rows[2][kMaxRanks];      // rows of a shard's tensor, per batch
  int32_t img_off[kMaxRanks + 1];        // image rows of the shards before
  int32_t heads[2];
  int32_t P, R, mode;
  float eps;
  // set by the launcher
  int64_t tasks_begin[3];           // warp tasks of the tensors before
  int32_t task_parts[2], task_heads;
  int32_t ctas[2];                  // backward: CTAs of q and of k
  float* partial;                   // backward: [ctas][D]
};
constexpr int kNormCtasPerSm = 2;  // norm_rope_backward_kernel (norm_rope.cu)

cudaError_t launch_attention_backward(const BwdParams& p, int D, cudaStream_t s);
cudaError_t launch_norm_rope(NormParams& p, int D, bool half_pairs, bool backward, int sm_count, cudaStream_t s);

}  // namespace uly
