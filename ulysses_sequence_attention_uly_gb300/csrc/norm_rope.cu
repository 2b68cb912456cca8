// norm_rope.cu -- RMS norm of every q and k head and the rotation by the
// row's position in one pass over the shards, and its gradient.
//
// Mathematics, per head x of D values with weight w, table row (cos, sin) and
// R the rotation of D/2 pairs:
//   rstd = 1 / sqrt(mean x^2 + eps)     n = x rstd w          y = R n
// and, for the gradient g of y (z = x rstd, dn = R^T g):
//   dw += dn z      dx = rstd (dn w - z mean(dn w z))
// both sums over a head, of x^2 and of dn w x, come from the same values, so
// the gradient needs one reduction step and one pass too.
//
// Bound by memory: 4 bytes an element forward, 6 backward.  D / 8 lanes hold a
// head, eight elements each, so that a lane holds whole pairs: [8l, 8l + 8) for
// the pairs (2i, 2i+1), and [4l, 4l + 4) with [D/2 + 4l, D/2 + 4l + 4) for the
// pairs (i, i + D/2).  A warp takes one row and walks its heads, 256 / D at a
// time and several of these at once, with the row's cosines, sines and the
// weights in registers.
// All arithmetic is f32; y and dx are rounded to bf16 once.
//
// Measured on q and k of 29328 rows of 40 heads of 128 (GB300, 6797 GB/s
// copy): forward 180.5 us = 6734 GB/s, backward 290 us = 6262 GB/s with
// the sum of the weight gradients.  Sixteen elements a lane: 196.9 and 404 us
// (160 registers: one CTA of the backward kernel on an SM).  Backward, CTAs an
// SM x head groups in flight: 2 x 4 287 us, 2 x 6 302, 3 x 2 315, 4 x 1 349,
// 2 x 2 345; three or more CTAs with four groups spill.
#include "grad.cuh"
#include "tc.cuh"

namespace uly {

__device__ unsigned long long g_norm_violations;

uint64_t norm_violations(bool reset) {
  if (!kChecked) return 0;
  unsigned long long v = 0;
  if (cudaMemcpyFromSymbol(&v, g_norm_violations, sizeof v) != cudaSuccess) return ~0ull;
  if (reset) {
    const unsigned long long z = 0;
    if (cudaMemcpyToSymbol(g_norm_violations, &z, sizeof z) != cudaSuccess) return ~0ull;
  }
  return v;
}

namespace {

constexpr int kNormWarps = 8;
constexpr int kNormUnroll = 4, kNormBwdUnroll = 4;  // head groups of a warp with loads in flight

struct RowAt {
  int t, shard, b;     // tensor (0 q, 1 k), shard, batch
  int64_t row;         // row of the shard's tensor, batches included
  int table;           // row of the cos / sin tables (global key order)
};

// Row i of tensor t's rows, counted over shards, batches and shard rows.
__device__ __forceinline__ RowAt decode_row(const NormParams& p, int t, int64_t i) {
  RowAt a;
  a.t = t;
  a.shard = 0;
  while (a.shard + 1 < p.P && i >= p.rows_begin[t][a.shard + 1]) ++a.shard;
  i -= p.rows_begin[t][a.shard];
  const int rows = p.shard_rows[t][a.shard];
  a.b = static_cast<int>(i / rows);
  const int r = static_cast<int>(i - static_cast<int64_t>(a.b) * rows);
  a.row = i;
  const int img = p.img_off[a.shard], len = p.img_off[a.shard + 1] - img;
  const int rep = rows - len;  // replicated rows of this tensor
  if (p.mode == ULY_REP_SUFFIX)
    a.table = r < len ? img + r : p.img_off[p.P] + (r - len);
  else
    a.table = r < rep ? r : p.R + img + (r - rep);
  return a;
}

// the lane's four cosines and sines
template <int D, bool HALF>
__device__ __forceinline__ void load_tables(const NormParams& p, const RowAt& a, int l, float4& c, float4& s) {
  c = make_float4(1.f, 1.f, 1.f, 1.f);
  s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!p.cos_table || !in_bounds(&g_norm_violations, a.table, 1, p.table_rows)) return;
  const int64_t at = a.b * p.table_batch_stride + static_cast<int64_t>(a.table) * (D / 2) + 4 * l;
  c = __ldg(reinterpret_cast<const float4*>(p.cos_table + at));
  s = __ldg(reinterpret_cast<const float4*>(p.sin_table + at));
}

// index of the lane's element j
template <int D, bool HALF>
__device__ __forceinline__ int element(int l, int j) {
  return HALF ? (j < 4 ? 4 * l + j : D / 2 + 4 * l + j - 4) : 8 * l + j;
}

template <int D, bool HALF>
__device__ __forceinline__ void load_weights(const float* w, int l, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = w ? __ldg(w + element<D, HALF>(l, j)) : 1.f;
}

// the lane's eight elements of the head at p (which includes the lane's offset)
template <int D, bool HALF>
__device__ __forceinline__ uint4 load_head(const uint8_t* p) {
  if (!HALF) return *reinterpret_cast<const uint4*>(p);
  const uint2 lo = *reinterpret_cast<const uint2*>(p), hi = *reinterpret_cast<const uint2*>(p + D);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
template <int D, bool HALF>
__device__ __forceinline__ void store_head(uint8_t* p, const float (&v)[8]) {
  const uint4 r = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7]));
  if (!HALF) {
    *reinterpret_cast<uint4*>(p) = r;
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(r.x, r.y);
    *reinterpret_cast<uint2*>(p + D) = make_uint2(r.z, r.w);
  }
}

__device__ __forceinline__ void unpack(const uint4 x, float (&v)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// v = R v (sign = 1) or R^T v (sign = -1) of the lane's four pairs
template <bool HALF>
__device__ __forceinline__ void rotate(float (&v)[8], const float4 c4, const float4 s4, float sign) {
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int a = HALF ? j : 2 * j, b = HALF ? 4 + j : 2 * j + 1;
    const float x = v[a], y = v[b], sj = sign * s[j];
    v[a] = fmaf(x, c[j], -(y * sj));
    v[b] = fmaf(x, sj, y * c[j]);
  }
}

// Forward.  A warp's task: heads [h0, h0 + heads_task) of one row.
template <int D, bool HALF>
__global__ void __launch_bounds__(32 * kNormWarps) norm_rope_kernel(const __grid_constant__ NormParams p) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // lanes of a head, heads of a warp at once
  const int lane = threadIdx.x & 31, l = lane % kLanes, hs = lane / kLanes;
  int64_t task = static_cast<int64_t>(blockIdx.x) * kNormWarps + (threadIdx.x >> 5);
  if (task >= p.tasks_begin[2]) return;
  const int t = task >= p.tasks_begin[1];
  task -= p.tasks_begin[t];
  const int64_t i = task / p.task_parts[t];
  const int h_lo = static_cast<int>(task - i * p.task_parts[t]) * p.task_heads;
  const int h_hi = min(h_lo + p.task_heads, p.heads[t]);
  const RowAt a = decode_row(p, t, i);
  if (!in_bounds(&g_norm_violations, a.row, 1, p.tensor_rows[t][a.shard])) return;
  float4 c, s;
  float w[8];
  load_tables<D, HALF>(p, a, l, c, s);
  load_weights<D, HALF>(p.weight[t], l, w);
  const int off = (HALF ? 8 : 16) * l;
  const uint8_t* x = p.x[t][a.shard] + a.row * p.row_bytes[t] + off;
  uint8_t* y = p.y[t][a.shard] + a.row * (static_cast<int64_t>(p.heads[t]) * D * 2) + off;
  constexpr int kUnroll = kNormUnroll;
  for (int h0 = h_lo; h0 < h_hi; h0 += kUnroll * kHeads) {
    uint4 in[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kHeads + hs;
      in[u] = make_uint4(0u, 0u, 0u, 0u);
      if (h < h_hi) in[u] = load_head<D, HALF>(x + h * (D * 2));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kHeads + hs;
      float v[8];
      unpack(in[u], v);
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(v[j], v[j], sq);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      const float rstd = rsqrtf(sq * (1.f / D) + p.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * w[j];
      rotate<HALF>(v, c, s, 1.f);
      if (h < h_hi) store_head<D, HALF>(y + h * (D * 2), v);
    }
  }
}

// Backward.  The CTAs [0, ctas[0]) share q's rows, the next ctas[1] k's; each
// warp walks rows with a fixed stride and keeps its lanes' part of dw in
// registers.  The CTA's sum goes to its own row of `partial`, which
// weight_grad_kernel adds up in a fixed order: the result does not depend on
// which CTA finishes first.
template <int D, bool HALF>
__global__ void __launch_bounds__(32 * kNormWarps, kNormCtasPerSm)
    norm_rope_backward_kernel(const __grid_constant__ NormParams p) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  __shared__ float sums[kNormWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % kLanes, hs = lane / kLanes;
  const int t = blockIdx.x >= p.ctas[0];
  const int cta = blockIdx.x - (t ? p.ctas[0] : 0);
  float w[8], dw[8];
  load_weights<D, HALF>(p.weight[t], l, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = 0.f;
  const int64_t dense = static_cast<int64_t>(p.heads[t]) * D * 2;
  const int off = (HALF ? 8 : 16) * l;
  for (int64_t task = static_cast<int64_t>(cta) * kNormWarps + warp; task < p.tasks_begin[t + 1] - p.tasks_begin[t];
       task += static_cast<int64_t>(p.ctas[t]) * kNormWarps) {
    const int64_t i = task / p.task_parts[t];
    const int h_lo = static_cast<int>(task - i * p.task_parts[t]) * p.task_heads;
    const int h_hi = min(h_lo + p.task_heads, p.heads[t]);
    const RowAt a = decode_row(p, t, i);
    if (!in_bounds(&g_norm_violations, a.row, 1, p.tensor_rows[t][a.shard])) continue;
    float4 c, s;
    load_tables<D, HALF>(p, a, l, c, s);
    const uint8_t* x = p.x[t][a.shard] + a.row * p.row_bytes[t] + off;
    const uint8_t* g = p.g[t][a.shard] + a.row * dense + off;
    uint8_t* y = p.y[t][a.shard] + a.row * dense + off;
    constexpr int kUnroll = kNormBwdUnroll;
    for (int h0 = h_lo; h0 < h_hi; h0 += kUnroll * kHeads) {
      uint4 xi[kUnroll], gi[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kHeads + hs;
        xi[u] = gi[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h < h_hi) {
          xi[u] = load_head<D, HALF>(x + h * (D * 2));
          gi[u] = load_head<D, HALF>(g + h * (D * 2));
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kHeads + hs;
        float v[8], dn[8];
        unpack(xi[u], v);
        unpack(gi[u], dn);
        rotate<HALF>(dn, c, s, -1.f);
        float sq = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sq = fmaf(v[j], v[j], sq);
          dot = fmaf(dn[j] * w[j], v[j], dot);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) {
          sq += __shfl_xor_sync(0xffffffffu, sq, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float rstd = rsqrtf(sq * (1.f / D) + p.eps);
        const float mean = dot * rstd * (1.f / D);  // of dn w z
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float z = v[j] * rstd;
          dw[j] = fmaf(dn[j], z, dw[j]);
          v[j] = rstd * (dn[j] * w[j] - z * mean);
        }
        if (h < h_hi) store_head<D, HALF>(y + h * (D * 2), v);
      }
    }
  }
  if (!p.partial) return;  // no weight gradient wanted
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
    if (hs == 0) sums[warp][element<D, HALF>(l, j)] = dw[j];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kNormWarps; ++k) v += sums[k][threadIdx.x];
    p.partial[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = v;
  }
}

// dw = the sum of its tensor's partial rows: 32 columns a CTA, 32 rows at a
// time.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* partial, int n_q, int n_k, int D, float* dwq,
                                                           float* dwk) {
  __shared__ float s[32][33];
  const int t = blockIdx.y, col = blockIdx.x * 32 + threadIdx.x;
  const int lo = t ? n_q : 0, hi = lo + (t ? n_k : n_q);
  float* out = t ? dwk : dwq;
  if (!out) return;
  float v = 0.f;
  for (int r = lo + threadIdx.y; r < hi; r += 32) v += partial[static_cast<int64_t>(r) * D + col];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += s[k][threadIdx.x];
    out[col] = v;
  }
}

// Heads of a task: a whole row's, unless there are too few rows for every
// SM's warps; then one pass's (256 / D heads) each.
void split_tasks(NormParams& p, int D, int sm_count) {
  const int pass = 256 / D;
  const int64_t rows = p.rows_begin[0][p.P] + p.rows_begin[1][p.P];
  const int most = p.heads[0] > p.heads[1] ? p.heads[0] : p.heads[1];
  p.task_heads = rows < static_cast<int64_t>(sm_count) * kNormWarps * 4 ? pass : (most + pass - 1) / pass * pass;
  p.tasks_begin[0] = 0;
  for (int t = 0; t < 2; ++t) {
    p.task_parts[t] = (p.heads[t] + p.task_heads - 1) / p.task_heads;
    if (p.task_parts[t] < 1) p.task_parts[t] = 1;
    p.tasks_begin[t + 1] = p.tasks_begin[t] + p.rows_begin[t][p.P] * p.task_parts[t];
  }
}

template <int D, bool HALF>
cudaError_t launch(NormParams& p, bool backward, int sm_count, cudaStream_t s) {
  split_tasks(p, D, sm_count);
  const int64_t tasks = p.tasks_begin[2];
  if (!backward) {
    const int64_t grid = (tasks + kNormWarps - 1) / kNormWarps;
    if (grid == 0) return cudaSuccess;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    norm_rope_kernel<D, HALF><<<static_cast<unsigned>(grid), 32 * kNormWarps, 0, s>>>(p);
    return cudaGetLastError();
  }
  // CTAs in proportion to the tensors' work, at least one where there is any
  const int64_t most = static_cast<int64_t>(sm_count) * kNormCtasPerSm;
  int64_t want[2];
  const int64_t all = p.rows_begin[0][p.P] * p.heads[0] + p.rows_begin[1][p.P] * p.heads[1];
  for (int t = 0; t < 2; ++t) {
    const int64_t n = p.tasks_begin[t + 1] - p.tasks_begin[t];
    const int64_t share = most * p.rows_begin[t][p.P] * p.heads[t] / (all > 0 ? all : 1);
    want[t] = (n + kNormWarps - 1) / kNormWarps;
    if (want[t] > share) want[t] = share > 1 ? share : (n > 0 ? 1 : 0);
    p.ctas[t] = static_cast<int32_t>(want[t]);
  }
  if (p.ctas[0] + p.ctas[1] == 0) return cudaSuccess;
  norm_rope_backward_kernel<D, HALF><<<p.ctas[0] + p.ctas[1], 32 * kNormWarps, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!p.dweight[0] && !p.dweight[1])) return e;
  weight_grad_kernel<<<dim3(D / 32, 2), dim3(32, 32), 0, s>>>(p.partial, p.ctas[0], p.ctas[1], D, p.dweight[0],
                                                               p.dweight[1]);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(NormParams& p, int D, bool half_pairs, bool backward, int sm_count, cudaStream_t s) {
  if (D == 128)
    return half_pairs ? launch<128, true>(p, backward, sm_count, s) : launch<128, false>(p, backward, sm_count, s);
  return half_pairs ? launch<64, true>(p, backward, sm_count, s) : launch<64, false>(p, backward, sm_count, s);
}

}  // namespace uly
