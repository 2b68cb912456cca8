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
// Bound by memory: 4 bytes an element forward, 6 backward.  D / 16 lanes hold
// a head: lane l has the elements [8l, 8l + 8) and [D/2 + 8l, D/2 + 8l + 8), so
// that both pairings, (2i, 2i+1) and (i, i + D/2), stay inside a lane and every
// load and store is 16 bytes.  A warp takes one row and walks its heads, 512 /
// D at a time, with the row's cosines, sines and the weights in registers.
// All arithmetic is f32; y and dx are rounded to bf16 once.
#include "internal.cuh"
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

template <bool HALF>
__device__ __forceinline__ void load_tables(const NormParams& p, const RowAt& a, int D, int l, float (&c)[8], float (&s)[8]) {
  const int half = D / 2;
  if (!p.cos_table || !in_bounds(&g_norm_violations, a.table, 1, p.table_rows)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = 1.f;
      s[j] = 0.f;
    }
    return;
  }
  const int64_t at = a.b * p.table_batch_stride + static_cast<int64_t>(a.table) * half;
  const int i0 = HALF ? 8 * l : 4 * l, i1 = HALF ? 8 * l + 4 : half / 2 + 4 * l;
  const float4 c0 = __ldg(reinterpret_cast<const float4*>(p.cos_table + at + i0));
  const float4 c1 = __ldg(reinterpret_cast<const float4*>(p.cos_table + at + i1));
  const float4 s0 = __ldg(reinterpret_cast<const float4*>(p.sin_table + at + i0));
  const float4 s1 = __ldg(reinterpret_cast<const float4*>(p.sin_table + at + i1));
  c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
  s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
}

__device__ __forceinline__ void load_weights(const float* w, int D, int l, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = 1.f;
  if (!w) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = __ldg(w + 8 * l + j);
    v[8 + j] = __ldg(w + D / 2 + 8 * l + j);
  }
}

__device__ __forceinline__ void unpack(const uint4 lo, const uint4 hi, float (&v)[16]) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// y = R v (sign = 1) or R^T v (sign = -1) of the lane's eight pairs
template <bool HALF>
__device__ __forceinline__ void rotate(float (&v)[16], const float (&c)[8], const float (&s)[8], float sign) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int a = HALF ? j : 2 * j, b = HALF ? 8 + j : 2 * j + 1;
    const float x = v[a], y = v[b], sj = sign * s[j];
    v[a] = fmaf(x, c[j], -(y * sj));
    v[b] = fmaf(x, sj, y * c[j]);
  }
}

// Forward.  A warp's task: heads [h0, h0 + heads_task) of one row.
template <int D, bool HALF>
__global__ void __launch_bounds__(32 * kNormWarps) norm_rope_kernel(const __grid_constant__ NormParams p) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // lanes of a head, heads of a warp pass
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
  float c[8], s[8], w[16];
  load_tables<HALF>(p, a, D, l, c, s);
  load_weights(p.weight[t], D, l, w);
  const uint8_t* x = p.x[t][a.shard] + a.row * p.row_bytes[t] + 16 * l;
  uint8_t* y = p.y[t][a.shard] + a.row * (static_cast<int64_t>(p.heads[t]) * D * 2) + 16 * l;
  constexpr int kUnroll = 4;
  for (int h0 = h_lo; h0 < h_hi; h0 += kUnroll * kHeads) {
    uint4 lo[kUnroll], hi[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kHeads + hs;
      lo[u] = hi[u] = make_uint4(0u, 0u, 0u, 0u);
      if (h < h_hi) {
        lo[u] = *reinterpret_cast<const uint4*>(x + h * (D * 2));
        hi[u] = *reinterpret_cast<const uint4*>(x + h * (D * 2) + D);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kHeads + hs;
      float v[16];
      unpack(lo[u], hi[u], v);
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) sq = fmaf(v[j], v[j], sq);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      const float rstd = rsqrtf(sq * (1.f / D) + p.eps);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = v[j] * rstd * w[j];
      rotate<HALF>(v, c, s, 1.f);
      if (h < h_hi) {
        *reinterpret_cast<uint4*>(y + h * (D * 2)) = pack8(v);
        *reinterpret_cast<uint4*>(y + h * (D * 2) + D) = pack8(v + 8);
      }
    }
  }
}

// Backward.  The CTAs [0, ctas[0]) share q's rows, the next ctas[1] k's; each
// warp walks rows with a fixed stride and keeps its lanes' part of dw in
// registers.  The CTA's sum goes to its own row of `partial`, which
// weight_grad_kernel adds up in a fixed order: the result does not depend on
// which CTA finishes first.
template <int D, bool HALF>
__global__ void __launch_bounds__(32 * kNormWarps) norm_rope_backward_kernel(const __grid_constant__ NormParams p) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
  __shared__ float sums[kNormWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % kLanes, hs = lane / kLanes;
  const int t = blockIdx.x >= p.ctas[0];
  const int cta = blockIdx.x - (t ? p.ctas[0] : 0);
  float w[16], dw[16];
  load_weights(p.weight[t], D, l, w);
#pragma unroll
  for (int j = 0; j < 16; ++j) dw[j] = 0.f;
  const int64_t dense = static_cast<int64_t>(p.heads[t]) * D * 2;
  for (int64_t task = static_cast<int64_t>(cta) * kNormWarps + warp; task < p.tasks_begin[t + 1] - p.tasks_begin[t];
       task += static_cast<int64_t>(p.ctas[t]) * kNormWarps) {
    const int64_t i = task / p.task_parts[t];
    const int h_lo = static_cast<int>(task - i * p.task_parts[t]) * p.task_heads;
    const int h_hi = min(h_lo + p.task_heads, p.heads[t]);
    const RowAt a = decode_row(p, t, i);
    if (!in_bounds(&g_norm_violations, a.row, 1, p.tensor_rows[t][a.shard])) continue;
    float c[8], s[8];
    load_tables<HALF>(p, a, D, l, c, s);
    const uint8_t* x = p.x[t][a.shard] + a.row * p.row_bytes[t] + 16 * l;
    const uint8_t* g = p.g[t][a.shard] + a.row * dense + 16 * l;
    uint8_t* y = p.y[t][a.shard] + a.row * dense + 16 * l;
    constexpr int kUnroll = 2;
    for (int h0 = h_lo; h0 < h_hi; h0 += kUnroll * kHeads) {
      uint4 xlo[kUnroll], xhi[kUnroll], glo[kUnroll], ghi[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kHeads + hs;
        xlo[u] = xhi[u] = glo[u] = ghi[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h < h_hi) {
          xlo[u] = *reinterpret_cast<const uint4*>(x + h * (D * 2));
          xhi[u] = *reinterpret_cast<const uint4*>(x + h * (D * 2) + D);
          glo[u] = *reinterpret_cast<const uint4*>(g + h * (D * 2));
          ghi[u] = *reinterpret_cast<const uint4*>(g + h * (D * 2) + D);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kHeads + hs;
        float v[16], dn[16];
        unpack(xlo[u], xhi[u], v);
        unpack(glo[u], ghi[u], dn);
        rotate<HALF>(dn, c, s, -1.f);
        float sq = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
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
        for (int j = 0; j < 16; ++j) {
          const float z = v[j] * rstd;
          dw[j] = fmaf(dn[j], z, dw[j]);
          v[j] = rstd * (dn[j] * w[j] - z * mean);
        }
        if (h < h_hi) {
          *reinterpret_cast<uint4*>(y + h * (D * 2)) = pack8(v);
          *reinterpret_cast<uint4*>(y + h * (D * 2) + D) = pack8(v + 8);
        }
      }
    }
  }
  if (!p.partial) return;  // no weight gradient wanted
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
    if (hs == 0) sums[warp][(j < 8 ? 0 : D / 2) + 8 * l + (j & 7)] = dw[j];
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
// SM's warps; then one pass's (512 / D heads) each.
void split_tasks(NormParams& p, int D, int sm_count) {
  const int pass = 512 / D;
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
