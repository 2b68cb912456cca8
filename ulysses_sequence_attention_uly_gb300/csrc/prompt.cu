// prompt.cu -- causal attention over packed sequences on the seq-sharded shards.
//
// For row i of a sequence: softmax over its rows j <= i of scale * q_i.k_j,
// times v_j; q head h uses kv head h / (Hq/Hkv).
#include <cuda_bf16.h>

#include "serve.cuh"
#include "tc.cuh"

namespace uly {

__device__ unsigned long long g_prompt_violations;

uint64_t prompt_violations(bool reset) {
  if (!kChecked) return 0;
  unsigned long long v = 0;
  if (cudaMemcpyFromSymbol(&v, g_prompt_violations, sizeof v) != cudaSuccess) return ~0ull;
  if (reset) {
    const unsigned long long z = 0;
    if (cudaMemcpyToSymbol(g_prompt_violations, &z, sizeof z) != cudaSuccess) return ~0ull;
  }
  return v;
}

// One warp per row and q head; the lanes share the head's elements.
template <int D>
__global__ void __launch_bounds__(256) prompt_kernel(const __grid_constant__ PromptParams p) {
  constexpr int E = D / 32;  // elements a lane
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x, h = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int N = p.shard_begin[p.P];
  if (h >= p.Hq) return;
  // the last sequence that begins at or before the row
  int lo = 0, hi = p.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (min(max(p.seq_starts[mid + 1], 0), N) > row)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (lo >= p.n_seqs) return;
  const int first = min(max(p.seq_starts[lo], 0), N);
  if (row < first) return;
  int sh = 0;
  while (row >= p.shard_begin[sh + 1]) ++sh;
  const int64_t q_row = static_cast<int64_t>(p.Hq) * D * 2, kv_row = static_cast<int64_t>(p.Hkv) * D * 2;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q[sh] + (row - p.shard_begin[sh]) * q_row) + h * D;
  float qf[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = __bfloat162float(q[lane + 32 * e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  int ks = 0;
  for (int j = first; j <= row; ++j) {
    while (j >= p.shard_begin[ks + 1]) ++ks;
    const int64_t off = (j - p.shard_begin[ks]) * kv_row + (h / p.G) * D * 2;
    const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(p.k[ks] + off);
    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.v[ks] + off);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += qf[e] * __bfloat162float(k[lane + 32 * e]);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), a = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * __bfloat162float(v[lane + 32 * e]);
  }
  const int64_t orow = row - p.shard_begin[sh];
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out[sh] + orow * q_row) + h * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + 32 * e] = __float2bfloat16(o[e] / l);
  if (lane == 0 && p.lse_out) p.lse[sh][orow * p.Hq + h] = (m + log2f(l)) * 0.6931471805599453f;
}

cudaError_t launch_prompt(const PromptParams& p, int D, cudaStream_t s) {
  const dim3 grid(p.shard_begin[p.P], (p.Hq + 7) / 8);
  if (D == 128)
    prompt_kernel<128><<<grid, 256, 0, s>>>(p);
  else
    prompt_kernel<64><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace uly
