// cache.cu -- the 8-bit paged cache: k and v rows of new tokens into its pages,
// and the attention of the newest tokens over it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "serve.cuh"
#include "tc.cuh"

namespace uly {

__device__ unsigned long long g_cache_violations;

uint64_t cache_violations(bool reset) {
  if (!kChecked) return 0;
  unsigned long long v = 0;
  if (cudaMemcpyFromSymbol(&v, g_cache_violations, sizeof v) != cudaSuccess) return ~0ull;
  if (reset) {
    const unsigned long long z = 0;
    if (cudaMemcpyToSymbol(g_cache_violations, &z, sizeof z) != cudaSuccess) return ~0ull;
  }
  return v;
}

// two e4m3 codes (low byte first) -> f16x2, exact
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// two floats -> two e4m3 codes (RNE, saturating), lo in the low byte
__device__ __forceinline__ uint16_t e4m3x2_of_f32(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- append --
constexpr int kLeastExponent = -60;

// 2^e for the least e >= -60 with amax <= 448 * 2^e.  448 = 1.75 * 2^8, so e is
// the exponent of amax less 8, and one more where its mantissa is above 1.75.
// (An infinity, all exponent bits set, gives 2^120.)
__device__ __forceinline__ float scale_of(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, kLeastExponent);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The rows [a, b) of sequence `s`, clamped to the tensor.
__device__ __forceinline__ void seq_rows(const CacheParams& c, int s, int& a, int& b) {
  a = min(max(c.starts[s], 0), c.n_rows);
  b = min(max(c.starts[s + 1], a), c.n_rows);
}

// One CTA looks after `group` new rows of one head of k (blockIdx.z 0) or v (1).
// A page's first new row leads: whoever has it quantises all new rows of that
// page, so that the page's scale is one CTA's business.  The rows stay in
// registers between the maximum and the codes: one read, one write.
//   PASSES rows of 16 bytes a thread: page_rows * D * 2 / (16 * 128).
// Bound by HBM for prompts, by latency for single tokens.
template <int D, int PASSES>
__global__ void __launch_bounds__(128) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8;             // threads a row
  constexpr int kRows = 128 / kLanes;       // rows a pass
  const CacheParams& c = p.c;
  const int tid = threadIdx.x, h = blockIdx.y, t = blockIdx.z;
  __shared__ int4 task[128];                // page, slot, rows, first row
  __shared__ int n_task;
  __shared__ float top[4];
  if (tid == 0) n_task = 0;
  __syncthreads();
  const int64_t row64 = static_cast<int64_t>(blockIdx.x) * p.group + tid;
  if (tid < p.group && row64 < c.n_rows) {
    const int row = static_cast<int>(row64);
    int lo = 0, hi = c.n_seqs;  // the first sequence that ends behind the row
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (c.starts[mid + 1] > row)
        hi = mid;
      else
        lo = mid + 1;
    }
    if (lo < c.n_seqs) {
      int a, b;
      seq_rows(c, lo, a, b);
      const int64_t pos = static_cast<int64_t>(c.lens[lo]) - (b - a) + (row - a);
      const int slot = static_cast<int>(pos & (c.page_rows - 1));
      if (row >= a && pos >= 0 && (pos >> c.page_shift) < c.table_width && (row == a || slot == 0)) {
        const int page = c.table[static_cast<int64_t>(lo) * c.table_width + (pos >> c.page_shift)];
        if (page >= 0 && page < c.n_pages)
          task[atomicAdd(&n_task, 1)] = make_int4(page, slot, min(b - row, c.page_rows - slot), row);
      }
    }
  }
  __syncthreads();
  const int n = n_task;  // (the tasks do not depend on one another: any order)
  const int sub = tid / kLanes, piece = tid % kLanes;
  for (int i = 0; i < n; ++i) {
    const int page = task[i].x, slot0 = task[i].y, rows = task[i].z, row0 = task[i].w;
    const uint8_t* x = p.x[t] + static_cast<int64_t>(h) * D * 2 + piece * 16;
    uint4 v[PASSES];
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < PASSES; ++q) {
      const int r = q * kRows + sub;
      v[q] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && in_bounds(&g_cache_violations, row0 + r, 1, c.n_rows))
        v[q] = *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(row0 + r) * p.row_bytes[t]);
      const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)  // (fmaxf leaves a NaN out)
        m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((tid & 31) == 0) top[tid >> 5] = m;
    float* const scale = (t ? c.v_scale : c.k_scale) + static_cast<int64_t>(page) * c.H + h;
    const float have = slot0 ? *scale : 0.f;
    __syncthreads();
    m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const float now = fmaxf(scale_of(m), have);
    uint8_t* const codes = (t ? c.v_pages : c.k_pages) + (static_cast<int64_t>(page) * c.H + h) * c.page_rows * D;
    if (slot0 && now != have) {
      // the page's older codes to the larger scale
      const float f = have / now;
      for (int e = tid; e < slot0 * (D / 8); e += 128) {
        uint2* const at = reinterpret_cast<uint2*>(codes) + e;
        uint2 b = *at;
        uint32_t* w = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float f0, f1, f2, f3;
          f16x2_to_f32(f16x2_of_e4m3(static_cast<uint16_t>(w[k])), f0, f1);
          f16x2_to_f32(f16x2_of_e4m3(static_cast<uint16_t>(w[k] >> 16)), f2, f3);
          w[k] = pack_b16x2(e4m3x2_of_f32(f0 * f, f1 * f), e4m3x2_of_f32(f2 * f, f3 * f));
        }
        *at = b;
      }
    }
    const float inv = 1.f / now;  // (exact: a power of two, unless the page came with another scale)
#pragma unroll
    for (int q = 0; q < PASSES; ++q) {
      const int r = q * kRows + sub;
      if (r >= rows || !in_bounds(&g_cache_violations, slot0 + r, 1, c.page_rows)) continue;
      const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
      uint16_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = e4m3x2_of_f32(__uint_as_float(w[k] << 16) * inv, __uint_as_float(w[k] & 0xFFFF0000u) * inv);
      *reinterpret_cast<uint2*>(codes + (slot0 + r) * D + piece * 8) =
          make_uint2(pack_b16x2(o[0], o[1]), pack_b16x2(o[2], o[3]));
    }
    if (tid == 0) *scale = now;
    __syncthreads();  // `top` is free again
  }
}

template <int D>
static cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  const dim3 grid((p.c.n_rows + p.group - 1) / p.group, p.c.H, 2);
  switch (p.c.page_rows * D / 1024) {
    case 1: append_kernel<D, 1><<<grid, 128, 0, s>>>(p); break;
    case 2: append_kernel<D, 2><<<grid, 128, 0, s>>>(p); break;
    case 4: append_kernel<D, 4><<<grid, 128, 0, s>>>(p); break;
    case 8: append_kernel<D, 8><<<grid, 128, 0, s>>>(p); break;
    case 16: append_kernel<D, 16><<<grid, 128, 0, s>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_append(const AppendParams& p, int D, cudaStream_t s) {
  return D == 128 ? launch_append<128>(p, s) : launch_append<64>(p, s);
}

// ------------------------------------------------------------- attention --
// One warp per row and q head; the lanes share the head's elements.
template <int D>
__global__ void __launch_bounds__(256) cached_kernel(const __grid_constant__ CachedParams p) {
  constexpr int E = D / 32;
  const CacheParams& c = p.c;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x, h = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (h >= p.Hq) return;
  int lo = 0, hi = c.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c.starts[mid + 1] > row)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (lo >= c.n_seqs) return;
  int a, b;
  seq_rows(c, lo, a, b);
  if (row < a) return;
  const int64_t cap = static_cast<int64_t>(c.table_width) * c.page_rows;
  const int64_t limit = min(static_cast<int64_t>(c.lens[lo]) - (b - a) + (row - a) + 1, cap);
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(p.q + row * p.q_row_bytes) + h * D;
  float qf[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = __bfloat162float(q[lane * E + e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t j = 0; j < limit; ++j) {
    const int page = c.table[static_cast<int64_t>(lo) * c.table_width + (j >> c.page_shift)];
    if (page < 0 || page >= c.n_pages) continue;
    const int64_t ph = static_cast<int64_t>(page) * c.H + h / p.G;
    const int64_t off = (ph * c.page_rows + (j & (c.page_rows - 1))) * D + lane * E;
    float s = 0.f, vf[E];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      float k0, k1;
      f16x2_to_f32(f16x2_of_e4m3(*reinterpret_cast<const uint16_t*>(c.k_pages + off + e)), k0, k1);
      f16x2_to_f32(f16x2_of_e4m3(*reinterpret_cast<const uint16_t*>(c.v_pages + off + e)), vf[e], vf[e + 1]);
      s += qf[e] * k0 + qf[e + 1] * k1;
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2 * c.k_scale[ph];
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn), vs = c.v_scale[ph];
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * vs * vf[e];
  }
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + (static_cast<int64_t>(row) * p.Hq + h) * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane * E + e] = __float2bfloat16(l > 0.f ? o[e] / l : 0.f);
  if (lane == 0 && p.lse)
    p.lse[static_cast<int64_t>(row) * p.Hq + h] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

cudaError_t launch_cache_attention(const CachedParams& p, int D, cudaStream_t s) {
  const dim3 grid(p.c.n_rows, (p.Hq + 7) / 8);
  if (D == 128)
    cached_kernel<128><<<grid, 256, 0, s>>>(p);
  else
    cached_kernel<64><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace uly
