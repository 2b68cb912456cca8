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
// Bound by the reading of the cache: for every code of k and v there are G * T
// multiplications (G q heads a cache head, T new rows a sequence), which is far
// below what the tensor cores do in the time that HBM takes for it.
//
// A unit is (sequence, 8 NT rows of its queries, cache head); a row is (token, q
// head of the group).  All units' blocks of 64 keys, in a row, are cut into as
// many equal parts as there are CTAs, so that a long sequence beside short ones
// keeps every SM busy and no SM more than the others.  A CTA's part covers some
// units whole, whose rows it stores, and up to two in part, whose sums it leaves
// in the workspace; combine_kernel adds those up, in order.
//
// A warp takes 16 keys at a time (they are in one page), straight from memory
// into the registers that the matrix instructions want, two steps ahead:
//   S^T = K Q^T   A = K: a lane has bytes 16 c to 16 c + 15 (and 64 on) of keys g
//                 and g + 8 (lane = 4 g + c); which of a row's elements meet in
//                 one instruction does not matter, as long as Q's are the same.
//   O^T = V^T P^T A = V^T: a lane has a piece of keys 2c, 2c+1, 2c+8, 2c+9, whose
//                 codes it pairs up by byte permutation before the conversion;
//                 P^T is S^T transposed in registers (movmatrix).
// e4m3 codes are exact in f16.  q goes to f16 with a power of two taken out of
// each row (so that no element overflows, and none matters that underflows), and
// P is rounded to f16, whose 11 bits are finer than what k and v have left.
// The scales of k multiply the scores.  Those of v go into P: its weight is
// 2^(s - M + log2 v_scale) with a reference maximum M of s + log2 v_scale, beside
// the sum of 2^(s - m), whose reference is m; so f16 holds the weights whatever
// the scales are.
namespace {

constexpr int kBlockKeys = 64;   // keys of a block: 16 for each of a CTA's warps
constexpr int kBuffers = 2;      // a warp's steps in registers: one worked on, the others on their way

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of 16-bit values, a row of which four lanes hold, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint4 load16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// What a sequence has to do: rows, key limit of its last row, blocks, units of
// one head.
struct SeqWork {
  int a, rows, len, blocks, tiles;
};
template <int RT>
__device__ __forceinline__ SeqWork seq_work(const CachedParams& p, int s) {
  const CacheParams& c = p.c;
  SeqWork w;
  int b;
  seq_rows(c, s, w.a, b);
  w.rows = b - w.a;
  const int64_t cap = static_cast<int64_t>(c.table_width) << c.page_shift;
  w.len = static_cast<int>(min(max(static_cast<int64_t>(c.lens[s]), int64_t{0}), min(cap, int64_t{0x7FFF0000})));
  // (a sequence without a key has a block all the same: its rows get zeros)
  w.blocks = max((w.len + kBlockKeys - 1) / kBlockKeys, 1);
  const int64_t rows = static_cast<int64_t>(w.rows) * p.G;
  w.tiles = static_cast<int>((rows + RT - 1) / RT);
  return w;
}

// Four elements of a finished row: o = O 2^(M - m) / l, and once a row its
// log-sum-exp; zero and -inf where no key was seen.
template <int D>
__device__ __forceinline__ void store_row(const CachedParams& p, const SeqWork& w, int64_t r, int h, int d,
                                          const float4& sum, float M, float m, float l) {
  if (r >= static_cast<int64_t>(w.rows) * p.G) return;
  const int token = static_cast<int>(r / p.G), head = h * p.G + static_cast<int>(r % p.G);
  const int64_t at = static_cast<int64_t>(w.a + token) * p.Hq + head;
  if (!in_bounds(&g_cache_violations, at, 1, static_cast<int64_t>(p.c.n_rows) * p.Hq)) return;
  const bool any = l > 0.f || l != l;
  const float f = any ? ex2_approx(M - m) / l : 0.f;
  uint2 v = make_uint2(0u, 0u);
  if (any) v = make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
  *reinterpret_cast<uint2*>(p.out + (at * D + d) * 2) = v;
  if (d == 0 && p.lse) p.lse[at] = any ? (m + lg2_approx(l)) * 0.6931471805599453f : -INFINITY;
}

__device__ __forceinline__ void wait_for_previous_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 16 keys of one head, as a lane holds them.
template <int D>
struct Step {
  uint4 k[2][D / 64];  // keys g and g + 8
  uint32_t v[4][D / 32];  // keys 2c, 2c + 1, 2c + 8, 2c + 9
  float ks, vs;
  bool there;          // in a real page
};

template <int D, int NT>
__global__ void __launch_bounds__(128, kCachedPerSm[NT - 1]) cached_kernel(const __grid_constant__ CachedParams p) {
  constexpr int RT = 8 * NT, KS = D / 16, MT = D / 16;
  const CacheParams& c = p.c;
  __shared__ int64_t sums[4];
  __shared__ int first_seq;
  __shared__ int64_t first_before;
  __shared__ float part[4][RT][D + 4];  // a warp's sums: O, then M, m, l
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cc = lane & 3;

  // ---- this CTA's part of all blocks
  const int per = (c.n_seqs + 127) / 128, s0 = min(tid * per, c.n_seqs), s1 = min(s0 + per, c.n_seqs);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    const SeqWork w = seq_work<RT>(p, s);
    mine += static_cast<int64_t>(w.tiles) * w.blocks * c.H;
  }
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int64_t before = upto - mine, total = 0;
  for (int i = 0; i < 4; ++i) {
    if (i < warp) before += sums[i];
    total += sums[i];
  }
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
  CachedPart* const note = p.parts + blockIdx.x;
  if (blockIdx.x >= ctas) {
    if (tid == 0) note->n = 0;
    return;
  }
  // (total is below 2^50, see the host; ctas below 2^10)
  int64_t lo = total * blockIdx.x / ctas;
  const int64_t hi = total * (blockIdx.x + 1) / ctas;
  if (before <= lo && lo < before + mine) {
    int64_t at = before;
    for (int s = s0; s < s1; ++s) {
      const SeqWork w = seq_work<RT>(p, s);
      const int64_t n = static_cast<int64_t>(w.tiles) * w.blocks * c.H;
      if (lo < at + n) {
        first_seq = s;
        first_before = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  int s = first_seq;
  int64_t off = lo - first_before;  // the part's first block among the sequence's
  SeqWork w = seq_work<RT>(p, s);
  int left_parts = 0;               // of a unit that others finish: how many parts it has
  CachedPart left = {};

  while (lo < hi) {
    const int64_t unit = off / w.blocks;
    const int b0 = static_cast<int>(off - unit * w.blocks);
    const int b1 = static_cast<int>(min(static_cast<int64_t>(w.blocks), b0 + (hi - lo)));
    const int tile = static_cast<int>(unit / c.H), h = static_cast<int>(unit - static_cast<int64_t>(tile) * c.H);

    // ---- the queries: lane 4 g + c has elements 16 c on of rows g (+ 8) for
    // the scores; of the sums it has rows 2 c and 2 c + 1
    uint32_t qf[NT][KS][2];
    float rf[NT][2];   // what turns a row's product into log2 scores, without k's scale
    int lim[NT][2];    // keys that a row sees
    int least = 0x7FFFFFFF, most = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t r = static_cast<int64_t>(tile) * RT + 8 * t + g;
      const bool live = r < static_cast<int64_t>(w.rows) * p.G;
      const int token = live ? static_cast<int>(r / p.G) : 0, head = h * p.G + static_cast<int>(live ? r % p.G : 0);
      uint4 x[D / 64][2];
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[i][j] = make_uint4(0u, 0u, 0u, 0u);
          if (live && in_bounds(&g_cache_violations, w.a + token, 1, c.n_rows))
            x[i][j] = *reinterpret_cast<const uint4*>(p.q + (w.a + token) * p.q_row_bytes +
                                                      (static_cast<int64_t>(head) * D + 64 * i + 16 * cc + 8 * j) * 2);
        }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t e[4] = {x[i][j].x, x[i][j].y, x[i][j].z, x[i][j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(e[k] << 16)), fabsf(__uint_as_float(e[k] & 0xFFFF0000u))));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e2 = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -126), 126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23) * p.scale_log2;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const uint4& y = x[j / 4][(j % 4) / 2];
        const uint32_t e0 = j % 2 ? y.z : y.x, e1 = j % 2 ? y.w : y.y;
        qf[t][j][0] = pack_f16x2(__uint_as_float(e0 << 16) * down, __uint_as_float(e0 & 0xFFFF0000u) * down);
        qf[t][j][1] = pack_f16x2(__uint_as_float(e1 << 16) * down, __uint_as_float(e1 & 0xFFFF0000u) * down);
      }
      // (a position below zero sees nothing; a row past the sequence's what it likes)
      const int64_t see = static_cast<int64_t>(c.lens[s]) - w.rows + token + 1;
      const int my_lim = live ? static_cast<int>(min(max(see, int64_t{0}), static_cast<int64_t>(w.len))) : 0x7FFFFFFF;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        rf[t][i] = __shfl_sync(0xffffffffu, up, (2 * cc + i) * 4);
        lim[t][i] = __shfl_sync(0xffffffffu, my_lim, (2 * cc + i) * 4);
      }
      least = min(least, __reduce_min_sync(0xffffffffu, my_lim));
      most = max(most, __reduce_max_sync(0xffffffffu, live ? my_lim : 0));
    }

    float o[NT][MT][4] = {};
    float m[NT][2], M[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[t][i] = M[t][i] = -INFINITY;
        l[t][i] = 0.f;
      }

    const int32_t* const table = c.table + static_cast<int64_t>(s) * c.table_width;
    const int end = min(b1 * kBlockKeys, most);  // keys of this piece that some row sees
    auto page_of = [&](int key) { return key < end ? __ldg(table + (key >> c.page_shift)) : -1; };
    auto fetch = [&](Step<D>& st, int key, int page) {
      st.there = key < end && page >= 0 && page < c.n_pages;
      if (!st.there) return;
      const int64_t ph = static_cast<int64_t>(page) * c.H + h;
      const int slot = key & (c.page_rows - 1);
      const uint8_t* const k = c.k_pages + (ph * c.page_rows + slot) * D;
      const uint8_t* const v = c.v_pages + (ph * c.page_rows + slot) * D;
      st.ks = __ldg(c.k_scale + ph);
      st.vs = __ldg(c.v_scale + ph);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < D / 64; ++j) st.k[i][j] = load16(k + (g + 8 * i) * D + 64 * j + 16 * cc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // (codes behind the last key may be NaN, and 0 times that would be)
        const int row = 2 * cc + (i & 1) + 8 * (i >> 1);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) st.v[i][j] = 0u;
        if (key + row < end) {
          if constexpr (D == 128) {
            const uint4 x = load16(v + row * D + 16 * g);
            st.v[i][0] = x.x;
            st.v[i][1] = x.y;
            st.v[i][2] = x.z;
            st.v[i][3] = x.w;
          } else {
            const uint2 x = load8(v + row * D + 8 * g);
            st.v[i][0] = x.x;
            st.v[i][1] = x.y;
          }
        }
      }
    };
    auto work = [&](const Step<D>& st, int key) {
      if (!st.there) return;
      float sc[NT][4] = {};
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const uint4 &x = st.k[0][j / 4], &y = st.k[1][j / 4];
        const uint32_t u = j % 4 == 0 ? x.x : j % 4 == 1 ? x.y : j % 4 == 2 ? x.z : x.w;
        const uint32_t z = j % 4 == 0 ? y.x : j % 4 == 1 ? y.y : j % 4 == 2 ? y.z : y.w;
        const uint32_t a0 = f16x2_of_e4m3(static_cast<uint16_t>(u)), a2 = f16x2_of_e4m3(static_cast<uint16_t>(u >> 16));
        const uint32_t a1 = f16x2_of_e4m3(static_cast<uint16_t>(z)), a3 = f16x2_of_e4m3(static_cast<uint16_t>(z >> 16));
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_f16(sc[t], a0, a1, a2, a3, qf[t][j][0], qf[t][j][1]);
      }
      const float lv = lg2_approx(st.vs);
      uint32_t pb[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float f0 = rf[t][0] * st.ks, f1 = rf[t][1] * st.ks;
        float x[4] = {sc[t][0] * f0, sc[t][1] * f1, sc[t][2] * f0, sc[t][3] * f1};  // keys g, g, g + 8, g + 8
        if (key + 16 > least) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key + g + 8 * (i >> 1) >= lim[t][i & 1]) x[i] = -INFINITY;
        }
        const float t0 = fmaxf(x[0], x[2]), t1 = fmaxf(x[1], x[3]);
        if (__any_sync(0xffffffffu, t0 > m[t][0] + 8.f || t1 > m[t][1] + 8.f || t0 + lv > M[t][0] + 8.f ||
                                        t1 + lv > M[t][1] + 8.f)) {
          float r[2] = {t0, t1};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) r[i] = fmaxf(r[i], __shfl_xor_sync(0xffffffffu, r[i], d));
            if (r[i] > m[t][i]) {
              l[t][i] *= ex2_approx(m[t][i] - r[i]);
              m[t][i] = r[i];
            }
            if (r[i] + lv > M[t][i]) {
              const float f = ex2_approx(M[t][i] - (r[i] + lv));
              M[t][i] = r[i] + lv;
#pragma unroll
              for (int q = 0; q < MT; ++q) {
                o[t][q][i] *= f;
                o[t][q][2 + i] *= f;
              }
            }
          }
        }
        float e[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = m[t][i] == -INFINITY ? 0.f : -m[t][i], b = lv - (M[t][i] == -INFINITY ? 0.f : M[t][i]);
          l[t][i] += ex2_approx(x[i] + a) + ex2_approx(x[2 + i] + a);
          e[i] = ex2_approx(x[i] + b);
          e[2 + i] = ex2_approx(x[2 + i] + b);
        }
        pb[t][0] = transpose8(pack_f16x2(e[0], e[1]));
        pb[t][1] = transpose8(pack_f16x2(e[2], e[3]));
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        // four elements of a lane's piece: two of the products' tiles
        const uint32_t a01 = __byte_perm(st.v[0][q], st.v[1][q], 0x5140), a23 = __byte_perm(st.v[0][q], st.v[1][q], 0x7362);
        const uint32_t b01 = __byte_perm(st.v[2][q], st.v[3][q], 0x5140), b23 = __byte_perm(st.v[2][q], st.v[3][q], 0x7362);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a = i ? a23 : a01, b = i ? b23 : b01;
          const uint32_t x0 = f16x2_of_e4m3(static_cast<uint16_t>(a)), x1 = f16x2_of_e4m3(static_cast<uint16_t>(a >> 16));
          const uint32_t x2 = f16x2_of_e4m3(static_cast<uint16_t>(b)), x3 = f16x2_of_e4m3(static_cast<uint16_t>(b >> 16));
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * q + i], x0, x1, x2, x3, pb[t][0], pb[t][1]);
        }
      }
    };

    // ---- steps of this warp, two loads ahead of the arithmetic
    {
      constexpr int kStride = kBlockKeys, kAhead = kBuffers - 1;
      int key = b0 * kBlockKeys + 16 * warp;
      Step<D> st[kBuffers];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(st[i], key + i * kStride, page_of(key + i * kStride));
      int page = page_of(key + kAhead * kStride);
      while (key < end) {
#pragma unroll
        for (int i = 0; i < kBuffers; ++i) {
          const int next = page_of(key + (kAhead + 1) * kStride);
          fetch(st[(i + kAhead) % kBuffers], key + kAhead * kStride, page);
          page = next;
          work(st[i], key);
          key += kStride;
        }
      }
    }

    // ---- the four warps' sums
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* const row = part[warp][8 * t + 2 * cc + i];
        float x = l[t][i];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (g == 0) {
          row[D] = M[t][i];
          row[D + 1] = m[t][i];
          row[D + 2] = x;
        }
        // (a lane has D / 8 elements of the row in a row)
#pragma unroll
        for (int q = 0; q < MT; q += 2)
          *reinterpret_cast<float4*>(row + (D / 8) * g + 2 * q) =
              make_float4(o[t][q][i], o[t][q][2 + i], o[t][q + 1][i], o[t][q + 1][2 + i]);
      }
    __syncthreads();
    const bool whole = b0 == 0 && b1 == w.blocks;
    float* const slot = p.sums + (static_cast<int64_t>(2 * blockIdx.x + (b0 == 0)) * RT) * (D + 4);
    for (int i = tid; i < RT * (D / 4); i += 128) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float Mx = -INFINITY, mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        Mx = fmaxf(Mx, part[k][r][D]);
        mx = fmaxf(mx, part[k][r][D + 1]);
      }
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float ls = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(&part[k][r][d]);
        const float f = part[k][r][D] == -INFINITY ? 0.f : ex2_approx(part[k][r][D] - Mx);
        const float f2 = part[k][r][D + 1] == -INFINITY ? 0.f : ex2_approx(part[k][r][D + 1] - mx);
        sum.x += f * x.x;
        sum.y += f * x.y;
        sum.z += f * x.z;
        sum.w += f * x.w;
        ls += f2 * part[k][r][D + 2];
      }
      if (whole) {
        store_row<D>(p, w, static_cast<int64_t>(tile) * RT + r, h, d, sum, Mx, mx, ls);
      } else {
        *reinterpret_cast<float4*>(slot + r * (D + 4) + d) = sum;
        if (d == 0) *reinterpret_cast<float4*>(slot + r * (D + 4) + D) = make_float4(Mx, mx, ls, 0.f);
      }
    }
    __syncthreads();  // `part` is free again
    if (b0 == 0 && !whole) {
      // the unit's last block is in the part of the CTA that has block lo + blocks - 1
      const int64_t last = lo + w.blocks - 1;
      int64_t cta = last * ctas / total;
      while (cta + 1 < ctas && total * (cta + 1) / ctas <= last) ++cta;
      while (total * cta / ctas > last) --cta;
      left = CachedPart{static_cast<int32_t>(cta - blockIdx.x + 1), s, tile, h};
    }
    lo += b1 - b0;
    off += b1 - b0;
    while (lo < hi && off >= static_cast<int64_t>(w.tiles) * w.blocks * c.H) {
      off -= static_cast<int64_t>(w.tiles) * w.blocks * c.H;
      w = seq_work<RT>(p, ++s);
    }
  }
  if (tid == 0) *note = left;
}

// The rows of a unit that several CTAs have parts of: one CTA a row, its warps
// taking the parts in turn.
template <int D, int NT>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ CachedParams p) {
  constexpr int RT = 8 * NT;
  __shared__ float4 sums[8][D / 4];
  __shared__ float ref[8][4];
  wait_for_previous_launch();
  const CachedPart part = p.parts[blockIdx.x];
  if (!part.n) return;
  const SeqWork w = seq_work<RT>(p, part.seq);
  const int64_t r = static_cast<int64_t>(part.tile) * RT + blockIdx.y;
  if (r >= static_cast<int64_t>(w.rows) * p.G) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto slot = [&](int k) {
    return p.sums + (static_cast<int64_t>(2 * (blockIdx.x + k) + (k == 0)) * RT + blockIdx.y) * (D + 4);
  };
  // references first, then the sums against them
  float Mx = -INFINITY, mx = -INFINITY;
  for (int k = threadIdx.x; k < part.n; k += 256) {
    const float* const x = slot(k) + D;
    Mx = fmaxf(Mx, x[0]);
    mx = fmaxf(mx, x[1]);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, d));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  }
  if (lane == 0) {
    ref[warp][0] = Mx;
    ref[warp][1] = mx;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    Mx = fmaxf(Mx, ref[k][0]);
    mx = fmaxf(mx, ref[k][1]);
  }
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  float ls = 0.f;
  for (int k = warp; k < part.n; k += 8) {
    const float* const x = slot(k);
    const float4 h = *reinterpret_cast<const float4*>(x + D);
    const float f = h.x == -INFINITY ? 0.f : ex2_approx(h.x - Mx), f2 = h.y == -INFINITY ? 0.f : ex2_approx(h.y - mx);
    if (lane < D / 4) {
      const float4 y = *reinterpret_cast<const float4*>(x + 4 * lane);
      sum.x += f * y.x;
      sum.y += f * y.y;
      sum.z += f * y.z;
      sum.w += f * y.w;
    }
    ls += f2 * h.z;
  }
  if (lane < D / 4) sums[warp][lane] = sum;
  if (lane == 0) ref[warp][2] = ls;
  __syncthreads();
  if (warp == 0 && lane < D / 4) {
    ls = 0.f;
    sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float4 y = sums[k][lane];
      sum.x += y.x;
      sum.y += y.y;
      sum.z += y.z;
      sum.w += y.w;
      ls += ref[k][2];
    }
    store_row<D>(p, w, r, part.head, 4 * lane, sum, Mx, mx, ls);
  }
}

template <int D, int NT>
cudaError_t launch_cached(const CachedParams& p, cudaStream_t s) {
  cached_kernel<D, NT><<<p.grid, 128, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid, 8 * NT);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<D, NT>, p);
}

}  // namespace

cudaError_t launch_cache_attention(const CachedParams& p, int D, cudaStream_t s) {
  if (D == 128) return p.row_tiles == 1 ? launch_cached<128, 1>(p, s) : launch_cached<128, 2>(p, s);
  return p.row_tiles == 1 ? launch_cached<64, 1>(p, s) : launch_cached<64, 2>(p, s);
}

}  // namespace uly
