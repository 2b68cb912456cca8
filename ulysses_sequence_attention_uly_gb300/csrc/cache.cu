// cache.cu -- the 8-bit paged cache: k and v rows of new tokens into its pages,
// and the attention of the newest tokens over it.
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

// Does `row` lead, that is, is it the first new row of its page?  Then its page,
// slot and the number of the page's new rows.
__device__ __forceinline__ bool leads(const CacheParams& c, int row, int& page, int& slot, int& rows) {
  int lo = 0, hi = c.n_seqs;  // the first sequence that ends behind the row
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c.starts[mid + 1] > row)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (lo >= c.n_seqs) return false;
  int a, b;
  seq_rows(c, lo, a, b);
  const int64_t pos = static_cast<int64_t>(c.lens[lo]) - (b - a) + (row - a);
  slot = static_cast<int>(pos & (c.page_rows - 1));
  if (row < a || pos < 0 || (pos >> c.page_shift) >= c.table_width || (row != a && slot != 0)) return false;
  page = c.table[static_cast<int64_t>(lo) * c.table_width + (pos >> c.page_shift)];
  rows = min(b - row, c.page_rows - slot);
  return page >= 0 && page < c.n_pages;
}

// Largest magnitude of eight bf16 values (fmaxf leaves a NaN out).
__device__ __forceinline__ float largest(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
  return m;
}

// Eight bf16 values times f, as codes.
__device__ __forceinline__ uint2 codes_of(const uint4& v, float f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint16_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    o[k] = e4m3x2_of_f32(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f);
  return make_uint2(pack_b16x2(o[0], o[1]), pack_b16x2(o[2], o[3]));
}

// Eight codes brought from one scale to another, f their ratio.
__device__ __forceinline__ void bring(uint2* at, float f) {
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

// One CTA looks after `group` new rows of one head of k (blockIdx.z 0) or v (1).
// A page's first new row leads: whoever has it quantises all new rows of that
// page, so that the page's scale is one CTA's business.  The rows stay in
// registers between the maximum and the codes: one read, one write.
//   PASSES rows of 16 bytes a thread: page_rows * D * 2 / (16 * 128).
// Bound by HBM; what a row's place hangs on is three accesses in a row, so that
// many CTAs an SM count (16384 rows, 8 heads of 128, pages of 64: with five 22.0
// us, with seven 20.6, 4900 GB/s).
template <int D, int PASSES>
__global__ void __launch_bounds__(128, PASSES <= 4 ? 12 : PASSES == 8 ? 7 : 4)
    append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8;             // threads a row
  constexpr int kRows = 128 / kLanes;       // rows a pass
  const CacheParams& c = p.c;
  const int tid = threadIdx.x, h = blockIdx.y, t = blockIdx.z;
  __shared__ int4 task[128];                // page, slot, rows, first row
  __shared__ int n_task;
  __shared__ float top[4];
  if (tid == 0) n_task = 0;
  __syncthreads();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * p.group + tid;
  int page, slot, rows;
  if (tid < p.group && row < c.n_rows && leads(c, static_cast<int>(row), page, slot, rows))
    task[atomicAdd(&n_task, 1)] = make_int4(page, slot, rows, static_cast<int>(row));
  __syncthreads();
  const int n = n_task;  // (the tasks do not depend on one another: any order)
  const int sub = tid / kLanes, piece = tid % kLanes;
  for (int i = 0; i < n; ++i) {
    const int page = task[i].x, slot0 = task[i].y, rows = task[i].z, row0 = task[i].w;
    const uint8_t* const x = p.x[t] + static_cast<int64_t>(h) * D * 2 + piece * 16;
    uint4 v[PASSES];
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < PASSES; ++q) {
      const int r = q * kRows + sub;
      v[q] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && in_bounds(&g_cache_violations, row0 + r, 1, c.n_rows))
        v[q] = *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(row0 + r) * p.row_bytes[t]);
    }
#pragma unroll
    for (int q = 0; q < PASSES; ++q) m = fmaxf(m, largest(v[q]));
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((tid & 31) == 0) top[tid >> 5] = m;
    const int64_t ph = static_cast<int64_t>(page) * c.H + h;
    float* const scale = (t ? c.v_scale : c.k_scale) + ph;
    const float have = slot0 ? *scale : 0.f;
    __syncthreads();
    const float now = fmaxf(scale_of(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]))), have);
    uint8_t* const codes = (t ? c.v_pages : c.k_pages) + ph * c.page_rows * D;
    if (slot0 && now != have)  // the page's older codes to the larger scale
      for (int e = tid; e < slot0 * (D / 8); e += 128) bring(reinterpret_cast<uint2*>(codes) + e, have / now);
    const float inv = 1.f / now;  // (exact: a power of two, unless the page came with another scale)
#pragma unroll
    for (int q = 0; q < PASSES; ++q) {
      const int r = q * kRows + sub;
      if (r < rows && in_bounds(&g_cache_violations, slot0 + r, 1, c.page_rows))
        *reinterpret_cast<uint2*>(codes + (slot0 + r) * D + piece * 8) = codes_of(v[q], inv);
    }
    if (tid == 0) *scale = now;
    __syncthreads();  // `top` is free again
  }
}

// The same for a few tokens a sequence: a warp for each row and head, half of it
// for k and half for v, where the row leads.  Up to kHeld rows a lane stay in
// registers; of more, all are read again for their codes.
template <int D>
__global__ void __launch_bounds__(128) append_few_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8;        // lanes a row
  constexpr int kRows = 16 / kLanes;   // rows that half a warp takes at once
  constexpr int kHeld = 4;
  const CacheParams& c = p.c;
  const int lane = threadIdx.x & 31, h = blockIdx.y * 4 + (threadIdx.x >> 5), t = lane >> 4;
  const int sub = (lane & 15) / kLanes, piece = lane % kLanes;
  int page, slot0, rows;
  if (h >= c.H || !leads(c, blockIdx.x, page, slot0, rows)) return;
  const int row0 = blockIdx.x;
  const uint8_t* const x = (t ? p.x[1] : p.x[0]) + static_cast<int64_t>(h) * D * 2 + piece * 16;
  const int64_t row_bytes = t ? p.row_bytes[1] : p.row_bytes[0];
  const int64_t ph = static_cast<int64_t>(page) * c.H + h;
  float* const scale = (t ? c.v_scale : c.k_scale) + ph;
  const float have = slot0 ? *scale : 0.f;
  auto load = [&](int r) {
    return r < rows && in_bounds(&g_cache_violations, row0 + r, 1, c.n_rows)
               ? *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(row0 + r) * row_bytes)
               : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 v[kHeld];
  float m = 0.f;
#pragma unroll
  for (int q = 0; q < kHeld; ++q) v[q] = load(q * kRows + sub);
#pragma unroll
  for (int q = 0; q < kHeld; ++q) m = fmaxf(m, largest(v[q]));
#pragma unroll 4
  for (int r = kHeld * kRows; r < rows; r += kRows) m = fmaxf(m, largest(load(r + sub)));
#pragma unroll
  for (int d = 8; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float now = fmaxf(scale_of(m), have);
  __syncwarp();  // every lane has read the scale before one writes it (shuffles order no memory)
  uint8_t* const codes = (t ? c.v_pages : c.k_pages) + ph * c.page_rows * D;
  if (slot0 && now != have)
    for (int e = lane & 15; e < slot0 * (D / 8); e += 16) bring(reinterpret_cast<uint2*>(codes) + e, have / now);
  const float inv = 1.f / now;
  auto store = [&](int r, const uint4& y) {
    if (r < rows && in_bounds(&g_cache_violations, slot0 + r, 1, c.page_rows))
      *reinterpret_cast<uint2*>(codes + (slot0 + r) * D + piece * 8) = codes_of(y, inv);
  };
#pragma unroll
  for (int q = 0; q < kHeld; ++q) store(q * kRows + sub, v[q]);
#pragma unroll 4
  for (int r = kHeld * kRows; r < rows; r += kRows) store(r + sub, load(r + sub));
  if ((lane & 15) == 0) *scale = now;
}

template <int D>
static cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  if (!p.group) {
    append_few_kernel<D><<<dim3(p.c.n_rows, (p.c.H + 3) / 4), 128, 0, s>>>(p);
    return cudaGetLastError();
  }
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
// below what even mma.sync does in the time that HBM takes for it (tensor pipe 16%
// of cycles).  32 heads on 8 of 128: two sequences of 120 and 131 thousand tokens
// 86 us, 6.0 TB/s (the loads alone, without arithmetic: 82); 64 sequences of 200 to
// 8000 tokens 67 us, 5.0 TB/s; one of 499 tokens 8 us.
//
// A unit is (sequence, 8 NT rows of its queries, cache head); a row is (token, q
// head of the group).  A unit's keys, in blocks of 64, are cut into equal parts of
// about the same length for all units, up to twice as many as CTAs run at once:
// SMs differ by a third in how fast they get data, so the GPU gives the next part
// to whoever is done.  A part that is a whole unit stores its rows; the sums of the
// others go through the workspace, and combine_kernel adds them up, in order.
//
// A warp takes 16 keys at a time (they are in one page) through a ring of its own
// in shared memory, and from there as the matrix instructions want them:
//   S^T = K Q^T   A = K: a lane has bytes 16 c to 16 c + 15 (and 64 on) of keys g
//                 and g + 8 (lane = 4 g + c); which of a row's elements meet in
//                 one instruction does not matter, as long as Q's are the same.
//   O^T = V^T P^T A = V^T: a lane has a piece of keys 2c, 2c+1, 2c+8, 2c+9, whose
//                 codes it pairs up by byte permutation before the conversion;
//                 P^T is S^T transposed in registers (movmatrix).
// e4m3 codes are exact in f16.  q goes to f16 with a power of two taken out of
// each row, so that no element overflows and those down to 2^-31 of the largest are
// exact, and P is rounded to f16, whose 11 bits are finer than what k and v have left.
// The scales of k multiply the scores.  Those of v go into P: its weight is
// 2^(s - M + log2 v_scale) with a reference M that follows the maximum of s + log2
// v_scale, beside the sum of 2^(s - m), whose reference is m.  M is kRoom below that
// maximum when it is raised, and is raised when a weight would pass 2^(8 + kRoom):
// f16's upper orders are used, and weights down to 2^-21 of the largest keep its 11
// bits (with a page's scale 2^20 above the others', the others' weights do); one
// that is smaller is off by 2^-32 of the largest at most.
namespace {

constexpr int kBlockKeys = 64;   // keys of a block: 16 for each of a CTA's warps
constexpr float kRoom = 7.f;     // 2^(8 + kRoom), with the exponential's error, is in f16's range
constexpr int kLongPart = 320 << 10;  // bytes of codes

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
// 16 (4) bytes from global to shared memory, asynchronously; `there` false: zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// wait for the launch before this one in the stream (a programmatic dependency)
__device__ __forceinline__ void wait_for_previous_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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

// A unit's row r: its place among all rows and heads of q (first_row: the
// sequence's first).
__device__ __forceinline__ int64_t row_place(const CachedParams& p, int first_row, int h, int64_t r) {
  return (first_row + r / p.G) * p.Hq + h * p.G + r % p.G;
}

// Four elements of a finished row: o = O 2^(M - m) / l, and once a row its
// log-sum-exp; zero and -inf where no key was seen.
template <int D>
__device__ __forceinline__ void store_row(const CachedParams& p, int64_t at, int d, const float4& sum, float M, float m,
                                          float l) {
  if (!in_bounds(&g_cache_violations, at, 1, static_cast<int64_t>(p.c.n_rows) * p.Hq)) return;
  const bool any = l > 0.f || l != l;
  const float f = any ? ex2_approx(M - m) / l : 0.f;
  uint2 v = make_uint2(0u, 0u);
  if (any) v = make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
  *reinterpret_cast<uint2*>(p.out + (at * D + d) * 2) = v;
  if (d == 0 && p.lse) p.lse[at] = any ? (m + lg2_approx(l)) * 0.6931471805599453f : -INFINITY;
}

// A warp's ring in shared memory: a stage has 16 keys' codes of k, then of v, in
// 16-byte pieces, and the two scales.  Piece i of row r is at piece i ^ (r mod 8)
// (64-wide rows: i ^ (r / 2 mod 4)), so that the reads below go without bank
// conflicts (64-wide v: two lanes a bank).
template <int D, int NT>
struct CachedCfg {
  // one worked on, the others on their way: 4 KB a warp, either way (more is
  // slower: two contexts of 120 to 131 thousand tokens with two stages 85 us, with
  // three 92)
  static constexpr int kStages = D == 128 ? 2 : 3;
  static constexpr int kHalf = 16 * D;                  // codes of k (or v)
  static constexpr int kStageBytes = 2 * kHalf + 16;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kPart = 8 * NT * (D + 4);        // floats: a warp's sums, which take the ring's place
  static constexpr int kSmem = 4 * (kWarpBytes > 4 * kPart ? kWarpBytes : 4 * kPart);
  static_assert(kSmem <= 48 * 1024, "no attribute is set for more");
  __device__ static __forceinline__ uint32_t piece(int row, int i) {
    return D == 128 ? row * 128 + ((i ^ (row & 7)) << 4) : row * 64 + ((i ^ ((row >> 1) & 3)) << 4);
  }
};

// ---- parts
// Parts of a unit, for `total` blocks of all units.  Few units have many parts
// each: as many in all as CTAs run at once, and none more, since one more would
// run alone.  Of many units the parts cannot be that even, and where they are
// long (kLongPart and more of codes), half of that length keeps the last ones from
// running alone.  64 ragged sequences, 8 heads, us with parts of a slot's share and
// of half of it, by the share:
//   128-wide   53 KB 23.1, 23.9   95 KB 28.3, 27.7   185 KB 37.7, 34.9   363 KB 58.6, 51.6   719 KB 101, 84
//    64-wide   48 KB 18.8, 23.3   93 KB 25.3, 27.7   181 KB 35.7, 36.8   359 KB 58.4, 55.8   715 KB 104, 93
// So 64-wide heads cross between 180 and 360 KB, 128-wide ones near 90 already; one
// constant for both gives the latter up to 8% away in between.  200 sequences are
// within 2% either way.
template <int D>
__device__ __forceinline__ int unit_parts(const CachedParams& p, const SeqWork& w, int64_t total) {
  int64_t n;
  if (p.whole) return 1;
  if (p.few) {
    n = static_cast<int64_t>(w.blocks) * p.slots / max(total, int64_t{1});
  } else {
    const int64_t slots = total > p.slots * (kLongPart / (kBlockKeys * 2 * D)) ? 2 * p.slots : p.slots;
    const int64_t blocks = max((total + slots - 1) / slots, int64_t{1});
    n = (w.blocks + blocks / 2) / blocks;
  }
  return static_cast<int>(min(max(n, int64_t{1}), static_cast<int64_t>(min(w.blocks, max_unit_parts(p.few)))));
}

// Sums over the CTA's 128 threads, exclusive; *total receives the whole.
__device__ __forceinline__ int64_t sum_before(int64_t v, int64_t* shared, int64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t upto = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 31) shared[warp] = upto;
  __syncthreads();
  int64_t before = upto - v, all = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < warp) before += shared[i];
    all += shared[i];
  }
  __syncthreads();
  *total = all;
  return before;
}

// More than 128 sequences: the parts before each of them, [n_seqs + 1], and the
// blocks of all units, by one CTA.
template <int D, int RT>
__global__ void __launch_bounds__(128) parts_kernel(const __grid_constant__ CachedParams p) {
  __shared__ int64_t shared[4];
  let_next_launch_start();
  const CacheParams& c = p.c;
  int64_t mine = 0, total;
  for (int s = threadIdx.x; s < c.n_seqs; s += 128) {
    const SeqWork w = seq_work<RT>(p, s);
    mine += static_cast<int64_t>(w.tiles) * w.blocks * c.H;
  }
  sum_before(mine, shared, &total);
  int64_t done = 0;
  for (int s0 = 0; s0 < c.n_seqs; s0 += 128) {
    const int s = s0 + threadIdx.x;
    int64_t n = 0, all;
    if (s < c.n_seqs) {
      const SeqWork w = seq_work<RT>(p, s);
      n = static_cast<int64_t>(w.tiles) * unit_parts<D>(p, w, total) * c.H;
    }
    const int64_t at = done + sum_before(n, shared, &all);
    if (s < c.n_seqs) p.before[s] = at;
    done += all;
  }
  if (threadIdx.x == 0) {
    p.before[c.n_seqs] = done;
    p.before[c.n_seqs + 1] = total;
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(128, kCachedPerSm[NT - 1]) cached_kernel(const __grid_constant__ CachedParams p) {
  using C = CachedCfg<D, NT>;
  constexpr int RT = 8 * NT, KS = D / 16, MT = D / 16;
  const CacheParams& c = p.c;
  extern __shared__ __align__(16) uint8_t ring_raw[];
  __shared__ int64_t shared[4];
  __shared__ int my_seq;
  __shared__ int64_t my_before, my_total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cc = lane & 3;
  float(*const part)[RT][D + 4] = reinterpret_cast<float(*)[RT][D + 4]>(ring_raw);  // a warp's sums: O, then M, m, l
  const uint32_t ring = smem_u32(ring_raw) + warp * C::kWarpBytes;
  CachedPart* const note = p.parts + blockIdx.x;
  let_next_launch_start();

  // ---- which part
  wait_for_previous_launch();
  if (tid == 0) my_seq = -1;
  if (c.n_seqs <= 128) {
    // a sequence a thread
    SeqWork w = {};
    int64_t total, all;
    if (tid < c.n_seqs) w = seq_work<RT>(p, tid);
    sum_before(static_cast<int64_t>(w.tiles) * w.blocks * c.H, shared, &total);
    const int64_t n = tid < c.n_seqs ? static_cast<int64_t>(w.tiles) * unit_parts<D>(p, w, total) * c.H : 0;
    const int64_t at = sum_before(n, shared, &all);
    if (at <= blockIdx.x && blockIdx.x < at + n) {
      my_seq = tid;
      my_before = at;
      my_total = total;
    }
  } else {
    __syncthreads();
    if (warp == 0 && blockIdx.x < p.before[c.n_seqs]) {
      // the last sequence that begins at or before the part, 32 ways at a time
      int lo = 0, n = c.n_seqs;
      while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const uint32_t yes = __ballot_sync(0xffffffffu, i < n && p.before[lo + i] <= blockIdx.x);
        const int k = 31 - __clz(yes);  // (lane 0 always)
        lo += k * step;
        n = min(step, n - k * step);
      }
      if (lane == 0) {
        my_seq = lo;
        my_before = p.before[lo];
        my_total = p.before[c.n_seqs + 1];
      }
    }
  }
  __syncthreads();
  const int s = my_seq;
  if (s < 0) {
    if (tid == 0 && !p.whole) note->n = 0;
    return;
  }
  const SeqWork w = seq_work<RT>(p, s);
  const int parts = unit_parts<D>(p, w, my_total);
  // (the heads of a page are next to each other in memory: neighbouring CTAs take
  // them, at the same time)
  const int64_t off = blockIdx.x - my_before, units = static_cast<int64_t>(w.tiles) * c.H, unit = off % units;
  // starts that fall give rows to several sequences, and more parts than the grid
  // has been made for: units that are not all there are left out, so that
  // combine_kernel finds every part it looks for
  if (my_before + units * parts > gridDim.x) {
    if (tid == 0 && !p.whole) note->n = 0;
    return;
  }
  const int idx = static_cast<int>(off / units);
  const int tile = static_cast<int>(unit / c.H), h = static_cast<int>(unit - static_cast<int64_t>(tile) * c.H);
  const int b0 = static_cast<int>(static_cast<int64_t>(w.blocks) * idx / parts);
  const int b1 = static_cast<int>(static_cast<int64_t>(w.blocks) * (idx + 1) / parts);
  const int64_t row0 = static_cast<int64_t>(tile) * RT;  // the unit's rows among the sequence's
  const int live = static_cast<int>(min(static_cast<int64_t>(w.rows) * p.G - row0, int64_t{RT}));
  if (tid == 0 && !p.whole) *note = CachedPart{parts, idx, static_cast<int32_t>(units), live, row_place(p, w.a, h, row0), row0};

  {
    const int32_t* const table = c.table + static_cast<int64_t>(s) * c.table_width;
    // (its last row sees most; a position below zero sees nothing)
    const int64_t all_see = static_cast<int64_t>(c.lens[s]) - w.rows + 1;
    auto sees = [&](int token) { return static_cast<int>(min(max(all_see + token, int64_t{0}), static_cast<int64_t>(w.len))); };
    const int end = min(b1 * kBlockKeys, sees(static_cast<int>((row0 + live - 1) / p.G)));  // keys that some row sees
    auto page_of = [&](int key) { return key < end ? __ldg(table + (key >> c.page_shift)) : -1; };
    // copies of the step at `key` into a stage; is there anything in it?
    auto fetch = [&](int stage, int key, int page) {
      const bool there = key < end && page >= 0 && page < c.n_pages;
      if (there) {
        const int64_t ph = static_cast<int64_t>(page) * c.H + h;
        const int64_t at = (ph * c.page_rows + (key & (c.page_rows - 1))) * D;
        const uint32_t to = ring + stage * C::kStageBytes;
        constexpr int kPieces = D / 16, kRows = 32 / kPieces;  // pieces of a row; rows that a warp copies at once
        const int i = lane % kPieces;
#pragma unroll
        for (int r0 = 0; r0 < 16; r0 += kRows) {
          const int r = r0 + lane / kPieces;
          const uint32_t x = C::piece(r, i);
          copy16(to + x, c.k_pages + at + r * D + 16 * i, true);
          // (codes behind the last key may be NaN, and 0 times that would be)
          copy16(to + C::kHalf + x, c.v_pages + at + r * D + 16 * i, key + r < end);
        }
        if (lane < 2) copy4(to + 2 * C::kHalf + 4 * lane, (lane ? c.v_scale : c.k_scale) + ph);
      }
      copies_commit();
      return there;
    };
    // the first steps' copies, before anything else
    constexpr int kAhead = C::kStages - 1;
    int key = b0 * kBlockKeys + 16 * warp;
    uint32_t there = 0;  // by stage
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      there |= fetch(i, key + i * kBlockKeys, page_of(key + i * kBlockKeys)) ? 1u << i : 0u;
    int page = page_of(key + kAhead * kBlockKeys);

    // ---- the queries: lane 4 g + c has elements 16 c on of rows g (+ 8) for
    // the scores; of the sums it has rows 2 c and 2 c + 1
    uint32_t qf[NT][KS][2];
    float rf[NT][2];   // what turns a row's product into log2 scores, without k's scale
    int lim[NT][2];    // keys that a row sees
    int least = 0x7FFFFFFF;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const bool mine = 8 * t + g < live;
      const int64_t r = mine ? row0 + 8 * t + g : 0;
      const int token = static_cast<int>(r / p.G), head = h * p.G + static_cast<int>(r % p.G);
      uint4 x[D / 64][2];
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[i][j] = make_uint4(0u, 0u, 0u, 0u);
          if (mine && in_bounds(&g_cache_violations, w.a + token, 1, c.n_rows))
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
      // the largest element to between 2^14 and 2^15, near f16's end: elements down to
      // 2^-31 of it are exact
      const int e2 = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112), 127) - 14;
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23) * p.scale_log2;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const uint4& y = x[j / 4][(j % 4) / 2];
        const uint32_t e0 = j % 2 ? y.z : y.x, e1 = j % 2 ? y.w : y.y;
        qf[t][j][0] = pack_f16x2(__uint_as_float(e0 << 16) * down, __uint_as_float(e0 & 0xFFFF0000u) * down);
        qf[t][j][1] = pack_f16x2(__uint_as_float(e1 << 16) * down, __uint_as_float(e1 & 0xFFFF0000u) * down);
      }
      // (a row past the sequence's sees what it likes)
      const int my_lim = mine ? sees(token) : 0x7FFFFFFF;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        rf[t][i] = __shfl_sync(0xffffffffu, up, (2 * cc + i) * 4);
        lim[t][i] = __shfl_sync(0xffffffffu, my_lim, (2 * cc + i) * 4);
      }
      least = min(least, __reduce_min_sync(0xffffffffu, my_lim));
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

    auto work = [&](uint32_t st, int key) {
      float sc[NT][4] = {};
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const uint4 x = ld_shared_v4(st + C::piece(g, 4 * j + cc)), y = ld_shared_v4(st + C::piece(g + 8, 4 * j + cc));
        const uint32_t u[4] = {x.x, x.y, x.z, x.w}, z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = f16x2_of_e4m3(static_cast<uint16_t>(u[i])), a2 = f16x2_of_e4m3(static_cast<uint16_t>(u[i] >> 16));
          const uint32_t a1 = f16x2_of_e4m3(static_cast<uint16_t>(z[i])), a3 = f16x2_of_e4m3(static_cast<uint16_t>(z[i] >> 16));
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16(sc[t], a0, a1, a2, a3, qf[t][4 * j + i][0], qf[t][4 * j + i][1]);
        }
      }
      const float ks = ld_shared_f32(st + 2 * C::kHalf), lv = lg2_approx(ld_shared_f32(st + 2 * C::kHalf + 4));
      const float lr = lv - kRoom;  // from a score to the reference that it asks for
      uint32_t pb[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float f0 = rf[t][0] * ks, f1 = rf[t][1] * ks;
        float x[4] = {sc[t][0] * f0, sc[t][1] * f1, sc[t][2] * f0, sc[t][3] * f1};  // keys g, g, g + 8, g + 8
        if (key + 16 > least) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key + g + 8 * (i >> 1) >= lim[t][i & 1]) x[i] = -INFINITY;
        }
        const float t0 = fmaxf(x[0], x[2]), t1 = fmaxf(x[1], x[3]);
        if (__any_sync(0xffffffffu, t0 > m[t][0] + 8.f || t1 > m[t][1] + 8.f || t0 + lr > M[t][0] + 8.f ||
                                        t1 + lr > M[t][1] + 8.f)) {
          float r[2] = {t0, t1};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) r[i] = fmaxf(r[i], __shfl_xor_sync(0xffffffffu, r[i], d));
            if (r[i] > m[t][i]) {
              l[t][i] *= ex2_approx(m[t][i] - r[i]);
              m[t][i] = r[i];
            }
            if (r[i] + lr > M[t][i]) {
              const float f = ex2_approx(M[t][i] - (r[i] + lr));
              M[t][i] = r[i] + lr;
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
      uint32_t v[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 2 * cc + (i & 1) + 8 * (i >> 1);
        if constexpr (D == 128) {
          const uint4 x = ld_shared_v4(st + C::kHalf + C::piece(row, g));
          v[i][0] = x.x;
          v[i][1] = x.y;
          v[i][2] = x.z;
          v[i][3] = x.w;
        } else {
          const uint2 x = ld_shared_v2(st + C::kHalf + C::piece(row, g >> 1) + 8 * (g & 1));
          v[i][0] = x.x;
          v[i][1] = x.y;
        }
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        // four elements of a lane's piece: two of the products' tiles
        const uint32_t a01 = __byte_perm(v[0][q], v[1][q], 0x5140), a23 = __byte_perm(v[0][q], v[1][q], 0x7362);
        const uint32_t b01 = __byte_perm(v[2][q], v[3][q], 0x5140), b23 = __byte_perm(v[2][q], v[3][q], 0x7362);
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

    // ---- steps of this warp: copies of the next stages under way
    {
      int stage = 0, to = kAhead;
      for (; key < end; key += kBlockKeys) {
        copies_wait<kAhead - 1>();
        __syncwarp();
        // (the stage that is filled now was read in the step before)
        const int next = page_of(key + (kAhead + 1) * kBlockKeys);
        there = (there & ~(1u << to)) | (fetch(to, key + kAhead * kBlockKeys, page) ? 1u << to : 0u);
        page = next;
        if ((there >> stage) & 1u) work(ring + stage * C::kStageBytes, key);
        __syncwarp();
        stage = stage + 1 == C::kStages ? 0 : stage + 1;
        to = to + 1 == C::kStages ? 0 : to + 1;
      }
      copies_wait<0>();
    }
    __syncthreads();  // the sums take the ring's place

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
    float* const slot = p.sums + static_cast<int64_t>(blockIdx.x) * RT * (D + 4);
    for (int i = tid; i < live * (D / 4); i += 128) {
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
      if (parts == 1) {
        store_row<D>(p, row_place(p, w.a, h, static_cast<int64_t>(tile) * RT + r), d, sum, Mx, mx, ls);
      } else {
        *reinterpret_cast<float4*>(slot + r * (D + 4) + d) = sum;
        if (d == 0) *reinterpret_cast<float4*>(slot + r * (D + 4) + D) = make_float4(Mx, mx, ls, 0.f);
      }
    }
  }
}

// The sums of a row's parts [k0, k1), at most 32 of them, by a warp: O against the
// largest M in four elements a lane (D / 4 lanes), l against the largest m in
// every lane.  A lane looks after a part's references; the parts' sums come eight
// at a time.
struct RowSum {
  float4 o;
  float M, m, l;
};
template <int D>
__device__ __forceinline__ RowSum sum_parts(const float* first, int64_t step, int k0, int k1, int lane) {
  float4 h = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
  if (k0 + lane < k1) h = *reinterpret_cast<const float4*>(first + (k0 + lane) * step + D);
  RowSum r = {make_float4(0.f, 0.f, 0.f, 0.f), h.x, h.y, 0.f};
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    r.M = fmaxf(r.M, __shfl_xor_sync(0xffffffffu, r.M, d));
    r.m = fmaxf(r.m, __shfl_xor_sync(0xffffffffu, r.m, d));
  }
  // (a part without a key has references of -inf and sums of 0)
  const float f = h.x == -INFINITY ? 0.f : ex2_approx(h.x - r.M);
  r.l = h.y == -INFINITY ? h.z : h.z * ex2_approx(h.y - r.m);
#pragma unroll
  for (int d = 16; d; d >>= 1) r.l += __shfl_xor_sync(0xffffffffu, r.l, d);
  for (int k = k0; k < k1; k += 8) {
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = *reinterpret_cast<const float4*>(first + min(k + i, k1 - 1) * step + 4 * (lane % (D / 4)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (k + i >= k1) continue;
      const float g = __shfl_sync(0xffffffffu, f, k + i - k0);
      r.o.x += g * x[i].x;
      r.o.y += g * x[i].y;
      r.o.z += g * x[i].z;
      r.o.w += g * x[i].w;
    }
  }
  return r;
}

// The rows of units in several parts: a CTA for each part, which takes the rows
// idx, idx + parts, ... of the unit: a warp a row, or, of more than 16 parts (then
// there is one row at most), all warps one row.
template <int D, int NT, int W>
__global__ void __launch_bounds__(32 * W) combine_kernel(const __grid_constant__ CachedParams p) {
  constexpr int kStep = 8 * NT * (D + 4);
  __shared__ float4 sums[W][D / 4];
  __shared__ float4 ref[W];
  static_assert(8 * NT <= 16 && max_unit_parts(W / 8) == 32 * W, "rows of a CTA, parts of a warp");
  wait_for_previous_launch();
  const CachedPart note = p.parts[blockIdx.x];
  if (note.n <= 1 || note.idx >= note.live) return;
  const int64_t left = static_cast<int64_t>(note.n - 1 - note.idx) * note.stride;  // parts behind this one's
  if (!in_bounds(&g_cache_violations, blockIdx.x, left + 1, gridDim.x)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(note.stride) * kStep;  // from a part to the next
  const float* const first = p.sums + blockIdx.x * static_cast<int64_t>(kStep) - note.idx * step;
  auto store = [&](int r, const RowSum& x) {
    // (row r of the unit is r places on in the tokens' order of heads)
    const int64_t u = note.row0 + r;
    if (lane < D / 4)
      store_row<D>(p, note.place + (u / p.G - note.row0 / p.G) * p.Hq + (u % p.G - note.row0 % p.G), 4 * lane, x.o, x.M,
                   x.m, x.l);
  };
  if (note.n <= 16) {
    for (int r = note.idx + warp * note.n; r < note.live; r += W * note.n)
      store(r, sum_parts<D>(first + r * (D + 4), step, 0, note.n, lane));
    return;
  }
  const int per = (note.n + W - 1) / W, k0 = min(warp * per, note.n);
  const RowSum mine = sum_parts<D>(first + note.idx * (D + 4), step, k0, min(k0 + per, note.n), lane);
  if (lane < D / 4) sums[warp][lane] = mine.o;
  if (lane == 0) ref[warp] = make_float4(mine.M, mine.m, mine.l, 0.f);
  __syncthreads();
  if (warp) return;
  RowSum all = {make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, -INFINITY, 0.f};
#pragma unroll
  for (int k = 0; k < W; ++k) {
    all.M = fmaxf(all.M, ref[k].x);
    all.m = fmaxf(all.m, ref[k].y);
  }
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const float4 x = sums[k][lane % (D / 4)];
    const float f = ref[k].x == -INFINITY ? 0.f : ex2_approx(ref[k].x - all.M);
    all.o.x += f * x.x;
    all.o.y += f * x.y;
    all.o.z += f * x.z;
    all.o.w += f * x.w;
    all.l += ref[k].y == -INFINITY ? ref[k].z : ref[k].z * ex2_approx(ref[k].y - all.m);
  }
  store(note.idx, all);
}

template <int D, int NT>
cudaError_t launch_cached(const CachedParams& p, cudaStream_t s) {
  using C = CachedCfg<D, NT>;
  cudaError_t e = cudaSuccess;
  // (each launch may come up while the one before it ends)
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (p.c.n_seqs > 128) {
    parts_kernel<D, 8 * NT><<<1, 128, 0, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(p.grid);
  cfg.dynamicSmemBytes = C::kSmem;
  e = cudaLaunchKernelEx(&cfg, cached_kernel<D, NT>, p);
  if (e != cudaSuccess || p.whole) return e;
  cfg.dynamicSmemBytes = 0;
  cfg.blockDim = dim3(max_unit_parts(p.few));
  return p.few == 2   ? cudaLaunchKernelEx(&cfg, combine_kernel<D, NT, 16>, p)
         : p.few == 1 ? cudaLaunchKernelEx(&cfg, combine_kernel<D, NT, 8>, p)
                      : cudaLaunchKernelEx(&cfg, combine_kernel<D, NT, 4>, p);
}

}  // namespace

cudaError_t launch_cache_attention(const CachedParams& p, int D, cudaStream_t s) {
  if (D == 128) return p.row_tiles == 1 ? launch_cached<128, 1>(p, s) : launch_cached<128, 2>(p, s);
  return p.row_tiles == 1 ? launch_cached<64, 1>(p, s) : launch_cached<64, 2>(p, s);
}

}  // namespace uly
