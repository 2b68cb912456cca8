// attn_bwd.cu -- the gradient of the attention in attn.cu for sm_103a
// (tcgen05 + TMEM + TMA), the probabilities recomputed from the log-sum-exp.
//
// Mathematics, per batch and q head (kv head h / G), over admitted (query n,
// key m) pairs:
//   P_nm  = exp(scale q_n.k_m - lse_n)          delta_n = o_n . do_n
//   dP    = dO V^T                              dS = P o (dP - delta)
//   dV_m  = sum_n P_nm do_n      dK_m = scale sum_n dS_nm q_n
//   dQ_n  = scale sum_m dS_nm k_m
// dK and dV also sum over the G query heads of a kv head.
//
// Two main kernels, each with its sums in TMEM from first to last term, so
// that no sum passes through memory and none depends on the order in which
// CTAs run (the results are the same bits on every call):
//   dkdv_kernel  one CTA per (batch, kv head, 128 keys), over every query
//                head of the group and every 128-query tile: four products a
//                tile pair (S, dP, dV, dK);
//   dq_kernel    one CTA per (batch, q head, 128 queries), over every 128-key
//                tile with an admitted key: three products (S, dP, dQ).
// One kernel with five products would have to add dQ through f32 atomics in
// memory, whose order changes the bits; the price of the two is 7/5 of the
// tensor work.
//
// Rounding: P, dS and (replicated rows of the fused call) the sum of the
// shards' do are rounded to bf16, since they are operands of bf16 MMAs; dS is
// formed from the f32 P, every sum is f32, the outputs are rounded once.
//
// Every mbarrier wait is bounded, as in attn.cu.
#include <atomic>

#include "internal.cuh"
#include "tc.cuh"

namespace uly {

__device__ unsigned long long g_bwd_violations;

uint64_t bwd_violations(bool reset) {
  if (!kChecked) return 0;
  unsigned long long v = 0;
  if (cudaMemcpyFromSymbol(&v, g_bwd_violations, sizeof v) != cudaSuccess) return ~0ull;
  if (reset) {
    const unsigned long long z = 0;
    if (cudaMemcpyToSymbol(g_bwd_violations, &z, sizeof z) != cudaSuccess) return ~0ull;
  }
  return v;
}

namespace {

template <int D>
struct BCfg {
  static constexpr int kPanels = D / 64;                   // 128-byte swizzle panels of a row
  static constexpr int kPanelBytes = kTileRows * 128;      // 16 KB
  static constexpr int kTileBytes = kPanels * kPanelBytes; // one 128-row tile
  static constexpr int kDSteps = D / 16;                   // MMAs of a product over D
  static constexpr int kRowSteps = kTileRows / 16;         // MMAs of a product over 128 rows
  static constexpr uint32_t kIdescS = make_idesc(1u, 128, 128, 0, 0);
  static constexpr uint32_t kIdescO = make_idesc(1u, 128, D, 0, 1);
  // dkdv_kernel: K, V and two stages of (Q, dO, row statistics)
  static constexpr int kStatBytes = 3 * kTileRows * 4;     // -lse (admitted keys, masked keys), -delta
  static constexpr int kStages = 2;
  static constexpr int kSmemKv = 1024 + (2 + 2 * kStages) * kTileBytes + kStages * kStatBytes;
  // dq_kernel: Q, dO, three K and two V slots
  static constexpr int kKSlots = 3, kVSlots = 2;
  static constexpr int kSmemQ = 1024 + (2 + kKSlots + kVSlots) * kTileBytes;
};
constexpr int kBwdThreads = 320;  // 8 warps of elementwise work, a TMA warp, an MMA warp

__device__ __forceinline__ void bwd_timeout(const BwdParams& p, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(p.status, kStatusTimeout);
}

__device__ __forceinline__ uint32_t bits_word(const uint4 b, int w) {
  return w == 0 ? b.x : w == 1 ? b.y : w == 2 ? b.z : b.w;
}
__device__ __forceinline__ bool bits_full(const uint4 b) { return (b.x & b.y & b.z & b.w) == 0xFFFFFFFFu; }

__device__ __forceinline__ void ld_shared_2b64(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// run of tile t (runs in order, `first` = first tile)
__device__ __forceinline__ int seg_of(const Seg* segs, int n, int t) {
  int s = 0;
  while (s + 1 < n && t >= segs[s + 1].first) ++s;
  return s;
}

// 128 rows x D of one head to shared memory (128-byte swizzle panels)
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* m, uint32_t bar, int head, int row, int b) {
#pragma unroll
  for (int pn = 0; pn < BCfg<D>::kPanels; ++pn)
    tma_load_4d(dst + pn * BCfg<D>::kPanelBytes, m, bar, pn * 64, head, row, b);
}

// Shared-memory descriptors (128-byte swizzle; tc.cuh): the upper word is the
// same for every operand here, the lower one is the start address / 16 and the
// leading byte offset.  One thread issues every MMA, and what it does between
// two of them delays the tensor core, so the lower words are a base and a
// constant.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_rows(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_cols(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | ((static_cast<uint32_t>(kTileRows) * 128u >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(alo), "r"(blo), "r"(idesc), "r"(acc), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(blo), "r"(idesc), "r"(acc), "r"(kDescHi)
      : "memory");
}

// D[tmem] = A B^T of two 128-row tiles in shared memory, both K-major (the
// sum runs over D); alo, blo from desc_rows
template <int D>
__device__ __forceinline__ void issue_rows(uint32_t d, uint32_t alo, uint32_t blo) {
  using C = BCfg<D>;
#pragma unroll
  for (int k = 0; k < C::kDSteps; ++k) {
    constexpr uint32_t kPanel = C::kPanelBytes >> 4;
    const uint32_t off = (k >> 2) * kPanel + (k & 3) * 2;
    mma_ss(d, alo + off, blo + off, C::kIdescS, k > 0);
  }
}

// D[tmem] (+)= A B with A a 128 x 128 bf16 matrix in TMEM (entries 0..63 of a
// row in the columns [a, a + 32), 64..127 in [a + 64, a + 96)) and B a
// 128-row tile in shared memory (MN-major; the sum runs over the rows); blo
// from desc_cols
template <int D>
__device__ __forceinline__ void issue_cols(uint32_t d, uint32_t a, uint32_t blo, bool acc) {
  using C = BCfg<D>;
#pragma unroll
  for (int k = 0; k < C::kRowSteps; ++k)
    mma_ts(d, a + 64 * (k >> 2) + 8 * (k & 3), blo + k * 128, C::kIdescO, acc || k > 0);
}

// Zero the rows of a 128-row tile whose bit in `live` is clear (one warp's
// share: rows [row0, row0 + 16)).
template <int D>
__device__ __forceinline__ void zero_dead_rows(uint32_t tile, const uint4 live, int row0, int lane) {
  const uint32_t w = bits_word(live, row0 >> 5) >> (row0 & 31);
  for (int r = 0; r < 16; ++r) {
    if ((w >> r) & 1u) continue;
    if (lane < 8 * BCfg<D>::kPanels)
      st_shared_v4(tile + (lane >> 3) * BCfg<D>::kPanelBytes + (row0 + r) * 128 + (lane & 7) * 16, 0u, 0u, 0u, 0u);
  }
}

// A 128 x D f32 accumulator in TMEM -> bf16 rows in the shared-memory buffer
// `stage` (2D bytes a row, 16-byte chunk c of row r at chunk c ^ (r mod
// chunks)); the thread's row, columns [c_lo, c_hi).
template <int D>
__device__ __forceinline__ void stage_rows(uint32_t t, float mul, uint32_t stage, int row, int c_lo, int c_hi, bool zero) {
  constexpr int kChunks = 2 * D / 16;
  const uint32_t my_row = stage + row * 2 * D;
  const uint32_t sw = row & (kChunks - 1);
  for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
    uint32_t o[32];
    if (!zero) {
      tmem_ld32(t + c0, o);
      tmem_wait_ld();
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 8 * k + 2 * e;
        v[e] = zero ? 0u : pack_bf16x2(__uint_as_float(o[c]) * mul, __uint_as_float(o[c + 1]) * mul);
      }
      st_shared_v4(my_row + ((static_cast<uint32_t>(c0 / 8 + k) ^ sw) << 4), v[0], v[1], v[2], v[3]);
    }
  }
}

// One warp's 32 staged rows (tile rows [32 q4, 32 q4 + 32), those below
// n_rows) of one head to the output tensors, 16-byte chunks [ch_lo, ch_lo +
// CH) of each; `run` says where they go.  A replicated run of the fused path
// goes to the owning rank's shard, and the other shards' copies, which the
// forward did not read for this head, get zero.
template <int D, int CH>
__device__ __forceinline__ void store_rows(const BwdParams& p, uint8_t* const* out, const int64_t* batch_stride,
                                           int64_t row_stride, const Seg& run, int row0, int n_rows, int head,
                                           int owner, int b, uint32_t stage, int q4, int ch_lo, int lane) {
  constexpr int kChunks = 2 * D / 16;
  constexpr int kPer = 32 / CH;  // rows stored at once
  const bool all = p.fused && run.out_shard < 0;
  const int lo = all ? 0 : (p.fused ? run.out_shard : owner), hi = all ? p.P : lo + 1;
  const int ch = ch_lo + lane % CH;
  if (!in_bounds(&g_bwd_violations, static_cast<int64_t>(head) * D * 2, D * 2, row_stride)) return;
  for (int sh = lo; sh < hi; ++sh) {
    const int base_row = (run.out_row0 < 0 ? p.shard_len[sh] : run.out_row0) + row0;
    uint8_t* const base = out[sh] + static_cast<int64_t>(b) * batch_stride[sh] + static_cast<int64_t>(head) * D * 2 + ch * 16;
    const bool zero = all && sh != owner;
#pragma unroll 4
    for (int k = 0; k < 32; k += kPer) {
      const int i = 32 * q4 + k + lane / CH;
      const int64_t off = static_cast<int64_t>(base_row + i) * row_stride;
      if (i >= n_rows || !in_bounds(&g_bwd_violations, off, row_stride, batch_stride[sh])) continue;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (!zero)
        v = ld_shared_v4(stage + i * 2 * D + ((static_cast<uint32_t>(ch) ^ static_cast<uint32_t>(i & (kChunks - 1))) << 4));
      *reinterpret_cast<uint4*>(base + off) = v;
    }
  }
}

// ----------------------------------------------------- row statistics --
// Per (batch, q head, 128-row tile of a run): -lse log2(e) and -delta, padded
// to whole tiles, which the main kernels read in tiles.  A row that takes
// part in nothing (past its run's end, no admitted key, or zero by the
// masked-row convention) has -inf, whose exponential is 0.  ULY_ROWS_SELF: the
// first array holds it for the admitted keys (rows that are admitted keys
// themselves), the second for the masked keys.  Fused, replicated rows: do is
// the sum of every shard's copy, since each received the output; the sum is
// rounded to bf16 into do_rep (the MMA's operand) and delta uses that value.
// Bound by memory: o and do are read once.  32 rows x 8 heads a CTA; 16 (D =
// 128) or 8 lanes share a row, the results go through shared memory so that
// they are written along rows.
template <int D>
__global__ void __launch_bounds__(256) stats_kernel(const __grid_constant__ BwdParams p) {
  constexpr int kLanes = D / 8, kUnits = 256 / kLanes, kRows = 32, kHeads = 8;
  __shared__ float s_dl[kHeads][kRows + 1];
  const int t = blockIdx.x / (kTileRows / kRows), r_lo = (blockIdx.x % (kTileRows / kRows)) * kRows;
  const int h0 = blockIdx.y * kHeads, b = blockIdx.z;
  const int s = seg_of(p.qseg, p.n_qseg, t);
  const Seg run = p.qseg[s];
  const int row0 = (t - run.first) * kTileRows + r_lo;  // first row inside the run
  const int lane = threadIdx.x % kLanes, unit = threadIdx.x / kLanes;
  const bool rep = p.fused && run.out_shard < 0;
#pragma unroll 4
  for (int i = unit; i < kRows * kHeads; i += kUnits) {
    const int r = i / kHeads, hh = i % kHeads, h = h0 + hh;
    float sum = 0.f;
    if (h < p.Hq && row0 + r < run.len) {
      const int owner = h / p.Hq_l;
      const int sh = p.fused ? (rep ? owner : run.out_shard) : owner;
      const int64_t col = (static_cast<int64_t>(p.fused ? h : h % p.Hq_l) * D + lane * 8) * 2;
      const int64_t row = (run.out_row0 < 0 ? p.shard_len[sh] : run.out_row0) + row0 + r;
      if (in_bounds(&g_bwd_violations, row * p.q_row_stride, p.q_row_stride, p.q_batch_stride[sh])) {
        const uint4 ov = *reinterpret_cast<const uint4*>(p.o[sh] + b * p.q_batch_stride[sh] + row * p.q_row_stride + col);
        uint4 dv;
        if (!rep) {
          dv = *reinterpret_cast<const uint4*>(p.dout[sh] + b * p.q_batch_stride[sh] + row * p.q_row_stride + col);
        } else {
          float acc[8] = {};
          for (int q = 0; q < p.P; ++q) {
            const int64_t rq = (run.out_row0 < 0 ? p.shard_len[q] : run.out_row0) + row0 + r;
            const uint4 x = *reinterpret_cast<const uint4*>(p.dout[q] + b * p.q_batch_stride[q] + rq * p.q_row_stride + col);
            const uint32_t* xw = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              acc[2 * k] += __uint_as_float(xw[k] << 16);
              acc[2 * k + 1] += __uint_as_float(xw[k] & 0xFFFF0000u);
            }
          }
          dv = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                          pack_bf16x2(acc[6], acc[7]));
          *reinterpret_cast<uint4*>(p.do_rep + ((static_cast<int64_t>(b) * run.len + row0 + r) * p.Hq + h) * D * 2 +
                                    lane * 16) = dv;
        }
        const uint32_t *ow = reinterpret_cast<const uint32_t*>(&ov), *dw = reinterpret_cast<const uint32_t*>(&dv);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sum = fmaf(__uint_as_float(ow[k] << 16), __uint_as_float(dw[k] << 16), sum);
          sum = fmaf(__uint_as_float(ow[k] & 0xFFFF0000u), __uint_as_float(dw[k] & 0xFFFF0000u), sum);
        }
      }
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_dl[hh][r] = sum;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kHeads; i += 256) {
    const int hh = i / kRows, r = i % kRows, h = h0 + hh;
    if (h >= p.Hq) continue;
    const int64_t at = ((static_cast<int64_t>(b) * p.Hq + h) * p.n_q_tiles + t) * kTileRows + r_lo + r;
    float nl = -INFINITY, nl2 = -INFINITY, dl = 0.f;
    const int lrow = row0 + r;
    if (lrow < run.len) {
      const int owner = h / p.Hq_l;
      const int sh = p.fused ? (rep ? owner : run.out_shard) : owner;
      const int64_t row = (run.out_row0 < 0 ? p.shard_len[sh] : run.out_row0) + lrow;
      const int64_t li = row * p.lse_row_stride + (p.fused ? h : h % p.Hq_l);
      float lse = -INFINITY;
      if (in_bounds(&g_bwd_violations, li, 1, p.lse_batch_stride[sh])) lse = p.lse[sh][b * p.lse_batch_stride[sh] + li];
      bool own_ok = true;
      if (p.masked_rows != ULY_ROWS_SDPA && run.kv_seg >= 0) {
        const Seg& ks = p.kseg[run.kv_seg];
        const int c = lrow % kTileRows;
        const uint4 kb = p.tile_bits[static_cast<int64_t>(b) * p.n_kv_tiles + ks.first + lrow / kTileRows];
        own_ok = (bits_word(kb, c >> 5) >> (c & 31)) & 1u;
      }
      const bool live = lse != -INFINITY && (own_ok || p.masked_rows != ULY_ROWS_ZERO);
      if (live) {
        const float v = -lse * 1.4426950408889634f;
        if (p.masked_rows != ULY_ROWS_SELF)
          nl = v;
        else if (own_ok)
          nl = v;
        else
          nl2 = v;
        dl = -s_dl[hh][r];
      }
    }
    p.nl[at] = nl;
    if (p.masked_rows == ULY_ROWS_SELF) p.nl[p.stat_stride + at] = nl2;
    p.dl[at] = dl;
  }
}

// The 64 entries of a thread's half row, two to a register pair.
//
// p = 2^(s sl2 + nl) from the scores at TMEM t, kept in f32 in pr.  NL: the
// addend is a row's (nl2) or, in shared memory at nl_addr, one per column.
// MASKED: entries whose bit in w0 (columns 0..31) or w1 (32..63) is clear are
// 0 whatever the score is.  The masked form is a path of its own, taken by
// whole warps: a test in the unmasked loop would cut it into pieces that the
// compiler cannot interleave.
template <bool COLS, bool MASKED>
__device__ __forceinline__ void half_row_p(uint32_t t, uint64_t mul, uint64_t nl2, uint32_t nl_addr, uint32_t w0,
                                           uint32_t w1, uint64_t (&pr)[32]) {
  uint32_t a[2][32];
  tmem_ld32(t, a[0]);
  tmem_ld32(t + 32, a[1]);
  tmem_wait_ld();
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    uint64_t n[2] = {nl2, nl2};
    if (COLS) ld_shared_2b64(nl_addr + 16 * k, n[0], n[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * k + e;  // pair: entries 2i, 2i + 1
      float x0, x1;
      f2_split(f2_fma(f2(__uint_as_float(a[i >> 4][(2 * i) & 31]), __uint_as_float(a[i >> 4][(2 * i + 1) & 31])), mul,
                      n[e]),
               x0, x1);
      x0 = ex2_approx(x0);
      x1 = ex2_approx(x1);
      if (MASKED) {
        const uint32_t w = (i < 16 ? w0 : w1) >> ((2 * i) & 31);
        x0 = w & 1u ? x0 : 0.f;
        x1 = w & 2u ? x1 : 0.f;
      }
      pr[i] = f2(x0, x1);
    }
  }
}

// ds = p (dp + ndl), rounded to bf16, from dP at TMEM t; ndl as nl above.
// `loaded` is called once dP is in registers.
template <bool COLS, bool MASKED, typename F>
__device__ __forceinline__ void half_row_ds(uint32_t t, uint64_t dl2, uint32_t dl_addr, uint32_t w0, uint32_t w1,
                                            const uint64_t (&pr)[32], uint32_t (&pk)[32], F loaded) {
  uint32_t a[2][32];
  tmem_ld32(t, a[0]);
  tmem_ld32(t + 32, a[1]);
  tmem_wait_ld();
  loaded();
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    uint64_t n[2] = {dl2, dl2};
    if (COLS) ld_shared_2b64(dl_addr + 16 * k, n[0], n[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * k + e;
      float x0, x1;
      f2_split(f2_mul(f2_add(f2(__uint_as_float(a[i >> 4][(2 * i) & 31]), __uint_as_float(a[i >> 4][(2 * i + 1) & 31])),
                             n[e]),
                      pr[i]),
               x0, x1);
      if (MASKED) {
        const uint32_t w = (i < 16 ? w0 : w1) >> ((2 * i) & 31);
        x0 = w & 1u ? x0 : 0.f;
        x1 = w & 2u ? x1 : 0.f;
      }
      pk[i] = pack_bf16x2(x0, x1);
    }
  }
}

__device__ __forceinline__ void pack_half_row(const uint64_t (&pr)[32], uint32_t (&pk)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    float x0, x1;
    f2_split(pr[i], x0, x1);
    pk[i] = pack_bf16x2(x0, x1);
  }
}

struct KvBars {
  uint64_t kv_full;
  uint64_t q_full[2], do_full[2], free[2];
  uint64_t s_full, dp_full;   // S, dP of the tile in TMEM
  uint64_t p_full, ds_full;   // P, dS stored to TMEM (8 warps)
  uint64_t done, drain;
  uint32_t tmem_base;
  int abort_flag;
};

// dK and dV of 128 keys of one kv head.
//   warp 8   TMA: K and V once, then Q, dO and the row statistics of every
//            128-query tile of every query head of the group (two stages).
//   warp 9   MMA: S = K Q^T and dP = V dO^T (keys are TMEM lanes), dV += P dO
//            and dK += dS Q with P, dS read from TMEM, in the order
//              S(0) dP(0) | dV(i) S(i+1) dK(i) dP(i+1) ...
//            so that two products (~1024 tensor cycles) run while P(i+1) is
//            computed and two while dS(i+1) is.
//   warps 0-7: one thread per key and half of the queries: P from S, stored
//            over S's columns; dS from dP, stored over dP's.
// TMEM: S [0,128) dP [128,256) dV [256,256+D) dK [256+D,256+2D).
template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1) dkdv_kernel(const __grid_constant__ BwdParams p) {
  using C = BCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ KvBars bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
  const int r = hk / p.Hkv_l;  // owning rank
  const Seg run = p.kseg[seg_of(p.kseg, p.n_kseg, t)];
  const int row0 = (t - run.first) * kTileRows;
  const uint4 bits = p.tile_bits[static_cast<int64_t>(b) * p.n_kv_tiles + t];
  const bool self = p.masked_rows == ULY_ROWS_SELF;
  const bool any = self || (bits.x | bits.y | bits.z | bits.w) != 0u;
  const int n_it = any ? p.G * p.n_q_tiles : 0;

  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sK = sbase, sV = sbase + C::kTileBytes, sSt = sbase + 2 * C::kTileBytes;  // stage: Q, dO
  const uint32_t sStat = sSt + 2 * C::kStages * C::kTileBytes;
  volatile int* abort_flag = &bars.abort_flag;
  if (tid == 0) {
    mbar_init(smem_u32(&bars.kv_full), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.q_full[i]), 1);
      mbar_init(smem_u32(&bars.do_full[i]), 1);
      mbar_init(smem_u32(&bars.free[i]), 1);
    }
    mbar_init(smem_u32(&bars.s_full), 1);
    mbar_init(smem_u32(&bars.dp_full), 1);
    mbar_init(smem_u32(&bars.p_full), 8);
    mbar_init(smem_u32(&bars.ds_full), 8);
    mbar_init(smem_u32(&bars.done), 1);
    mbar_init(smem_u32(&bars.drain), 1);
    bars.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&bars.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const uint32_t tS = tmem, tDP = tmem + 128, tDV = tmem + 256, tDK = tmem + 256 + D;
  const uint64_t deadline = globaltimer_ns() + p.wait_ns;

  if (warp == 8) {
    if (lane == 0 && n_it > 0) {
      const int kvhead = p.fused ? hk : hk % p.Hkv_l;
      const int kmap = run.src < 0 ? r : run.src;
      const int krow = (run.row0 < 0 ? p.shard_len[kmap] : run.row0) + row0;
      const uint32_t bkv = smem_u32(&bars.kv_full);
      mbar_arrive_expect_tx(bkv, 2 * C::kTileBytes);
      load_tile<D>(sK, &p.tk[kmap], bkv, kvhead, krow, b);
      load_tile<D>(sV, &p.tv[kmap], bkv, kvhead, krow, b);
      const uint32_t stat = kTileRows * 4;
      int g = 0, qs = 0, qt = 0, it = 0;  // q head of the group, run, tile inside the run
      for (; it < n_it; ++it) {
        const int st = it & 1;
        if (it >= 2 && !mbar_wait(smem_u32(&bars.free[st]), ((it >> 1) - 1) & 1, deadline, abort_flag)) {
          bwd_timeout(p, abort_flag);
          break;
        }
        const int h = hk * p.G + g;
        const Seg& q = p.qseg[qs];
        const bool rep = p.fused && q.out_shard < 0;
        const int qmap = q.src < 0 ? r : q.src;
        const int qhead = p.fused ? h : h % p.Hq_l;
        const int qrow = (q.row0 < 0 ? p.shard_len[qmap] : q.row0) + qt * kTileRows;
        const uint32_t bq = smem_u32(&bars.q_full[st]), bd = smem_u32(&bars.do_full[st]);
        const uint32_t sq = sSt + 2 * st * C::kTileBytes, sd = sq + C::kTileBytes, ss = sStat + st * C::kStatBytes;
        const int64_t at = ((static_cast<int64_t>(b) * p.Hq + h) * p.n_q_tiles + q.first + qt) * kTileRows;
        mbar_arrive_expect_tx(bq, C::kTileBytes + (self ? 2 : 1) * stat);
        if (it != p.withhold_fill) load_tile<D>(sq, &p.tq[qmap], bq, qhead, qrow, b);
        bulk_load(ss, p.nl + at, stat, bq);
        if (self) bulk_load(ss + stat, p.nl + p.stat_stride + at, stat, bq);
        mbar_arrive_expect_tx(bd, C::kTileBytes + stat);
        if (rep)
          load_tile<D>(sd, &p.tdo_rep, bd, h, qt * kTileRows, b);
        else
          load_tile<D>(sd, &p.tdo[qmap], bd, qhead, qrow, b);
        bulk_load(ss + 2 * stat, p.dl + at, stat, bd);
        if (++qt * kTileRows >= q.len) {
          qt = 0;
          if (++qs == p.n_qseg) {
            qs = 0;
            ++g;
          }
        }
      }
      if (*abort_flag) {
        // drain: no copy may land after the CTA has left (a withheld one
        // never completes and only costs the bound)
        const uint64_t dl2 = globaltimer_ns() + 100000000ull;
        volatile int never = 0;
        for (int f = (it > 2 ? it - 2 : 0); f < it; ++f) {
          mbar_wait(smem_u32(&bars.q_full[f & 1]), (f >> 1) & 1, dl2, &never);
          mbar_wait(smem_u32(&bars.do_full[f & 1]), (f >> 1) & 1, dl2, &never);
        }
        mbar_wait(smem_u32(&bars.kv_full), 0, dl2, &never);
      }
    }
  } else if (warp == 9) {
    if (lane == 0 && n_it > 0) {
      const uint32_t dk = desc_rows(sK), dv = desc_rows(sV);
      uint32_t q_r[2], q_c[2], o_r[2], o_c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q_r[i] = desc_rows(sSt + 2 * i * C::kTileBytes);
        q_c[i] = desc_cols(sSt + 2 * i * C::kTileBytes);
        o_r[i] = desc_rows(sSt + (2 * i + 1) * C::kTileBytes);
        o_c[i] = desc_cols(sSt + (2 * i + 1) * C::kTileBytes);
      }
      bool ok = mbar_wait(smem_u32(&bars.kv_full), 0, deadline, abort_flag) &&
                mbar_wait(smem_u32(&bars.q_full[0]), 0, deadline, abort_flag);
      tc_fence_after();
      if (ok) {
        issue_rows<D>(tS, dk, q_r[0]);
        mma_commit(smem_u32(&bars.s_full));
        ok = mbar_wait(smem_u32(&bars.do_full[0]), 0, deadline, abort_flag);
        tc_fence_after();
      }
      if (ok) {
        issue_rows<D>(tDP, dv, o_r[0]);
        mma_commit(smem_u32(&bars.dp_full));
      }
      for (int it0 = 0; ok && it0 < n_it; it0 += 2) {
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const int it = it0 + st, nx = st ^ 1;
          if (!ok || it >= n_it) break;
          const bool more = it + 1 < n_it;
          if (!(ok = mbar_wait(smem_u32(&bars.p_full), st, deadline, abort_flag))) break;
          tc_fence_after();
          issue_cols<D>(tDV, tS, o_c[st], it > 0);
          if (more) {
            if (!(ok = mbar_wait(smem_u32(&bars.q_full[nx]), ((it + 1) >> 1) & 1, deadline, abort_flag))) break;
            issue_rows<D>(tS, dk, q_r[nx]);
            mma_commit(smem_u32(&bars.s_full));
          }
          if (!(ok = mbar_wait(smem_u32(&bars.ds_full), st, deadline, abort_flag))) break;
          tc_fence_after();
          issue_cols<D>(tDK, tDP, q_c[st], it > 0);
          mma_commit(more ? smem_u32(&bars.free[st]) : smem_u32(&bars.done));
          if (more) {
            if (!(ok = mbar_wait(smem_u32(&bars.do_full[nx]), ((it + 1) >> 1) & 1, deadline, abort_flag))) break;
            issue_rows<D>(tDP, dv, o_r[nx]);
            mma_commit(smem_u32(&bars.dp_full));
          }
        }
      }
      if (!ok) bwd_timeout(p, abort_flag);
      mma_commit(smem_u32(&bars.drain));
      volatile int never = 0;
      if (!mbar_wait(smem_u32(&bars.drain), 0, globaltimer_ns() + p.wait_ns, &never)) bwd_timeout(p, abort_flag);
    }
  } else {
    const int wg = warp >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;  // key of the tile = TMEM lane
    const uint32_t off = (static_cast<uint32_t>(q4 * 32) << 16) + 64 * wg;
    const uint32_t mS = tS + off, mDP = tDP + off;
    const bool key_ok = (bits_word(bits, q4) >> lane) & 1u;
    const bool dead = row0 + row >= run.len || (!self && !key_ok);
    const bool any_dead = __any_sync(0xffffffffu, dead);
    const uint32_t stat = kTileRows * 4;
    const uint32_t nl_off = (self && !key_ok ? stat : 0u) + 64 * wg * 4;
    const uint64_t mul = f2(p.scale_log2, p.scale_log2);
    const bool zero_rows = p.masked_rows == ULY_ROWS_ZERO;
    bool ok = true;
    int qs = 0, qt = 0;
    for (int it = 0; it < n_it; ++it) {
      const int st = it & 1;
      const uint32_t ss = sStat + st * C::kStatBytes;
      uint4 live = make_uint4(~0u, ~0u, ~0u, ~0u);
      if (zero_rows) {
        // queries that take part in nothing may hold anything: their rows of
        // Q and dO are zeroed before the sums over queries read them
        const Seg& q = p.qseg[qs];
        live = q.kv_seg < 0 ? live
                            : p.tile_bits[static_cast<int64_t>(b) * p.n_kv_tiles + p.kseg[q.kv_seg].first + qt];
        if (++qt * kTileRows >= q.len) {
          qt = 0;
          if (++qs == p.n_qseg) qs = 0;
        }
      }
      const bool fix = !bits_full(live);
      ok = mbar_wait(smem_u32(&bars.q_full[st]), (it >> 1) & 1, deadline, abort_flag) &&
           mbar_wait(smem_u32(&bars.s_full), it & 1, deadline, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // entries that take part: every query, none for a dead key
      const uint32_t w0 = dead ? 0u : bits_word(live, 2 * wg), w1 = dead ? 0u : bits_word(live, 2 * wg + 1);
      uint64_t pr[32];
      uint32_t pk[32];
      if (!(any_dead || fix))
        half_row_p<true, false>(mS, mul, 0, ss + nl_off, w0, w1, pr);
      else
        half_row_p<true, true>(mS, mul, 0, ss + nl_off, w0, w1, pr);
      pack_half_row(pr, pk);
      tmem_st32(mS, pk);
      // (the stage's dO landed: its statistics are read below, and dead rows
      // are zeroed here)
      ok = mbar_wait(smem_u32(&bars.do_full[st]), (it >> 1) & 1, deadline, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const uint32_t sq = sSt + 2 * st * C::kTileBytes;
      if (fix) {
        zero_dead_rows<D>(sq, live, 16 * warp, lane);
        zero_dead_rows<D>(sq + C::kTileBytes, live, 16 * warp, lane);
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.p_full));
      ok = mbar_wait(smem_u32(&bars.dp_full), it & 1, deadline, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t dl_addr = ss + 2 * stat + 64 * wg * 4;
      if (!(any_dead || fix))
        half_row_ds<true, false>(mDP, 0, dl_addr, w0, w1, pr, pk, [] {});
      else
        half_row_ds<true, true>(mDP, 0, dl_addr, w0, w1, pr, pk, [] {});
      tmem_st32(mDP, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.ds_full));
    }
    if (ok && n_it > 0) {
      ok = mbar_wait(smem_u32(&bars.done), 0, deadline, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) ok = false;
      tc_fence_after();
    }
    if (!ok) {
      bwd_timeout(p, abort_flag);
    } else {
      // warps 0-3: dV, warps 4-7: dK; each warp stages and stores its 32 rows
      const uint32_t stage = sSt + wg * (2 * C::kTileBytes);
      stage_rows<D>((wg ? tDK : tDV) + (static_cast<uint32_t>(q4 * 32) << 16), wg ? p.scale : 1.f, stage, row, 0, D,
                    n_it == 0);
      __syncwarp();
      store_rows<D, 2 * D / 16>(p, wg ? p.dk : p.dv, p.kv_batch_stride, p.kv_row_stride, run, row0, run.len - row0,
                                p.fused ? hk : hk % p.Hkv_l, r, b, stage, q4, 0, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct QBars {
  uint64_t q_full;
  uint64_t k_full[3], k_free[3], v_full[2], v_free[2];
  uint64_t s_full[2], dp_full, dp_free, ds_full[2];
  uint64_t done, drain;
  uint32_t tmem_base;
  int abort_flag;
};

// dQ of 128 queries of one q head.
//   warp 8   TMA: Q and dO once, K (three slots) and V (two) of every kv tile
//            with an admitted key.
//   warp 9   MMA: S = Q K^T, dP = dO V^T (queries are TMEM lanes), dQ += dS K
//            with dS read from TMEM, in the order
//              S(0) dP(0) S(1) | dP(j+1) dQ(j) S(j+2) ...
//   warps 0-7: one thread per query and half of the keys: dS from S and dP,
//            stored over S's columns (two S buffers, so that the next tile's
//            scores are there when this one's are done).
// TMEM: S0 [0,128) S1 [128,256) dP [256,384) dQ [384,384+D).
template <int D>
__global__ void __launch_bounds__(kBwdThreads, 1) dq_kernel(const __grid_constant__ BwdParams p) {
  using C = BCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ QBars bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int r = h / p.Hq_l, hk = h / p.G;
  const Seg run = p.qseg[seg_of(p.qseg, p.n_qseg, t)];
  const int row0 = (t - run.first) * kTileRows;
  const int n_it = p.n_active[b];
  const int32_t* active = p.active + static_cast<int64_t>(b) * p.n_kv_tiles;

  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = sbase, sDO = sbase + C::kTileBytes, sK = sbase + 2 * C::kTileBytes;
  const uint32_t sV = sK + C::kKSlots * C::kTileBytes;
  volatile int* abort_flag = &bars.abort_flag;
  if (tid == 0) {
    mbar_init(smem_u32(&bars.q_full), 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(smem_u32(&bars.k_full[i]), 1);
      mbar_init(smem_u32(&bars.k_free[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.v_full[i]), 1);
      mbar_init(smem_u32(&bars.v_free[i]), 1);
      mbar_init(smem_u32(&bars.s_full[i]), 1);
      mbar_init(smem_u32(&bars.ds_full[i]), 8);
    }
    mbar_init(smem_u32(&bars.dp_full), 1);
    mbar_init(smem_u32(&bars.dp_free), 8);
    mbar_init(smem_u32(&bars.done), 1);
    mbar_init(smem_u32(&bars.drain), 1);
    bars.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&bars.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const uint32_t tDP = tmem + 256, tDQ = tmem + 384;
  const uint64_t deadline = globaltimer_ns() + p.wait_ns;

  if (warp == 8) {
    if (lane == 0 && n_it > 0) {
      const bool rep = p.fused && run.out_shard < 0;
      const int qmap = run.src < 0 ? r : run.src;
      const int qhead = p.fused ? h : h % p.Hq_l, kvhead = p.fused ? hk : hk % p.Hkv_l;
      const int qrow = (run.row0 < 0 ? p.shard_len[qmap] : run.row0) + row0;
      const uint32_t bq = smem_u32(&bars.q_full);
      mbar_arrive_expect_tx(bq, 2 * C::kTileBytes);
      load_tile<D>(sQ, &p.tq[qmap], bq, qhead, qrow, b);
      if (rep)
        load_tile<D>(sDO, &p.tdo_rep, bq, h, row0, b);
      else
        load_tile<D>(sDO, &p.tdo[qmap], bq, qhead, qrow, b);
      int nk = 0, nv = 0;  // K and V fills issued
      for (int it = 0; it < n_it; ++it) {
        const int e = active[it];
        const bool good = in_bounds(&g_bwd_violations, e >> 20, 1, p.n_kseg);
        const Seg& k = p.kseg[good ? e >> 20 : 0];
        const int kmap = k.src < 0 ? r : k.src;
        const int krow = (k.row0 < 0 ? p.shard_len[kmap] : k.row0) + (e & 0xFFFFF) * kTileRows;
        const int ks = it % C::kKSlots, vs = it % C::kVSlots;
        if (it >= C::kKSlots &&
            !mbar_wait(smem_u32(&bars.k_free[ks]), (it / C::kKSlots - 1) & 1, deadline, abort_flag)) {
          bwd_timeout(p, abort_flag);
          break;
        }
        const uint32_t bk = smem_u32(&bars.k_full[ks]);
        mbar_arrive_expect_tx(bk, C::kTileBytes);
        if (good && it != p.withhold_fill) load_tile<D>(sK + ks * C::kTileBytes, &p.tk[kmap], bk, kvhead, krow, b);
        ++nk;
        if (it >= C::kVSlots &&
            !mbar_wait(smem_u32(&bars.v_free[vs]), (it / C::kVSlots - 1) & 1, deadline, abort_flag)) {
          bwd_timeout(p, abort_flag);
          break;
        }
        const uint32_t bv = smem_u32(&bars.v_full[vs]);
        mbar_arrive_expect_tx(bv, C::kTileBytes);
        if (good) load_tile<D>(sV + vs * C::kTileBytes, &p.tv[kmap], bv, kvhead, krow, b);
        ++nv;
      }
      if (*abort_flag) {
        const uint64_t dl2 = globaltimer_ns() + 100000000ull;
        volatile int never = 0;
        for (int f = max(0, nk - C::kKSlots); f < nk; ++f)
          mbar_wait(smem_u32(&bars.k_full[f % C::kKSlots]), (f / C::kKSlots) & 1, dl2, &never);
        for (int f = max(0, nv - C::kVSlots); f < nv; ++f)
          mbar_wait(smem_u32(&bars.v_full[f % C::kVSlots]), (f / C::kVSlots) & 1, dl2, &never);
        mbar_wait(bq, 0, dl2, &never);
      }
    }
  } else if (warp == 9) {
    if (lane == 0 && n_it > 0) {
      const uint32_t dq = desc_rows(sQ), ddo = desc_rows(sDO);
      uint32_t k_r[C::kKSlots], k_c[C::kKSlots], v_r[C::kVSlots];
#pragma unroll
      for (int i = 0; i < C::kKSlots; ++i) {
        k_r[i] = desc_rows(sK + i * C::kTileBytes);
        k_c[i] = desc_cols(sK + i * C::kTileBytes);
      }
#pragma unroll
      for (int i = 0; i < C::kVSlots; ++i) v_r[i] = desc_rows(sV + i * C::kTileBytes);
      bool ok = mbar_wait(smem_u32(&bars.q_full), 0, deadline, abort_flag) &&
                mbar_wait(smem_u32(&bars.k_full[0]), 0, deadline, abort_flag);
      tc_fence_after();
      if (ok) {
        issue_rows<D>(tmem, dq, k_r[0]);
        mma_commit(smem_u32(&bars.s_full[0]));
        ok = mbar_wait(smem_u32(&bars.v_full[0]), 0, deadline, abort_flag);
      }
      if (ok) {
        issue_rows<D>(tDP, ddo, v_r[0]);
        mma_commit(smem_u32(&bars.dp_full));
        mma_commit(smem_u32(&bars.v_free[0]));
        if (n_it > 1) {
          ok = mbar_wait(smem_u32(&bars.k_full[1]), 0, deadline, abort_flag);
          if (ok) {
            issue_rows<D>(tmem + 128, dq, k_r[1]);
            mma_commit(smem_u32(&bars.s_full[1]));
          }
        }
      }
      // unrolled over a turn of both rings, so that every slot is a constant
      constexpr int kTurn = C::kKSlots * C::kVSlots;
      static_assert(kTurn % 2 == 0, "S buffers alternate");
      for (int it0 = 0; ok && it0 < n_it; it0 += kTurn) {
#pragma unroll
        for (int u = 0; u < kTurn; ++u) {
          const int it = it0 + u, buf = u & 1, ks = u % C::kKSlots, vs = (u + 1) % C::kVSlots,
                    ks2 = (u + 2) % C::kKSlots;
          if (!ok || it >= n_it) break;
          if (it + 1 < n_it) {
            if (!(ok = mbar_wait(smem_u32(&bars.dp_free), it & 1, deadline, abort_flag) &&
                       mbar_wait(smem_u32(&bars.v_full[vs]), ((it + 1) / C::kVSlots) & 1, deadline, abort_flag)))
              break;
            tc_fence_after();
            issue_rows<D>(tDP, ddo, v_r[vs]);
            mma_commit(smem_u32(&bars.dp_full));
            mma_commit(smem_u32(&bars.v_free[vs]));
          }
          if (!(ok = mbar_wait(smem_u32(&bars.ds_full[buf]), (it >> 1) & 1, deadline, abort_flag))) break;
          tc_fence_after();
          issue_cols<D>(tDQ, tmem + 128 * buf, k_c[ks], it > 0);
          mma_commit(it + 1 < n_it ? smem_u32(&bars.k_free[ks]) : smem_u32(&bars.done));
          if (it + 2 < n_it) {
            if (!(ok = mbar_wait(smem_u32(&bars.k_full[ks2]), ((it + 2) / C::kKSlots) & 1, deadline, abort_flag))) break;
            issue_rows<D>(tmem + 128 * buf, dq, k_r[ks2]);
            mma_commit(smem_u32(&bars.s_full[buf]));
          }
        }
      }
      if (!ok) bwd_timeout(p, abort_flag);
      mma_commit(smem_u32(&bars.drain));
      volatile int never = 0;
      if (!mbar_wait(smem_u32(&bars.drain), 0, globaltimer_ns() + p.wait_ns, &never)) bwd_timeout(p, abort_flag);
    }
  } else {
    const int wg = warp >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;  // query of the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t mDP = tDP + lane_off + 64 * wg;
    const bool self = p.masked_rows == ULY_ROWS_SELF;
    // a masked row under ULY_ROWS_SELF attends to the masked keys
    bool invert = false;
    if (self && run.kv_seg >= 0) {
      const uint4 qb = p.tile_bits[static_cast<int64_t>(b) * p.n_kv_tiles + p.kseg[run.kv_seg].first + row0 / kTileRows];
      invert = !((bits_word(qb, q4) >> lane) & 1u);
    }
    const int64_t at = ((static_cast<int64_t>(b) * p.Hq + h) * p.n_q_tiles + t) * kTileRows + row;
    const float nl = p.nl[(invert ? p.stat_stride : 0) + at], dl = p.dl[at];
    const bool dead = nl == -INFINITY;
    const bool any_dead = __any_sync(0xffffffffu, dead);
    const uint64_t mul = f2(p.scale_log2, p.scale_log2), nl2 = f2(nl, nl), dl2 = f2(dl, dl);
    const uint4* row_bits = (invert ? p.active_inv : p.active_bits) + static_cast<int64_t>(b) * p.n_kv_tiles;
    uint4 bits_next = n_it > 0 ? __ldg(row_bits) : make_uint4(0u, 0u, 0u, 0u);
    bool ok = true;
    int ks = 0;
    for (int it = 0; it < n_it; ++it) {
      const int buf = it & 1;
      const uint32_t mS = tmem + lane_off + 128 * buf + 64 * wg;
      const uint4 bits = bits_next;
      if (it + 1 < n_it) bits_next = __ldg(row_bits + it + 1);
      // some entry of the warp is not admitted
      const bool part = any_dead || __any_sync(0xffffffffu, !bits_full(bits));
      const uint32_t w0 = dead ? 0u : bits_word(bits, 2 * wg), w1 = dead ? 0u : bits_word(bits, 2 * wg + 1);
      ok = mbar_wait(smem_u32(&bars.s_full[buf]), (it >> 1) & 1, deadline, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint64_t pr[32];
      if (!part)
        half_row_p<false, false>(mS, mul, nl2, 0, w0, w1, pr);
      else
        half_row_p<false, true>(mS, mul, nl2, 0, w0, w1, pr);
      ok = mbar_wait(smem_u32(&bars.dp_full), it & 1, deadline, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t pk[32];
      // (dP is in registers: the next tile's may overwrite it)
      const auto loaded = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.dp_free));
      };
      if (!part)
        half_row_ds<false, false>(mDP, dl2, 0, w0, w1, pr, pk, loaded);
      else
        half_row_ds<false, true>(mDP, dl2, 0, w0, w1, pr, pk, loaded);
      tmem_st32(mS, pk);
      if (part && !self) {
        // keys that are not admitted may hold anything: their rows of K are
        // zeroed before the sum over keys reads them (S has read them)
        zero_dead_rows<D>(sK + ks * C::kTileBytes, __ldg(p.active_bits + static_cast<int64_t>(b) * p.n_kv_tiles + it),
                          16 * warp, lane);
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.ds_full[buf]));
      if (++ks == C::kKSlots) ks = 0;
    }
    if (ok && n_it > 0) {
      ok = mbar_wait(smem_u32(&bars.done), 0, deadline, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) ok = false;
      tc_fence_after();
    }
    if (!ok) {
      bwd_timeout(p, abort_flag);
    } else {
      // warps 0-3: the first half of the columns, warps 4-7 the second
      stage_rows<D>(tDQ + lane_off, p.scale, sQ, row, wg * (D / 2), (wg + 1) * (D / 2), n_it == 0);
      __syncwarp();
      store_rows<D, D / 16>(p, p.dq, p.q_batch_stride, p.q_row_stride, run, row0, run.len - row0,
                            p.fused ? h : h % p.Hq_l, r, b, sQ, q4, wg * (D / 16), lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The shared-memory limit of a kernel is set once on every device that
// launches it (setting it twice is harmless).
template <int D>
cudaError_t configure() {
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (bit && (configured.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  using C = BCfg<D>;
  if ((e = cudaFuncSetAttribute(dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemKv)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemQ)) != cudaSuccess)
    return e;
  configured.fetch_or(bit, std::memory_order_relaxed);
  return cudaSuccess;
}

template <int D>
cudaError_t launch(const BwdParams& p, cudaStream_t s) {
  using C = BCfg<D>;
  cudaError_t e = configure<D>();
  if (e != cudaSuccess) return e;
  stats_kernel<D><<<dim3(p.n_q_tiles * 4, (p.Hq + 7) / 8, p.B), 256, 0, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  dkdv_kernel<D><<<dim3(p.n_kv_tiles, p.Hkv, p.B), kBwdThreads, C::kSmemKv, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  dq_kernel<D><<<dim3(p.n_q_tiles, p.Hq, p.B), kBwdThreads, C::kSmemQ, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_backward(const BwdParams& p, int D, cudaStream_t s) {
  return D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace uly
