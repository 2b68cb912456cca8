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
// Two kinds of CTA in one launch, each with its sums in TMEM from first to last
// term, so that no sum passes through memory and none depends on the order in
// which CTAs run (the results are the same bits on every call):
//   dkdv_cta  one for a (batch, kv head, 128 keys), over every query head of the
//             group and every 128-query tile: four products a tile pair (S, dP,
//             dV, dK);
//   dq_cta    one for a (batch, q head, 128 queries), over every 128-key tile
//             with an admitted key: three products (S, dP, dQ).
// With five products in one, dQ would have to be added up in memory, by atomics
// whose order changes the bits or by CTAs in turn; the price of the two is 7/5
// of the tensor work.
//
// Bound by the tensor cores where loops are long and D is 128 (8 heads of 8192
// rows: 537 us, 1792 TFLOP/s of the seven products, 94% of 1912 measured with
// one large matrix product; larger calls run into the power limit: 40 heads of
// 27792 rows 31.4 ms, 1745 TFLOP/s, which is what a matrix product sustains).
// With 64-wide heads, or masks, by the elementwise work and the issue of MMAs:
// 406 us, 1185 TFLOP/s (tensor pipe active 49% of cycles, issue slots 39%).  Short loops, by what surrounds them: about 5.5 us a
// CTA, of which 2.5 pass before its first scores are there.
//
// Rounding: P and dS are rounded to bf16, since they are operands of bf16 MMAs;
// dS is formed from the f32 P, every sum is f32, the outputs are rounded once.
// Replicated rows of the fused call, whose do is the sum over the shards: that
// sum enters as two bf16 parts, the products being linear in do, so these
// rows' tiles are gone through twice.
//
// Every mbarrier wait is bounded, as in attn.cu.
#include <atomic>

#include "grad.cuh"
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
  // No static shared memory and no slack: the buffer starts on a 1024-byte
  // boundary (the kernel checks it), and at D = 128 it is all that a CTA can
  // have.
  // dK, dV: K, V, three Q and two dO slots with their row statistics, barriers
  static constexpr int kQSlots = 3, kOSlots = 2;
  // dK, dV: a tile's P has columns of TMEM to itself, which 64-wide heads leave
  // free, and is stored while dP is computed (8 heads of 8192 rows 413 -> 406
  // us, 12 on 4 of 2300 rows 69.8 -> 65.9); not where the queries' own tokens
  // mask (78.6 -> 81.9: it takes registers that the masks need)
  template <bool OWN>
  static constexpr bool kOwnP = D == 64 && !OWN;
  static constexpr int kStatBytes = kTileRows * 4;         // -lse log2(e) or -delta of a tile's rows
  static constexpr int kKvBars = (2 + kQSlots + kOSlots) * kTileBytes + (kQSlots + kOSlots) * kStatBytes;
  // dQ: Q, dO, three K and two V slots, barriers
  static constexpr int kKSlots = 3, kVSlots = 2;
  static constexpr int kQBars = (2 + kKSlots + kVSlots) * kTileBytes;
  static constexpr int kSmem = kKvBars + 256;
  static_assert(kQBars <= kKvBars && kSmem <= 227 * 1024, "shared memory of a CTA");
};
constexpr int kBwdThreads = 352;  // 8 warps of elementwise work, a TMA warp, two MMA warps

// first of n iterations that are part k of `parts`
__device__ __forceinline__ int share(int n, int k, int parts) {
  return static_cast<int>(static_cast<int64_t>(n) * k / parts);
}

// barrier 1 of a CTA: the TMA warp arrives (its barriers are initialised) and
// goes on, the others wait
__device__ __forceinline__ void ready_arrive() { asm volatile("bar.arrive 1, %0;" ::"n"(kBwdThreads) : "memory"); }
__device__ __forceinline__ void ready_wait() { asm volatile("bar.sync 1, %0;" ::"n"(kBwdThreads) : "memory"); }

__device__ __forceinline__ void bwd_timeout(const BwdParams& p, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(p.status, kStatusTimeout);
}

// What is in flight when a CTA gives up ends in its shared memory or TMEM, which
// the next CTA gets, so it is waited for whatever the plan's limit: the products
// on their barrier (a limit that is never reached), the copies by time, since
// the barriers that they arrive on may lack other arrivals for good.
constexpr uint64_t kDrainNs = 100000000ull, kCopiesNs = 50000000ull;

__device__ __forceinline__ void drain_products(const BwdParams& p, uint64_t* bar, volatile int* abort_flag) {
  mma_commit(smem_u32(bar));
  volatile int never = 0;
  if (!mbar_wait(smem_u32(bar), 0, globaltimer_ns() + kDrainNs, &never)) bwd_timeout(p, abort_flag);
}
// (by one warp, once every thread of the CTA has come past its last copy)
__device__ __forceinline__ void drain_copies(volatile int* abort_flag) {
  if (!*abort_flag) return;
  const uint64_t until = globaltimer_ns() + kCopiesNs;
  while (globaltimer_ns() < until) {
  }
}

// As mbar_wait in as little code as possible, for the elementwise loops, which
// jump over it several times a tile (8 heads of 8192 rows of 64: 488 us with
// mbar_wait, 481 with this, when it was taken).
__device__ __forceinline__ bool ew_wait(uint32_t bar, uint32_t parity, uint64_t deadline_ns, volatile int* abort_flag) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 r;\n\t.reg .b64 t;\n"
      "EW_LOOP_%=:\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra EW_DONE_%=;\n\t"
      "ld.volatile.shared.b32 r, [%3];\n\t"
      "setp.ne.b32 q, r, 0;\n\t"
      "@q bra EW_DONE_%=;\n\t"
      "mov.u64 t, %%globaltimer;\n\t"
      "setp.gt.u64 q, t, %4;\n\t"
      "@!q bra EW_LOOP_%=;\n"
      "EW_DONE_%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity), "r"(smem_u32(const_cast<int*>(abort_flag))), "l"(deadline_ns) : "memory");
  return ok != 0;
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

// tensor map of run s for the heads of rank r, and the run's first row in it
__device__ __forceinline__ int map_of(const Seg& s, int r) { return s.src < 0 ? r - 1 - s.src : s.src; }
__device__ __forceinline__ int first_row(const BwdParams& p, const Seg& s, int r) {
  return s.row0 < 0 ? p.shard_len[r] : s.row0;
}

// 128 rows x D of one head to shared memory, panels of 64 columns one behind
// the other (the map's fourth dimension), in one instruction
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* m, uint32_t bar, int head, int row, int b) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %3, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(head), "r"(row), "r"(b)
      : "memory");
}

// Shared-memory descriptors (128-byte swizzle; tc.cuh): the upper word is the
// same for every operand here, the lower one is the start address / 16 and the
// leading byte offset.  What an issuing thread does between two MMAs delays the
// tensor core, so the lower words are a base and a constant.
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
// row in the columns [a, a + 32), 64..127 in [a + HALF, a + HALF + 32)) and B a
// 128-row tile in shared memory (MN-major; the sum runs over the rows); blo
// from desc_cols
template <int D, int HALF = 64>
__device__ __forceinline__ void issue_cols(uint32_t d, uint32_t a, uint32_t blo, bool acc) {
  using C = BCfg<D>;
#pragma unroll
  for (int k = 0; k < C::kRowSteps; ++k)
    mma_ts(d, a + HALF * (k >> 2) + 8 * (k & 3), blo + k * 128, C::kIdescO, acc || k > 0);
}

// Zero the rows of a 128-row tile whose bit in `live` is clear: one warp's
// share, rows [row0, row0 + 16) (four of them at a time), bits 0..15.
template <int D>
__device__ __forceinline__ void zero_dead_rows(uint32_t tile, uint32_t live, int row0, int lane) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 4 * k + (lane >> 3);
    if (!((live >> r) & 1u))
#pragma unroll
      for (int pn = 0; pn < BCfg<D>::kPanels; ++pn)
        st_shared_v4(tile + pn * BCfg<D>::kPanelBytes + (row0 + r) * 128 + (lane & 7) * 16, 0u, 0u, 0u, 0u);
  }
}
// that share of warp `warp`, from the two words of its half of the tile's bits
__device__ __forceinline__ uint32_t warp_rows(const uint2 half, int warp) {
  return ((warp & 2 ? half.y : half.x) >> (16 * (warp & 1))) & 0xFFFFu;
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

// ------------------------------------------------------------- split --
// Where there are too few tiles for the SMs, a tile's loop is shared by the
// CTAs of a cluster, a part of the iterations each.  Each leaves its f32 sums
// in its shared memory, and each adds up a share of the rows of all of them in
// the order of the CTAs: the same bits on every call.  A read of another CTA's
// shared memory takes hundreds of cycles, so eight of a lane's are under way,
// along the rows.  All of it, the launch in clusters included, costs a call 3
// to 5 us (128-wide heads; reads of two pieces in turn 2 us more, writes to the
// CTA that adds up 4 more).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// address of 16-byte piece c of row r of an f32 matrix [][D]
template <int D>
__device__ __forceinline__ uint32_t f32_at(uint32_t base, int r, int c) {
  constexpr int kPieces = D / 4;
  return base + static_cast<uint32_t>(r * kPieces + (c ^ (r & (kPieces - 1)))) * 16u;
}

// piece c of row r of the matrix in the shared memory of CTA `rank` of the cluster
template <int D>
__device__ __forceinline__ float4 ld_peer(uint32_t base, int r, int c, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(f32_at<D>(base, r, c)), "r"(rank)
      : "memory");
  return v;
}

// the thread's row of an f32 accumulator in TMEM, columns [c_lo, c_hi), to
// shared memory
template <int D>
__device__ __forceinline__ void keep_rows(uint32_t t, uint32_t base, int row, int c_lo, int c_hi, bool zero) {
  for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
    uint32_t o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0u;
    if (!zero) {
      tmem_ld32(t + c0, o);
      tmem_wait_ld();
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      st_shared_v4(f32_at<D>(base, row, c0 / 4 + k), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
  }
}

// This CTA's share of the rows of a matrix at `base`: the sum over the
// cluster's CTAs, times mul, to the output tensors as store_rows writes them.
template <int D>
__device__ __forceinline__ void join_rows(const BwdParams& p, uint8_t* const* out, const int64_t* batch_stride,
                                          int64_t row_stride, const Seg& run, int row0, int head, int owner, int b,
                                          uint32_t base, float mul, int part) {
  constexpr int kPieces = D / 4, kSets = 8;
  const int log = p.parts >> 1, rows = kTileRows >> log;  // (parts: 2 or 4)
  const int n = min(rows, run.len - row0 - part * rows) * kPieces, lane_off = head * D * 2;
  if (!in_bounds(&g_bwd_violations, lane_off, D * 2, row_stride)) return;
  const bool all = p.fused && run.out_shard < 0;
  const int lo = all ? 0 : (p.fused ? run.out_shard : owner), hi = all ? p.P : lo + 1;
  for (int sh = lo; sh < hi; ++sh) {
    const int64_t r0 = (run.out_row0 < 0 ? p.shard_len[sh] : run.out_row0) + row0 + part * rows;
    if (n > 0 && !in_bounds(&g_bwd_violations, r0 * row_stride, n / kPieces * row_stride, batch_stride[sh])) continue;
    uint8_t* dst = out[sh] + b * batch_stride[sh] + r0 * row_stride + lane_off;
    const bool zero = all && sh != owner;
    for (int i0 = threadIdx.x; i0 < n; i0 += kBwdThreads * (kSets >> log)) {
      float4 u[kSets];
#pragma unroll
      for (int s = 0; s < kSets; ++s) {
        const int i = min(i0 + (s >> log) * kBwdThreads, n - 1);
        u[s] = ld_peer<D>(base, part * rows + i / kPieces, i % kPieces, s & (p.parts - 1));
      }
#pragma unroll
      for (int s = 0; s < kSets; ++s) {
        const int i = i0 + (s >> log) * kBwdThreads;
        if (s & (p.parts - 1))
          u[s] = make_float4(u[s - 1].x + u[s].x, u[s - 1].y + u[s].y, u[s - 1].z + u[s].z, u[s - 1].w + u[s].w);
        if ((s & (p.parts - 1)) == p.parts - 1 && i < n) {
          const uint2 w = make_uint2(pack_bf16x2(u[s].x * mul, u[s].y * mul), pack_bf16x2(u[s].z * mul, u[s].w * mul));
          *reinterpret_cast<uint2*>(dst + i / kPieces * row_stride + i % kPieces * 8) = zero ? make_uint2(0u, 0u) : w;
        }
      }
    }
  }
}

// ------------------------------------------------------- preparation --
// Is the key of global index `key` admitted in batch b?
__device__ __forceinline__ bool admitted(const BwdParams& p, int b, int key) {
  if (!in_bounds(&g_bwd_violations, key, 1, p.Nk)) return false;
  if (p.key_mask) return p.key_mask[static_cast<int64_t>(b) * p.Nk + key] != 0;
  if (!p.key_ranges) return true;
  const int32_t* rg = p.key_ranges + static_cast<int64_t>(b) * p.n_ranges * 2;
  for (int q = 0; q < p.n_ranges; ++q)
    if (key >= rg[2 * q] && key < rg[2 * q + 1]) return true;
  return false;
}

// global index of the first key of kv run s
__device__ __forceinline__ int first_key(const BwdParams& p, int s) {
  int k = 0;
  for (int i = 0; i < s; ++i) k += p.kseg[i].len;
  return k;
}

// sum over eight bf16 pairs of products
__device__ __forceinline__ float dot8(const uint4 a, const uint4 b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    s = fmaf(__uint_as_float(x[k] << 16), __uint_as_float(y[k] << 16), s);
    s = fmaf(__uint_as_float(x[k] & 0xFFFF0000u), __uint_as_float(y[k] & 0xFFFF0000u), s);
  }
  return s;
}

// first row of tile i of the replicated run in dl_lo
__device__ __forceinline__ int64_t lo_at(const BwdParams& p, int b, int h, int i) {
  return ((static_cast<int64_t>(b) * p.Hq + h) * p.n_lo + i) * kTileRows;
}

constexpr int kPrepThreads = 256;

// The kv tile tables of batch b: the admitted keys of every tile, and the list
// of tiles that a query attends to: those whose 128 keys are all admitted from
// the front, in key order, and the others from the back, so that dQ's loop over
// the former needs no masks (ULY_ROWS_SELF: all from the back).  One CTA, a
// warp a tile.
struct TableSmem {
  uint4 bits[kPrepThreads], inv[kPrepThreads];
  int32_t packed[kPrepThreads];
  int2 warp_sum[kPrepThreads / 32];
};
__device__ __forceinline__ void build_tables(const BwdParams& p, int b, TableSmem& sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(b) * p.n_kv_tiles;
  int n_full = 0, n_part = 0;
  // the run of the warp's tile, and the keys before it
  int s = 0, seg_first = 0, seg_len = p.kseg[0].len, key_base = 0;
  int seg_end = p.n_kseg > 1 ? p.kseg[1].first : p.n_kv_tiles;
  for (int t0 = 0; t0 < p.n_kv_tiles; t0 += kPrepThreads) {
    for (int k = warp; k < kPrepThreads && t0 + k < p.n_kv_tiles; k += kPrepThreads / 32) {
      while (t0 + k >= seg_end) {
        key_base += seg_len;
        ++s;
        seg_first = p.kseg[s].first;
        seg_len = p.kseg[s].len;
        seg_end = s + 1 < p.n_kseg ? p.kseg[s + 1].first : p.n_kv_tiles;
      }
      const int i = t0 + k - seg_first, key0 = key_base + i * kTileRows, n_in = min(kTileRows, seg_len - i * kTileRows);
      uint32_t w[4], in[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = lane + 32 * j;
        const bool ok = c < n_in && admitted(p, b, key0 + c);
        w[j] = __ballot_sync(0xffffffffu, ok);
        in[j] = __ballot_sync(0xffffffffu, c < n_in);
      }
      if (lane == 0) {
        const uint4 wb = make_uint4(w[0], w[1], w[2], w[3]);
        p.tile_bits[row + t0 + k] = wb;
        sm.bits[k] = wb;
        sm.inv[k] = make_uint4(~w[0] & in[0], ~w[1] & in[1], ~w[2] & in[2], ~w[3] & in[3]);
        sm.packed[k] = (s << 20) | i;
      }
    }
    __syncthreads();
    const int k = threadIdx.x;
    bool any = false, full = false;
    if (t0 + k < p.n_kv_tiles) {
      const uint4 wb = sm.bits[k];
      const bool self = p.masked_rows == ULY_ROWS_SELF;
      any = self || (wb.x | wb.y | wb.z | wb.w) != 0u;
      full = !self && bits_full(wb);
    }
    const uint32_t vf = __ballot_sync(0xffffffffu, full), vp = __ballot_sync(0xffffffffu, any && !full);
    if (lane == 0) sm.warp_sum[warp] = make_int2(__popc(vf), __popc(vp));
    __syncthreads();
    const uint32_t below = (1u << lane) - 1u;
    int front = n_full + __popc(vf & below), back = n_part + __popc(vp & below);
    for (int i = 0; i < kPrepThreads / 32; ++i) {
      if (i < warp) {
        front += sm.warp_sum[i].x;
        back += sm.warp_sum[i].y;
      }
      n_full += sm.warp_sum[i].x;
      n_part += sm.warp_sum[i].y;
    }
    const int slot = full ? front : p.n_kv_tiles - 1 - back;
    if (any && in_bounds(&g_bwd_violations, slot, 1, p.n_kv_tiles)) {
      p.active[row + slot] = sm.packed[k];
      p.active_bits[row + slot] = sm.bits[k];
      p.active_inv[row + slot] = sm.inv[k];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    p.n_active[b] = n_full + n_part;
    p.n_full[b] = n_full;
  }
}

// The first B CTAs build the kv tile tables.  The others: per (batch, q head,
// 128-row tile of a run) -lse log2(e) and -delta, padded to whole tiles, which
// the main kernel reads in tiles.  A row that takes part in nothing (past its
// run's end, no admitted key, or zero by the masked-row convention) has -inf,
// whose exponential is 0.  Fused, replicated rows: do is the sum of every
// shard's copy, since each received the output, written as two bf16 operands
// (do_hi, do_lo) with a delta each.
// Bound by memory: o and do are read once (40 heads of 29328 rows of 128, 616
// MB with the summed rows: 114 us, 5.4 TB/s; small calls 4 to 8 us, the longest
// of its dependent steps).  ROWS rows x 8 heads a CTA; 16 (D = 128) or 8 lanes
// share a row, the results go through shared memory so that they are written
// along rows.
template <int D, int ROWS>
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(const __grid_constant__ BwdParams p) {
  constexpr int kLanes = D / 8, kUnits = kPrepThreads / kLanes, kRows = ROWS, kHeads = 8;
  constexpr int kParts = kTileRows / kRows;
  __shared__ union {
    TableSmem table;
    struct {
      float hi[kHeads][kRows + 1], lo[kHeads][kRows + 1];
    } dl;
  } sm;
  if (blockIdx.x < static_cast<uint32_t>(p.B)) {
    build_tables(p, blockIdx.x, sm.table);
    return;
  }
  uint32_t i0 = blockIdx.x - p.B;
  const int hg = (p.Hq + kHeads - 1) / kHeads;
  const int h0 = static_cast<int>(i0 % hg) * kHeads;
  i0 /= hg;
  const int t = static_cast<int>(i0 / kParts % p.n_q_tiles), r_lo = static_cast<int>(i0 % kParts) * kRows;
  const int b = static_cast<int>(i0 / kParts / p.n_q_tiles);
  const Seg run = p.qseg[seg_of(p.qseg, p.n_qseg, t)];
  const int row0 = (t - run.first) * kTileRows + r_lo;  // first row inside the run
  const int lane = threadIdx.x % kLanes, unit = threadIdx.x / kLanes;
  const bool rep = p.fused && run.out_shard < 0;
#pragma unroll 8
  for (int i = unit; i < kRows * kHeads; i += kUnits) {
    const int r = i / kHeads, hh = i % kHeads, h = h0 + hh;
    float sum = 0.f, sum_lo = 0.f;
    if (h < p.Hq && row0 + r < run.len) {
      const int owner = h / p.Hq_l;
      const int sh = p.fused ? (rep ? owner : run.out_shard) : owner;
      const int64_t col = (static_cast<int64_t>(p.fused ? h : h % p.Hq_l) * D + lane * 8) * 2;
      const int64_t row = (run.out_row0 < 0 ? p.shard_len[sh] : run.out_row0) + row0 + r;
      if (in_bounds(&g_bwd_violations, row * p.q_row_stride, p.q_row_stride, p.q_batch_stride[sh])) {
        const uint4 ov = *reinterpret_cast<const uint4*>(p.o[sh] + b * p.q_batch_stride[sh] + row * p.q_row_stride + col);
        uint4 dv, dlo = make_uint4(0u, 0u, 0u, 0u);
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
          // the sum as two bf16 values, whose own sum is off by at most 2^-17
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            hi[k] = pack_bf16x2(acc[2 * k], acc[2 * k + 1]);
            lo[k] = pack_bf16x2(acc[2 * k] - __uint_as_float(hi[k] << 16),
                                acc[2 * k + 1] - __uint_as_float(hi[k] & 0xFFFF0000u));
          }
          dv = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          dlo = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          const int64_t at = ((static_cast<int64_t>(b) * run.len + row0 + r) * p.Hq + h) * D * 2 + lane * 16;
          *reinterpret_cast<uint4*>(p.do_hi + at) = dv;
          if (p.n_lo) *reinterpret_cast<uint4*>(p.do_lo + at) = dlo;
        }
        sum = dot8(ov, dv);
        if (rep) sum_lo = dot8(ov, dlo);
      }
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      sum_lo += __shfl_xor_sync(0xffffffffu, sum_lo, o);
    }
    if (lane == 0) {
      sm.dl.hi[hh][r] = sum;
      sm.dl.lo[hh][r] = sum_lo;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kHeads; i += kPrepThreads) {
    const int hh = i / kRows, r = i % kRows, h = h0 + hh;
    if (h >= p.Hq) continue;
    const int64_t at = ((static_cast<int64_t>(b) * p.Hq + h) * p.n_q_tiles + t) * kTileRows + r_lo + r;
    float nl = -INFINITY, dl = 0.f, dl_lo = 0.f;
    const int lrow = row0 + r;
    if (lrow < run.len) {
      const int owner = h / p.Hq_l;
      const int sh = p.fused ? (rep ? owner : run.out_shard) : owner;
      const int64_t row = (run.out_row0 < 0 ? p.shard_len[sh] : run.out_row0) + lrow;
      const int64_t li = row * p.lse_row_stride + (p.fused ? h : h % p.Hq_l);
      float lse = -INFINITY;
      if (in_bounds(&g_bwd_violations, li, 1, p.lse_batch_stride[sh])) lse = p.lse[sh][b * p.lse_batch_stride[sh] + li];
      // (ULY_ROWS_ZERO: a row whose own token is a masked key)
      const bool zero = p.masked_rows == ULY_ROWS_ZERO && run.kv_seg >= 0 &&
                        !admitted(p, b, first_key(p, run.kv_seg) + lrow);
      const bool live = lse != -INFINITY && !zero;
      if (live) {
        nl = -lse * 1.4426950408889634f;
        dl = -sm.dl.hi[hh][r];
        dl_lo = -sm.dl.lo[hh][r];
      }
    }
    p.nl[at] = nl;
    p.dl[at] = dl;
    if (rep && p.n_lo) p.dl_lo[lo_at(p, b, h, t - run.first) + r_lo + r] = dl_lo;
  }
}

// A thread works on 64 entries of a tile's row, two to a register pair.
//
// Entries that do not attend are cleared in the packed bf16 pairs, so that
// neither an infinity nor a NaN in a masked place gets through and the f32
// arithmetic is the same for all.  A mask word's even and odd bits are first
// drawn apart within each half (bit 2i + e of a half to bit 8e + i), so that
// one shift puts the two bits of two pairs at the tops of bytes and one byte
// permutation, which can repeat a byte's top bit, makes a pair's mask.
__device__ __forceinline__ uint32_t pair_bits(uint32_t x) {
  uint32_t t = (x ^ (x >> 1)) & 0x22222222u;
  x ^= t ^ (t << 1);
  t = (x ^ (x >> 2)) & 0x0C0C0C0Cu;
  x ^= t ^ (t << 2);
  t = (x ^ (x >> 4)) & 0x00F000F0u;
  return x ^ t ^ (t << 4);
}
// the mask of pair i (0..31) from the two words' pair_bits
template <int I>
__device__ __forceinline__ uint32_t pair_mask(uint32_t u0, uint32_t u1) {
  uint32_t m;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(m) : "r"((I < 16 ? u0 : u1) << (7 - (I & 7))), "n"((I & 8) ? 0xBBAA : 0x9988));
  return m;
}
template <int N, int I = 0>
__device__ __forceinline__ void mask_pairs(uint32_t (&pk)[N], uint32_t u0, uint32_t u1) {
  if constexpr (I < N) {
    pk[I] &= pair_mask<I>(u0, u1);
    mask_pairs<N, I + 1>(pk, u0, u1);
  }
}

// p = 2^(s sl2 + nl) from the scores at TMEM t, kept in f32 in pr.  COLS: the
// addend is one per column, in shared memory at nl_addr; otherwise the row's,
// nl2.  `loaded` is called once the scores are in registers.
template <bool COLS, typename F>
__device__ __forceinline__ void half_row_p(uint32_t t, uint64_t mul, uint64_t nl2, uint32_t nl_addr,
                                           uint64_t (&pr)[32], F loaded) {
  uint32_t a[2][32];
  tmem_ld32(t, a[0]);
  tmem_ld32(t + 32, a[1]);
  tmem_wait_ld();
  loaded();
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
      pr[i] = f2(ex2_approx(x0), ex2_approx(x1));
    }
  }
}

// ds = p (dp + ndl), rounded to bf16, from the loaded dP; ndl as nl above.
template <bool COLS>
__device__ __forceinline__ void half_row_ds(const uint32_t (&a)[2][32], uint64_t dl2, uint32_t dl_addr,
                                            const uint64_t (&pr)[32], uint32_t (&pk)[32]) {
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
      pk[i] = pack_bf16x2(x0, x1);
    }
  }
}

// p rounded to bf16, 32 entries to the 16 TMEM columns from t on
template <bool MASKED, int C>
__device__ __forceinline__ void store_p(uint32_t t, const uint64_t (&pr)[32], uint32_t u) {
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1;
    f2_split(pr[16 * C + i], x0, x1);
    pk[i] = pack_bf16x2(x0, x1);
  }
  if (MASKED) mask_pairs(pk, u, u);
  tmem_st16(t + 16 * C, pk);
}

struct KvBars {
  uint64_t kq_full, q1_full;  // K and Q(0); Q(1)
  uint64_t nl_full[3];        // -lse log2(e) of a tile's rows
  uint64_t s_full[2];         // S(i) in region i mod 2
  uint64_t s_go;              // phase i: S(i) read out of TMEM (8 warps); dO(i), -delta (and V) landed
  uint64_t dp_full;           // phase i: dP(i) in region i mod 2
  uint64_t dp_issued;         // phase i: dP(i) issued
  uint64_t ds_full[2];        // dS(i) stored (8 warps): i mod 2, as dP(i+1) does not wait for dK(i)
  uint64_t p_go[2];           // P(i) stored (8 warps), Q(i+2) landed: i mod 2, since a warp may store
                              // P(i+1) before Q(i+2) is there
  uint64_t v_done[2];         // dV(i), and with it dK(i), complete: i mod 2, as dV(i+1) does not wait for S(i+2)
  uint64_t done, drain[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(KvBars) <= 256, "room for the barriers");

// What the elementwise warps of dkdv_cta share.
struct KvWork {
  KvBars* bars;
  uint32_t tmem, sQ, sDO, sNl, sDl;
  int n_it, b, first_tile;  // of the head's tiles
  uint64_t deadline;
};

// The elementwise loop of dkdv_cta: one thread per key and half of the
// queries.  MODE 0: every pair of the warp attends.  1: `dead` keys do not.
// 2: it goes by the queries' own tokens too (ULY_ROWS_ZERO, _SELF).  Loops of
// their own, so that the common one has no test in it and all but fits the
// registers (at D = 128 up to 8 bytes are spilled).  (A test that jumps over
// a tile's masking costs more than the masking: 64-wide heads, scattered mask,
// 177 us with it and 157 without, when it was taken.)
template <int D, int MODE>
__device__ __forceinline__ bool kv_loop(const BwdParams& p, const KvWork& k, int warp, int lane, bool key_ok, bool dead) {
  using C = BCfg<D>;
  KvBars& bars = *k.bars;
  volatile int* abort_flag = &bars.abort_flag;
  const int wg = warp >> 2, q4 = warp & 3;
  const uint32_t off = (static_cast<uint32_t>(q4 * 32) << 16) + 64 * wg;
  const uint64_t mul = f2(p.scale_log2, p.scale_log2);
  const bool self = p.masked_rows == ULY_ROWS_SELF, zero_rows = p.masked_rows == ULY_ROWS_ZERO;
  uint2 live_next = make_uint2(0u, 0u);
  // The queries' own tokens, a tile ahead of their use.  The q runs are kv runs
  // of the same tokens, in order, so their kv tiles follow one another.
  const uint2* own = reinterpret_cast<const uint2*>(
                         p.tile_bits + static_cast<int64_t>(k.b) * p.n_kv_tiles +
                         (MODE == 2 && p.qseg[0].kv_seg >= 0 ? p.kseg[p.qseg[0].kv_seg].first : 0)) +
                     wg;  // (the warp's half of a tile's bits)
  const int rep_tile = p.qseg[p.rep_qseg].first;  // (the replicated run's once more, with do_lo)
  int own_tile = k.first_tile;
  const auto next_live = [&] {
    live_next = __ldg(own + 2 * (own_tile < p.n_q_tiles ? own_tile : rep_tile + own_tile - p.n_q_tiles));
    if (++own_tile == p.n_q_tiles + p.n_lo) own_tile = 0;
  };
  if (MODE == 2) next_live();
  int qslot = 0, qturn = 0;
  for (int it = 0; it < k.n_it; ++it) {
    const uint32_t mR = k.tmem + off + 128 * (it & 1);
    const uint32_t nl_addr = k.sNl + qslot * C::kStatBytes + 64 * wg * 4;
    const uint32_t dl_addr = k.sDl + (it & 1) * C::kStatBytes + 64 * wg * 4;
    uint32_t u0 = 0u, u1 = 0u, rows = 0xFFFFu;
    if (MODE == 2) {
      const uint2 live = live_next;
      rows = warp_rows(live, warp);
      if (it + 1 < k.n_it) next_live();
      // queries that attend to the thread's key: those whose own token is
      // admitted (ULY_ROWS_ZERO), those of the key's own kind (ULY_ROWS_SELF;
      // past the run's end the statistics exclude)
      u0 = live.x;
      u1 = live.y;
      if (self && !key_ok) {
        u0 = ~u0;
        u1 = ~u1;
      }
      if (dead) u0 = u1 = 0u;
      u0 = pair_bits(u0);
      u1 = pair_bits(u1);
    } else if (MODE == 1) {
      u0 = u1 = dead ? 0u : ~0u;
    }
    bool ok = ew_wait(smem_u32(&bars.nl_full[qslot]), qturn & 1, k.deadline, abort_flag) &
              ew_wait(smem_u32(&bars.s_full[it & 1]), (it >> 1) & 1, k.deadline, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return false;
    tc_fence_after();
    uint64_t pr[32];
    const auto s_loaded = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.s_go));
    };
    half_row_p<true>(mR, mul, 0, nl_addr, pr, s_loaded);
    constexpr bool kOwnP = C::template kOwnP<MODE == 2>;
    const uint32_t mP =
        kOwnP ? k.tmem + 384 + (static_cast<uint32_t>(q4 * 32) << 16) + 64 * (it & 1) + 32 * wg : mR + 32;
    if (kOwnP) {
      store_p<MODE != 0, 0>(mP, pr, u0);
      store_p<MODE != 0, 1>(mP, pr, u1);
    }
    ok = ew_wait(smem_u32(&bars.s_go), it & 1, k.deadline, abort_flag) &
         ew_wait(smem_u32(&bars.dp_full), it & 1, k.deadline, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return false;
    tc_fence_after();
    uint32_t a[2][32], pk[32];
    tmem_ld32(mR, a[0]);
    tmem_ld32(mR + 32, a[1]);
    if (MODE == 2 && zero_rows && rows != 0xFFFFu) {
      // queries that take part in nothing may hold anything: their rows of Q
      // and dO are zeroed before the sums over queries read them (S and dP
      // have read them)
      zero_dead_rows<D>(k.sQ + qslot * C::kTileBytes, rows, 16 * warp, lane);
      zero_dead_rows<D>(k.sDO + (it & 1) * C::kTileBytes, rows, 16 * warp, lane);
      fence_proxy_async_smem();
    }
    tmem_wait_ld();
    half_row_ds<true>(a, 0, dl_addr, pr, pk);
    if (MODE == 1) {
#pragma unroll
      for (int i = 0; i < 32; ++i) pk[i] &= u0;
    } else if (MODE == 2) {
      mask_pairs(pk, u0, u1);
    }
    tmem_st32(mR, pk);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.ds_full[it & 1]));
    if (!kOwnP) {
      store_p<MODE != 0, 0>(mP, pr, u0);
      store_p<MODE != 0, 1>(mP, pr, u1);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
    }
    if (lane == 0) mbar_arrive(smem_u32(&bars.p_go[it & 1]));
    if (++qslot == C::kQSlots) {
      qslot = 0;
      ++qturn;
    }
  }
  if (k.n_it > 0) {
    const bool ok = ew_wait(smem_u32(&bars.done), 0, k.deadline, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return false;
    tc_fence_after();
  }
  return true;
}

// dK and dV of 128 keys of one kv head.
//   warp 8   TMA: K and V once, then Q, dO and the row statistics of every
//            128-query tile of every query head of the group.
//   warp 9   MMA: S = K Q^T (keys are TMEM lanes), dK += dS Q and dV += P do
//            with dS and P read from TMEM, in the order
//              S(0) S(1) | dK(i) dV(i) S(i+2) ...
//   warp 10  MMA: dP(i) = V dO^T, as soon as S(i) is in registers.  Where the
//            tile has masks, so that the elementwise work is what everything
//            waits for, dV(i - 1) and S(i + 1) come after it.
//   warps 0-7: P from S, dS from dP.
// Two query tiles are under way in two TMEM regions of 128 columns.  A region
// holds in turn a tile's S, then (once S is in registers) its dP, then (once dP
// is) its dS and P in bf16, half a row's P in the 32 columns behind its dS.
// A thread spends about 47 cycles on issuing an MMA (64 on the tensor core for
// 128-wide heads, 32 for the sums of 64-wide ones), 75 on a commit and 85 on a
// wait for a barrier that has completed.  So there are two of them: one thread
// for all four products, 578 us, two 537 (8 heads of 8192 rows; 64-wide 459 and
// 408); S on the second thread, which then waits for dV(i), 625.  And the copy
// of a tile is one more arrival on a barrier that its first reader waits for
// anyway.  Slots: Q(i) over Q(i-3) once dV(i-3), issued after dK(i-3), is
// complete; dO(i) over dO(i-2) once dV(i-2) is.
// TMEM: regions [0,128) [128,256), dV [256,256+D), dK [256+D,256+2D); 64-wide
// heads: P of the two tiles [384,448) [448,512).
template <int D, bool OWN, bool SPLIT>
__device__ __forceinline__ void dkdv_cta(const BwdParams& p, uint8_t* smem_raw, int t, int hk, int b, int part) {
  using C = BCfg<D>;
  KvBars& bars = *reinterpret_cast<KvBars*>(smem_raw + C::kKvBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = hk / p.Hkv_l;  // owning rank
  const Seg run = p.kseg[seg_of(p.kseg, p.n_kseg, t)];
  const int row0 = (t - run.first) * kTileRows;
  const uint4 bits = p.tile_bits[static_cast<int64_t>(b) * p.n_kv_tiles + t];
  const bool self = p.masked_rows == ULY_ROWS_SELF;
  const bool any = self || (bits.x | bits.y | bits.z | bits.w) != 0u;
  const int n_all = any ? p.G * (p.n_q_tiles + p.n_lo) : 0;
  // SPLIT: this CTA's share of them
  const int it_lo = SPLIT ? share(n_all, part, p.parts) : 0;
  const int n_it = SPLIT ? share(n_all, part + 1, p.parts) - it_lo : n_all;

  const uint32_t sK = smem_u32(smem_raw), sV = sK + C::kTileBytes, sQ = sK + 2 * C::kTileBytes;
  const uint32_t sDO = sQ + C::kQSlots * C::kTileBytes, sNl = sDO + C::kOSlots * C::kTileBytes;
  const uint32_t sDl = sNl + C::kQSlots * C::kStatBytes;
  volatile int* abort_flag = &bars.abort_flag;
  const uint64_t deadline = globaltimer_ns() + p.wait_ns;

  if (warp == 8) {
    if (lane == 0) {
      mbar_init(smem_u32(&bars.kq_full), 1);
      mbar_init(smem_u32(&bars.q1_full), 1);
      for (int i = 0; i < C::kQSlots; ++i) mbar_init(smem_u32(&bars.nl_full[i]), 1);
      mbar_init(smem_u32(&bars.s_full[0]), 1);
      mbar_init(smem_u32(&bars.s_full[1]), 1);
      mbar_init(smem_u32(&bars.s_go), 9);
      mbar_init(smem_u32(&bars.dp_full), 1);
      mbar_init(smem_u32(&bars.dp_issued), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&bars.ds_full[i]), 8);
        mbar_init(smem_u32(&bars.p_go[i]), 9);
        mbar_init(smem_u32(&bars.v_done[i]), 1);
        mbar_init(smem_u32(&bars.drain[i]), 1);
      }
      mbar_init(smem_u32(&bars.done), 1);
      bars.abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    ready_arrive();
    if (lane == 0 && n_it > 0) {
      const int kvhead = p.fused ? hk : hk % p.Hkv_l;
      const int kmap = map_of(run, r), krow = first_row(p, run, r) + row0;
      const uint32_t b_sgo = smem_u32(&bars.s_go);
      // Where tiles come from is worked out ahead, so that their loads follow at
      // once when a slot is free: mq .. for the next Q, mo .. for the next dO
      // (the tile before it).
      // A head's tiles: every run's, then the replicated run's again with do_lo
      // (run n_qseg here).
      int g = 0, qs = 0, qt = 0;  // q head of the group, run, tile inside the run
      const int n_runs = p.n_qseg + (p.n_lo ? 1 : 0);
      if (SPLIT) {
        g = it_lo / (p.n_q_tiles + p.n_lo);
        const int i = it_lo % (p.n_q_tiles + p.n_lo);
        qs = i < p.n_q_tiles ? seg_of(p.qseg, p.n_qseg, i) : p.n_qseg;
        qt = i - (i < p.n_q_tiles ? p.qseg[qs].first : p.n_q_tiles);
      }
      int qhead = 0, qrow = 0, ohead = 0, orow = 0, ohead_n = 0, orow_n = 0;
      const CUtensorMap *mq = nullptr, *mo = nullptr, *mo_n = nullptr;
      const float *nl = nullptr, *dl = nullptr, *dl_n = nullptr;
      const auto next = [&] {
        mo = mo_n;
        ohead = ohead_n;
        orow = orow_n;
        dl = dl_n;
        const int h = hk * p.G + g;
        if (g == p.G) return;
        const bool lo = qs == p.n_qseg;
        const Seg& q = p.qseg[lo ? p.rep_qseg : qs];
        const bool rep = p.fused && q.out_shard < 0;
        const int qmap = map_of(q, r);
        qhead = p.fused ? h : h % p.Hq_l;
        qrow = first_row(p, q, r) + qt * kTileRows;
        ohead_n = rep ? h : qhead;
        orow_n = rep ? qt * kTileRows : qrow;
        mq = &p.tq[qmap];
        mo_n = rep ? (lo ? &p.tdo_lo : &p.tdo_hi) : &p.tdo[qmap];
        const int64_t at = ((static_cast<int64_t>(b) * p.Hq + h) * p.n_q_tiles + q.first + qt) * kTileRows;
        nl = p.nl + at;
        dl_n = lo ? p.dl_lo + lo_at(p, b, h, qt) : p.dl + at;
        if (++qt * kTileRows >= q.len) {
          qt = 0;
          if (++qs == n_runs) {
            qs = 0;
            ++g;
          }
        }
      };
      // Q(it): its slot is free since v_done(it - 3); p_go(it - 4) is complete
      // for the same reason
      const auto load_q = [&](int it) {
        const uint32_t slot = it % C::kQSlots;
        const uint32_t bq = smem_u32(it == 0 ? &bars.kq_full : it == 1 ? &bars.q1_full : &bars.p_go[it & 1]);
        const uint32_t bn = smem_u32(&bars.nl_full[slot]);
        mbar_arrive_expect_tx(bq, (it == 0 ? 2 : 1) * C::kTileBytes);
        if (it == 0) load_tile(sK, &p.tk[kmap], bq, kvhead, krow, b);
        if (it != p.withhold_fill) load_tile(sQ + slot * C::kTileBytes, mq, bq, qhead, qrow, b);
        mbar_arrive_expect_tx(bn, C::kStatBytes);
        bulk_load(sNl + slot * C::kStatBytes, nl, C::kStatBytes, bn);
      };
      // dO(it): its slot is free since v_done(it - 2); phase it - 1 of s_go is
      // complete
      const auto load_o = [&](int it) {
        const uint32_t slot = it & 1;
        mbar_arrive_expect_tx(b_sgo, (it == 0 ? 2 : 1) * C::kTileBytes + C::kStatBytes);
        if (it == 0) load_tile(sV, &p.tv[kmap], b_sgo, kvhead, krow, b);
        load_tile(sDO + slot * C::kTileBytes, mo, b_sgo, ohead, orow, b);
        bulk_load(sDl + slot * C::kStatBytes, dl, C::kStatBytes, b_sgo);
      };
      bool ok = true;
      next();
      load_q(0);
      next();
      load_o(0);
      if (n_it > 1) {
        load_q(1);
        next();
        ok = mbar_wait(b_sgo, 0, deadline, abort_flag);
        if (ok) load_o(1);
      }
      if (ok && n_it > 2) {
        load_q(2);
        next();
        // dO(it) and Q(it + 1) follow v_done(it - 2) and s_go(it - 1)
        for (int it = 2; it < n_it; ++it) {
          if (!(ok = mbar_wait(smem_u32(&bars.v_done[it & 1]), ((it - 2) >> 1) & 1, deadline, abort_flag) &&
                     mbar_wait(b_sgo, ~it & 1, deadline, abort_flag)))
            break;
          load_o(it);
          if (it + 1 < n_it) load_q(it + 1);
          next();
        }
      }
      if (ok) {
        // the last two of p_go have no copy
        if (n_it > 1) mbar_arrive(smem_u32(&bars.p_go[n_it & 1]));
        mbar_arrive(smem_u32(&bars.p_go[(n_it - 1) & 1]));
      } else {
        bwd_timeout(p, abort_flag);
      }
    }
  } else if (warp == 9) {
    tmem_alloc(smem_u32(&bars.tmem_base), 512);
    tmem_relinquish();
    tc_fence_before();
    ready_wait();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base, tDV = tmem + 256, tDK = tmem + 256 + D;
    if (lane == 0 && n_it > 0) {
      uint32_t q_c[C::kQSlots], o_c[C::kOSlots];
#pragma unroll
      for (int i = 0; i < C::kQSlots; ++i) q_c[i] = desc_cols(sQ + i * C::kTileBytes);
#pragma unroll
      for (int i = 0; i < C::kOSlots; ++i) o_c[i] = desc_cols(sDO + i * C::kTileBytes);
      const bool ordered = OWN || run.len - row0 < kTileRows || !bits_full(bits);
      const uint32_t dk = desc_rows(sK);
      uint32_t q_r[C::kQSlots];
#pragma unroll
      for (int i = 0; i < C::kQSlots; ++i) q_r[i] = desc_rows(sQ + i * C::kTileBytes);
      bool ok = mbar_wait(smem_u32(&bars.kq_full), 0, deadline, abort_flag);
      tc_fence_after();
      if (ok) {
        issue_rows<D>(tmem, dk, q_r[0]);
        mma_commit(smem_u32(&bars.s_full[0]));
      }
      if (ok && n_it > 1) {
        ok = mbar_wait(smem_u32(&bars.q1_full), 0, deadline, abort_flag);
        if (ok) {
          issue_rows<D>(tmem + 128, dk, q_r[1]);
          mma_commit(smem_u32(&bars.s_full[1]));
        }
      }
      // unrolled over a turn of the rings, so that every operand is a constant
      constexpr int kTurn = C::kQSlots * C::kOSlots;
      static_assert(kTurn % 2 == 0 && C::kOSlots == 2, "regions and phases alternate");
      for (int it0 = 0; ok && it0 < n_it; it0 += kTurn) {
#pragma unroll
        for (int u = 0; u < kTurn; ++u) {
          const int it = it0 + u;
          if (!ok || it >= n_it) break;
          const uint32_t tR = tmem + 128 * (u & 1);
          if (!(ok = mbar_wait(smem_u32(&bars.ds_full[u & 1]), (it >> 1) & 1, deadline, abort_flag))) break;
          tc_fence_after();
          issue_cols<D>(tDK, tR, q_c[u % C::kQSlots], it > 0);
          // (measured, 12 heads on 4 of 2304 rows: by the queries' own masks 99 us
          // without this order and 89 with it, no masks 80 and 83)
          if (ordered && it + 1 < n_it &&
              !(ok = mbar_wait(smem_u32(&bars.dp_issued), ~u & 1, deadline, abort_flag)))
            break;
          if (!(ok = mbar_wait(smem_u32(&bars.p_go[u & 1]), (it >> 1) & 1, deadline, abort_flag))) break;
          tc_fence_after();
          if constexpr (C::template kOwnP<OWN>)
            issue_cols<D, 32>(tDV, tmem + 384 + 64 * (u & 1), o_c[u % C::kOSlots], it > 0);
          else
            issue_cols<D>(tDV, tR + 32, o_c[u % C::kOSlots], it > 0);
          if (it + 2 < n_it) {
            mma_commit(smem_u32(&bars.v_done[u & 1]));
            issue_rows<D>(tR, dk, q_r[(u + 2) % C::kQSlots]);
            mma_commit(smem_u32(&bars.s_full[u & 1]));
          } else if (it + 1 == n_it)
            mma_commit(smem_u32(&bars.done));
        }
      }
      if (!ok) bwd_timeout(p, abort_flag);
      drain_products(p, &bars.drain[0], abort_flag);
    }
  } else if (warp == 10) {
    tc_fence_before();
    ready_wait();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;
    if (lane == 0 && n_it > 0) {
      const uint32_t dv = desc_rows(sV);
      uint32_t o_r[C::kOSlots];
#pragma unroll
      for (int i = 0; i < C::kOSlots; ++i) o_r[i] = desc_rows(sDO + i * C::kTileBytes);
      bool ok = true;
      ok = ok && mbar_wait(smem_u32(&bars.s_go), 0, deadline, abort_flag);
      tc_fence_after();
      if (ok) {
        issue_rows<D>(tmem, dv, o_r[0]);
        mbar_arrive(smem_u32(&bars.dp_issued));
        mma_commit(smem_u32(&bars.dp_full));
      }
      for (int it0 = 0; ok && it0 + 1 < n_it; it0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int it = it0 + u;
          if (!ok || it + 1 >= n_it) break;
          if (!(ok = mbar_wait(smem_u32(&bars.s_go), ~u & 1, deadline, abort_flag))) break;
          tc_fence_after();
          issue_rows<D>(tmem + 128 * (~u & 1), dv, o_r[~u & 1]);
          mbar_arrive(smem_u32(&bars.dp_issued));
          mma_commit(smem_u32(&bars.dp_full));
        }
      }
      if (!ok) bwd_timeout(p, abort_flag);
      drain_products(p, &bars.drain[1], abort_flag);
    }
  } else {
    tc_fence_before();
    ready_wait();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base, tDV = tmem + 256, tDK = tmem + 256 + D;
    const int wg = warp >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;  // key of the tile = TMEM lane
    const bool key_ok = (bits_word(bits, q4) >> lane) & 1u;
    const bool dead = row0 + row >= run.len || (!self && !key_ok);
    const KvWork k = {&bars, tmem, sQ, sDO, sNl, sDl, n_it, b, n_it > 0 ? it_lo % (p.n_q_tiles + p.n_lo) : 0, deadline};
    bool ok;
    if constexpr (OWN)
      ok = kv_loop<D, 2>(p, k, warp, lane, key_ok, dead);
    else if (__any_sync(0xffffffffu, dead))
      ok = kv_loop<D, 1>(p, k, warp, lane, key_ok, dead);
    else
      ok = kv_loop<D, 0>(p, k, warp, lane, key_ok, dead);
    if (!ok) {
      tmem_wait_st();  // (P may be on its way)
      bwd_timeout(p, abort_flag);
    } else if (SPLIT) {
      // warps 0-3: dV, warps 4-7: dK, in f32 from the buffer's start on (every
      // copy into it has been read)
      keep_rows<D>((wg ? tDK : tDV) + (static_cast<uint32_t>(q4 * 32) << 16), sK + wg * (kTileRows * D * 4), row, 0, D,
                   n_it == 0);
    } else {
      // warps 0-3: dV, warps 4-7: dK; each warp stages and stores its 32 rows
      // (in two slots of Q: every copy into them has been read)
      const uint32_t stage = sQ + wg * C::kTileBytes;
      stage_rows<D>((wg ? tDK : tDV) + (static_cast<uint32_t>(q4 * 32) << 16), wg ? p.scale : 1.f, stage, row, 0, D,
                    n_it == 0);
      __syncwarp();
      store_rows<D, 2 * D / 16>(p, wg ? p.dk : p.dv, p.kv_batch_stride, p.kv_row_stride, run, row0, run.len - row0,
                                p.fused ? hk : hk % p.Hkv_l, r, b, stage, q4, 0, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) drain_copies(abort_flag);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(bars.tmem_base, 512);
  }
  if (SPLIT) {
    cluster_sync();
    const int head = p.fused ? hk : hk % p.Hkv_l;
    for (int m = 0; m < 2; ++m)
      join_rows<D>(p, m ? p.dk : p.dv, p.kv_batch_stride, p.kv_row_stride, run, row0, head, r, b,
                   sK + m * (kTileRows * D * 4), m ? p.scale : 1.f, part);
    cluster_sync();  // no CTA leaves while another reads its sums
  }
}

struct QBars {
  uint64_t q_full, lo_full;   // Q and dO; do_lo in dO's place
  uint64_t full[3];           // K and V of a tile (K's slot)
  uint64_t s_full[2], dp_full, dp_free, ds_full[2];
  uint64_t v_free[2];         // dP(i) complete
  uint64_t k_done[2];         // dQ(i) complete: i mod 2, as dQ(i+1) does not wait for S(i+2)
  uint64_t done, drain[2];
  uint32_t tmem_base;
  int abort_flag;
};

// slot in the tile list of the it'th tile of dQ's loop
__device__ __forceinline__ int listed(const BwdParams& p, int it, int n_full) {
  return it < n_full ? it : p.n_kv_tiles - 1 - (it - n_full);
}

// What the elementwise warps of dq_cta share.
struct QWork {
  QBars* bars;
  uint32_t tmem, sK;
  int n_it, n_full, b, j_lo;  // j_lo: first tile of the list
  uint64_t deadline;
};

// The elementwise loop of dq_cta over the tiles [it0, it1) (base: 0, or the
// number of tiles when they are gone through again): one thread per
// query and half of the keys.  MASKED: keys that are not admitted, and dead
// rows.
template <int D, bool MASKED>
__device__ __forceinline__ bool q_loop(const BwdParams& p, const QWork& k, int warp, int lane, int base, int it0, int it1,
                                       float nl, float dl, bool dead, const uint4* row_bits) {
  using C = BCfg<D>;
  QBars& bars = *k.bars;
  volatile int* abort_flag = &bars.abort_flag;
  const int wg = warp >> 2, q4 = warp & 3;
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const uint32_t mDP = k.tmem + 256 + lane_off + 64 * wg;
  const uint64_t mul = f2(p.scale_log2, p.scale_log2), nl2 = f2(nl, nl), dl2 = f2(dl, dl);
  const uint2* tile_bits = reinterpret_cast<const uint2*>(p.active_bits + static_cast<int64_t>(k.b) * p.n_kv_tiles) + wg;
  const uint2* half_bits = reinterpret_cast<const uint2*>(row_bits) + wg;
  const bool zero_keys = p.masked_rows != ULY_ROWS_SELF;
  uint2 bits_next = make_uint2(0u, 0u), keys_next = bits_next;
  if (MASKED && it0 < it1) {
    bits_next = __ldg(half_bits + 2 * listed(p, k.j_lo + it0, k.n_full));
    keys_next = __ldg(tile_bits + 2 * listed(p, k.j_lo + it0, k.n_full));
  }
  for (int j = it0; j < it1; ++j) {
    const int it = base + j, buf = it & 1;
    const uint32_t mS = k.tmem + lane_off + 128 * buf + 64 * wg;
    const uint2 bits = bits_next, keys = keys_next;
    if (MASKED && j + 1 < it1) {
      bits_next = __ldg(half_bits + 2 * listed(p, k.j_lo + j + 1, k.n_full));
      keys_next = __ldg(tile_bits + 2 * listed(p, k.j_lo + j + 1, k.n_full));
    }
    bool ok = ew_wait(smem_u32(&bars.s_full[buf]), (it >> 1) & 1, k.deadline, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return false;
    tc_fence_after();
    uint64_t pr[32];
    half_row_p<false>(mS, mul, nl2, 0, pr, [] {});
    ok = ew_wait(smem_u32(&bars.dp_full), it & 1, k.deadline, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return false;
    tc_fence_after();
    uint32_t a[2][32], pk[32];
    tmem_ld32(mDP, a[0]);
    tmem_ld32(mDP + 32, a[1]);
    tmem_wait_ld();
    // dP is in registers: the next tile's may overwrite it
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.dp_free));
    half_row_ds<false>(a, dl2, 0, pr, pk);
    if (MASKED)
      mask_pairs(pk, pair_bits(dead ? 0u : bits.x), pair_bits(dead ? 0u : bits.y));
    tmem_st32(mS, pk);
    if (MASKED && zero_keys) {
      // keys that are not admitted may hold anything: their rows of K are
      // zeroed before the sum over keys reads them (S has read them)
      zero_dead_rows<D>(k.sK + (it % C::kKSlots) * C::kTileBytes, warp_rows(keys, warp), 16 * warp, lane);
      fence_proxy_async_smem();
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.ds_full[buf]));
  }
  return true;
}

// dQ of 128 queries of one q head.
//   warp 8   TMA: Q and dO once, K (three slots) and V (two) of every kv tile
//            with an admitted key.
//   warp 9   MMA: S = Q K^T (queries are TMEM lanes), dQ += dS K with dS read
//            from TMEM, in the order  S(0) S(1) | dQ(j) S(j+2) ...
//   warp 10  MMA: dP(j) = dO V^T, as soon as dP(j-1) is in registers.
//   warps 0-7: one thread per query and half of the keys: dS from S and dP,
//            stored over S's columns (two S buffers, so that the next tile's
//            scores are there when this one's are done).
// A step takes about 1900 cycles at D = 128 (1536 of them on the tensor core;
// dK/dV 2450 of 2048), 1350 with 64-wide heads.
// TMEM: S0 [0,128) S1 [128,256) dP [256,384) dQ [384,384+D).
template <int D, bool SPLIT>
__device__ __forceinline__ void dq_cta(const BwdParams& p, uint8_t* smem_raw, int t, int h, int b, int part) {
  using C = BCfg<D>;
  QBars& bars = *reinterpret_cast<QBars*>(smem_raw + C::kQBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = h / p.Hq_l, hk = h / p.G;
  const Seg run = p.qseg[seg_of(p.qseg, p.n_qseg, t)];
  const int row0 = (t - run.first) * kTileRows;
  // replicated rows of the fused call: every tile with do_hi, then with do_lo
  const bool rep = p.fused && run.out_shard < 0, twice = rep && p.n_lo > 0;
  const int n_all = p.n_active[b], n_full = p.n_full[b];
  // SPLIT: this CTA's share of the list
  const int j_lo = SPLIT ? share(n_all, part, p.parts) : 0;
  const int n = SPLIT ? share(n_all, part + 1, p.parts) - j_lo : n_all;
  const int n_it = twice ? 2 * n : n;
  const int32_t* active = p.active + static_cast<int64_t>(b) * p.n_kv_tiles;

  const uint32_t sQ = smem_u32(smem_raw), sDO = sQ + C::kTileBytes, sK = sQ + 2 * C::kTileBytes;
  const uint32_t sV = sK + C::kKSlots * C::kTileBytes;
  volatile int* abort_flag = &bars.abort_flag;
  const uint64_t deadline = globaltimer_ns() + p.wait_ns;

  if (warp == 8) {
    if (lane == 0) {
      mbar_init(smem_u32(&bars.q_full), 1);
      mbar_init(smem_u32(&bars.lo_full), 1);
      for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&bars.full[i]), 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&bars.s_full[i]), 1);
        mbar_init(smem_u32(&bars.ds_full[i]), 8);
        mbar_init(smem_u32(&bars.k_done[i]), 1);
        mbar_init(smem_u32(&bars.v_free[i]), 1);
        mbar_init(smem_u32(&bars.drain[i]), 1);
      }
      mbar_init(smem_u32(&bars.dp_full), 1);
      mbar_init(smem_u32(&bars.dp_free), 8);
      mbar_init(smem_u32(&bars.done), 1);
      bars.abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    ready_arrive();
    if (lane == 0 && n_it > 0) {
      const int qmap = map_of(run, r);
      const int qhead = p.fused ? h : h % p.Hq_l, kvhead = p.fused ? hk : hk % p.Hkv_l;
      const int qrow = first_row(p, run, r) + row0;
      const uint32_t bq = smem_u32(&bars.q_full);
      mbar_arrive_expect_tx(bq, 2 * C::kTileBytes);
      load_tile(sQ, &p.tq[qmap], bq, qhead, qrow, b);
      if (rep)
        load_tile(sDO, &p.tdo_hi, bq, h, row0, b);
      else
        load_tile(sDO, &p.tdo[qmap], bq, qhead, qrow, b);
      // (where a tile comes from is worked out before its slots are free)
      const CUtensorMap *mk, *mv;
      int krow;
      bool good;
      const auto next = [&](int it) {
        const int e = active[listed(p, j_lo + (it < n ? it : it - n), n_full)];
        good = in_bounds(&g_bwd_violations, e >> 20, 1, p.n_kseg);
        const Seg& k = p.kseg[good ? e >> 20 : 0];
        const int kmap = map_of(k, r);
        krow = first_row(p, k, r) + (e & 0xFFFFF) * kTileRows;
        mk = &p.tk[kmap];
        mv = &p.tv[kmap];
      };
      next(0);
      for (int it = 0; it < n_it; ++it) {
        const int ks = it % C::kKSlots, vs = it % C::kVSlots;
        // the slots' last readers are dQ(it-3) and dP(it-2)
        if ((it >= 2 && !mbar_wait(smem_u32(&bars.v_free[it & 1]), ((it - 2) >> 1) & 1, deadline, abort_flag)) ||
            (it >= 3 && !mbar_wait(smem_u32(&bars.k_done[(it - 3) & 1]), ((it - 3) >> 1) & 1, deadline, abort_flag))) {
          bwd_timeout(p, abort_flag);
          break;
        }
        const uint32_t bf = smem_u32(&bars.full[ks]);
        mbar_arrive_expect_tx(bf, 2 * C::kTileBytes);
        if (good && it != p.withhold_fill) load_tile(sK + ks * C::kTileBytes, mk, bf, kvhead, krow, b);
        if (good) load_tile(sV + vs * C::kTileBytes, mv, bf, kvhead, krow, b);
        if (twice && it == n) {
          // do_lo over do_hi once dP(n - 1) is complete (dP(n - 2) is: the
          // waits above; dP(n) waits for this copy)
          if (!mbar_wait(smem_u32(&bars.v_free[(n - 1) & 1]), ((n - 1) >> 1) & 1, deadline, abort_flag)) {
            bwd_timeout(p, abort_flag);
            break;
          }
          const uint32_t bl = smem_u32(&bars.lo_full);
          mbar_arrive_expect_tx(bl, C::kTileBytes);
          load_tile(sDO, &p.tdo_lo, bl, h, row0, b);
        }
        if (it + 1 < n_it) next(it + 1);
      }
    }
  } else if (warp == 9) {
    tmem_alloc(smem_u32(&bars.tmem_base), 512);
    tmem_relinquish();
    tc_fence_before();
    ready_wait();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base, tDQ = tmem + 384;
    if (lane == 0 && n_it > 0) {
      uint32_t k_c[C::kKSlots];
#pragma unroll
      for (int i = 0; i < C::kKSlots; ++i) k_c[i] = desc_cols(sK + i * C::kTileBytes);
      const uint32_t dq = desc_rows(sQ);
      uint32_t k_r[C::kKSlots];
#pragma unroll
      for (int i = 0; i < C::kKSlots; ++i) k_r[i] = desc_rows(sK + i * C::kTileBytes);
      bool ok = mbar_wait(smem_u32(&bars.q_full), 0, deadline, abort_flag) &&
                mbar_wait(smem_u32(&bars.full[0]), 0, deadline, abort_flag);
      tc_fence_after();
      if (ok) {
        issue_rows<D>(tmem, dq, k_r[0]);
        mma_commit(smem_u32(&bars.s_full[0]));
        if (n_it > 1) {
          ok = mbar_wait(smem_u32(&bars.full[1]), 0, deadline, abort_flag);
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
          const int it = it0 + u, buf = u & 1;
          if (!ok || it >= n_it) break;
          if (!(ok = mbar_wait(smem_u32(&bars.ds_full[buf]), (it >> 1) & 1, deadline, abort_flag))) break;
          tc_fence_after();
          issue_cols<D>(tDQ, tmem + 128 * buf, k_c[u % C::kKSlots], it > 0);
          if (it + 2 < n_it) {
            const int ks2 = (u + 2) % C::kKSlots;
            if (it + 3 < n_it) mma_commit(smem_u32(&bars.k_done[buf]));
            if (!(ok = mbar_wait(smem_u32(&bars.full[ks2]), ((it + 2) / C::kKSlots) & 1, deadline, abort_flag))) break;
            issue_rows<D>(tmem + 128 * buf, dq, k_r[ks2]);
            mma_commit(smem_u32(&bars.s_full[buf]));
          } else if (it + 1 == n_it)
            mma_commit(smem_u32(&bars.done));
        }
      }
      if (!ok) bwd_timeout(p, abort_flag);
      drain_products(p, &bars.drain[0], abort_flag);
    }
  } else if (warp == 10) {
    tc_fence_before();
    ready_wait();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base, tDP = tmem + 256;
    if (lane == 0 && n_it > 0) {
      const uint32_t ddo = desc_rows(sDO);
      uint32_t v_r[C::kVSlots];
#pragma unroll
      for (int i = 0; i < C::kVSlots; ++i) v_r[i] = desc_rows(sV + i * C::kTileBytes);
      bool ok = mbar_wait(smem_u32(&bars.q_full), 0, deadline, abort_flag) &&
                mbar_wait(smem_u32(&bars.full[0]), 0, deadline, abort_flag);
      tc_fence_after();
      if (ok) {
        issue_rows<D>(tDP, ddo, v_r[0]);
        mma_commit(smem_u32(&bars.dp_full));
        mma_commit(smem_u32(&bars.v_free[0]));
      }
      int slot = 1, turn = 0;  // of tile it + 1
      for (int it0 = 0; ok && it0 + 1 < n_it; it0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int it = it0 + u;
          if (!ok || it + 1 >= n_it) break;
          if (!(ok = mbar_wait(smem_u32(&bars.dp_free), u, deadline, abort_flag) &&
                     mbar_wait(smem_u32(&bars.full[slot]), turn & 1, deadline, abort_flag)))
            break;
          if (twice && it + 1 == n && !(ok = mbar_wait(smem_u32(&bars.lo_full), 0, deadline, abort_flag))) break;
          tc_fence_after();
          issue_rows<D>(tDP, ddo, v_r[~u & 1]);
          mma_commit(smem_u32(&bars.dp_full));
          mma_commit(smem_u32(&bars.v_free[~u & 1]));
          if (++slot == C::kKSlots) {
            slot = 0;
            ++turn;
          }
        }
      }
      if (!ok) bwd_timeout(p, abort_flag);
      drain_products(p, &bars.drain[1], abort_flag);
    }
  } else {
    tc_fence_before();
    ready_wait();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base, tDQ = tmem + 384;
    const int wg = warp >> 2, q4 = warp & 3;
    const int row = q4 * 32 + lane;  // query of the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const bool self = p.masked_rows == ULY_ROWS_SELF;
    // a masked row under ULY_ROWS_SELF attends to the masked keys
    bool invert = false;
    if (self && run.kv_seg >= 0) {
      const uint4 qb = p.tile_bits[static_cast<int64_t>(b) * p.n_kv_tiles + p.kseg[run.kv_seg].first + row0 / kTileRows];
      invert = !((bits_word(qb, q4) >> lane) & 1u);
    }
    const int64_t at = ((static_cast<int64_t>(b) * p.Hq + h) * p.n_q_tiles + t) * kTileRows + row;
    const float nl = p.nl[at], dl = p.dl[at];
    const bool dead = nl == -INFINITY;
    const uint4* row_bits = (invert ? p.active_inv : p.active_bits) + static_cast<int64_t>(b) * p.n_kv_tiles;
    const QWork k = {&bars, tmem, sK, n_it, n_full, b, j_lo, deadline};
    // the tiles without masks, then the others; all of them with masks where a
    // row of the warp takes part in nothing
    const int plain = __any_sync(0xffffffffu, dead) ? 0 : min(max(n_full - j_lo, 0), n);
    bool ok = true;
    for (int base = 0; ok && base < n_it; base += n) {
      const float d = base == 0 ? dl : p.dl_lo[lo_at(p, b, h, row0 / kTileRows) + row];
      ok = q_loop<D, false>(p, k, warp, lane, base, 0, plain, nl, d, dead, row_bits) &&
           q_loop<D, true>(p, k, warp, lane, base, plain, n, nl, d, dead, row_bits);
    }
    if (ok && n_it > 0) {
      ok = mbar_wait(smem_u32(&bars.done), 0, deadline, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) ok = false;
      tc_fence_after();
    }
    if (!ok) {
      tmem_wait_st();  // (P may be on its way)
      bwd_timeout(p, abort_flag);
    } else if (SPLIT) {
      keep_rows<D>(tDQ + lane_off, sQ, row, wg * (D / 2), (wg + 1) * (D / 2), n_it == 0);
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
  if (warp == 8) drain_copies(abort_flag);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(bars.tmem_base, 512);
  }
  if (SPLIT) {
    cluster_sync();
    join_rows<D>(p, p.dq, p.q_batch_stride, p.q_row_stride, run, row0, p.fused ? h : h % p.Hq_l, r, b, sQ, p.scale, part);
    cluster_sync();
  }
}

// One launch for both kinds of CTA: they need nothing from each other, so that
// dQ's fill the SMs that the last ones of dK and dV leave idle (8 heads of 8192
// rows: 649 us in two launches, 580 in one).
template <int D, bool OWN, bool SPLIT>
__global__ void __launch_bounds__(kBwdThreads, 1) backward_kernel(const __grid_constant__ BwdParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {  // (never: the buffer is placed on a 1024-byte boundary)
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  // longest first: dQ of tiles that are gone through twice, dK and dV, dQ
  uint32_t i = blockIdx.x, part = 0;
  if (SPLIT) {
    part = i % p.parts;
    i /= p.parts;
  }
  const uint32_t n_lo = p.n_lo, n_twice = n_lo * p.Hq * p.B, lo0 = p.qseg[p.rep_qseg].first;
  if (i >= n_twice && i - n_twice < p.n_kv_ctas) {
    i -= n_twice;
    const uint32_t t = i % p.n_kv_tiles;
    i /= p.n_kv_tiles;
    dkdv_cta<D, OWN, SPLIT>(p, smem_raw, t, i % p.Hkv, i / p.Hkv, part);
  } else {
    uint32_t n, t;  // tiles of this kind, and which
    if (i < n_twice) {
      n = n_lo;
      t = lo0 + i % n;
    } else {
      i -= n_twice + p.n_kv_ctas;
      n = p.n_q_tiles - n_lo;
      t = i % n;
      if (t >= lo0) t += n_lo;
    }
    i /= n;
    dq_cta<D, SPLIT>(p, smem_raw, t, i % p.Hq, i / p.Hq, part);
  }
}

template <int D, bool OWN, bool SPLIT>
cudaError_t launch_main(const BwdParams& p, unsigned grid, cudaStream_t s) {
  // the shared-memory limit is set once on every device that launches the
  // kernel (setting it twice is harmless)
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!bit || !(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(backward_kernel<D, OWN, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             BCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  if (!SPLIT) {
    backward_kernel<D, OWN, SPLIT><<<grid, kBwdThreads, BCfg<D>::kSmem, s>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid * p.parts);
  cfg.blockDim = dim3(kBwdThreads);
  cfg.dynamicSmemBytes = BCfg<D>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.parts;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, backward_kernel<D, OWN, SPLIT>, p);
}

template <int D>
cudaError_t launch(const BwdParams& p, cudaStream_t s) {
  // 16 rows a CTA of the preparation, 8 where an SM would get less than two of
  // these (8 heads of 2048 rows: 6.3 us with 16, 4.6 with 8; 40 heads of 29328
  // rows 114 and 123)
  const unsigned prep = static_cast<unsigned>(p.n_q_tiles) * ((p.Hq + 7) / 8) * p.B, n16 = prep * (kTileRows / 16);
  if (n16 < 2u * static_cast<unsigned>(p.sms))
    prep_kernel<D, 8><<<p.B + prep * (kTileRows / 8), kPrepThreads, 0, s>>>(p);
  else
    prep_kernel<D, 16><<<p.B + n16, kPrepThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned grid = p.n_kv_ctas + static_cast<unsigned>(p.n_q_tiles) * p.Hq * p.B;
  const bool own = p.masked_rows != ULY_ROWS_SDPA;
  if (p.parts > 1) return own ? launch_main<D, true, true>(p, grid, s) : launch_main<D, false, true>(p, grid, s);
  return own ? launch_main<D, true, false>(p, grid, s) : launch_main<D, false, false>(p, grid, s);
}

}  // namespace

cudaError_t launch_attention_backward(const BwdParams& p, int D, cudaStream_t s) {
  return D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace uly
