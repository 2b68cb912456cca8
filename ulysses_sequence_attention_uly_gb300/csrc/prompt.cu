// prompt.cu -- causal attention over packed sequences on the seq-sharded shards
// (tcgen05 + TMEM + TMA).
//
// For row i of a sequence: softmax over its rows j <= i of scale * q_i.k_j,
// times v_j; q head h uses kv head h / (Hq/Hkv).
//
// tables_kernel cuts the sequences into runs (a sequence's rows in one shard)
// and the runs into units of query rows, those with most keys first.  The
// attention kernel is persistent, one CTA an SM; an item is a unit and a head
// (pair), taken from a counter, so that a CTA that is done early takes more.
//
// An item has two 128-row query tiles that walk the same keys: one tile of two
// q heads of a kv head where the group is even, else two tiles of one head
// (then the first ends a key tile before the second).  Key tiles are 128 rows
// from a run's first row on, as are query tiles, so that only a tile's last key
// tile is cut by the diagonal and only a run's last one is short.
//   warp 8      TMA producer: takes items, loads Q tiles, and K and V tiles
//               through a ring of slots, in groups (V_s-1, K_s) of one step
//               each; it goes on to the next item while this one is finished.
//   warp 9      one thread issues the MMAs, in the order
//                 PV0(s) S0(s+1) PV1(s) S1(s+1)
//               and at an item's end PV0 PV1 S0 S1, the scores being the next
//               item's: they are done by the time the softmax warps have stored
//               this item's output.
//   warps 0-7   softmax of the two tiles, one thread a row, as in attn.cu: log2
//               domain, a lazily raised reference maximum, P in bf16 over S in
//               TMEM.  The epilogue stages its rows in shared memory of its own,
//               so that Q's slot is free for the next item.
// Rows of V behind a run's end (another sequence's, or nothing's) are zeroed in
// shared memory before P V: their P is 0, but 0 times a NaN is not.
// TMEM: S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [256+D,256+2D).
//
// The arithmetic of an item does not depend on which CTA takes it: the same
// bits on every call.  Every wait is bounded, each for itself (a CTA may be at
// work for seconds): its clock is first read when it has been waited for a while,
// since a reading before every wait cost up to a tenth.
//
// What bounds it (ncu, 8192 rows of 32 heads on 8): long items run at 2500 to 2600
// cycles a step, of which the four products take 2048 and the operands' way through
// shared memory 2000 (S reads both operands from there); tensor pipe active 74% of
// cycles, DRAM 5%.  27280 rows of 40 heads 4.39 ms after a pause, 1737 TFLOP/s of
// admitted pairs (for seconds on end 5.1 ms, 1500, at the power limit).  Short items: what is around the steps, about 3 us an item, that
// follows one upon the other (the last product, the store, the next softmax): 24
// prompts of 30 to 900 rows 58 to 59 us, tensor pipe 32%, DRAM 20%.
#include <atomic>

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

namespace {

constexpr int kItems = 4;  // items under way between the roles of a CTA

template <int D>
struct PCfg {
  static constexpr int kPanelBytes = kTileRows * 128;
  static constexpr int kTileBytes = D / 64 * kPanelBytes;
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kHalf = kSlots / 2;  // groups in the ring
  static constexpr int kQkSteps = D / 16;
  static constexpr int kPvSteps = 8;
  static constexpr uint32_t kIdescS = make_idesc(1, 128, 128, 0, 0);
  static constexpr uint32_t kIdescO = make_idesc(1, 128, D, 0, 1);
  static constexpr int kStageBytes = 32 * 128;  // a warp's 32 rows, 64 columns at a time
  static constexpr int kSmem = 1024 + (2 + kSlots) * kTileBytes + 8 * kStageBytes;
  static constexpr int kThreads = 320;
  static_assert(kSmem + 1024 <= 232448, "shared memory");
};

struct Item {
  int32_t run;      // -1: no more
  int32_t tile;     // first q tile (128 rows) inside the run
  int32_t head;     // first q head
  int32_t n[2];     // key tiles of the two q tiles (0: no such tile)
  int32_t shard, row0, len, first_run;
  int32_t first_len;  // rows of the sequence's first run
  int32_t pad[2];
};

struct PBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t full[4], empty[4];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t drain;
  Item item[kItems];
  PromptRun run[kDirectItems * kMaxRanks];  // direct: the runs of the sequences of the CTA's items
  PromptUnit unit[kDirectItems];            // direct: the items' units, their runs among them
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ void tma_load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int head, int row) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(head), "r"(row), "r"(0), "r"(0)
      : "memory");
}

// A wait on a barrier that gives up after limit_ns, or when another role has.  The
// limit counts from the 64th try on (each is waited for by the hardware a while).
// Out of line: the roles wait in many places of unrolled code, which has to stay
// small (24 prompts of 30 to 900 rows: inline 62.5 us, out of line 59.4).
__device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                           volatile int* abort_flag) {
  uint32_t spins = 0;
  uint64_t since = 0;
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((++spins & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = globaltimer_ns();
      if (!since) since = now;
      if (now - since > limit_ns) return false;
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || bar_wait_long(bar, parity, limit_ns, abort_flag);
}

// wait for the launch before this one in the stream (a programmatic dependency)
__device__ __forceinline__ void wait_for_previous_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- tables --
// Exclusive sum over the block's 1024 threads; *total receives the whole.
__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t* shared, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) shared[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint64_t w = shared[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    shared[lane] = w;
  }
  __syncthreads();
  const uint64_t before = warp ? shared[warp - 1] : 0;
  *total = shared[31];
  __syncthreads();
  return before + x - v;
}

// Largest of the values (none negative) up to this thread's.
__device__ __forceinline__ int block_max(int v, uint64_t* shared64) {
  int* const shared = reinterpret_cast<int*>(shared64);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v = max(v, y);
  }
  if (lane == 31) shared[warp] = v;
  __syncthreads();
  const int before = __reduce_max_sync(0xffffffffu, lane < warp ? shared[lane] : 0);
  __syncthreads();
  return max(v, before);
}

__device__ __forceinline__ int units_of(int len, int pair) {
  return pair ? (len + kTileRows - 1) / kTileRows : (len + 2 * kTileRows - 1) / (2 * kTileRows);
}

// One CTA (6 us, beside which the attention's CTAs come up): runs and units of all
// sequences.  The units are put in order of
// their key tiles (counting sort, largest first; which of two alike comes first
// is chance and changes nothing).
__global__ void __launch_bounds__(1024) tables_kernel(const __grid_constant__ PromptCut p) {
  __shared__ uint64_t sums[32];
  __shared__ int32_t run_unit_s[kSortBuckets];
  __shared__ int32_t bucket[kSortBuckets];
  __shared__ int32_t last_end;
  let_next_launch_start();
  const PromptTables& t = p.t;
  const int tid = threadIdx.x, N = p.shard_begin[p.P];
  int n_runs = 0, n_units = 0, reached = 0;
  for (int s0 = 0; s0 < p.n_seqs; s0 += 1024) {
    // rows [a, b) of sequence s.  A start below an earlier one counts as that
    // one, so that no row is in two sequences and the tables hold them all.
    const int s = s0 + tid;
    const int start = s < p.n_seqs ? min(max(p.seq_starts[s], 0), N) : 0;
    const int end = s < p.n_seqs ? min(max(p.seq_starts[s + 1], 0), N) : 0;
    const int a = max(block_max(start, sums), reached), b = s < p.n_seqs ? max(a, end) : a;
    if (tid == 1023) last_end = b;
    int runs = 0, units = 0;
    for (int i = 0; i < p.P; ++i) {
      const int len = min(b, p.shard_begin[i + 1]) - max(a, p.shard_begin[i]);
      if (len > 0) {
        ++runs;
        units += units_of(len, p.pair);
      }
    }
    uint64_t total;
    const uint64_t before = block_sum((static_cast<uint64_t>(runs) << 32) | static_cast<uint32_t>(units), sums, &total);
    int r = n_runs + static_cast<int>(before >> 32), u = n_units + static_cast<int>(before & 0xFFFFFFFFu);
    const int first = r;
    int kv = 0;
    for (int i = 0; i < p.P; ++i) {
      const int lo = max(a, p.shard_begin[i]), len = min(b, p.shard_begin[i + 1]) - lo;
      if (len <= 0 || !in_bounds(&g_prompt_violations, r, 1, t.max_runs)) continue;
      t.runs[r] = PromptRun{i, lo - p.shard_begin[i], len, first};
      t.run_unit[r] = u;
      if (r < kSortBuckets) run_unit_s[r] = u;
      t.run_kv[r] = kv;
      kv += (len + kTileRows - 1) / kTileRows;
      u += units_of(len, p.pair);
      ++r;
    }
    n_runs += static_cast<int>(total >> 32);
    n_units += static_cast<int>(total & 0xFFFFFFFFu);
    reached = last_end;
  }
  for (int i = tid; i < kSortBuckets; i += 1024) bucket[i] = 0;
  __syncthreads();
  const int32_t* const run_unit = n_runs <= kSortBuckets ? run_unit_s : t.run_unit;
  // unit i of the sequences' order: its run (the last that begins at or before it)
  auto unit = [&](int i) {
    int lo = 0, hi = n_runs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (run_unit[mid] <= i)
        lo = mid;
      else
        hi = mid;
    }
    const int len = t.runs[lo].len, tiles = (len + kTileRows - 1) / kTileRows;
    const int tile = (i - run_unit[lo]) * (p.pair ? 1 : 2);
    const int last = p.pair ? tile : min(tile + 1, tiles - 1);
    return PromptUnit{lo, tile, t.run_kv[lo] + last + 1, 0};
  };
  for (int i = tid; i < n_units; i += 1024)
    atomicAdd(&bucket[kSortBuckets - 1 - min(unit(i).n_kv >> p.sort_shift, kSortBuckets - 1)], 1);
  __syncthreads();
  const int c0 = bucket[2 * tid], c1 = bucket[2 * tid + 1];
  uint64_t total;
  const int at = static_cast<int>(block_sum(static_cast<uint64_t>(c0 + c1), sums, &total));
  bucket[2 * tid] = at;
  bucket[2 * tid + 1] = at + c0;
  __syncthreads();
  for (int i = tid; i < n_units; i += 1024) {
    const PromptUnit u = unit(i);
    const int place = atomicAdd(&bucket[kSortBuckets - 1 - min(u.n_kv >> p.sort_shift, kSortBuckets - 1)], 1);
    if (in_bounds(&g_prompt_violations, place, 1, t.max_units)) t.units[place] = u;
  }
  if (tid == 0) {
    t.head[0] = n_units;
    t.head[1] = p.grid;  // (CTA b's first item is item b)
  }
}

// ------------------------------------------------------------- attention --
__device__ __forceinline__ void record_timeout(const PromptParams& p, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicOr(p.status, kStatusTimeout);
}

// p = 2^(s * sl2 + neg) for 32 scores of a row, in bf16 to TMEM at tP as part of
// the A operand of P V; adds the f32 values to acc.
__device__ __forceinline__ void exp_store(const uint32_t (&a)[32], float sl2, float neg, uint32_t tP,
                                          uint64_t (&acc)[4]) {
  const uint64_t mul = f2(sl2, sl2), add = f2(neg, neg);
  uint32_t pk[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    float x0, x1;
    f2_split(f2_fma(f2(__uint_as_float(a[2 * q]), __uint_as_float(a[2 * q + 1])), mul, add), x0, x1);
    const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
    acc[q & 3] = f2_add(acc[q & 3], f2(e0, e1));
    pk[q] = pack_bf16x2(e0, e1);
  }
  tmem_st16(tP, pk);
}

// The running output to a new reference maximum.
template <int D>
__device__ __forceinline__ void rescale(uint32_t tO, float alpha) {
#pragma unroll
  for (int c0 = 0; c0 < D; c0 += 16) {
    uint32_t o[16];
    tmem_ld16(tO + c0, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
    tmem_st16(tO + c0, o);
  }
}

// The reference maximum (log2 domain) after a tile whose largest score is m_row:
// raised only when that grows by more than 2^8.  Returns what is then to be
// multiplied into the running sum and output.
__device__ __forceinline__ float raise(float m_row, float sl2, float& m_ref) {
  const float m_new = m_row * sl2;
  if (!(m_new > m_ref + 8.f)) return 1.f;
  const float alpha = ex2_approx(m_ref - m_new);
  m_ref = m_new;
  return alpha;
}

// One row of a 128 x 128 tile of scores (TMEM at tS) to its exponentials in place,
// with the running reference maximum, sum and output (TMEM at tO) brought along.
// (The product before these scores, which used O, has completed with them.)
template <int D>
__device__ __forceinline__ void whole_row(uint32_t tS, uint32_t tO, float sl2, bool first, float& m_ref, float& l_run) {
  uint32_t a[4][32];
  float mc[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32_max(tS + 32 * c, a[c], mc[c]);
  tmem_wait_ld();
  const float alpha = raise(fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3])), sl2, m_ref);
  const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
  float sum = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
    exp_store(a[2 * h], sl2, neg, tS + 32 * h, acc);
    exp_store(a[2 * h + 1], sl2, neg, tS + 32 * h + 16, acc);
    float s0, s1;
    f2_split(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
    sum += s0 + s1;
    if (h == 0 && !first && __any_sync(0xffffffffu, alpha != 1.f)) rescale<D>(tO, alpha);
  }
  l_run = l_run * alpha + sum;
}

// The same where the row sees the columns before `limit` only: of the warp's
// first `chunks` chunks of 32 columns all but the last whole, and nothing of the
// others.  A chunk at a time, twice, in little code: short prompts go through it
// once an item and wait for instructions as much as for anything.  (P of a chunk
// takes columns of chunks that are done.)
template <int D>
__device__ __forceinline__ void edge_row(uint32_t tS, uint32_t tO, float sl2, bool first, int limit, int chunks,
                                         float& m_ref, float& l_run) {
  uint32_t a[32];
  float m_row = -INFINITY;
#pragma unroll 1
  for (int c = 0; c + 1 < chunks; ++c) {
    float m;
    tmem_ld32_max(tS + 32 * c, a, m);
    tmem_wait_ld();
    m_row = fmaxf(m_row, m);
  }
  tmem_ld32(tS + 32 * (chunks - 1), a);
  tmem_wait_ld();
  const int cut = limit - 32 * (chunks - 1);
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < cut) m_row = fmaxf(m_row, __uint_as_float(a[i]));
  const float alpha = raise(m_row, sl2, m_ref);
  const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
  uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    tmem_ld32(tS + 32 * c, a);
    tmem_wait_ld();
    const int n = limit - 32 * c;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= n) a[i] = __float_as_uint(-INFINITY);
    exp_store(a, sl2, neg, tS + 16 * c, acc);
  }
#pragma unroll 1
  for (int c = chunks; c < 4; ++c) {
    const uint32_t none[16] = {};
    tmem_st16(tS + 16 * c, none);
  }
  if (!first && __any_sync(0xffffffffu, alpha != 1.f)) rescale<D>(tO, alpha);
  float s0, s1;
  f2_split(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
  l_run = l_run * alpha + (s0 + s1);
}

// Key tiles of an item in order: the runs of its sequence from the first on.
struct KeyTiles {
  const PromptRun* runs;
  int run, left;  // left: rows of the run from this tile on
  int shard, row0;
  // `first`: the sequence's first run
  __device__ __forceinline__ void begin(const PromptRun* r, int first_run, const int4& first) {
    runs = r;
    run = first_run;
    enter(first);
  }
  __device__ __forceinline__ void enter(const int4& v) {
    shard = v.x;
    row0 = v.y;
    left = v.z;
  }
  // (not after the item's last tile: there may be no run behind it)
  __device__ __forceinline__ void next() {
    if (left > kTileRows) {
      left -= kTileRows;
      row0 += kTileRows;
    } else {
      ++run;
      enter(*reinterpret_cast<const int4*>(runs + run));
    }
  }
};

// Direct, by one warp: the CTA's items among all in the order of the sequences.
// CTA b has item b and, where there are more items than CTAs, the one as far from
// the end: of one sequence a short one and a long one.
__device__ __forceinline__ void find_items(const PromptCut& p, int n_hp, PBars& bars, int lane) {
  const int N = p.shard_begin[p.P];
  int total = 0;
  if (lane < kDirectItems) bars.unit[lane].run = -1;
  __syncwarp();  // before another lane puts an item there (shuffles order no memory)
  // first how many units there are, then the items' own
  for (int k = -1; k < kDirectItems; ++k) {
    const int idx = k <= 0 ? static_cast<int>(blockIdx.x) : total * n_hp - 1 - static_cast<int>(blockIdx.x);
    if (k >= 0 && (idx >= total * n_hp || (k > 0 && idx < p.grid))) break;
    const int w = k < 0 ? -1 : idx / n_hp;
    int reached = 0, units_before = 0;
    for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
      // rows [a, b) of sequence s0 + lane, as in tables_kernel
      const int s = s0 + lane;
      int a = s < p.n_seqs ? min(max(p.seq_starts[s], 0), N) : 0;
      const int end = s < p.n_seqs ? min(max(p.seq_starts[s + 1], 0), N) : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, a, d);
        if (lane >= d) a = max(a, y);
      }
      a = max(a, reached);
      const int b = s < p.n_seqs ? max(a, end) : a;
      int units = 0;
      for (int i = 0; i < p.P; ++i) {
        const int len = min(b, p.shard_begin[i + 1]) - max(a, p.shard_begin[i]);
        if (len > 0) units += units_of(len, p.pair);
      }
      int upto = units;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
      }
      upto += units_before;
      if (upto - units <= w && w < upto) {  // one lane's sequence has it
        const int first = k * kMaxRanks;
        int r = first, kv = 0, at = upto - units;
        for (int i = 0; i < p.P; ++i) {
          const int lo = max(a, p.shard_begin[i]), len = min(b, p.shard_begin[i + 1]) - lo;
          if (len <= 0) continue;
          bars.run[r] = PromptRun{i, lo - p.shard_begin[i], len, first};
          const int here = units_of(len, p.pair), tiles = (len + kTileRows - 1) / kTileRows;
          if (w >= at && w < at + here) {
            const int tile = (w - at) * (p.pair ? 1 : 2);
            bars.unit[k] = PromptUnit{r, tile, kv + (p.pair ? tile : min(tile + 1, tiles - 1)) + 1, idx - w * n_hp};
          }
          at += here;
          kv += tiles;
          ++r;
        }
      }
      reached = __shfl_sync(0xffffffffu, b, 31);
      units_before = __shfl_sync(0xffffffffu, upto, 31);
    }
    if (k < 0) total = units_before;
  }
}

template <int D>
__device__ __forceinline__ void producer(const PromptParams& p, PBars& bars, uint32_t sQ, uint32_t sKV,
                                         int n_items, const PromptRun* runs, uint64_t wait_ns) {
  using C = PCfg<D>;
  volatile int* abort_flag = &bars.abort_flag;
  bool ok = true;
  int g = 0;                // groups issued (= steps begun)
  int n_q[2] = {0, 0};      // Q tiles loaded
  int v_shard = 0, v_row = 0, v_head = 0;
  // group g: V of step g - 1 and K of step g
  auto group = [&](bool has_k, int shard, int row, int head) {
    const int bi = g % C::kHalf;
    if (g >= C::kHalf && !bar_wait(smem_u32(&bars.empty[bi]), (g / C::kHalf - 1) & 1, wait_ns, abort_flag))
      return false;
    const uint32_t bf = smem_u32(&bars.full[bi]);
    mbar_arrive_expect_tx(bf, (g > 0 && has_k ? 2 : 1) * C::kTileBytes);
    if (g > 0 && 2 * g - 1 != p.withhold_fill)
      tma_load_tile(sKV + (2 * g - 1) % C::kSlots * C::kTileBytes, &p.tv[v_shard], bf, v_head, v_row);
    if (has_k && 2 * g != p.withhold_fill)
      tma_load_tile(sKV + 2 * g % C::kSlots * C::kTileBytes, &p.tk[shard], bf, head, row);
    v_shard = shard;
    v_row = row;
    v_head = head;
    ++g;
    return true;
  };
  int idx = p.direct ? 0 : blockIdx.x, known = -1;
  int4 u, r, f;  // the item's unit, its run, its sequence's first run
  for (int k = 0; ok; ++k) {
    const int slot = k % kItems;
    if (k >= kItems &&
        !(ok = bar_wait(smem_u32(&bars.item_empty[slot]), (k / kItems - 1) & 1, wait_ns, abort_flag)))
      break;
    Item it = {};
    it.run = -1;
    if (idx < n_items) {
      const int w = idx / p.n_hp;
      int hp = idx - w * p.n_hp;
      if (w != known || p.direct) {
        known = w;
        u = *reinterpret_cast<const int4*>(p.direct ? &bars.unit[k] : &p.cut.t.units[w]);
        if (p.direct) hp = u.w;
        f = r = *reinterpret_cast<const int4*>(runs + u.x);
        if (r.w != u.x) f = *reinterpret_cast<const int4*>(runs + r.w);
      }
      it.run = u.x;
      it.tile = u.y;
      it.shard = r.x;
      it.row0 = r.y;
      it.len = r.z;
      it.first_run = r.w;
      it.first_len = f.z;
      if (p.cut.pair) {
        it.head = 2 * hp;
        it.n[0] = it.n[1] = u.z;
      } else {
        it.head = hp;
        const bool two = (u.y + 1) * kTileRows < r.z;
        it.n[0] = two ? u.z - 1 : u.z;
        it.n[1] = two ? u.z : 0;
      }
    }
    bars.item[slot] = it;
    mbar_arrive(smem_u32(&bars.item_full[slot]));
    if (it.run < 0) break;
    const int n = max(it.n[0], it.n[1]), kv_head = it.head / p.G;
    KeyTiles kt;
    kt.begin(runs, it.first_run, f);
    int next = idx + 1;  // direct
    for (int s = 0; s < n; ++s) {
      // the next item is taken late, so that whoever is behind takes less; the
      // steps under way cover what finding out about it costs
      if (s == max(n - 3, 0) && !p.direct) next = atomicAdd(&p.cut.t.head[1], 1);
      if (!(ok = group(true, kt.shard, kt.row0, kv_head))) break;
      if (s == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!ok || !it.n[i]) continue;
          if (n_q[i] && !(ok = bar_wait(smem_u32(&bars.q_empty[i]), (n_q[i] - 1) & 1, wait_ns, abort_flag)))
            continue;
          const uint32_t bq = smem_u32(&bars.q_full[i]);
          mbar_arrive_expect_tx(bq, C::kTileBytes);
          tma_load_tile(sQ + i * C::kTileBytes, &p.tq[it.shard], bq, p.cut.pair ? it.head + i : it.head,
                        it.row0 + (p.cut.pair ? it.tile : it.tile + i) * kTileRows);
          ++n_q[i];
        }
        if (!ok) break;
      }
      if (s + 1 < n) kt.next();
    }
    idx = next;
  }
  if (ok && g > 0) ok = group(false, 0, 0, 0);
  if (!ok) record_timeout(p, abort_flag);
  if (*abort_flag) {
    // no copy lands in shared memory after the CTA has left (a withheld one
    // costs the bound)
    const uint64_t dl = globaltimer_ns() + 100000000ull;
    volatile int never = 0;
    for (int f = g > C::kHalf ? g - C::kHalf : 0; f < g; ++f)
      mbar_wait(smem_u32(&bars.full[f % C::kHalf]), (f / C::kHalf) & 1, dl, &never);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (n_q[i]) mbar_wait(smem_u32(&bars.q_full[i]), (n_q[i] - 1) & 1, dl, &never);
  }
}

template <int D>
__device__ __forceinline__ void issuer(const PromptParams& p, PBars& bars, uint32_t sQ, uint32_t sKV, uint32_t tmem,
                                       uint64_t wait_ns) {
  using C = PCfg<D>;
  volatile int* abort_flag = &bars.abort_flag;
  // descriptors as in attn.cu: a fixed high part and the start address / 16
  const uint64_t hi_s = sdesc_sw128(0, 16, 1024);              // Q and K: K-major
  const uint64_t hi_v = sdesc_sw128(0, C::kPanelBytes, 1024);  // V: MN-major
  const uint32_t q_lo = (sQ & 0x3FFFFu) >> 4, kv_lo = (sKV & 0x3FFFFu) >> 4;
  constexpr uint32_t kTileLo = C::kTileBytes >> 4;
  uint64_t dq[2][C::kQkSteps], dk[C::kHalf][C::kQkSteps], dv[C::kHalf][C::kPvSteps];
#pragma unroll
  for (int k = 0; k < C::kQkSteps; ++k) {
    const uint32_t off = ((k >> 2) * C::kPanelBytes + (k & 3) * 32) >> 4;
    dq[0][k] = hi_s | (q_lo + off);
    dq[1][k] = hi_s | (q_lo + kTileLo + off);
#pragma unroll
    for (int u = 0; u < C::kHalf; ++u) dk[u][k] = hi_s | (kv_lo + ((2 * u + 2) % C::kSlots) * kTileLo + off);
  }
#pragma unroll
  for (int u = 0; u < C::kHalf; ++u)
#pragma unroll
    for (int k = 0; k < C::kPvSteps; ++k) dv[u][k] = hi_v | (kv_lo + (2 * u + 1) * kTileLo + ((k * 16 * 128) >> 4));

  int n_item = 0;                // items read
  int left0 = 0, left1 = 0;      // steps of this item that a tile still has, this one included
  uint32_t par_p = 0, par_q = 0;  // parities of the two tiles' barriers, a bit each
  uint32_t acc = 0;              // the item has had a step
  uint32_t turn = 0;             // turns of the ring
  constexpr int kUnroll = 4;     // steps a turn of the plain loop: the jump back costs the issuer
  constexpr int kPlain = 8;
  static_assert(kUnroll % C::kHalf == 0, "whole turns of the ring");
  bool ok = true, more = false;
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    ok = bar_wait(smem_u32(&bar), parity & 1, wait_ns, abort_flag);
    tc_fence_after();
    return ok;
  };
  auto read_item = [&](int& n0, int& n1) {
    const int slot = n_item % kItems;
    if (!wait(bars.item_full[slot], n_item / kItems)) return false;
    const bool end = bars.item[slot].run < 0;
    n0 = end ? 0 : bars.item[slot].n[0];
    n1 = end ? 0 : bars.item[slot].n[1];
    mbar_arrive(smem_u32(&bars.item_empty[slot]));
    ++n_item;
    return true;
  };
  // Scores of a tile (constants: every descriptor is ready, since what the issuer
  // spends between two instructions the tensor core waits for), and its product
  // with V.  `steps`: that the tile has from these scores (this product) on, 0: more
  // than one.
#define ULY_SCORES(i, kd, steps, fresh)                                                                       \
  do {                                                                                                       \
    if (fresh) {                                                                                             \
      if (!wait(bars.q_full[i], par_q >> i)) break;                                                          \
      par_q ^= 1u << i;                                                                                      \
    }                                                                                                        \
    _Pragma("unroll") for (int k = 0; k < C::kQkSteps; ++k)                                                  \
        mma_bf16_ss(tmem + 128 * i, dq[i][k], kd[k], C::kIdescS, k > 0);                                     \
    mma_commit(smem_u32(&bars.s_full[i]));                                                                   \
    if ((steps) == 1) mma_commit(smem_u32(&bars.q_empty[i]));                                                \
  } while (0)
#define ULY_VALUES(i, vd, steps)                                                                              \
  do {                                                                                                       \
    if (!wait(bars.p_full[i], par_p >> i)) break;                                                            \
    par_p ^= 1u << i;                                                                                        \
    _Pragma("unroll") for (int k = 0; k < C::kPvSteps; ++k)                                                  \
        mma_bf16_ts(tmem + 256 + D * i, tmem + 128 * i + 8 * k, vd[k], C::kIdescO, acc | (k > 0));           \
    if ((steps) == 1) mma_commit(smem_u32(&bars.o_done[i]));                                                 \
  } while (0)
  if (read_item(left0, left1) && (left0 || left1)) {
    more = true;
    if (wait(bars.full[0], 0)) {
      // (K of step 0 is in slot 0, which is dk[kHalf - 1])
      if (left0) ULY_SCORES(0, dk[C::kHalf - 1], left0, true);
      if (ok && left1) ULY_SCORES(1, dk[C::kHalf - 1], left1, true);
      if (ok) mma_commit(smem_u32(&bars.empty[0]));
    }
  }
  while (ok && more) {
    // Steps in the middle of an item, both tiles going on: nothing to decide (a
    // 16384-row sequence: 1.49 ms without this loop, 1.29 with it).  Whole turns of
    // the ring, and kPlain steps at least: items of few stay in one piece of code,
    // since what a CTA's roles go through does not stay in the instruction cache
    // when it is long (512-row prompts 59.0 -> 54.5 us; from four steps on, 1024-row
    // ones take 83 us, from eight 76).
    int plain = min(left0, left1) - 2;  // (the last scores of a tile free its queries' slot)
    plain = plain < kPlain ? 0 : plain - plain % C::kHalf;
    left0 -= plain;
    left1 -= plain;
    while (ok && plain > 0) {
#pragma unroll
      for (int w = 0; w < kUnroll; ++w) {
        const int u = w % C::kHalf, bi = (u + 1) % C::kHalf;
        if (plain == 0) break;
        if (!wait(bars.full[bi], u == C::kHalf - 1 ? turn + 1 : turn)) break;
        ULY_VALUES(0, dv[u], 0);
        ULY_SCORES(0, dk[u], 0, false);
        if (!ok) break;
        ULY_VALUES(1, dv[u], 0);
        ULY_SCORES(1, dk[u], 0, false);
        if (!ok) break;
        mma_commit(smem_u32(&bars.empty[bi]));
        acc = 1;
        if (u == C::kHalf - 1) ++turn;
        --plain;
      }
    }
    // Any step s = turn * kHalf + u: a tile may end, or begin the next item.
#pragma unroll
    for (int u = 0; u < C::kHalf; ++u) {
      if (!ok || !more) break;
      const int bi = (u + 1) % C::kHalf;
      int next0 = left0 - 1, next1 = left1 - 1;
      bool last = false;
      if (min(next0, next1) <= 0) {  // a tile ends
        last = max(next0, next1) <= 0;
        if (last) {
          if (!read_item(next0, next1)) break;
          more = next0 || next1;
        } else {
          next0 = max(next0, 0);
          next1 = max(next1, 0);
        }
      }
      if (!wait(bars.full[bi], u == C::kHalf - 1 ? turn + 1 : turn)) break;
      if (left0) ULY_VALUES(0, dv[u], left0);
      // (an item's last product does not wait for the next one's queries)
      if (last && ok && left1) ULY_VALUES(1, dv[u], left1);
      if (ok && next0) ULY_SCORES(0, dk[u], next0, last);
      if (!last && ok && left1) ULY_VALUES(1, dv[u], left1);
      if (ok && next1) ULY_SCORES(1, dk[u], next1, last);
      if (!ok) break;
      if (more) mma_commit(smem_u32(&bars.empty[bi]));
      left0 = next0;
      left1 = next1;
      acc = last ? 0 : 1;
    }
    ++turn;
  }
#undef ULY_SCORES
#undef ULY_VALUES
  if (!ok) record_timeout(p, abort_flag);
  // every MMA has completed before TMEM is released
  mma_commit(smem_u32(&bars.drain));
  volatile int never = 0;
  if (!mbar_wait(smem_u32(&bars.drain), 0, globaltimer_ns() + 100000000ull, &never)) record_timeout(p, abort_flag);
}

template <int D>
__device__ __forceinline__ void softmax(const PromptParams& p, PBars& bars, uint32_t sKV, uint32_t sStage,
                                        uint32_t tmem, const PromptRun* runs, int warp, int lane, uint64_t wait_ns) {
  using C = PCfg<D>;
  volatile int* abort_flag = &bars.abort_flag;
  const int wg = warp >> 2, q4 = warp & 3, row = q4 * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const uint32_t tS = tmem + lane_off + 128 * wg, tO = tmem + lane_off + 256 + D * wg;
  const uint32_t stage = sStage + warp * C::kStageBytes;
  const float sl2 = p.scale_log2;
  int n_s = 0, n_o = 0, step0 = 0;  // S tiles and O tiles waited for; steps of the items before
  int idle = 0;  // steps of the item before in which these warps had no tile
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const int slot = k % kItems;
    // The next item comes near the end of this one.  Warps without a tile in this one
    // wait as long as the other roles may in its steps, where up to four waits (for
    // K and V, scores, P, a free slot) follow upon each other; when one of those gives
    // up, so do they.
    bool there = false;
    for (int i = 0; i <= 4 * idle && !there && !*abort_flag; ++i)
      there = bar_wait(smem_u32(&bars.item_full[slot]), (k / kItems) & 1, wait_ns, abort_flag);
    if (!__all_sync(0xffffffffu, there)) {
      ok = false;
      break;
    }
    const Item& it = bars.item[slot];
    if (it.run < 0) break;
    const int n = wg ? it.n[1] : it.n[0];
    if (n > 0) {
      float m_ref = -INFINITY, l_run = 0.f;
      int run = it.first_run, left = it.first_len;  // rows of the run from tile s on
      auto scores_ready = [&]() {
        if (!__all_sync(0xffffffffu, bar_wait(smem_u32(&bars.s_full[wg]), n_s & 1, wait_ns, abort_flag))) return false;
        ++n_s;
        tc_fence_after();
        return true;
      };
      auto probabilities_ready = [&]() {
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.p_full[wg]));
      };
      int s = 0;
      while (ok) {
        // tiles that every row sees whole
        const int whole = min(left / kTileRows, n - 1 - s);
        left -= whole * kTileRows;
        for (const int end = s + whole; s < end; ++s) {
          if (!(ok = scores_ready())) break;
          whole_row<D>(tS, tO, sl2, s == 0, m_ref, l_run);
          probabilities_ready();
        }
        if (!ok) break;
        const bool diagonal = s + 1 == n;
        if (left == 0) {  // (only before the diagonal: the next run)
          left = runs[++run].len;
          continue;
        }
        // the diagonal, where a row sees the columns up to its own, or a run's
        // short last tile, where it sees those up to the run's end (rows behind
        // that end, which are not stored, see what they like)
        if (!(ok = scores_ready())) break;
        edge_row<D>(tS, tO, sl2, s == 0, diagonal ? row + 1 : left, diagonal ? q4 + 1 : (left + 31) >> 5, m_ref, l_run);
        if (left < kTileRows) {
          // V's rows behind the run's end: zero (both tiles' warps do it, each
          // before its own product)
          const int st = step0 + s, gr = st + 1;
          if (!__all_sync(0xffffffffu, bar_wait(smem_u32(&bars.full[gr % C::kHalf]), (gr / C::kHalf) & 1, wait_ns,
                                                 abort_flag))) {
            tmem_wait_st();  // (P is on its way: TMEM is not freed before it is there)
            ok = false;
            break;
          }
          if (row >= left) {
            const uint32_t v = sKV + (2 * st + 1) % C::kSlots * C::kTileBytes + row * 128;
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
#pragma unroll
              for (int c = 0; c < 8; ++c) st_shared_v4(v + i * C::kPanelBytes + 16 * c, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        probabilities_ready();
        ++s;
        if (diagonal) break;
        left = runs[++run].len;
      }
      if (!ok) break;
      // ---- epilogue
      const int shard = it.shard, first_row = it.row0;
      const int tile = p.cut.pair ? it.tile : it.tile + wg, head = p.cut.pair ? it.head + wg : it.head;
      const int row0 = tile * kTileRows + q4 * 32;  // the warp's first row inside the run
      const int rows = it.len - row0;               // the warp's rows that there are (may be 32 and more, or none)
      const int64_t row_bytes = static_cast<int64_t>(p.Hq) * D * 2;
      uint8_t* const base = p.out[shard] + (first_row + row0 + (lane >> 3)) * row_bytes +
                            static_cast<int64_t>(head) * D * 2 + (lane & 7) * 16;
      const int shard_rows = p.cut.shard_begin[shard + 1] - p.cut.shard_begin[shard];
      const float inv = 1.f / l_run;  // (a row has itself: l_run > 0, NaN inputs aside)
      if (!__all_sync(0xffffffffu, bar_wait(smem_u32(&bars.o_done[wg]), n_o & 1, wait_ns, abort_flag))) {
        ok = false;
        break;
      }
      ++n_o;
      tc_fence_after();
      uint32_t o[D / 32][32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) tmem_ld32(tO + 32 * c, o[c]);
      tmem_wait_ld();
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        // 64 columns of the warp's rows through shared memory: 16-byte piece c
        // of row r at piece c ^ (r mod 8); stored eight lanes a row
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t(&x)[32] = o[2 * h + c / 4];
          const int e = 8 * (c % 4);
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = pack_bf16x2(__uint_as_float(x[e + 2 * i]) * inv, __uint_as_float(x[e + 2 * i + 1]) * inv);
          st_shared_v4(stage + lane * 128 + ((c ^ (lane & 7)) << 4), v[0], v[1], v[2], v[3]);
        }
        __syncwarp();
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3);
          v[i] = ld_shared_v4(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
        }
        uint8_t* at = base + h * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i, at += 4 * row_bytes)
          if (4 * i + (lane >> 3) < rows &&
              in_bounds(&g_prompt_violations, first_row + row0 + 4 * i + (lane >> 3), 1, shard_rows))
            *reinterpret_cast<uint4*>(at) = v[i];
        __syncwarp();
      }
      if (p.lse_out && lane < rows && in_bounds(&g_prompt_violations, first_row + row0 + lane, 1, shard_rows))
        p.lse[shard][static_cast<int64_t>(first_row + row0 + lane) * p.Hq + head] =
            (m_ref + lg2_approx(l_run)) * 0.6931471805599453f;
    }
    idle = n > 0 ? 0 : max(it.n[0], it.n[1]);
    step0 += max(it.n[0], it.n[1]);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars.item_empty[slot]));
  }
  if (!ok) record_timeout(p, abort_flag);
}

template <int D>
__global__ void __launch_bounds__(320, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = PCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PBars bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = sbase, sKV = sbase + 2 * C::kTileBytes, sStage = sKV + C::kSlots * C::kTileBytes;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.q_full[i]), 1);
      mbar_init(smem_u32(&bars.q_empty[i]), 1);
      mbar_init(smem_u32(&bars.s_full[i]), 1);
      mbar_init(smem_u32(&bars.p_full[i]), 4);
      mbar_init(smem_u32(&bars.o_done[i]), 1);
    }
    for (int i = 0; i < C::kHalf; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 1);
      mbar_init(smem_u32(&bars.empty[i]), 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(smem_u32(&bars.item_full[i]), 1);
      mbar_init(smem_u32(&bars.item_empty[i]), 9);  // the softmax warps and the issuer
    }
    mbar_init(smem_u32(&bars.drain), 1);
    bars.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&bars.tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == 8 && p.direct) find_items(p.cut, p.n_hp, bars, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!p.direct) wait_for_previous_launch();  // the tables
  const uint32_t tmem = bars.tmem_base;
  const int n_items = p.direct ? (bars.unit[0].run >= 0) + (bars.unit[1].run >= 0) : p.cut.t.head[0] * p.n_hp;
  static_assert(kDirectItems == 2, "items are counted above");
  const PromptRun* const runs = p.direct ? bars.run : p.cut.t.runs;
  if ((p.direct ? 0 : static_cast<int>(blockIdx.x)) < n_items) {
    if (warp == 8) {
      if (lane == 0) producer<D>(p, bars, sQ, sKV, n_items, runs, p.wait_ns);
    } else if (warp == 9) {
      if (lane == 0) issuer<D>(p, bars, sQ, sKV, tmem, p.wait_ns);
    } else {
      softmax<D>(p, bars, sKV, sStage, tmem, runs, warp, lane, p.wait_ns);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const PromptParams& p, cudaStream_t s) {
  using C = PCfg<D>;
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!bit || !(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  if (p.direct) {
    prompt_kernel<D><<<p.cut.grid, C::kThreads, C::kSmem, s>>>(p);
    return cudaGetLastError();
  }
  tables_kernel<<<1, 1024, 0, s>>>(p.cut);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the attention's CTAs come up while the tables are written
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.cut.grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_kernel<D>, p);
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& p, int D, cudaStream_t s) {
  return D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace uly
