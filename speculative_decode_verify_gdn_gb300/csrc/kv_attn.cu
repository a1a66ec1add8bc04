// Attention of verify windows over the paged cache (contract in include/gdn_kv.h), on the tensor
// cores.
//
// Mathematics: softmax over a row's keys in one pass with a running maximum m and sum l, and joined
// over disjoint sets of keys by their log-sum-exps: with (o_i, e_i) of set i,
// e = log sum exp(e_i), o = sum exp(e_i - e) o_i.  So a row's prefix, its own sequence and any
// pieces of either can be computed apart.
//
// The work is cut into items: (prefix run, kv head, block of up to 256 rows) for the prefixes, a
// run being consecutive sequences with the same prefix, and (sequence, kv head, block) for what a
// sequence does not share.  A row is one query head of one window token; a block's rows all meet
// the same keys, so the prefix is read and multiplied once for every sequence on it.  An item's
// keys come in tiles of 128.  Prefix items are in the order run, head, block; the sequences' in
// the order head, sequence, block, so that CTAs at work at the same time read the same tokens'
// other heads, which lie beside each other in memory (B=256 K=1: 163 us, 173 with a sequence's heads
// one after the other).  All tiles of all items, in order, are dealt to the CTAs (one per SM) in
// equal contiguous stretches: a CTA's part of an item is a segment, it yields the
// softmax-weighted sum and the log-sum-exp of its own keys (f32, in the workspace), and a last
// kernel joins a row's segments.  Few rows over a long axis are split over the card by that, and
// many over a short one are not.  Which CTA computes what depends on the lengths alone, and no
// sum is formed by atomics, so results repeat bit for bit.
//
// Kernels: plan (one CTA: lengths -> items and stretches; up to 32 sequences the tile kernel's
// schedulers do that), tiles (persistent, tcgen05), join.
//
// The tile kernel: a producer warp brings keys and values by TMA (128-byte swizzle) into a ring
// of tiles; a warp per stream issues S = Q K^T and O += P V (tcgen05, M = 128, accumulators in
// tensor memory, P read from tensor memory); one warp deals out segments and fetches their
// queries; two groups of four warps, one per stream, turn S into P, a row per thread.  A block of
// more rows than a tile's uses the two streams for its two halves on the same keys (32 KB of
// keys or values serve 256 rows, half the L2 traffic of one stream each); a smaller one gives them
// alternate tiles of the same rows.  While one stream's softmax runs, the tensor core works for
// the other.
//
// Measured on one GB300 (plan + tiles + join; peaks: 6796 GB/s copy, 1957 TFLOP/s cuBLAS bf16, 1733
// when the power cap sets the clock):
//   B=64 K=16 Hq=32 Hkv=4 D=128 behind 32768 tokens   383-409 us, 1350-1450 TFLOP/s: bound by the tensor
//     core's wait for a stream's chain (S, softmax, P, O), a tile pair every ~3000 cycles where its
//     products take 2048
//   B=1 K=16 Hq=32 Hkv=8 over 131072 tokens           94 us, 5710 GB/s: HBM, then the join
//   B=32 K=16 Hq=32 Hkv=8 behind 8192 + 1..2048       99-100 us: prefix tiles 45, own tiles 25 (latency
//     of a 5-tile ring), start, ends and join the rest
//   B=256 K=1 Hq=32 Hkv=8, 4 prefixes of 3001 + 5..1024  151 us, 3930 GB/s
//   B=1 K=1 over 700 tokens                           14-15 us: two dependent launches
// The loops over boxes and over scores are kept rolled: the kernel's code is more than the
// instruction cache holds, and unrolling them costs more in misses than it saves.
#include <atomic>

#include "kv_index.h"
#include "kv_kernels.h"
#include "kv_tile.cuh"

namespace gdn {

namespace {

constexpr int kPlanThreads = 512, kPlanRuns = 512;
constexpr int kJoinWarps = 4, kJoinRowsMax = 32;  // (four warps: four lists)

// ---------------------------------------------------------------- the plan
struct SeqRec {       // a sequence: what it does not share, and where its rows are in its prefix run
  long long off;      // its first tile among those of one kv head
  long long pre_off;  // the run's first tile
  long long pre_row;  // the run's first row of partial results
  long long pre_rows; // the run's rows per kv head
  long long pre_at;   // the sequence's first of them
  int32_t tiles;      // per item (0: nothing to do)
  int32_t pre_tiles;  // per item of the run (0: no prefix)
  int32_t keys;       // cached tokens
  int32_t win;        // window tokens, clamped to 0..K
};
struct RunRec {       // consecutive sequences on one prefix
  long long off;
  long long row;
  int32_t tiles;
  int32_t keys;
  int32_t slot;
  int32_t b0, n;      // sequences b0 .. b0 + n - 1
  int32_t pad[3];
};
struct PlanHead {
  long long tiles, prefix_tiles;  // in all; those of the runs come first
  long long own_row;              // first row of the sequences' partial results
  long long head_tiles;           // the sequences' tiles of one kv head
  int32_t runs;
  int32_t split;                  // prefixes and sequences are dealt out apart from each other
};
struct StartRec {
  int32_t own, idx;  // where a stretch begins: run or sequence idx
};

struct AttnWs {
  PlanHead* head;
  StartRec* start;  // [2][kCtas]
  SeqRec* seq;      // [B]
  RunRec* run;      // [B]
  float* lse;       // [rows] log2 units
  float* o;         // [rows, D]
};

__host__ __device__ inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Rows of partial results of a block, with `tile` rows to a stream: one per row when the streams
// hold its halves, else two (one per stream).
__host__ __device__ inline int block_width(int rows, int tile) { return rows > tile ? rows : 2 * rows; }
// Rows of partial results of all blocks of `rows` rows.
template <typename T>
__host__ __device__ inline T rows_width(T rows, int tile) {
  const T full = (rows - 1) / (2 * tile);
  return full * 2 * tile + block_width(int(rows - full * 2 * tile), tile);
}

__host__ __device__ inline AttnWs carve_attn(void* base, const gdn_kv_dims& d, size_t* total) {
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t o = 0;
  // a segment of CTA c and item i starts at row 256 c + (rows of the items before i); every row of
  // the batch has at most two rows here from its prefix and two from its own sequence
  const size_t rows = 2 * size_t(kBlockRows) * kCtas + 4 * size_t(d.B) * d.K * d.Hq;
  AttnWs w;
  w.head = reinterpret_cast<PlanHead*>(p + o), o += 256;
  w.start = reinterpret_cast<StartRec*>(p + o), o += up256(2 * sizeof(StartRec) * kCtas);
  w.seq = reinterpret_cast<SeqRec*>(p + o), o += up256(sizeof(SeqRec) * size_t(d.B));
  w.run = reinterpret_cast<RunRec*>(p + o), o += up256(sizeof(RunRec) * size_t(d.B));
  w.lse = reinterpret_cast<float*>(p + o), o += up256(4 * rows);
  w.o = reinterpret_cast<float*>(p + o), o += 4 * rows * size_t(d.D);
  if (total) *total = o;
  return w;
}

// A deal gives CTA c tiles [first_tile(c), first_tile(c + 1)) of `tiles`; the CTA of tile x.
//
// With at least kSplitTiles tiles, the prefixes' and the sequences' are two deals, and every CTA
// gets its share of both - even CTAs in this order, odd ones in the other: a prefix tile costs
// tensor-core time and a sequence's tile memory time, so a CTA that had one kind alone would end
// early or late, and at any time half the CTAs wait for memory while half compute.  With fewer,
// one deal over all tiles puts them on as many CTAs as there are.  (B=64 behind 32768 tokens: 543 us in
// two deals, 849 in one.)
constexpr long long kSplitTiles = 4 * kCtas;
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* sums, T& total) {  // exclusive, kPlanThreads threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  T s = lane < kPlanThreads / 32 ? sums[lane] : T(0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const T before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return x - v + (warp > 0 ? before : 0);
}

// A slot's length, 0 (and a status bit) when it is negative or beyond the table's columns.
__device__ __forceinline__ int slot_len(const AttnParams& p, int slot) {
  const int n = p.seq_len[slot];
  if (n < 0 || (long long)n > (long long)p.d.max_pages * p.d.page_size) {
    atomicOr(p.err, GDN_DEVERR_KV_LEN);
    return 0;
  }
  return n;
}

__device__ __forceinline__ int prefix_slot(const AttnParams& p, int b) {
  if (!p.prefix_of) return -1;
  const int s = p.prefix_of[b];
  return s < 0 || s >= p.d.n_slots ? -1 : s;
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnWs w) {
  __shared__ long long sums[32];
  // runs and first tiles, where they fit here: what one step of the plan hands to the next would
  // otherwise be a trip to L2
  __shared__ RunRec runs[kPlanRuns];
  __shared__ long long seq_off[kPlanThreads];
  pdl_launch_dependents();
  pdl_wait();
  const gdn_kv_dims& d = p.d;
  const int tid = int(threadIdx.x), KG = d.K * (d.Hq / d.Hkv);
  long long n_runs = 0;
  auto run_at = [&](long long r) -> RunRec& { return r < kPlanRuns ? runs[r] : w.run[r]; };
  // (one step of threads, the usual case, keeps what it knows of its sequence for the steps below)
  const bool once = d.B <= kPlanThreads;
  int win = 0, keys = 0, slot = -1;
  long long run = -1;
  for (int b0 = 0; b0 < d.B; b0 += kPlanThreads) {  // sequences: lengths, and the runs' ends
    const int b = b0 + tid;
    bool first = false, last = false;
    int run_keys = 0;
    win = 0, keys = 0, slot = -1;
    if (b < d.B) {
      const int before = b > 0 ? prefix_slot(p, b - 1) : -1, after = b + 1 < d.B ? prefix_slot(p, b + 1) : -1;
      slot = prefix_slot(p, b);
      keys = slot_len(p, d.slot0 + b);
      win = p.win_len ? p.win_len[b] : d.K;
      if (win < 0 || win > d.K) {
        atomicOr(p.err, GDN_DEVERR_KV_WINDOW);
        win = win < 0 ? 0 : d.K;
      }
      if (slot < 0 && p.prefix_of && p.prefix_of[b] != -1) atomicOr(p.err, GDN_DEVERR_KV_SLOT);
      first = slot >= 0 && before != slot;
      last = slot >= 0 && after != slot;
      if (first) run_keys = slot_len(p, slot);
    }
    long long total;
    run = n_runs + block_scan<long long>(first ? 1 : 0, sums, total) - (first ? 0 : 1);
    if (slot < 0) run = -1;
    if (b < d.B) {
      if (!once) {
        w.seq[b].keys = keys;
        w.seq[b].win = win;
        w.seq[b].pre_off = run;  // (for now)
      }
      if (first) {
        RunRec x{};
        x.b0 = b;
        x.slot = slot;
        x.keys = run_keys;
        x.tiles = (run_keys + kTileKeys - 1) / kTileKeys;
        run_at(run) = x;
      }
    }
    __syncthreads();
    if (last) run_at(run).n = b + 1;  // (its end; the length follows)
    n_runs += total;
  }
  __syncthreads();
  long long tiles = 0, row = 0;
  for (int r0 = 0; r0 < n_runs; r0 += kPlanThreads) {
    const int r = r0 + tid;
    long long mine = 0, rows = 0;
    RunRec x{};
    if (r < n_runs) {
      x = run_at(r);
      x.n -= x.b0;
      const long long block = (long long)x.n * KG;
      mine = (block + 2 * p.tile_rows - 1) / (2 * p.tile_rows) * d.Hkv * x.tiles;
      rows = d.Hkv * rows_width(block, p.tile_rows);
    }
    long long total, total_rows;
    x.off = tiles + block_scan<long long>(mine, sums, total);
    x.row = row + block_scan<long long>(rows, sums, total_rows);
    if (r < n_runs) {
      w.run[r] = x;
      if (r < kPlanRuns) runs[r] = x;
    }
    tiles += total;
    row += total_rows;
  }
  __syncthreads();
  const long long prefix_tiles = tiles;
  const int own_blocks = (KG + 2 * p.tile_rows - 1) / (2 * p.tile_rows);
  long long head_tiles = 0;
  for (int b0 = 0; b0 < d.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    SeqRec q{};
    if (b < d.B) {
      if (!once) win = w.seq[b].win, keys = w.seq[b].keys, run = w.seq[b].pre_off;
      q.keys = keys;
      q.win = win;
      q.tiles = win > 0 ? ((keys + 15) / 16 + 1 + 7) / 8 : 0;  // units of 16 keys; the window is one unit
      if (run >= 0) {
        const RunRec r = run_at(run);
        q.pre_off = r.off;
        q.pre_row = r.row;
        q.pre_rows = (long long)r.n * KG;
        q.pre_at = (long long)(b - r.b0) * KG;
        q.pre_tiles = r.tiles;
      }
    }
    long long total;
    q.off = head_tiles + block_scan<long long>((long long)own_blocks * q.tiles, sums, total);
    if (b < d.B) w.seq[b] = q;
    if (once) seq_off[tid] = q.off;
    head_tiles += total;
  }
  tiles += head_tiles * d.Hkv;
  const bool split = tiles >= kSplitTiles;
  if (tid == 0) {
    w.head->tiles = tiles;
    w.head->prefix_tiles = prefix_tiles;
    w.head->own_row = row + (split ? kBlockRows * kCtas : 0);
    w.head->runs = int(n_runs);
    w.head->split = split;
    w.head->head_tiles = head_tiles;
  }
  __syncthreads();
  if (tid < 2 * kCtas) {  // where each stretch begins: the last record that starts at or before it
    const int own = tid / kCtas, c = tid % kCtas;
    const long long x = !split ? first_tile(c, tiles) : own ? prefix_tiles + first_tile(c, tiles - prefix_tiles) : first_tile(c, prefix_tiles);
    StartRec s{0, 0};
    if (x < tiles) {
      s.own = x >= prefix_tiles;
      const long long y = s.own ? (x - prefix_tiles) % head_tiles : x;
      int lo = 0, hi = (s.own ? d.B : int(n_runs)) - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if ((!s.own ? run_at(mid).off : once ? seq_off[mid] : w.seq[mid].off) <= y)
          lo = mid;
        else
          hi = mid - 1;
      }
      s.idx = lo;
    }
    w.start[tid] = s;
  }
}

// ---------------------------------------------------------------- segments
struct Seg {
  int own, idx, h, row0, rows;  // rows row0 .. row0 + rows - 1 of the run's or sequence's rows
  int pair;                     // they fill more than one row tile: both streams take every tile of keys
  int tok0;                     // its first window token (of all B K)
  int slot, keys, win;          // cached tokens; own: window tokens (prefix: -1)
  int units;                    // of 16 keys, the window's included
  int t0, t1;                   // tiles of the item
  int parity;                   // of tile t0 in the order of all tiles
  long long part;               // first row of its partial results
  __device__ __forceinline__ bool paired() const { return pair != 0; }
  struct Tiles {
    int all;
    __device__ __forceinline__ int units(int t) const { return all - 8 * t < 8 ? all - 8 * t : 8; }
  };
  __device__ __forceinline__ Tiles tiles() const { return Tiles{int(uniform(uint32_t(units)))}; }  // (a converged warp)
};

// The plan of a batch of at most 32 sequences, by one converged warp: lane b has sequence b's record
// and lane r run r's.  The tile kernel's scheduler makes it for itself, which saves the plan kernel's
// launch (B=1 decode: 17.1 us with it, 14.8 without).
constexpr int kWarpPlan = 32;
__device__ __forceinline__ long long warp_scan(long long v, int lane, long long& total) {  // exclusive
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  total = __shfl_sync(0xffffffffu, x, 31);
  return x - v;
}
__device__ __forceinline__ void warp_plan(const AttnParams& p, int lane, PlanHead& head, SeqRec& q, RunRec& r) {
  const gdn_kv_dims& d = p.d;
  const int KG = d.K * (d.Hq / d.Hkv), block = 2 * p.tile_rows;
  const bool there = lane < d.B;
  q = SeqRec{};
  r = RunRec{};
  int slot = -1;
  if (there) {
    slot = prefix_slot(p, lane);
    if (slot < 0 && p.prefix_of && p.prefix_of[lane] != -1) atomicOr(p.err, GDN_DEVERR_KV_SLOT);
    q.keys = slot_len(p, d.slot0 + lane);
    q.win = p.win_len ? p.win_len[lane] : d.K;
    if (q.win < 0 || q.win > d.K) {
      atomicOr(p.err, GDN_DEVERR_KV_WINDOW);
      q.win = q.win < 0 ? 0 : d.K;
    }
    q.tiles = q.win > 0 ? ((q.keys + 15) / 16 + 1 + 7) / 8 : 0;  // units of 16 keys; the window is one unit
  }
  const int before = __shfl_up_sync(0xffffffffu, slot, 1), after = __shfl_down_sync(0xffffffffu, slot, 1);
  const uint32_t firsts = __ballot_sync(0xffffffffu, slot >= 0 && (lane == 0 || before != slot));
  const uint32_t lasts = __ballot_sync(0xffffffffu, slot >= 0 && (lane == 31 || after != slot));
  const int runs = __popc(firsts);
  const int b0 = lane < runs ? int(__fns(firsts, 0, lane + 1)) : 0;
  r.slot = __shfl_sync(0xffffffffu, slot, b0);
  long long mine = 0, rows = 0;
  if (lane < runs) {
    r.b0 = b0;
    r.n = int(__fns(lasts, 0, lane + 1)) + 1 - b0;
    r.keys = slot_len(p, r.slot);
    r.tiles = (r.keys + kTileKeys - 1) / kTileKeys;
    const long long all = (long long)r.n * KG;
    mine = (all + block - 1) / block * d.Hkv * r.tiles;
    rows = d.Hkv * rows_width(all, p.tile_rows);
  }
  long long prefix_tiles, prefix_rows, head_tiles;
  r.off = warp_scan(mine, lane, prefix_tiles);
  r.row = warp_scan(rows, lane, prefix_rows);
  q.off = warp_scan((long long)((KG + block - 1) / block) * q.tiles, lane, head_tiles);
  const int run = slot >= 0 ? __popc(firsts & ((2u << lane) - 1u)) - 1 : 0;
  const long long run_off = __shfl_sync(0xffffffffu, r.off, run), run_row = __shfl_sync(0xffffffffu, r.row, run);
  const int run_n = __shfl_sync(0xffffffffu, r.n, run), run_b0 = __shfl_sync(0xffffffffu, r.b0, run);
  const int run_tiles = __shfl_sync(0xffffffffu, r.tiles, run);
  if (slot >= 0) {
    q.pre_off = run_off;
    q.pre_row = run_row;
    q.pre_rows = (long long)run_n * KG;
    q.pre_at = (long long)(lane - run_b0) * KG;
    q.pre_tiles = run_tiles;
  }
  head.prefix_tiles = prefix_tiles;
  head.tiles = prefix_tiles + head_tiles * d.Hkv;
  head.split = head.tiles >= kSplitTiles;
  head.own_row = prefix_rows + (head.split ? kBlockRows * kCtas : 0);
  head.head_tiles = head_tiles;
  head.runs = runs;
}

// Walks a CTA's stretch segment by segment (a converged warp).
struct SegWalk {
  const AttnParams& p;
  const AttnWs& w;
  const bool small;  // the plan is the warp's own
  PlanHead head;
  SeqRec my_seq;
  RunRec my_run;
  long long x, end;
  int own, idx, h, cta, deal;  // (h: kv head of the sequences' items)
  __device__ __forceinline__ SegWalk(const AttnParams& p_, const AttnWs& w_, int cta_, int lane)
      : p(p_), w(w_), small(p_.d.B <= kWarpPlan), cta(cta_) {
    if (small) {
      warp_plan(p, lane, head, my_seq, my_run);
      if (cta == 0) {  // for the join
        if (lane < p.d.B) w.seq[lane] = my_seq;
        if (lane == 0) *w.head = head;
      }
    } else {
      head = *w.head;
    }
    deal = 0;
    begin();
  }
  // The last record that starts at or before a stretch's first tile (the plan kernel has looked for it).
  __device__ __forceinline__ StartRec start(int which) const {
    if (!small) return w.start[which * kCtas + cta];
    StartRec s{0, 0};
    if (x < head.tiles) {
      s.own = x >= head.prefix_tiles;
      const long long y = s.own ? (x - head.prefix_tiles) % head.head_tiles : x;
      const uint32_t at = s.own ? __ballot_sync(0xffffffffu, (threadIdx.x & 31) < unsigned(p.d.B) && my_seq.off <= y)
                                : __ballot_sync(0xffffffffu, (threadIdx.x & 31) < unsigned(head.runs) && my_run.off <= y);
      s.idx = 31 - __clz(int(at));
    }
    return s;
  }
  __device__ __forceinline__ void begin() {  // the CTA's stretch of its first or second deal
    const int which = head.split ? deal ^ (cta & 1) : 0;
    if (head.split) {
      const long long o = which ? head.prefix_tiles : 0, n = which ? head.tiles - head.prefix_tiles : head.prefix_tiles;
      x = o + first_tile(cta, n), end = o + first_tile(cta + 1, n);
    } else {
      x = deal ? 0 : first_tile(cta, head.tiles), end = deal ? 0 : first_tile(cta + 1, head.tiles);
    }
    const StartRec s = start(which);
    own = s.own, idx = s.idx;
    h = own && x < end ? int((x - head.prefix_tiles) / head.head_tiles) : 0;
  }
  __device__ __forceinline__ SeqRec seq(int i) const {
    if (!small) return w.seq[i];
    SeqRec q{};
    q.off = __shfl_sync(0xffffffffu, my_seq.off, i);
    q.tiles = __shfl_sync(0xffffffffu, my_seq.tiles, i);
    q.keys = __shfl_sync(0xffffffffu, my_seq.keys, i);
    q.win = __shfl_sync(0xffffffffu, my_seq.win, i);
    return q;
  }
  __device__ __forceinline__ RunRec run(int i) const {
    if (!small) return w.run[i];
    RunRec r{};
    r.off = __shfl_sync(0xffffffffu, my_run.off, i);
    r.row = __shfl_sync(0xffffffffu, my_run.row, i);
    r.tiles = __shfl_sync(0xffffffffu, my_run.tiles, i);
    r.keys = __shfl_sync(0xffffffffu, my_run.keys, i);
    r.slot = __shfl_sync(0xffffffffu, my_run.slot, i);
    r.b0 = __shfl_sync(0xffffffffu, my_run.b0, i);
    r.n = __shfl_sync(0xffffffffu, my_run.n, i);
    return r;
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (x >= end && deal == 0) deal = 1, begin();
    if (x >= end) return false;
    const gdn_kv_dims& d = p.d;
    const int KG = d.K * (d.Hq / d.Hkv);
    while (true) {
      if (!own && idx == head.runs) own = 1, idx = 0;
      if (own && idx >= d.B) {  // the next head's
        if (++h >= d.Hkv) return false;
        idx = 0;
      }
      long long off, rows, row;
      int tiles;
      if (own) {
        const SeqRec q = seq(idx);
        off = head.prefix_tiles + h * head.head_tiles + q.off, tiles = q.tiles, rows = KG;
        row = head.own_row + ((long long)h * d.B + idx) * rows_width(KG, p.tile_rows);
        s.slot = d.slot0 + idx, s.keys = q.keys, s.win = q.win, s.tok0 = idx * d.K;
        s.units = (q.keys + 15) / 16 + 1;
      } else {
        const RunRec r = run(idx);
        off = r.off, tiles = r.tiles, rows = (long long)r.n * KG, row = r.row;
        s.slot = r.slot, s.keys = r.keys, s.win = -1, s.tok0 = r.b0 * d.K;
        s.units = (r.keys + 15) / 16;
      }
      const int block = 2 * p.tile_rows;
      const int blocks = int((rows + block - 1) / block);
      const long long items = own ? blocks : (long long)blocks * d.Hkv;
      if (tiles == 0 || x >= off + items * tiles) {
        ++idx;
        continue;
      }
      const int item = int((x - off) / tiles);
      s.own = own, s.idx = idx;
      const int ph = own ? 0 : item / blocks, rb = item - ph * blocks;
      s.h = own ? h : ph;
      s.row0 = rb * block;
      s.rows = int(rows - s.row0 < block ? rows - s.row0 : block);
      s.pair = s.rows > p.tile_rows;
      s.t0 = int(x - off - (long long)item * tiles);
      const long long left = end - x;
      s.t1 = left < tiles - s.t0 ? s.t0 + int(left) : tiles;
      s.parity = int(x & 1);
      s.part = (long long)kBlockRows * cta + row + ph * rows_width(rows, p.tile_rows) + s.row0;
      x += s.t1 - s.t0;
      return true;
    }
  }
};

// ---------------------------------------------------------------- the tile kernel
struct TileMaps {
  // (D, token, kv head, page or sequence, layer), keys and values: boxes of 16 tokens of the cache, of
  // `box` tokens of it, and of 16 tokens of the window
  CUtensorMap few[2], many[2], window[2];
  // queries, (D, query head, token): boxes of G heads x the tokens of a row tile, and of a sequence's
  CUtensorMap qt, qs;
};

template <int D, bool F16>
__global__ void __launch_bounds__(kTileThreads, 1)
    attn_tile_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnWs w, const int box, const __grid_constant__ TileMaps maps) {
  using L = TileLayout<D, Seg>;
  constexpr int NS = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ int page_of_box[32][2];
  __shared__ volatile uint32_t gave_up, turns[2];  // (turns: taken so far by each tensor-core warp)
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - smem_addr(smem_raw));
  const TileBars bars = tile_bars<NS>(reinterpret_cast<uint64_t*>(smem + L::OFF_BAR));
  uint64_t *const full = bars.full, *const empty = bars.empty, *const q_ready = bars.q_ready, *const s_ready = bars.s_ready,
           *const p_ready = bars.p_ready, *const o_done = bars.o_done, *const q_free = bars.q_free, *const seg_full = bars.seg_full,
           *const seg_empty = bars.seg_empty;
  Seg* const segs = reinterpret_cast<Seg*>(smem + L::OFF_SEG);
  const int tid = int(threadIdx.x), warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const gdn_kv_dims& d = p.d;
  const int G = d.Hq / d.Hkv;

  if (tid == 0) {
    init_tile_bars<NS>(bars, 2);
    turns[0] = turns[1] = 0;
    gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(&tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  // Bounded wait of a whole warp, which goes on or gives up together; once one warp has given up,
  // all of the CTA's do.  (Every branch is on a vote: the tensor-core warp's operands stay in
  // uniform registers only as long as the compiler can see that its lanes stay together.)
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    for (uint32_t i = 0; !__all_sync(0xffffffffu, mbar_sleep(bar, parity)); ++i) {
      if (__any_sync(0xffffffffu, gave_up || i > kMaxLooks)) {
        if (i > kMaxLooks) {
          gave_up = 1;
          atomicOr(p.err, kDevErrTimeout);
        }
        return false;
      }
    }
    return true;
  };

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    // Copies go out as slots fall free; the page numbers of the tile behind are on their way to shared
    // memory meanwhile (into a register, the warp would wait for them at its next instruction).
    // Small pages make many copies (16 tokens each: 32 a tile of keys and values), so all that a copy
    // needs is in uniform registers when its turn comes; lane i looks up box i.
    uint32_t n = 0, issued = 0;  // tiles and ring uses so far; tile n's keys are use 2n, its values 2n + 1
    uint32_t k = 0;              // segments so far
    int t = 0, t1 = 0;           // of the present segment: next tile, end
    bool ok = true, more = true;
    uint32_t slot = 0, phase = 1;  // of the next use; the phase that its slot was emptied in
    // the segment at hand
    int seg_units = 0, seg_cached = 0, seg_h = 0, seg_b = 0;
    const int32_t* seg_pages = nullptr;
    // the tile behind the one at hand
    int units = 0, boxes = 0, in = 0;
    uint32_t ahead = 0;     // tiles looked up
    bool whole = false;     // all from the cache, in boxes of `box` tokens
    int window = -1;        // the unit that is the window (-1: none)
    int* const page = page_of_box[lane];  // of this tile and the next in turn
    auto next_tile = [&]() {
      while (ok && t == t1) {
        __syncwarp();
        if (k > 0 && lane == 0) mbar_arrive(seg_empty + (k - 1) % kSegRing);
        ok = wait_warp(seg_full + k % kSegRing, (k / kSegRing) & 1);
        const Seg& seg = segs[k % kSegRing];
        t = int(uniform(uint32_t(seg.t0))), t1 = int(uniform(uint32_t(seg.t1)));
        ++k;
        if (t1 < 0) more = false;
        if (t1 < 0 || !ok) return;
        seg_units = int(uniform(uint32_t(seg.units))), seg_cached = int(uniform(uint32_t((seg.keys + 15) >> 4)));
        seg_h = int(uniform(uint32_t(seg.h))), seg_b = int(uniform(uint32_t(seg.idx)));
        seg_pages = p.table + (long long)seg.slot * d.max_pages;
      }
      if (!ok) return;
      units = seg_units - 8 * t < 8 ? seg_units - 8 * t : 8;
      const int cached = seg_cached - 8 * t;  // units of this tile from the cache (may exceed 8)
      whole = cached >= 8;
      window = !whole && units > cached ? cached : -1;  // (the window is the unit behind the cached ones)
      boxes = whole ? kTileKeys / box : units;
      if (lane < boxes && lane != window) {
        const int token = t * kTileKeys + lane * (whole ? box : 16);
        const int col = page_column(token, p.page_inv);
        in = token - col * d.page_size;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(page + (ahead & 1))), "l"(seg_pages + col) : "memory");
      }
      ++t, ++ahead;
    };
    next_tile();
    while (ok && more) {
      const int now_units = units, now_boxes = boxes, now_in = in, now_window = window, now_h = seg_h, now_b = seg_b;
      const bool now_whole = whole;
      asm volatile("cp.async.wait_all;" ::: "memory");
      int now_page = page[n & 1];
      if (lane < now_boxes && lane != now_window && (now_page < 0 || now_page >= d.n_pages)) {  // reads zeros there
        atomicOr(p.err, GDN_DEVERR_KV_PAGE);
        now_page = d.n_pages;
      }
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        if (!wait_warp(empty + slot, phase)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(full + slot, uint32_t(now_units) * 16 * D * 2);
        __syncwarp();
        const uint32_t dst = base + L::OFF_RING + slot * L::BYTES, bar = smem_addr(full + slot), step = uint32_t(now_whole ? box : 16) * 128;
        const CUtensorMap* const m = now_whole ? &maps.many[v] : &maps.few[v];
#pragma unroll 1
        for (int b = 0; b < now_boxes; ++b) {
          const bool win = b == now_window;
          const int c1 = win ? 0 : int(uniform_from(uint32_t(now_in), b)), c3 = win ? now_b : int(uniform_from(uint32_t(now_page), b));
          tma_box<D>(dst + b * step, win ? &maps.window[v] : m, c1, now_h, c3, win ? 0 : p.layer, bar);
        }
        issued = 2 * n + v + 1;
        if (++slot == NS) slot = 0, phase ^= 1;
        if (v == 0) next_tile();
        if (!ok) break;
      }
      ++n;
    }
    // the last uses of the ring: the copies have landed and the tensor core has read them
    for (uint32_t use = issued > NS ? issued - NS : 0; use < issued; ++use) {
      if (ok) ok = wait_warp(empty + use % NS, (use / NS) & 1);
      if (!ok) mbar_drain(full + use % NS, (use / NS) & 1);
    }
  } else if (warp == 9 || warp == 10) {
    tensor_warp<D, F16>(warp - 9, lane, tmem, base, p.scale < 0.f, segs, bars, turns, wait_warp);
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax: stream s, one row per thread
    const int s = warp >> 2, r = tid & 127;
    const uint32_t lane_sel = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + tmem_s(s) + lane_sel, to = tmem + tmem_o(s) + lane_sel;
    const float c = fmaxf(fabsf(p.scale) * kLog2e, 1e-30f);  // (0 is as good as 1e-30)
    uint32_t n = 0, ns = 0, no = 0;  // tiles of the CTA, tiles of this stream, its segments
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      const Seg& seg = segs[k % kSegRing];
      if (!wait_warp(seg_full + k % kSegRing, (k / kSegRing) & 1)) {
        ok = false;
        break;
      }
      auto done = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty + k % kSegRing);
      };
      if (seg.t1 < 0) break;
      const bool paired = seg.paired();
      const uint32_t n0 = n;
      n += uint32_t(seg.t1 - seg.t0);
      int t = seg.t0;
      if (!paired && ((seg.parity ^ s) & 1)) ++t;
      if (t >= seg.t1) {
        done();
        continue;
      }
      const int step = paired ? 1 : 2;
      const int srow0 = paired ? s * p.tile_rows : 0;
      const int rows = seg.rows - srow0 < p.tile_rows ? seg.rows - srow0 : p.tile_rows;
      const bool idle = 32 * (warp & 3) >= rows;  // a warp without rows only keeps the barriers going

      uint32_t seen = 0;  // own: the window tokens that this row sees
      if (seg.own && seg.t1 == (seg.units + 7) / 8) {
        // each lane holds a node's parent; four doublings reach every ancestor of 16 nodes
        uint32_t anc = 0;
        if (p.parent) {
          int up = -1;
          if (lane < seg.win) {  // (a padding token has no parent)
            up = p.parent[(long long)seg.idx * d.K + lane];
            if (up < -1 || up >= lane) {
              atomicOr(p.err, kDevErrTreeParent);
              up = -1;
            }
          }
          anc = 1u << lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a = __shfl_sync(0xffffffffu, anc, up & 31);
            const int g = __shfl_sync(0xffffffffu, up, up & 31);
            if (up >= 0) anc |= a, up = g;
          }
        } else {
          anc = (2u << lane) - 1u;
        }
        const int tok = ((seg.row0 + srow0 + r) / G) % d.K;
        seen = __shfl_sync(0xffffffffu, anc, tok & 31) & ((1u << seg.win) - 1u);
      }

      float m = -INFINITY, l = 0.f;  // running maximum (unscaled) and sum
      bool first = true;
      for (; ok && t < seg.t1; t += step, ++ns) {
        if (!wait_warp(s_ready + s, ns & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int units = seg.units - 8 * t < 8 ? seg.units - 8 * t : 8;
        const int cached = seg.keys - t * kTileKeys;  // keys of this tile from the cache (may exceed 128)
        if (!idle) {
          const int wu = (cached + 15) & ~15;  // the window's unit (own; behind the tile for a prefix)
          softmax_tile<D, F16>(ts, to, c, r < rows, first, cached < kTileKeys, [&](int q, int g) {
            const int n_seen = cached - 64 * q - 32 * g;
            uint32_t see = n_seen >= 32 ? 0xffffffffu : n_seen <= 0 ? 0u : (1u << n_seen) - 1u;
            if (seg.own && (wu >> 5) == 2 * q + g) see |= seen << (wu & 31);
            return see;
          }, [] {}, m, l);  // (a tile's scores come behind the products of the tile before)
        }
        first = false;
        if (cached < kTileKeys && (seg.own || (cached & 15))) {
          // values behind the last cached token of its unit, and behind the window's last token, are
          // not the batch's: zero them, for 0 x NaN is NaN
          const uint32_t use = 2 * (n0 + uint32_t(t - seg.t0)) + 1, slot = use % NS;
          if (!wait_warp(full + slot, (use / NS) & 1)) {
            ok = false;
            break;
          }
          const int tail = cached > 0 ? cached : 0, wu = (tail + 15) / 16 * 16;
          const int end = units * 16;
          uint8_t* const v_tile = smem + L::OFF_RING + slot * L::BYTES;
          constexpr int C = D / 8;
          for (int i = r; i < (end - tail) * C; i += kGroupThreads) {
            const int row = tail + i / C, ch = i % C;
            if (row >= wu && row < wu + seg.win) continue;
            *reinterpret_cast<uint4*>(v_tile + (ch >> 3) * L::HALF + row * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(p_ready + s);
      }
      if (!ok) break;

      // the segment's result: O / l and the log-sum-exp in powers of two
      if (!wait_warp(o_done + s, no & 1)) {
        ok = false;
        break;
      }
      ++no;
      tc_fence_after();
      if (!idle) {
        const long long part = seg.part + (paired ? srow0 : s * seg.rows) + r;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float* const out = w.o + part * D;
#pragma unroll 1
        for (int q = 0; q < D; q += 32) {
          float o[32];
          tmem_ld32(to + q, o);
          if (r < rows) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= inv;
#pragma unroll
            for (int j = 0; j < 32; j += 8) store8(out + q + j, o + j);
          }
        }
        if (r < rows) w.lse[part] = l == 0.f ? -INFINITY : m * c + log2f(l);
      }
      tc_fence_before();
      done();
    }
  }
  else if (warp == 11) {
    // ------------------------------------------------------------ segments and queries, ahead of the rest
    // Walks the CTA's stretches and hands segments on as the ring has room, and fetches a segment's
    // queries as soon as the products with the ones before are done - whichever comes first.  Queries
    // come by TMA, whole tokens of G heads: rows behind the block's last hold other tokens' queries or
    // what was there, and nothing reads their results.
    SegWalk walk(p, w, int(blockIdx.x), lane);
    uint32_t k = 0, kq = 0;      // segments handed on; segment whose queries are next
    uint32_t nq0 = 0, nq1 = 0;   // segments of each stream
    int part = 0;                // of segment kq: its first or second stream
    uint32_t idle = 0;
    bool more = true, ok = true;
    while (ok && (more || kq < k)) {
      bool did = false;
      if (more && __all_sync(0xffffffffu, mbar_look(seg_empty + k % kSegRing, ((k / kSegRing) & 1) ^ 1))) {
        Seg seg;
        more = walk.next(seg);
        if (lane == 0) {
          if (!more) seg.t1 = -1;
          segs[k % kSegRing] = seg;
          mbar_arrive(seg_full + k % kSegRing);
        }
        __syncwarp();
        if (more) ++k;
        did = true;
      }
      if (kq < k) {
        const Seg& seg = segs[kq % kSegRing];
        const bool paired = seg.paired();
        const int s = paired ? part : (seg.parity + part) & 1;  // in the order of their first tiles
        const uint32_t nq = s ? nq1 : nq0;
        if (nq == 0 || __all_sync(0xffffffffu, mbar_look(q_free + s, (nq - 1) & 1))) {
          const int toks = seg.own && d.K < p.tile_toks ? d.K : p.tile_toks;
          if (lane == 0) mbar_arrive_expect_tx(q_ready + s, uint32_t(toks * G) * D * 2);
          __syncwarp();
          if (lane < D / 64)
            tma_load3(base + L::OFF_Q + s * L::BYTES + lane * L::HALF, seg.own ? &maps.qs : &maps.qt, lane * 64, seg.h * G,
                      seg.tok0 + seg.row0 / G + (paired ? s * p.tile_toks : 0), smem_addr(q_ready + s));
          if (s)
            ++nq1;
          else
            ++nq0;
          if (++part == 2 || (!paired && seg.t1 - seg.t0 == 1)) {
            part = 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(seg_empty + kq % kSegRing);
            ++kq;
          }
          did = true;
        }
      }
      idle = did ? 0 : idle + 1;
      if (__any_sync(0xffffffffu, gave_up || idle > kMaxIdle)) {
        if (idle > kMaxIdle) {
          gave_up = 1;
          atomicOr(p.err, kDevErrTimeout);
        }
        ok = false;
      }
    }
    // (the tensor core waits for every tile of queries; after a wait that gave up, they land first)
    if (!ok) {
      if (nq0 > 0) mbar_drain(q_ready, (nq0 - 1) & 1);
      if (nq1 > 0) mbar_drain(q_ready + 1, (nq1 - 1) & 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- join
// One CTA per (sequence, kv head, 4 to 32 of its rows): the segments of the sequence and of its prefix,
// weighted by their log-sum-exps.  Where the segments are follows from the plan and is listed once
// per CTA; then a warp takes a row at a time, without a division (document batch of the file's head:
// 384 us, 392 with 64-bit divisions by the block's rows for every row).  Bound by the latency of its loads (lengths, then
// log-sum-exps, then sums): the sums of a row are read together, and a CTA takes as many rows as
// leave eight CTAs to an SM, 4 at least (the whole call at B=32 K=16 behind 8192 tokens: 106 us, 117
// with two CTAs to an SM, 109 with sixteen; at B=1 K=16 with 40 segments a row a join with 32 rows to
// a CTA takes 63 us where 4 take 12).  A grid that is on the card at once has registers for sixteen
// rows of sums in flight instead of four (K=16 Hq=32 Hkv=8: one sequence of 131072 tokens 94.2 us, 99.2
// with four; four of 32768, 512 CTAs, 92.6 and 94.3; five of 26000, 640 CTAs and more than four to an SM,
// 94.2 and 93.9; sixteen of 8192 103.6 and 97.8).
template <int D, bool F16, int U>
__global__ void __launch_bounds__(32 * kJoinWarps, U == 4 ? 8 : 4)
    attn_join_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnWs w, const int join_rows) {
  constexpr int N = D / 32;
  // the partial results of a block's first row: of the sequence (0, 1) and of the prefix (2, 3), the
  // block that holds the CTA's first row and the one behind it
  __shared__ long long list[4][2 * kCtas];
  __shared__ int counts[4];
  __shared__ int row_at[kJoinWarps][32];
  __shared__ float row_w[kJoinWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const gdn_kv_dims& d = p.d;
  const int G = d.Hq / d.Hkv, KG = d.K * G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = (KG + join_rows - 1) / join_rows;
  const int r0 = int(blockIdx.x % unsigned(chunks)) * join_rows, bh = int(blockIdx.x / unsigned(chunks));
  const int h = bh % d.Hkv, b = bh / d.Hkv;
  const SeqRec q = w.seq[b];
  const PlanHead head = *w.head;
  const int rows = KG - r0 < join_rows ? KG - r0 : join_rows;
  const int pre0 = int(q.pre_at) + r0;  // the CTA's first row in the prefix's (rows in all: below 2^29)
  const int tile = p.tile_rows, block = 2 * tile;
  const int own_block = r0 / block, pre_block = pre0 / block;
  {
    const bool own = warp < 2;
    const int all = own ? KG : int(q.pre_rows), first = own ? r0 : pre0;
    const int n = own ? q.tiles : q.pre_tiles;
    const int rb = (own ? own_block : pre_block) + (warp & 1);
    int count = 0;
    if (n > 0 && ((warp & 1) == 0 || rb * block < first + rows)) {
      const long long deal = head.split && own ? head.prefix_tiles : 0;
      const long long size = !head.split ? head.tiles : own ? head.tiles - head.prefix_tiles : head.prefix_tiles;
      const int blocks = (all + block - 1) / block;
      const int width = all - rb * block < block ? all - rb * block : block;
      const bool paired = width > tile;
      const long long from = own ? head.prefix_tiles + h * head.head_tiles + q.off + (long long)rb * n : q.pre_off + ((long long)h * blocks + rb) * n;
      const int c0 = cta_of(from - deal, size), c1 = cta_of(from - deal + n - 1, size);
      const long long base = (own ? head.own_row + ((long long)h * d.B + b) * rows_width(KG, tile) : q.pre_row + (long long)h * rows_width(all, tile)) + rb * block;
      const int parts = (c1 - c0 + 1) * (paired ? 1 : 2);
      for (int i0 = 0; i0 < parts; i0 += 32) {
        const int i = i0 + lane, c = c0 + (paired ? i : i >> 1), s = paired ? 0 : i & 1;
        bool there = i < parts;
        if (there) {
          long long lo = deal + first_tile(c, size), hi = deal + first_tile(c + 1, size);
          lo = lo < from ? from : lo;
          hi = hi > from + n ? from + n : hi;
          there = hi > lo && (paired || hi - lo >= 2 || int(lo & 1) == s);  // (a single tile belongs to one stream)
        }
        const uint32_t some = __ballot_sync(0xffffffffu, there);
        if (there) list[warp][count + __popc(some & ((1u << lane) - 1u))] = (long long)kBlockRows * c + base + s * width;
        count += __popc(some);
      }
    }
    if (lane == 0) counts[warp] = count;
  }
  __syncthreads();
  for (int i = warp; i < rows; i += kJoinWarps) {
    const int r = r0 + i, t = r / G;
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    float M = -INFINITY, W = 0.f;
    const bool live = t < q.win;
    if (live) {
      // (a CTA's rows are fewer than a block's: in its first row's block or the next)
      int lr_own = r - own_block * block, lr_pre = pre0 + i - pre_block * block;
      const int side_own = lr_own >= block ? 1 : 0, side = lr_pre >= block ? 3 : 2;
      if (side_own == 1) lr_own -= block;
      if (side == 3) lr_pre -= block;
      const int n_own = counts[side_own], count = n_own + counts[side];
      for (int j0 = 0; j0 < count; j0 += 32) {
        const int j = j0 + lane;
        long long at = 0;
        float e = -INFINITY;
        if (j < count) {
          at = j < n_own ? list[side_own][j] + lr_own : list[side][j - n_own] + lr_pre;
          e = w.lse[at];
        }
        float mx = e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float Mn = fmaxf(M, mx), f = M == -INFINITY ? 0.f : exp2f(M - Mn);
        const float wt = e == -INFINITY ? 0.f : exp2f(e - (Mn == -INFINITY ? 0.f : Mn));  // (NaN stays NaN)
        M = Mn;
        W = W * f + warp_sum(wt);
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] *= f;
        const uint32_t some = __ballot_sync(0xffffffffu, wt != 0.f);
        __syncwarp();
        if (wt != 0.f) {
          const int k = __popc(some & ((1u << lane) - 1u));
          row_at[warp][k] = int(at);  // (rows of partial results: below 2^31)
          row_w[warp][k] = wt;
        }
        __syncwarp();
        const int m = __popc(some);
        for (int k0 = 0; k0 < m; k0 += U) {
          float v[U][N];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (k0 + u < m) {
              const float* o = w.o + (long long)row_at[warp][k0 + u] * D + lane * N;
              if (N == 4)
                *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(o);
              else
                *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(o);
            }
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (k0 + u < m) {
              const float wj = row_w[warp][k0 + u];
#pragma unroll
              for (int k = 0; k < N; ++k) acc[k] += wj * v[u][k];
            }
        }
      }
      const float inv = 1.f / W;
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] *= inv;
    }
    const long long row = ((long long)b * d.K + t) * d.Hq + h * G + (r - t * G);
    uint32_t* const o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D) + lane * (N / 2);
    if (N == 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(pack2<F16>(acc[0], acc[1]), pack2<F16>(acc[N - 2], acc[N - 1]));
    else
      *o = pack2<F16>(acc[0], acc[1]);
    if (p.lse && lane == 0) p.lse[row] = live ? (M + log2f(W)) * kLn2 : -INFINITY;
  }
}

// ---------------------------------------------------------------- launches
template <int D, bool F16>
cudaError_t launch(const AttnParams& p, const AttnWs& w, int box, const TileMaps& maps, cudaStream_t stream) {
  using L = TileLayout<D, Seg>;
  static_assert(L::TOTAL <= 232448 - 512, "shared memory");
  cudaError_t e = p.d.B <= kWarpPlan ? cudaSuccess : launch_dependent(attn_plan_kernel, 1u, kPlanThreads, 0, stream, p, w);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> allowed{0};  // a bit per device: the kernel may use its shared memory there
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(allowed.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(attn_tile_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::TOTAL);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(1ull << (dev & 63));
  }
  e = launch_dependent(attn_tile_kernel<D, F16>, unsigned(kCtas), kTileThreads, L::TOTAL, stream, p, w, box, maps);
  if (e != cudaSuccess) return e;
  const int KG = p.d.K * (p.d.Hq / p.d.Hkv);
  const long long heads = (long long)p.d.B * p.d.Hkv;
  int join_rows = kJoinRowsMax;
  while (join_rows > kJoinWarps && heads * ((KG + join_rows - 1) / join_rows) < 8 * kCtas) join_rows /= 2;
  const long long joins = heads * ((KG + join_rows - 1) / join_rows);
  return launch_dependent(joins <= 4 * kCtas ? attn_join_kernel<D, F16, 16> : attn_join_kernel<D, F16, 4>, unsigned(joins),
                    32 * kJoinWarps, 0, stream, p, w, join_rows);
}

}  // namespace

size_t attn_workspace_bytes(const gdn_kv_dims& d) {
  size_t n = 0;
  carve_attn(nullptr, d, &n);
  return n;
}

cudaError_t launch_attn(const AttnParams& params, cudaStream_t stream) {
  AttnParams p = params;
  const gdn_kv_dims& d = p.d;
  const int G = d.Hq / d.Hkv;
  p.tile_toks = kTileRows / G;
  p.tile_rows = p.tile_toks * G;
  p.page_inv = page_units_inv(d.page_size);
  const EncodeTiled encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  // Tokens per copy of a full tile: as many as lie together in a page, a divisor of the tile's 128.
  int box = 16;
  while (box < kTileKeys && d.page_size % (2 * box) == 0) box *= 2;
  const auto type = d.dtype ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  bool ok = true;
  auto map = [&](CUtensorMap* m, const void* at, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* boxes) {
    ok = ok && encode(m, type, cuuint32_t(rank), const_cast<void*>(at), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  TileMaps maps;
  const cuuint64_t cd[5] = {cuuint64_t(d.D), cuuint64_t(d.page_size), cuuint64_t(d.Hkv), cuuint64_t(d.n_pages), cuuint64_t(d.n_layers)};
  const cuuint64_t cs[4] = {2ull * d.cache_token_stride, 2ull * d.cache_head_stride, 2ull * d.cache_page_stride, 2ull * d.cache_layer_stride};
  const cuuint32_t b16[5] = {64, 16, 1, 1, 1}, bb[5] = {64, cuuint32_t(box), 1, 1, 1};
  map(&maps.few[0], p.k_cache, 5, cd, cs, b16);
  map(&maps.few[1], p.v_cache, 5, cd, cs, b16);
  map(&maps.many[0], p.k_cache, 5, cd, cs, bb);
  map(&maps.many[1], p.v_cache, 5, cd, cs, bb);
  // rows behind a window's K-th token read as zeros
  const cuuint64_t wd[5] = {cuuint64_t(d.D), cuuint64_t(d.K), cuuint64_t(d.Hkv), cuuint64_t(d.B), 1};
  const cuuint64_t wst[4] = {2ull * d.win_token_stride, 2ull * d.D, 2ull * d.K * d.win_token_stride, 2ull * d.K * d.win_token_stride};
  map(&maps.window[0], p.k_win, 5, wd, wst, b16);
  map(&maps.window[1], p.v_win, 5, wd, wst, b16);
  const cuuint64_t qd[3] = {cuuint64_t(d.D), cuuint64_t(d.Hq), cuuint64_t(d.B) * d.K};
  const cuuint64_t qst[2] = {2ull * d.D, 2ull * d.q_token_stride};
  const cuuint32_t bt[3] = {64, cuuint32_t(G), cuuint32_t(p.tile_toks)}, bs[3] = {64, cuuint32_t(G), cuuint32_t(d.K < p.tile_toks ? d.K : p.tile_toks)};
  map(&maps.qt, p.q, 3, qd, qst, bt);
  map(&maps.qs, p.q, 3, qd, qst, bs);
  if (!ok) return cudaErrorInvalidValue;
  const AttnWs w = carve_attn(p.ws, d, nullptr);
  if (d.D == 128) return d.dtype ? launch<128, true>(p, w, box, maps, stream) : launch<128, false>(p, w, box, maps, stream);
  return d.dtype ? launch<64, true>(p, w, box, maps, stream) : launch<64, false>(p, w, box, maps, stream);
}

}  // namespace gdn
