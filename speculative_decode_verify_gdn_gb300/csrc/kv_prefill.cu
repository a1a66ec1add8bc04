// Attention of packed queries over the paged cache (gdn_attn_prefill; contract in include/gdn_kv.h), on the
// tensor cores.
//
// Mathematics: softmax over a row's keys in one pass with a running maximum and sum, and joined over disjoint
// sets of keys by their log-sum-exps, as in kv_attn.cu, whose tiles (kv_tile.cuh) this uses.
//
// The work is cut into items (kv head, block): a block is up to 2 x 128 rows of consecutive tokens of one
// sequence - a row is one query head of one token, the head's whole group of tokens go together - and its
// keys are the prefix's, then those of its own slot that its last row sees, in tiles of 128.  All tiles of all
// items, head by head, are dealt to the CTAs (one per SM) in equal contiguous stretches, so every CTA has the
// same number of tiles whatever the lengths are.  An item that lies within a stretch is finished by its CTA; of
// one that is cut, each CTA writes the softmax-weighted sum and log-sum-exp of its own keys (f32, in the
// workspace: at most two such pieces a CTA), and a last kernel joins them.  Which CTA computes what depends on
// the lengths alone, and no sum is formed by atomics, so results repeat bit for bit.
//
// Kernels: tiles (persistent, tcgen05; every CTA plans for itself) or, for few rows to a sequence, a kernel of warps that
// work by themselves (below); join.  A batch of both kinds of sequences has both, one after the other in the same workspace.
//
// A block of more than 128 rows gives each stream half of them, on the same keys; a smaller one gives the
// streams alternate tiles of the same rows, and at its end the two sums are joined in tensor memory, each
// softmax group taking half of the columns.
//
// Measured on one GB300, calls in a row and, where it differs, in turn with other work (peaks: 6702 GB/s copy, 1903 TFLOP/s cuBLAS bf16, 1728 when the power cap sets
// the clock):
//   prompts of 4096..16384 tokens, Hq=32 Hkv=8 D=128     3.0-3.3 ms, 1250-1350 TFLOP/s: the chain scores, softmax, products of a
//     stream (a pair of tiles in 1.9 us) at the power cap
//   512 tokens behind 65536, Hq=32 Hkv=8 D=128           387-413 us, 1340-1430 TFLOP/s, in turn 444-458, 1210-1250: the same chain (14 % less with half of the
//     softmax left out).  Its 64 items read the same keys at different times, 2.2 GB from HBM where 0.28 would do; reading
//     them together (stretches dealt in rounds) gave 408, and 130 for 119 behind 16384
//   13 prompts of 1..901 tokens behind 1531 shared and 0..333 own, f16 Hq=24 Hkv=4 D=64   110 us, 660 TFLOP/s: the warp
//     that issues the products, a pair of tiles in 1.4 us; start, ends of segments and join 20 us
//   24 prompts of 3..448 tokens over 400..1500 states, Hq=Hkv=16 D=64   57.5 us, in turn 62: start, ends of 4.6 segments a CTA, join
//   64 single tokens over 1..1500 states, f16 Hq=Hkv=16 D=64   45-49 us, 4.0-4.4 TB/s (few rows)
//   one prompt of 37 tokens   14 us: the host's two launches and its tensor maps (three, five where 32 tokens of a page lie together)
#include <atomic>
#include <climits>

#include "kv_device.cuh"
#include "kv_index.h"
#include "kv_tile.cuh"

namespace gdn {

namespace {

constexpr int kJoinAlone = 4;   // pieces that the CTAs of one worker join by themselves
constexpr int kJoinChunks = 8;  // CTAs of the join to a CTA of the tile kernel (cross attention of prompts 59 us, 61 with 4, 60 with 16)
constexpr int kFewRows = 8;     // rows of a block of the kernel for few rows
constexpr int kFewThreads = 128;
__host__ __device__ constexpr int few_ctas(int D) { return D == 128 ? 3 : 4; }  // CTAs to an SM
__host__ __device__ constexpr int few_workers(int D) { return kCtas * few_ctas(D) * (kFewThreads / 32); }

struct alignas(16) JoinRec {  // of worker c: a cut item that begins in its stretch and ends in that of worker `end`
  int32_t tok0, rows;  // rows 0: there is none
  int32_t h, end, part0;
  int32_t before;      // the worker in whose stretch the item began that its own begins within; -1: it does not
  int32_t spare[2];
};

struct PackedWs {
  JoinRec* join;     // [workers]
  float* lse;        // [workers][2][rows] log2 units (kCtas workers with kBlockRows, or few_workers with kFewRows)
  float* o;          // [workers][2][rows][D]
};

__host__ __device__ inline size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

__host__ __device__ inline PackedWs carve_packed(void* base, const gdn_kv_dims& d, size_t* total) {
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t o = 0;
  const size_t parts = 2 * size_t(kBlockRows) * kCtas;
  static_assert(few_workers(64) * kFewRows <= kBlockRows * kCtas && few_workers(64) >= few_workers(128), "room for either kernel's pieces");
  PackedWs w;
  w.join = reinterpret_cast<JoinRec*>(p + o), o += round256(sizeof(JoinRec) * few_workers(64));
  w.lse = reinterpret_cast<float*>(p + o), o += round256(4 * parts);
  w.o = reinterpret_cast<float*>(p + o), o += 4 * parts * size_t(d.D);
  if (total) *total = o;
  return w;
}

// ---------------------------------------------------------------- the plan
// How the calls' rows are cut into blocks: all that depends on the heads alone.
struct Cut {
  int tile_toks, toks;  // tokens of a row tile, of a block
  int key_log;          // a tile has 2^key_log keys
  int period_log;       // after so many (2^period_log) blocks, their keys are a whole number of tiles more
  int causal;
  int workers;          // that the tiles are dealt to
  int least, most;      // sequences of so many tokens are taken; the others count for none here
  __host__ __device__ __forceinline__ long long tiles_of(long long keys) const { return (keys + (1 << key_log) - 1) >> key_log; }
};

struct SeqRows {
  int lo, n;       // its packed tokens
  int len;         // tokens in its slot
  int pre_slot, pre_keys;
  __device__ __forceinline__ int pre_tiles(const Cut& c) const { return int(c.tiles_of(pre_keys)); }
  __device__ __forceinline__ int blocks(const Cut& c) const { return int((unsigned(n) + unsigned(c.toks) - 1u) / unsigned(c.toks)); }
  // own keys that the last row of block k sees
  __device__ __forceinline__ int keys(const Cut& c, int k) const {
    if (!c.causal) return len;
    const long long e = (long long)len - n + (long long)c.toks * (k + 1);
    return e < 0 ? 0 : e < len ? int(e) : len;
  }
  // Tiles of the first k blocks: sums of their keys' tiles, period by period.
  __device__ __forceinline__ long long tiles(const Cut& c, int k) const {
    const long long pre = c.tiles_of(pre_keys) * k;
    if (!c.causal) return pre + c.tiles_of(len) * k;
    const long long off = (long long)len - n;
    const int i0 = off >= 0 ? 1 : int((unsigned long long)(-off) / unsigned(c.toks)) + 1;  // the first block with keys, counted from 1
    long long sum = 0;
    if (k >= i0) {
      const long long m = (long long)k - i0 + 1, first = off + (long long)c.toks * i0 + (1 << c.key_log) - 1;
      const int period = 1 << c.period_log, rest = int(m & (period - 1));
      const long long whole = m >> c.period_log, more = (long long)c.toks << c.period_log >> c.key_log;  // (tiles that a period adds)
      long long one = 0, part = 0;
      for (int i = 0; i < period && i < m; ++i) {
        const long long t = (first + (long long)c.toks * i) >> c.key_log;
        one += t;
        if (i < rest) part += t;
      }
      sum = (whole > 0 ? whole * one : 0) + (more * whole * (whole - 1) / 2 << c.period_log) + part + rest * more * whole;
    }
    if (k == blocks(c) && k > 0) {  // the last block is as long as it is
      const long long e = off + (long long)c.toks * k;
      sum += c.tiles_of(len) - (e > 0 ? c.tiles_of(e) : 0);
    }
    return pre + sum;
  }
  // Tokens in blocks without keys, the first ones.
  __device__ __forceinline__ int without_keys(const Cut& c) const {
    if (pre_keys > 0 || n == 0) return 0;
    if (len == 0) return n;
    if (!c.causal || len >= n) return 0;
    const int k = (n - len) / c.toks;
    return k * c.toks;
  }
};

__device__ __forceinline__ SeqRows load_sequence(const PackedAttnParams& p, const Cut& cut, int b, bool report) {
  const gdn_kv_dims& d = p.d;
  SeqRows s;
  const int lo = p.cu[b], hi = p.cu[b + 1], len = p.seq_len[d.slot0 + b], slot = p.prefix_of ? p.prefix_of[b] : -1;
  const int refused = p.refused && p.causal ? p.refused[d.slot0 + b] : -1;
  uint32_t bad = 0;
  s.lo = lo, s.n = hi > lo ? hi - lo : 0;
  s.len = len;
  if (len < 0 || (long long)len > (long long)d.max_pages * d.page_size) s.len = 0, bad |= GDN_DEVERR_KV_LEN;
  if (slot < -1 || slot >= d.n_slots) bad |= GDN_DEVERR_KV_SLOT;
  s.pre_slot = slot < 0 || slot >= d.n_slots ? -1 : slot;
  s.pre_keys = 0;
  if (s.pre_slot >= 0) {
    s.pre_keys = p.seq_len[s.pre_slot];
    if (s.pre_keys < 0 || (long long)s.pre_keys > (long long)d.max_pages * d.page_size) s.pre_keys = 0, bad |= GDN_DEVERR_KV_LEN;
  }
  // a slot that is as long as when room for its tokens was refused: its last tokens are others than the rows, which see nothing
  if (refused >= 0 && refused == len && s.n > 0) s.len = 0, s.pre_slot = -1, s.pre_keys = 0, bad |= GDN_DEVERR_KV_LEN;
  if (bad && report) atomicOr(p.err, bad);
  if (s.n < cut.least || s.n > cut.most) s.n = 0;
  return s;
}

// Every CTA plans for itself: each thread sums the tiles of a few consecutive sequences, and the CTA the sums of its
// threads.  A worker then looks for the thread, and that thread's sequence, with the first tile of its stretch.
struct Plan {
  long long head_tiles, tiles;  // of one kv head, and of all
  int32_t workers;              // that the tiles are dealt to: each has one at least
  int32_t empty;                // some rows have no keys
  // The deal gives worker i tiles [begin(i), begin(i + 1)); the worker of tile x.
  __device__ __forceinline__ long long begin(long long i) const { return i * tiles / workers; }
  __device__ __forceinline__ int worker_of(long long x) const {
    int i = int(float(x) * (float(workers) / float(tiles)));  // (within one of it)
    i = i < 0 ? 0 : i > workers - 1 ? workers - 1 : i;
    while (i > 0 && begin(i) > x) --i;
    while (i < workers - 1 && begin(i + 1) <= x) ++i;
    return i;
  }
};

// before[i]: tiles of the sequences of the threads before thread i (T + 32 of them: sums of the warps behind).
template <int T>
__device__ __forceinline__ void make_plan(const PackedAttnParams& p, const Cut& cut, Plan& plan, long long* before) {
  const gdn_kv_dims& d = p.d;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);
  const int each = (d.B + T - 1) / T;
  const int b0 = tid * each < d.B ? tid * each : d.B, b1 = b0 + each < d.B ? b0 + each : d.B;
  bool bad = tid == 0 && (p.cu[0] != 0 || p.cu[d.B] > p.n_tokens), empty = false;
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    bad |= p.cu[b] > p.cu[b + 1];
    const SeqRows s = load_sequence(p, cut, b, cta == 0);
    mine += s.tiles(cut, s.blocks(cut));
    empty |= s.without_keys(cut) > 0;
  }
  bad = __syncthreads_or(bad) != 0;
  empty = __syncthreads_or(empty) != 0;
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  long long* const sums = before + T;
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  long long sum = 0, all = 0;
#pragma unroll
  for (int i = 0; i < T / 32; ++i) {
    sum += i < warp ? sums[i] : 0;
    all += sums[i];
  }
  before[tid] = sum + x - mine;
  if (tid == 0) {
    if (bad) all = 0;
    if (bad && cta == 0) atomicOr(p.err, kDevErrSeqlens);
    plan.head_tiles = all, plan.tiles = all * d.Hkv;
    plan.workers = int(plan.tiles < cut.workers ? plan.tiles : cut.workers);
    plan.empty = empty && !bad;
  }
  __syncthreads();
}

// Outputs of rows without keys, whole blocks of them: 0 and -inf.
__device__ __noinline__ void write_empty(const PackedAttnParams& p, const Cut& cut) {
  const gdn_kv_dims& d = p.d;
  for (int b = int(blockIdx.x); b < d.B; b += int(gridDim.x)) {
    const SeqRows s = load_sequence(p, cut, b, false);
    const long long rows = (long long)s.without_keys(cut) * d.Hq, first = (long long)s.lo * d.Hq;
    uint4* const out = reinterpret_cast<uint4*>(p.out + first * d.D);
    for (long long k = threadIdx.x; k < rows * (d.D / 8); k += blockDim.x) out[k] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse)
      for (long long k = threadIdx.x; k < rows; k += blockDim.x) p.lse[first + k] = -INFINITY;
  }
}

// ---------------------------------------------------------------- segments
struct Seg {
  int tok0, rows;               // packed tokens, rows of the block
  int h;                        // kv head
  int pair;                     // they fill more than one row tile: both streams take every tile of keys
  int slot, keys;               // own slot, and the keys in it that the last row sees
  int lim;                      // the keys in it that the first row sees (causal: a token more each token; may be below 1)
  int pre_slot, pre_keys, pre_tiles;
  int t0, t1;                   // tiles of the item
  int parity;                   // of tile t0 in the order of all tiles
  int part;                     // first row of its partial results (-1: the whole item, which goes to the outputs)
  __device__ __forceinline__ bool paired() const { return pair != 0; }
  struct Tiles {
    int pre_tiles, pre_units, own_units;  // units of 16 keys
    __device__ __forceinline__ int units(int t) const {
      const int left = t < pre_tiles ? pre_units - 8 * t : own_units - 8 * (t - pre_tiles);
      return left < 8 ? left : 8;
    }
  };
  __device__ __forceinline__ Tiles tiles() const {  // (a converged warp)
    return Tiles{int(uniform(uint32_t(pre_tiles))), int(uniform(uint32_t((pre_keys + 15) >> 4))), int(uniform(uint32_t((keys + 15) >> 4)))};
  }
};

// Walks a worker's stretch segment by segment (a converged warp).  Lane i knows sequence from + i.
template <int T, int ROWS>  // threads that planned, rows of a piece's partial results
struct SegWalk {
  const PackedAttnParams& p;
  const PackedWs& w;
  const Cut& cut;
  const Plan& plan;
  const int id, lane, G;
  long long begin, x, end;
  int h, b, k, t_in;  // the item at hand: kv head, sequence, block; its tiles before x
  int from, before_me;
  SeqRows mine;
  __device__ __forceinline__ SeqRows sequence(int i) {
    if (i < from || i >= from + 32) {
      from = i;
      const int at = i + lane < p.d.B ? i + lane : p.d.B - 1;
      mine = load_sequence(p, cut, at, false);
    }
    const int l = i - from;
    SeqRows s;
    s.lo = __shfl_sync(0xffffffffu, mine.lo, l), s.n = __shfl_sync(0xffffffffu, mine.n, l);
    s.len = __shfl_sync(0xffffffffu, mine.len, l), s.pre_slot = __shfl_sync(0xffffffffu, mine.pre_slot, l);
    s.pre_keys = __shfl_sync(0xffffffffu, mine.pre_keys, l);
    return s;
  }
  __device__ __forceinline__ SegWalk(const PackedAttnParams& p_, const PackedWs& w_, const Cut& cut_, const Plan& plan_,
                                     const long long* before, int id_, int lane_)
      : p(p_), w(w_), cut(cut_), plan(plan_), id(id_), lane(lane_), G(p_.d.Hq / p_.d.Hkv) {
    begin = x = end = 0;
    h = b = k = t_in = 0;
    from = -64, before_me = -1;
    if (id >= plan.workers) {
      if (lane == 0) w.join[id].rows = 0, w.join[id].before = -1;
      return;
    }
    begin = x = plan.begin(id), end = plan.begin(id + 1);
    h = int(begin / plan.head_tiles);
    long long y = begin - h * plan.head_tiles;
    // the last thread, and then its last sequence, with at most y tiles before it
    int at = 0;
    for (int n = T, step = T / 32; step > 0; n = step, step = step / 32 > 0 ? step / 32 : step > 1 ? 1 : 0) {
      const uint32_t some = __ballot_sync(0xffffffffu, lane * step < n && before[at + lane * step] <= y);
      at += (31 - __clz(int(some))) * step;
    }
    y -= before[at];
    const int each = (p.d.B + T - 1) / T;
    for (b = at * each; b < p.d.B - 1; ++b) {
      const SeqRows s = sequence(b);
      const long long t = s.tiles(cut, s.blocks(cut));
      if (y < t) break;
      y -= t;
    }
    const SeqRows s = sequence(b);
    int n = s.blocks(cut);  // its last block with at most y tiles before it, 32 at a time
    while (n > 1) {
      const int step = (n + 31) / 32, i = lane * step;
      const uint32_t some = __ballot_sync(0xffffffffu, i < n && s.tiles(cut, k + i) <= y);
      const int j = 31 - __clz(int(some));
      k += j * step;
      n = n - j * step < step ? n - j * step : step;
    }
    t_in = int(y - s.tiles(cut, k));
    if (t_in > 0) before_me = plan.worker_of(begin - t_in);
    if (lane == 0) w.join[id].rows = 0, w.join[id].before = before_me;
  }
  __device__ __forceinline__ bool next(Seg& g) {
    if (x >= end) return false;
    while (true) {
      if (b == p.d.B) b = 0, ++h;
      const SeqRows s = sequence(b);
      if (k >= s.blocks(cut)) {
        ++b, k = 0;
        continue;
      }
      const int pre = s.pre_tiles(cut), keys = s.keys(cut, k), tiles = pre + int(cut.tiles_of(keys));
      if (tiles == 0) {
        ++k;
        continue;
      }
      const int j0 = k * cut.toks, toks = s.n - j0 < cut.toks ? s.n - j0 : cut.toks;
      g.tok0 = s.lo + j0, g.rows = toks * G, g.h = h;
      g.pair = toks > cut.tile_toks;
      g.slot = p.d.slot0 + b, g.keys = keys, g.lim = cut.causal ? s.len - s.n + j0 + 1 : s.len;
      g.pre_slot = s.pre_slot, g.pre_keys = s.pre_keys, g.pre_tiles = pre;
      g.t0 = t_in;
      g.t1 = end - x < tiles - t_in ? t_in + int(end - x) : tiles;
      g.parity = int(x & 1);
      const int second = x == begin ? 0 : 1;  // (of the worker's pieces: one that its stretch begins with, one that it ends with)
      g.part = g.t0 == 0 && g.t1 == tiles ? -1 : (2 * id + second) * ROWS;
      if (g.t0 == 0 && g.t1 < tiles && lane == 0)
        w.join[id] = JoinRec{g.tok0, g.rows, h, plan.worker_of(x + tiles - 1), g.part, before_me, {0, 0}};
      x += g.t1 - g.t0;
      t_in = 0, ++k;  // (an item that goes on ends the stretch)
      return true;
    }
  }
};

// ---------------------------------------------------------------- the tile kernel
struct PackedMaps {
  // (D, token, kv head, page, 1), keys and values: boxes of 16 tokens, and of `box` tokens
  CUtensorMap few[2], many[2];
  // queries, (D, query head, token): boxes of G heads x the tokens of a row tile
  CUtensorMap queries;
};

// At D = 64 tensor memory has room for a third tile of scores, and the products of a stream's next scores need not wait
// until its probabilities have been multiplied (256 rows of 32 heads over 92160 keys: 219 us, 242 with two tiles and a warp
// per stream).  What then sets the pace is this warp: 1470 cycles a use, 256 + 256 of them the tensor core's, before a
// tile's second stream stopped waiting for keys and values that the first had seen (235 us).  A warp each for scores and
// products takes 204 us there, but 71 where this takes 65 on the cross attention of prompts.  All uses of the tensor core are in one order, n = 0, 1, 2, ..: a tile's scores
// of stream 0 and of stream 1, or a stream's alone; use n has buffer n % 3.  One warp issues
//   S(0) S(1) S(2) O(0) S(3) O(1) S(4) ..
// Barriers: s_ready, a stream's i-th use on its barrier i % 4 (three uses may be under way that the stream's softmax
// has not looked at yet; a fourth one comes behind products that need its probabilities); p_ready by buffer, and the
// issuing warp sees every phase of it; o_step, a stream's sums after each tile, for a softmax that has to rescale them; a
// tile's slots are released once.
template <int D>
struct Ahead {
  static constexpr bool ON = D == 64;
  static constexpr int BUFFERS = 3;
  static __device__ __forceinline__ uint32_t o_col(int s) { return ON ? 384u + 64u * uint32_t(s) : tmem_o(s); }
};
struct AheadBars {
  uint64_t s_ready[2][4], p_ready[3], o_step[2];
};
template <int D, bool F16, typename Wait>
__device__ __forceinline__ void tensor_warp_ahead(const int lane, const uint32_t tmem, const uint32_t base, const bool negative,
                                                  const Seg* const segs, const TileBars& bars, AheadBars& ahead, Wait wait_warp) {
  using L = TileLayout<D, Seg>;
  constexpr int NS = L::STAGES, NB = Ahead<D>::BUFFERS;
  const uint32_t tm = uniform(tmem);
  const uint32_t values_idesc = idesc_f16<F16>(kTileKeys, D) | (1u << 16);  // B (values) MN-major
  const uint32_t scores_idesc = negative ? 1u << 13 : 0u;                   // a negative scale negates the queries
  struct Use {
    uint32_t units, slot, phase, flags;  // its values' slot; flags: 1 stream, 2 first of the stream's sums, 4 last, 8 the slot's last, 16 not its first
  };
  Use u0{}, u1{}, u2{};  // whose O += P V is still to be issued, the eldest first
  uint32_t pending = 0;
  uint32_t n_buf = 0, p_buf = 0, p_phase = 0;  // buffer of the next scores; of the eldest pending use, and its phase
  uint32_t slot = 0, phase = 0;                // of a tile's keys; its values are in the slot behind
  uint32_t uses0 = 0, uses1 = 0, nq0 = 0, nq1 = 0;  // scores and segments of each stream
  bool ok = true;
  auto values = [&]() {  // O += P V of the eldest
    ok = ((u0.flags & 16u) || wait_warp(bars.full + u0.slot, u0.phase)) && wait_warp(ahead.p_ready + p_buf, p_phase);
    if (!ok) return;
    tc_fence_after();
    const uint32_t s = u0.flags & 1u, to = tm + Ahead<D>::o_col(int(s)), ts = tm + 128u * p_buf;
    const uint32_t db = swizzled_desc_lo(base + L::OFF_RING + u0.slot * L::BYTES, L::HALF);
    umma_values_first(to, ts, db, values_idesc, u0.flags & 2u ? 0u : 1u);
    if (u0.units == 8) {
      umma_values_rest(to, ts, db, values_idesc);
    } else {
#pragma unroll 1
      for (uint32_t u = 1; u < u0.units; ++u) umma_values_first(to, ts + 8 * u, db + 128 * u, values_idesc, 1);
    }
    umma_commit_one(ahead.o_step + s);
    if (u0.flags & 8u) umma_commit_one(bars.empty + u0.slot);
    if (u0.flags & 4u) umma_commit_one(bars.o_done + s);
    u0 = u1, u1 = u2, --pending;
    if (++p_buf == NB) p_buf = 0, p_phase ^= 1;
  };
  for (uint32_t k = 0; ok; ++k) {
    const Seg& seg = segs[k % kSegRing];
    if (!wait_warp(bars.seg_full + k % kSegRing, (k / kSegRing) & 1)) {
      ok = false;
      break;
    }
    const int t0 = int(uniform(uint32_t(seg.t0))), t1 = int(uniform(uint32_t(seg.t1)));
    const auto tiles = seg.tiles();
    const uint32_t parity = uniform(uint32_t(seg.parity));
    const bool paired = uniform(seg.paired() ? 1u : 0u) != 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.seg_empty + k % kSegRing);
    if (t1 < 0) break;
#pragma unroll 1
    for (int t = t0; ok && t < t1; ++t) {
      const uint32_t vslot = slot + 1 < NS ? slot + 1 : 0, vphase = slot + 1 < NS ? phase : phase ^ 1;
      const uint32_t units = uint32_t(tiles.units(t));
      const bool first = paired ? t == t0 : t - t0 < 2, last = paired ? t == t1 - 1 : t1 - t <= 2;
#pragma unroll 1
      for (uint32_t i = 0; i < (paired ? 2u : 1u); ++i) {
        const uint32_t s = paired ? i : (parity + uint32_t(t - t0)) & 1u;
        const bool slot_last = !paired || i == 1;
        if (pending == NB) values();
        if (ok && first) ok = wait_warp(bars.q_ready + s, (s ? nq1 : nq0) & 1);
        ok = ok && (i == 1 || wait_warp(bars.full + slot, phase));
        if (!ok) break;
        tc_fence_after();
        umma_scores<D>(tm + 128u * n_buf, swizzled_desc_lo(base + L::OFF_Q + s * L::BYTES, 16),
                       swizzled_desc_lo(base + L::OFF_RING + slot * L::BYTES, 16), idesc_f16<F16>(kTileKeys, int(16 * units)) | scores_idesc);
        umma_commit_one(&ahead.s_ready[s][(s ? uses1 : uses0) & 3]);
        if (slot_last) umma_commit_one(bars.empty + slot);
        if (last) umma_commit_one(bars.q_free + s);
        if (first) nq0 += s ^ 1, nq1 += s;
        uses0 += s ^ 1, uses1 += s;
        const Use u{units, vslot, vphase, s | (first ? 2u : 0u) | (last ? 4u : 0u) | (slot_last ? 8u : 0u) | (i == 1 ? 16u : 0u)};
        if (pending == 0)
          u0 = u;
        else if (pending == 1)
          u1 = u;
        else
          u2 = u;
        ++pending;
        if (++n_buf == NB) n_buf = 0;
      }
      slot += 2, phase ^= slot >= NS ? 1u : 0u, slot -= slot >= NS ? NS : 0;
    }
  }
  while (ok && pending > 0) values();
  if (!ok) {  // what is under way finishes before tensor memory is freed
    umma_commit_one(bars.o_done);
    mbar_drain(bars.o_done, 0);
    mbar_drain(bars.o_done, 1);
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kTileThreads, 1)
    packed_tile_kernel(const __grid_constant__ PackedAttnParams p, const __grid_constant__ PackedWs w, const __grid_constant__ Cut cut, const int box,
                       const uint32_t page_inv, const __grid_constant__ PackedMaps maps) {
  using L = TileLayout<D, Seg>;
  constexpr int NS = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ int page_of_box[32][2];
  __shared__ volatile uint32_t gave_up, turns[2];  // (turns: taken so far by each tensor-core warp)
  __shared__ uint64_t merge_bar;                   // the two softmax groups, at the end of a segment that they share
  __shared__ Plan plan;
  __shared__ AheadBars ahead;
  __shared__ float2 merge_ml[kTileRows];           // maximum (log2 units) and sum of a row, one stream's and then the other's
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - smem_addr(smem_raw));
  const TileBars bars = tile_bars<NS>(reinterpret_cast<uint64_t*>(smem + L::OFF_BAR));
  Seg* const segs = reinterpret_cast<Seg*>(smem + L::OFF_SEG);
  const int tid = int(threadIdx.x), warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const gdn_kv_dims& d = p.d;
  const int G = d.Hq / d.Hkv, tile_toks = cut.tile_toks, tile_rows = tile_toks * G;

  if (tid == 0) {
    init_tile_bars<NS>(bars, Ahead<D>::ON ? 1 : 2);
    mbar_init(&merge_bar, 2 * kGroupThreads);
    if (Ahead<D>::ON) {
      for (int i = 0; i < 8; ++i) mbar_init(&ahead.s_ready[i / 4][i % 4], 1);
      for (int i = 0; i < 3; ++i) mbar_init(ahead.p_ready + i, kGroupThreads);
      for (int i = 0; i < 2; ++i) mbar_init(ahead.o_step + i, 1);
    }
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
  long long* const before = reinterpret_cast<long long*>(smem + L::OFF_SEG - 8 * 1024);  // (in the ring's last slot, which fills after the plan)
  make_plan<kTileThreads>(p, cut, plan, before);
  fence_proxy_async_smem();
  if (plan.empty) write_empty(p, cut);

  // Bounded wait of a whole warp, which goes on or gives up together; once one warp has given up, all of the
  // CTA's do.
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
    // As in kv_attn.cu: copies go out as slots fall free, the page numbers of the tile behind are on their way to
    // shared memory meanwhile, and lane i looks up box i.
    uint32_t n = 0, issued = 0;  // tiles and ring uses so far; tile n's keys are use 2n, its values 2n + 1
    uint32_t k = 0;              // segments so far
    int t = 0, t1 = 0;           // of the present segment: next tile, end
    bool ok = true, more = true;
    uint32_t slot = 0, phase = 1;  // of the next use; the phase that its slot was emptied in
    // the segment at hand
    Seg::Tiles tiles{};
    int seg_h = 0;
    const int32_t *own_pages = nullptr, *pre_pages = nullptr;
    // the tile behind the one at hand
    int units = 0, boxes = 0, in = 0;
    uint32_t ahead = 0;     // tiles looked up
    bool whole = false;     // in boxes of `box` tokens
    int* const page = page_of_box[lane];  // of this tile and the next in turn
    auto next_tile = [&]() {
      while (ok && t == t1) {
        __syncwarp();
        if (k > 0 && lane == 0) mbar_arrive(bars.seg_empty + (k - 1) % kSegRing);
        ok = wait_warp(bars.seg_full + k % kSegRing, (k / kSegRing) & 1);
        const Seg& seg = segs[k % kSegRing];
        t = int(uniform(uint32_t(seg.t0))), t1 = int(uniform(uint32_t(seg.t1)));
        ++k;
        if (t1 < 0) more = false;
        if (t1 < 0 || !ok) return;
        tiles = seg.tiles();
        seg_h = int(uniform(uint32_t(seg.h)));
        own_pages = p.table + (long long)seg.slot * d.max_pages;
        pre_pages = p.table + (long long)(seg.pre_slot < 0 ? 0 : seg.pre_slot) * d.max_pages;
      }
      if (!ok) return;
      units = tiles.units(t);
      whole = units == 8;
      boxes = whole ? kTileKeys / box : units;
      if (lane < boxes) {
        const bool own = t >= tiles.pre_tiles;
        const int token = (own ? t - tiles.pre_tiles : t) * kTileKeys + lane * (whole ? box : 16);
        const int col = page_column(token, page_inv);
        in = token - col * d.page_size;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(page + (ahead & 1))), "l"((own ? own_pages : pre_pages) + col) : "memory");
      }
      ++t, ++ahead;
    };
    next_tile();
    while (ok && more) {
      const int now_units = units, now_boxes = boxes, now_in = in, now_h = seg_h;
      const bool now_whole = whole;
      asm volatile("cp.async.wait_all;" ::: "memory");
      int now_page = page[n & 1];
      if (lane < now_boxes && (now_page < 0 || now_page >= d.n_pages)) {  // reads zeros there
        atomicOr(p.err, GDN_DEVERR_KV_PAGE);
        now_page = d.n_pages;
      }
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        if (!wait_warp(bars.empty + slot, phase)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(bars.full + slot, uint32_t(now_units) * 16 * D * 2);
        __syncwarp();
        const uint32_t dst = base + L::OFF_RING + slot * L::BYTES, bar = smem_addr(bars.full + slot), step = uint32_t(now_whole ? box : 16) * 128;
        const CUtensorMap* const m = now_whole ? &maps.many[v] : &maps.few[v];
#pragma unroll 1
        for (int b = 0; b < now_boxes; ++b)
          tma_box<D>(dst + b * step, m, int(uniform_from(uint32_t(now_in), b)), now_h, int(uniform_from(uint32_t(now_page), b)), 0, bar);
        issued = 2 * n + v + 1;
        if (++slot == NS) slot = 0, phase ^= 1;
        if (v == 0) next_tile();
        if (!ok) break;
      }
      ++n;
    }
    // the last uses of the ring: the copies have landed and the tensor core has read them
    for (uint32_t use = issued > NS ? issued - NS : 0; use < issued; ++use) {
      if (ok) ok = wait_warp(bars.empty + use % NS, (use / NS) & 1);
      if (!ok) mbar_drain(bars.full + use % NS, (use / NS) & 1);
    }
  } else if (warp == 9 || warp == 10) {
    if (!Ahead<D>::ON)
      tensor_warp<D, F16>(warp - 9, lane, tmem, base, p.scale < 0.f, segs, bars, turns, wait_warp);
    else if (warp == 9)
      tensor_warp_ahead<D, F16>(lane, tmem, base, p.scale < 0.f, segs, bars, ahead, wait_warp);
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax: stream s, one row per thread
    const int s = warp >> 2, r = tid & 127;
    const uint32_t lane_sel = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t to = tmem + Ahead<D>::o_col(s) + lane_sel;
    const float c = fmaxf(fabsf(p.scale) * kLog2e, 1e-30f);  // (0 is as good as 1e-30)
    uint32_t n = 0, ns = 0;          // tiles of the CTA, tiles of this stream
    uint32_t uses = 0;               // of the tensor core before this segment (Ahead)
    uint32_t no = 0, no_other = 0;   // segments of this stream and of the other
    uint32_t meets = 0;              // phases of the groups' barrier so far
    auto meet = [&] {
      mbar_arrive(&merge_bar);
      return wait_warp(&merge_bar, meets++ & 1);
    };
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      const Seg& seg = segs[k % kSegRing];
      if (!wait_warp(bars.seg_full + k % kSegRing, (k / kSegRing) & 1)) {
        ok = false;
        break;
      }
      auto done = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.seg_empty + k % kSegRing);
      };
      if (seg.t1 < 0) break;
      const bool paired = seg.paired();
      const uint32_t n0 = n, uses0 = uses;
      n += uint32_t(seg.t1 - seg.t0);
      uses += uint32_t(seg.t1 - seg.t0) << (paired ? 1 : 0);
      int t = seg.t0;
      if (!paired && ((seg.parity ^ s) & 1)) ++t;
      const bool shared = !paired && seg.t1 - seg.t0 > 1;  // both streams have tiles of the same rows
      if (t >= seg.t1) {
        ++no_other;
        done();
        continue;
      }
      const int step = paired ? 1 : 2;
      const int srow0 = paired ? s * tile_rows : 0;
      const int rows = seg.rows - srow0 < tile_rows ? seg.rows - srow0 : tile_rows;
      const bool idle = 32 * (warp & 3) >= rows;  // a warp without rows only keeps the barriers going
      // own keys that this row sees, and that the stream's first row sees
      const int tok = (srow0 + r) / G, tok_first = srow0 / G;
      const int lim = seg.lim + (p.causal ? tok : 0), lim_first = seg.lim + (p.causal ? tok_first : 0);

      float m = -INFINITY, l = 0.f;  // running maximum (unscaled) and sum
      bool first = true;
      for (; ok && t < seg.t1; t += step, ++ns) {
        const uint32_t use = uses0 + (paired ? 2 * uint32_t(t - seg.t0) + uint32_t(s) : uint32_t(t - seg.t0)), buffer = use % 3;
        const uint32_t ts = tmem + lane_sel + (Ahead<D>::ON ? 128u * buffer : tmem_s(s));
        if (!(Ahead<D>::ON ? wait_warp(&ahead.s_ready[s][ns & 3], (ns >> 2) & 1) : wait_warp(bars.s_ready + s, ns & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool own = t >= seg.pre_tiles;
        const int key0 = (own ? t - seg.pre_tiles : t) * kTileKeys;
        const int left = (own ? seg.keys : seg.pre_keys) - key0;  // keys of this tile that some row sees (may exceed 128)
        if (!idle) {
          const int mine = (own ? lim : seg.pre_keys) - key0, fewest = (own ? lim_first : seg.pre_keys) - key0;
          softmax_tile<D, F16>(ts, to, c, r < rows, first, fewest < kTileKeys, [&](int q, int g) {
            const int n_seen = mine - 64 * q - 32 * g;
            return n_seen >= 32 ? 0xffffffffu : n_seen <= 0 ? 0u : (1u << n_seen) - 1u;
          }, [&] {
            // Scores come before the products of the stream's tile before, which has to be done now.  (Those of the tile
            // before that are: use n's scores are behind the products of use n - 3, and a stream's uses are two apart.
            // So the phase's parity tells.)
            if (Ahead<D>::ON) {
              wait_warp(ahead.o_step + s, (ns - 1) & 1);
              tc_fence_after();
            }
          }, m, l);
        }
        first = false;
        if (left < kTileKeys && (left & 15)) {
          // values behind the last token of its unit may be anything: zero them, for 0 x NaN is NaN
          const uint32_t fill = 2 * (n0 + uint32_t(t - seg.t0)) + 1, slot = fill % NS;
          if (!wait_warp(bars.full + slot, (fill / NS) & 1)) {
            ok = false;
            break;
          }
          const int end = (left + 15) & ~15;
          uint8_t* const v_tile = smem + L::OFF_RING + slot * L::BYTES;
          constexpr int C = D / 8;
          for (int i = r; i < (end - left) * C; i += kGroupThreads) {
            const int row = left + i / C, ch = i % C;
            *reinterpret_cast<uint4*>(v_tile + (ch >> 3) * L::HALF + row * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(Ahead<D>::ON ? ahead.p_ready + buffer : bars.p_ready + s);
      }
      if (!ok) break;

      // the segment's result
      if (!wait_warp(bars.o_done + s, no & 1)) {
        ok = false;
        break;
      }
      ++no;
      float w_own = 1.f, w_other = 0.f, M = m == -INFINITY ? -INFINITY : m * c, sum = l;  // (log2 units)
      if (shared) {  // each group takes the sums of both streams, in half of the columns
        float2 other;
        if (s) merge_ml[r] = make_float2(M, l);
        ok = meet();
        if (!s && ok) other = merge_ml[r], merge_ml[r] = make_float2(M, l);
        ok = ok && meet() && wait_warp(bars.o_done + (s ^ 1), no_other & 1);
        if (!ok) break;
        if (s) other = merge_ml[r];
        ++no_other;
        const float top = fmaxf(M, other.x);
        w_own = M == -INFINITY ? 0.f : exp2f(M - top);
        w_other = other.x == -INFINITY ? 0.f : exp2f(other.x - top);
        M = top;
        sum = l * w_own + other.y * w_other;
      }
      if (paired) ++no_other;
      tc_fence_after();
      if (!idle) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float f_own = w_own * inv, f_other = w_other * inv;
        const uint32_t to_other = tmem + Ahead<D>::o_col(s ^ 1) + lane_sel;
        const int token = seg.tok0 + tok;
        const long long out_row = (long long)token * d.Hq + seg.h * G + (srow0 + r - tok * G);
        const int q0 = shared ? s * (D / 2) : 0, q1 = shared ? q0 + D / 2 : D;
#pragma unroll 1
        for (int q = q0; q < q1; q += 32) {
          float o[32];
          tmem_ld32(to + q, o);
          if (shared) {
            float x[32];
            tmem_ld32(to_other + q, x);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = (w_own == 0.f ? 0.f : o[j] * f_own) + (w_other == 0.f ? 0.f : x[j] * f_other);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = sum == 0.f ? 0.f : o[j] * inv;  // (a row without keys is 0, whatever values others see)
          }
          if (r < rows) {
            if (seg.part < 0) {
              uint4* const out = reinterpret_cast<uint4*>(p.out + out_row * D + q);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                out[j] = make_uint4(pack2<F16>(o[8 * j], o[8 * j + 1]), pack2<F16>(o[8 * j + 2], o[8 * j + 3]),
                                    pack2<F16>(o[8 * j + 4], o[8 * j + 5]), pack2<F16>(o[8 * j + 6], o[8 * j + 7]));
            } else {
              float* const out = w.o + (long long)(seg.part + srow0 + r) * D + q;
#pragma unroll
              for (int j = 0; j < 32; j += 8) store8(out + j, o + j);
            }
          }
        }
        if (r < rows && q0 == 0) {
          const float e = sum == 0.f ? -INFINITY : M + log2f(sum);
          if (seg.part >= 0)
            w.lse[seg.part + srow0 + r] = e;
          else if (p.lse)
            p.lse[out_row] = e * kLn2;
        }
      }
      tc_fence_before();
      // neither stream's next products overwrite sums that the other group still reads
      if (shared && !meet()) {
        ok = false;
        break;
      }
      done();
    }
  } else if (warp == 11) {
    // ------------------------------------------------------------ segments and queries, ahead of the rest
    // As in kv_attn.cu: segments go out as the ring has room, and a segment's queries as soon as the products with
    // the ones before are done.  Queries come by TMA, whole tokens of G heads: rows behind the block's last hold
    // other tokens' queries or what was there, and nothing reads their results.
    SegWalk<kTileThreads, kBlockRows> walk(p, w, cut, plan, before, int(blockIdx.x), lane);
    uint32_t k = 0, kq = 0;      // segments handed on; segment whose queries are next
    uint32_t nq0 = 0, nq1 = 0;   // segments of each stream
    int part = 0;                // of segment kq: its first or second stream
    uint32_t idle = 0;
    bool more = true, ok = true;
    while (ok && (more || kq < k)) {
      bool did = false;
      if (more && __all_sync(0xffffffffu, mbar_look(bars.seg_empty + k % kSegRing, ((k / kSegRing) & 1) ^ 1))) {
        Seg seg;
        more = walk.next(seg);
        if (lane == 0) {
          if (!more) seg.t1 = -1;
          segs[k % kSegRing] = seg;
          mbar_arrive(bars.seg_full + k % kSegRing);
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
        if (nq == 0 || __all_sync(0xffffffffu, mbar_look(bars.q_free + s, (nq - 1) & 1))) {
          if (lane == 0) mbar_arrive_expect_tx(bars.q_ready + s, uint32_t(tile_rows) * D * 2);
          __syncwarp();
          if (lane < D / 64)
            tma_load3(base + L::OFF_Q + s * L::BYTES + lane * L::HALF, &maps.queries, lane * 64, seg.h * G,
                      seg.tok0 + (paired ? s * tile_toks : 0), smem_addr(bars.q_ready + s));
          if (s)
            ++nq1;
          else
            ++nq0;
          if (++part == 2 || (!paired && seg.t1 - seg.t0 == 1)) {
            part = 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.seg_empty + kq % kSegRing);
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
      if (nq0 > 0) mbar_drain(bars.q_ready, (nq0 - 1) & 1);
      if (nq1 > 0) mbar_drain(bars.q_ready + 1, (nq1 - 1) & 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- few rows
// Where sequences have about eight rows to a kv head or fewer (single tokens, with their heads), a tile of 128 rows is all
// padding and its chain of products, not the memory, sets the pace (64 single tokens over 1..1500 keys: 71 us with it, 45
// here).
// Here a block is up to 8 rows, and a warp is a worker by itself: it takes 16 keys at a time, straight from
// memory into the registers that the warp-wide products (m16n8k16) read, and no shared memory or barrier is in the way.
// The elements of a head and the keys are summed in an order of the lanes' own, so that each lane's operands are
// 16 bytes that lie together:
//   S = Q K^T: lane (n, j) = (lane / 4, lane % 4) holds elements 32 c + 8 j .. + 7 of query n and of key n (and n + 8);
//   O^T = V^T P^T: it holds elements 64 c + 8 n .. + 7 of keys 2 j, 2 j + 1, 2 j + 8, 2 j + 9 - the keys whose scores of
//   row n it has from S - and gets elements 64 c + 8 n .. + 7 of rows 2 j and 2 j + 1.
// P is rounded to the type of V, as in the tiles.
// Keys of the round to come are fetched as soon as the products have read the ones before, and values likewise, so that
// one or the other is always on its way.  Bound: HBM (4000 keys at Hkv=8 D=128 5.9 TB/s), at short lengths the trips to
// memory that a segment begins with, one behind the other: bounds, page numbers, keys.  Four CTAs to an SM at D = 64 (122
// registers; 5 spill and are as fast, 3 take 53 us for 45), three at D = 128 (89 us at 4000 keys, 98 with two or four).
template <bool F16>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int D, bool F16>
__global__ void __launch_bounds__(kFewThreads, few_ctas(D))
    packed_few_kernel(const __grid_constant__ PackedAttnParams p, const __grid_constant__ PackedWs w, const __grid_constant__ Cut cut, const uint32_t page_inv) {
  constexpr int CK = D / 32, CV = D / 64;  // parts of a key and of a value in a lane
  __shared__ Plan plan;
  __shared__ long long before[kFewThreads + 32];
  pdl_launch_dependents();
  pdl_wait();
  make_plan<kFewThreads>(p, cut, plan, before);
  if (plan.empty) write_empty(p, cut);
  const gdn_kv_dims& d = p.d;
  const int lane = threadIdx.x & 31, n = lane >> 2, j = lane & 3, G = d.Hq / d.Hkv;
  // (neighbours of a stretch on different SMs: the last stretches of a short list are not all on a few)
  SegWalk<kFewThreads, kFewRows> walk(p, w, cut, plan, before, int(threadIdx.x >> 5) * int(gridDim.x) + int(blockIdx.x), lane);
  const float c = p.scale * kLog2e;
  Seg seg;
  while (walk.next(seg)) {
    const int rows = seg.rows, tiles = seg.t1 - seg.t0;
    // queries: zeros in rows that the block has not
    uint32_t q[CK][4];
#pragma unroll
    for (int i = 0; i < CK; ++i) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (n < rows) x = load16(p.q + (long long)(seg.tok0 + n / G) * d.q_token_stride + (seg.h * G + n % G) * D + 32 * i + 8 * j);
      q[i][0] = x.x, q[i][1] = x.y, q[i][2] = x.z, q[i][3] = x.w;
    }
    const int lim = seg.lim + (cut.causal ? n / G : 0);  // own keys that row n sees
    // Places of 16 tiles' keys: lane 2 i + e has those of keys 16 e .. 16 e + 15 of tile i
    long long place = 0;
    auto look_up = [&](int t) {
      const int mine = t + (lane >> 1);
      if (mine < seg.t1) {
        const bool own = mine >= seg.pre_tiles;
        const int token = (own ? mine - seg.pre_tiles : mine) * 32 + 16 * (lane & 1);
        if (token < (own ? seg.keys : seg.pre_keys)) {
          const int col = page_column(token, page_inv);
          int page = p.table[(long long)(own ? seg.slot : seg.pre_slot) * d.max_pages + col];
          if (page < 0 || page >= d.n_pages) {
            atomicOr(p.err, GDN_DEVERR_KV_PAGE);
            page = 0;
          }
          place = page * d.cache_page_stride + (token - col * d.page_size) * d.cache_token_stride + seg.h * d.cache_head_stride;
        }
      }
    };
    // keys of round r that some row sees (may exceed the round's)
    auto left_of = [&](int r) {
      const int t = seg.t0 + r / 2, in = r % 2 * 16;
      return t >= seg.pre_tiles ? seg.keys - 32 * (t - seg.pre_tiles) - in : seg.pre_keys - 32 * t - in;
    };
    auto place_of = [&](int r) { return __shfl_sync(0xffffffffu, place, r & 31); };
    uint4 kx[2][CK], vx[4][CV];
    auto fetch_keys = [&](int r) {
      const int left = left_of(r);
      const long long at = place_of(r);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < CK; ++i)
          kx[u][i] = left > 0 ? load16(p.k_cache + at + (8 * u + n) * d.cache_token_stride + 32 * i + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto fetch_values = [&](int r) {
      const int left = left_of(r);
      const long long at = place_of(r);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int key = 2 * j + (u & 1) + 8 * (u >> 1);
#pragma unroll
        for (int i = 0; i < CV; ++i)  // (values behind the last key may be anything, and 0 x NaN is NaN)
          vx[u][i] = key < left ? load16(p.v_cache + at + key * d.cache_token_stride + 64 * i + 8 * n) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    float o[CV][4][4];
#pragma unroll
    for (int i = 0; i < CV; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][t][x] = 0.f;
    float m = -INFINITY, l = 0.f;  // of row n: running maximum (log2 units), this lane's part of the sum
    const int rounds = 2 * tiles;
    look_up(seg.t0);
    fetch_keys(0);
    fetch_values(0);
#pragma unroll 1
    for (int r = 0; r < rounds; ++r) {
      const int t = seg.t0 + r / 2;
      float sc[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        sc[u][0] = sc[u][1] = sc[u][2] = sc[u][3] = 0.f;
#pragma unroll
        for (int i = 0; i < CK; ++i) {
          mma_16x8x16<F16>(sc[u], q[i][0], 0u, q[i][1], 0u, kx[u][i].x, kx[u][i].y);
          mma_16x8x16<F16>(sc[u], q[i][2], 0u, q[i][3], 0u, kx[u][i].z, kx[u][i].w);
        }
      }
      const bool more = r + 1 < rounds;
      const bool own = t >= seg.pre_tiles;
      const int sees = (own ? lim - 32 * (t - seg.pre_tiles) : seg.pre_keys - 32 * t) - r % 2 * 16;  // keys of this round that row n sees
      if (more) {
        if ((r + 1) % 32 == 0) look_up(seg.t0 + (r + 1) / 2);  // (the values of the round before are on their way already)
        fetch_keys(r + 1);
      }
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[i][e] = 8 * i + 2 * j + e < sees ? sc[i][e] * c : -INFINITY;
          top = fmaxf(top, sc[i][e]);
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const bool move = top > m && !(top - m <= kLag);  // (m = -inf: infinitely far)
      if (__any_sync(0xffffffffu, move)) {
        const float f = move ? exp2_fast(m - top) : 1.f;
        if (move) m = top;
        l *= f;
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * j), f1 = __shfl_sync(0xffffffffu, f, 8 * j + 4);  // of rows 2 j, 2 j + 1
#pragma unroll
        for (int i = 0; i < CV; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[i][x][0] *= f0, o[i][x][1] *= f1, o[i][x][2] *= f0, o[i][x][3] *= f1;
      }
      const float base = m == -INFINITY ? 0.f : m;
      uint32_t pr[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float w0 = exp2_fast(sc[u][0] - base), w1 = exp2_fast(sc[u][1] - base);
        l += w0 + w1;
        pr[u] = pack2<F16>(w0, w1);
      }
#pragma unroll
      for (int i = 0; i < CV; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // elements 64 i + 8 n + 2 x and the one behind
          const uint32_t w0 = word(vx[0][i], x), w1 = word(vx[1][i], x), w2 = word(vx[2][i], x), w3 = word(vx[3][i], x);
          mma_16x8x16<F16>(o[i][x], __byte_perm(w0, w1, 0x5410), __byte_perm(w0, w1, 0x7632), __byte_perm(w2, w3, 0x5410),
                           __byte_perm(w2, w3, 0x7632), pr[0], pr[1]);
        }
      if (more) fetch_values(r + 1);
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const float inv = l == 0.f ? 0.f : 1.f / l, e = l == 0.f ? -INFINITY : m + log2f(l);
    const int tok = n / G;
    if (j == 0 && n < rows) {
      if (seg.part >= 0)
        w.lse[seg.part + n] = e;
      else if (p.lse)
        p.lse[(long long)(seg.tok0 + tok) * d.Hq + seg.h * G + (n - tok * G)] = e * kLn2;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {  // rows 2 j and 2 j + 1
      const int r = 2 * j + u, rt = r / G;
      const float f = __shfl_sync(0xffffffffu, inv, 4 * r);
      if (r < rows) {
#pragma unroll
        for (int i = 0; i < CV; ++i) {
          float y[8];
#pragma unroll
          for (int x = 0; x < 4; ++x) y[2 * x] = f == 0.f ? 0.f : o[i][x][u] * f, y[2 * x + 1] = f == 0.f ? 0.f : o[i][x][2 + u] * f;
          if (seg.part >= 0)
            store8(w.o + (long long)(seg.part + r) * D + 64 * i + 8 * n, y);
          else
            *reinterpret_cast<uint4*>(p.out + ((long long)(seg.tok0 + rt) * d.Hq + seg.h * G + (r - rt * G)) * D + 64 * i + 8 * n) =
                make_uint4(pack2<F16>(y[0], y[1]), pack2<F16>(y[2], y[3]), pack2<F16>(y[4], y[5]), pack2<F16>(y[6], y[7]));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- join
// `chunks` CTAs for every PER workers.  An item of a few pieces is joined by those of the worker that it begins with, one of many
// by those of all its workers together.  D / 8 lanes sum a row's pieces; 2, 4, .. such groups of a CTA share a row where pieces
// are many and the rows do not keep all groups busy, and their sums are joined in shared memory.  Bound: the trips to L2 (the
// item, its pieces) and the start of its CTAs.  A warp to each row, all by the CTAs of the item's first worker, took 119 us where
// this takes 113 (prompts of 1..901 tokens behind 1531 shared and 0..333 own), 71 where this takes 54 (a token behind 65536, Hq=32
// Hkv=8 D=128) and 195 where this takes 35 (Hq=8 Hkv=1).
template <int D, bool F16, int ROWS, int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) packed_join_kernel(const __grid_constant__ PackedAttnParams p, const __grid_constant__ PackedWs w, const int chunks) {
  constexpr int LANES = D / 8, GROUPS = THREADS / LANES, U = ROWS == kFewRows ? 4 : 2;  // (pieces in flight: more are more registers)
  __shared__ float4 sums[GROUPS][2][LANES];
  __shared__ float2 weights[GROUPS];
  pdl_launch_dependents();
  pdl_wait();
  const gdn_kv_dims& d = p.d;
  __shared__ JoinRec recs[PER + 1];
  __shared__ int begins[PER + 1];  // the workers that the items begin with
  const int me = int(blockIdx.x) / chunks, chunk = int(blockIdx.x) - me * chunks;  // of the CTAs of workers PER me .. PER me + PER - 1
  const int G = d.Hq / d.Hkv, lane = int(threadIdx.x) % LANES, group = int(threadIdx.x) / LANES;
  if (int(threadIdx.x) < PER) {
    const int c = PER * me + int(threadIdx.x);
    const JoinRec rec = w.join[c];
    recs[threadIdx.x] = rec, begins[threadIdx.x] = c;
    if (threadIdx.x == 0) {
      JoinRec other{};
      if (rec.before >= 0) other = w.join[rec.before];
      recs[PER] = other, begins[PER] = rec.before;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i <= PER; ++i) {
    const JoinRec rec = recs[i];
    if (rec.rows == 0) continue;
    const int c0 = begins[i], parts = rec.end - c0 + 1, first = c0 / PER;
    const int ctas = (parts > kJoinAlone ? rec.end / PER - first + 1 : 1) * chunks, cta = (me - first) * chunks + chunk;
    if (cta >= ctas) continue;
    int log = 0;
    while ((1 << log) < GROUPS && (rec.rows << (log + 1)) <= ctas * GROUPS && (8 << log) <= parts) ++log;
    const int split = 1 << log, s = group & (split - 1), each = (parts + split - 1) >> log, rows = GROUPS >> log;
    // piece j's row: the first worker's piece, then the one that each stretch begins with
    for (int r0 = cta * rows; r0 < rec.rows; r0 += ctas * rows) {
      const int r = r0 + (group >> log);
      auto at = [&](int j) { return (j == 0 ? rec.part0 : 2 * (c0 + j) * ROWS) + r; };
      const int mine = r < rec.rows ? parts : 0;
      float4 v[U][2];
      auto load = [&](int i0) {  // this group's pieces i0, i0 + 1, ..
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (s + split * (i0 + u) < mine) {
            const float4* o = reinterpret_cast<const float4*>(w.o + (long long)at(s + split * (i0 + u)) * D) + 2 * lane;
            v[u][0] = o[0], v[u][1] = o[1];
          }
      };
      float acc[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.f;
      float M = -INFINITY, W = 0.f;
      for (int b0 = 0; b0 < each; b0 += LANES) {
        const int j = s + split * (b0 + lane), n = each - b0 < LANES ? each - b0 : LANES;
        const float e = j < mine ? w.lse[at(j)] : -INFINITY;
        load(b0);
        float mx = e;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float Mn = fmaxf(M, mx), f = M == -INFINITY ? 0.f : exp2_fast(M - Mn);
        const float wt = e == -INFINITY ? 0.f : exp2_fast(e - (Mn == -INFINITY ? 0.f : Mn));  // (NaN stays NaN)
        float all = wt;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        M = Mn, W = W * f + all;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= f;
        for (int i0 = 0; i0 < n; i0 += U) {
          if (i0 > 0) load(b0 + i0);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float wj = i0 + u < n ? __shfl_sync(0xffffffffu, wt, i0 + u, LANES) : 0.f;
            if (wj != 0.f) {
              acc[0] += wj * v[u][0].x, acc[1] += wj * v[u][0].y, acc[2] += wj * v[u][0].z, acc[3] += wj * v[u][0].w;
              acc[4] += wj * v[u][1].x, acc[5] += wj * v[u][1].y, acc[6] += wj * v[u][1].z, acc[7] += wj * v[u][1].w;
            }
          }
        }
      }
      if (split > 1) {
        __syncthreads();
        sums[group][0][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]), sums[group][1][lane] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (lane == 0) weights[group] = make_float2(M, W);
        __syncthreads();
        if (s == 0) {
          for (int x = 1; x < split; ++x) M = fmaxf(M, weights[group + x].x);
          W = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = 0.f;
          for (int x = 0; x < split; ++x) {
            const float2 mw = weights[group + x];
            const float f = mw.x == -INFINITY ? 0.f : exp2_fast(mw.x - M);
            const float4 a = sums[group + x][0][lane], b = sums[group + x][1][lane];
            W += f * mw.y;
            acc[0] += f * a.x, acc[1] += f * a.y, acc[2] += f * a.z, acc[3] += f * a.w;
            acc[4] += f * b.x, acc[5] += f * b.y, acc[6] += f * b.z, acc[7] += f * b.w;
          }
        }
      }
      if (s != 0 || r >= rec.rows) continue;
      const float inv = W == 0.f ? 0.f : __fdividef(1.f, W);
      const int tok = r / G;
      const long long row = (long long)(rec.tok0 + tok) * d.Hq + rec.h * G + (r - tok * G);
      *reinterpret_cast<uint4*>(p.out + row * D + 8 * lane) =
          make_uint4(pack2<F16>(acc[0] * inv, acc[1] * inv), pack2<F16>(acc[2] * inv, acc[3] * inv), pack2<F16>(acc[4] * inv, acc[5] * inv),
                     pack2<F16>(acc[6] * inv, acc[7] * inv));
      if (p.lse && lane == 0) p.lse[row] = W == 0.f ? -INFINITY : (M + log2f(W)) * kLn2;
    }
  }
}

// ---------------------------------------------------------------- launches
template <int D, bool F16>
cudaError_t launch(const PackedAttnParams& p, const PackedWs& w, const Cut& cut, int box, const PackedMaps& maps, cudaStream_t stream) {
  using L = TileLayout<D, Seg>;
  static_assert(L::TOTAL + 1536 <= 232448, "shared memory");
  static std::atomic<uint64_t> allowed{0};  // a bit per device: the kernel may use its shared memory there
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(allowed.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(packed_tile_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::TOTAL);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(1ull << (dev & 63));
  }
  e = launch_dependent(packed_tile_kernel<D, F16>, unsigned(kCtas), kTileThreads, L::TOTAL, stream, p, w, cut, box, page_units_inv(p.d.page_size), maps);
  if (e != cudaSuccess) return e;
  return launch_dependent(packed_join_kernel<D, F16, kBlockRows, 256, 1>, unsigned(kCtas * kJoinChunks), 256, 0, stream, p, w, kJoinChunks);
}

template <int D, bool F16>
cudaError_t launch_few(const PackedAttnParams& p, const PackedWs& w, const Cut& cut, cudaStream_t stream) {
  // Loads in flight need room in L1, which a kernel with all of the shared memory leaves little of, and a kernel that can do
  // with what it finds does not have it changed: 64 tokens behind 4000 157 us by themselves, 245 next to the tiles, 167 there
  // when asked for (10 % is room for all CTAs; with 0 a part of them waits at D = 64: 50 -> 73 us).
  static std::atomic<uint64_t> asked{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(asked.load() >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(packed_few_kernel<D, F16>, cudaFuncAttributePreferredSharedMemoryCarveout, 10);
    if (e != cudaSuccess) return e;
    asked.fetch_or(1ull << (dev & 63));
  }
  e = launch_dependent(packed_few_kernel<D, F16>, unsigned(kCtas * few_ctas(D)), kFewThreads, 0, stream, p, w, cut, page_units_inv(p.d.page_size));
  if (e != cudaSuccess) return e;
  // A token's items by wide CTAs for four workers, where they are few and in hundreds of pieces each, or by a small one for each
  // worker: 8 items behind 65536 keys 54 and 59 us, one 35 and 79, but 16 (D = 64) 57 and 54, and 1024 of 1..1500 keys 49 and 45.
  const long long blocks = p.n_tokens / cut.toks + p.d.B, items = (blocks < p.n_tokens ? blocks : p.n_tokens) * p.d.Hkv;  // at most
  if (items <= 8) return launch_dependent(packed_join_kernel<D, F16, kFewRows, 256, 4>, unsigned(cut.workers / 4), 256, 0, stream, p, w, 1);
  return launch_dependent(packed_join_kernel<D, F16, kFewRows, 64, 1>, unsigned(cut.workers), 64, 0, stream, p, w, 1);
}

// How rows are cut into blocks of `toks` tokens, and keys into tiles of 2^key_log, dealt to so many workers.
Cut make_cut(int tile_toks, int toks, int key_log, int causal, int workers, int least, int most) {
  Cut c{tile_toks, toks, key_log, 0, causal, workers, least, most};
  while ((c.toks << c.period_log) % (1 << key_log)) ++c.period_log;
  return c;
}

}  // namespace

size_t packed_attn_workspace_bytes(const gdn_kv_dims& d, int64_t) {
  size_t n = 0;
  carve_packed(nullptr, d, &n);
  return n;
}

cudaError_t launch_packed_attn(const PackedAttnParams& p, cudaStream_t stream) {
  const gdn_kv_dims& d = p.d;
  const int G = d.Hq / d.Hkv, toks = kTileRows / G;
  const PackedWs w = carve_packed(p.ws, d, nullptr);
  // Few rows or tiles: the host knows how many rows and sequences there are and how long a slot can be, the device alone how
  // the rows are distributed.  The kernel for few rows reads a sequence's keys once for every 8 rows, so it is for sequences
  // of that many: us with it and with tiles, 64 sequences of 1..1500 keys f16 Hkv=16 D=64 1 row 44 and 64, 8 rows 43 and 65;
  // bf16 Hkv=8 D=128 4 rows 39 and 46, 8 rows 40 and 48, 12 rows 67 and 52; 8 such sequences 15 and 19.  But 200 tokens of one
  // sequence behind 30000 1235 and 112, 16 behind 65536 218 and 55, 16 behind 1000 20 and 15.
  //  - It takes all that has at most 8 rows a sequence and kv head on average (of more than 512 tokens, a token), if what it
  //    would read should all tokens be one sequence's costs no more than it saves, a few us.  That they are as many as
  //    the sequences makes a token each likely, and more can be risked.
  //  - Else each kernel takes its sequences, one after the other: 255 tokens of as many sequences behind 1000 and 257 of one
  //    behind 65536 412 us (3790 with few rows alone).  The second pair of launches costs 7 us where it has nothing to do.
  //    Both and tiles alone: 64 x 8 rows D=64 51 and 65, 128 x 8 rows D=128 81 and 85, 32 x 8 rows 36 and 33, 16 x 8 rows 30 and
  //    23: below 32 sequences tiles take all.
  int least = 0;  // tokens of the sequences that the tiles take
  if (G <= kFewRows && (long long)p.n_tokens * G <= (long long)kFewRows * d.B && (p.n_tokens <= 512 || p.n_tokens <= d.B)) {
    const int few = kFewRows / G;
    const double slot = double(d.max_pages) * d.page_size * (p.prefix_of ? 2 : 1);
    const double read = ctas_of(p.n_tokens, few) * slot * d.Hkv * d.D * 4.0;  // bytes, at 10 TB/s
    const bool alone = p.n_tokens <= few || read <= (p.n_tokens == d.B ? 1e9 : 64e6);
    if (alone || (p.n_tokens >= 32 && d.B >= 32)) {
      const Cut cut = make_cut(few, few, 5, p.causal, few_workers(d.D), 0, alone ? INT_MAX : few);
      const cudaError_t e = d.D == 128 ? (d.dtype ? launch_few<128, true>(p, w, cut, stream) : launch_few<128, false>(p, w, cut, stream))
                                       : (d.dtype ? launch_few<64, true>(p, w, cut, stream) : launch_few<64, false>(p, w, cut, stream));
      if (e != cudaSuccess || alone) return e;
      least = few + 1;
    }
  }
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
  PackedMaps maps;
  const cuuint64_t cd[5] = {cuuint64_t(d.D), cuuint64_t(d.page_size), cuuint64_t(d.Hkv), cuuint64_t(d.n_pages), 1};
  const cuuint64_t cs[4] = {2ull * d.cache_token_stride, 2ull * d.cache_head_stride, 2ull * d.cache_page_stride, 2ull * d.cache_layer_stride};
  const cuuint32_t b16[5] = {64, 16, 1, 1, 1}, bb[5] = {64, cuuint32_t(box), 1, 1, 1};
  map(&maps.few[0], p.k_cache, 5, cd, cs, b16);
  map(&maps.few[1], p.v_cache, 5, cd, cs, b16);
  if (box > 16) {
    map(&maps.many[0], p.k_cache, 5, cd, cs, bb);
    map(&maps.many[1], p.v_cache, 5, cd, cs, bb);
  } else {
    maps.many[0] = maps.few[0], maps.many[1] = maps.few[1];
  }
  const cuuint64_t qd[3] = {cuuint64_t(d.D), cuuint64_t(d.Hq), cuuint64_t(p.n_tokens)};
  const cuuint64_t qst[2] = {2ull * d.D, 2ull * d.q_token_stride};
  const cuuint32_t bt[3] = {64, cuuint32_t(G), cuuint32_t(toks)};
  map(&maps.queries, p.q, 3, qd, qst, bt);
  if (!ok) return cudaErrorInvalidValue;
  const Cut cut = make_cut(toks, 2 * toks, 7, p.causal, kCtas, least, INT_MAX);
  if (d.D == 128) return d.dtype ? launch<128, true>(p, w, cut, box, maps, stream) : launch<128, false>(p, w, cut, box, maps, stream);
  return d.dtype ? launch<64, true>(p, w, cut, box, maps, stream) : launch<64, false>(p, w, cut, box, maps, stream);
}

}  // namespace gdn
