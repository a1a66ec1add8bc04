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
// Kernels: tiles (persistent, tcgen05; every CTA plans for itself), join.
//
// A block of more than 128 rows gives each stream half of them, on the same keys; a smaller one gives the
// streams alternate tiles of the same rows, and at its end the two sums are joined in tensor memory, each
// softmax group taking half of the columns.
#include <atomic>

#include "kv_device.cuh"
#include "kv_index.h"
#include "kv_tile.cuh"

namespace gdn {

namespace {

constexpr int kJoinWarps = 8, kJoinChunks = 8;  // CTAs to a cut item

struct JoinRec {       // a cut item, by the CTA c0 that it begins in; it ends in CTA c1
  int32_t tok0, rows;  // rows 0: there is none
  int32_t h, c0, c1, part0;
};

struct PackedWs {
  JoinRec* join;     // [kCtas]
  float* lse;        // [kCtas][2][kBlockRows] log2 units
  float* o;          // [kCtas][2][kBlockRows][D]
};

__host__ __device__ inline size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

__host__ __device__ inline PackedWs carve_packed(void* base, const gdn_kv_dims& d, size_t* total) {
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t o = 0;
  const size_t parts = 2 * size_t(kBlockRows) * kCtas;
  PackedWs w;
  w.join = reinterpret_cast<JoinRec*>(p + o), o += round256(sizeof(JoinRec) * kCtas);
  w.lse = reinterpret_cast<float*>(p + o), o += round256(4 * parts);
  w.o = reinterpret_cast<float*>(p + o), o += 4 * parts * size_t(d.D);
  if (total) *total = o;
  return w;
}

// ---------------------------------------------------------------- the plan
// How the calls' rows are cut into blocks: all that depends on the heads alone.
struct Cut {
  int tile_toks, toks;  // tokens of a row tile, of a block
  int period_log;       // after so many (2^period_log) blocks, their keys are a whole number of tiles more
  int causal;
};

struct SeqRows {
  int lo, n;       // its packed tokens
  int len;         // tokens in its slot
  int pre_slot, pre_keys;
  __device__ __forceinline__ int pre_tiles() const { return (pre_keys + kTileKeys - 1) / kTileKeys; }
  __device__ __forceinline__ int blocks(const Cut& c) const { return int((unsigned(n) + unsigned(c.toks) - 1u) / unsigned(c.toks)); }
  // own keys that the last row of block k sees
  __device__ __forceinline__ int keys(const Cut& c, int k) const {
    if (!c.causal) return len;
    const long long e = (long long)len - n + (long long)c.toks * (k + 1);
    return e < 0 ? 0 : e < len ? int(e) : len;
  }
  // Tiles of the first k blocks: sums of ceil(keys / 128), period by period.
  __device__ __forceinline__ long long tiles(const Cut& c, int k) const {
    const long long pre = (long long)pre_tiles() * k;
    if (!c.causal) return pre + (long long)((len + kTileKeys - 1) / kTileKeys) * k;
    const long long off = (long long)len - n;
    const int i0 = off >= 0 ? 1 : int((unsigned long long)(-off) / unsigned(c.toks)) + 1;  // the first block with keys, counted from 1
    long long sum = 0;
    if (k >= i0) {
      const long long m = (long long)k - i0 + 1, first = off + (long long)c.toks * i0 + kTileKeys - 1;
      const int period = 1 << c.period_log, rest = int(m & (period - 1));
      const long long whole = m >> c.period_log, more = (long long)c.toks << c.period_log >> 7;  // (tiles that a period adds)
      long long one = 0, part = 0;
      for (int i = 0; i < period && i < m; ++i) {
        const long long t = (first + (long long)c.toks * i) >> 7;
        one += t;
        if (i < rest) part += t;
      }
      sum = (whole > 0 ? whole * one : 0) + (more * whole * (whole - 1) / 2 << c.period_log) + part + rest * more * whole;
    }
    if (k == blocks(c) && k > 0) {  // the last block is as long as it is
      const long long e = off + (long long)c.toks * k;
      sum += (len + kTileKeys - 1) / kTileKeys - (e > 0 ? (e + kTileKeys - 1) >> 7 : 0);
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

__device__ __forceinline__ SeqRows load_sequence(const PackedAttnParams& p, int b, bool report) {
  const gdn_kv_dims& d = p.d;
  SeqRows s;
  const int lo = p.cu[b], hi = p.cu[b + 1], len = p.seq_len[d.slot0 + b], slot = p.prefix_of ? p.prefix_of[b] : -1;
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
  if (bad && report) atomicOr(p.err, bad);
  return s;
}

// Every CTA plans for itself: each thread sums the tiles of a few consecutive sequences, the CTA the sums of its
// threads, and the thread that has the first tile of the CTA's stretch among its own says in which sequence.
struct Plan {
  long long head_tiles, tiles;  // of one kv head, and of all
  long long into;               // the stretch begins so many tiles into
  int32_t b, h;                 // sequence b, kv head h
  int32_t ctas;                 // that the tiles are dealt to: each has one at least
  int32_t empty;                // some rows have no keys
  // The deal gives CTA c tiles [begin(c), begin(c + 1)); the CTA of tile x.
  __device__ __forceinline__ long long begin(long long c) const { return c * tiles / ctas; }
  __device__ __forceinline__ int cta_of(long long x) const {
    int c = int(float(x) * (float(ctas) / float(tiles)));  // (within one of it)
    c = c < 0 ? 0 : c > ctas - 1 ? ctas - 1 : c;
    while (c > 0 && begin(c) > x) --c;
    while (c < ctas - 1 && begin(c + 1) <= x) ++c;
    return c;
  }
};

__device__ __forceinline__ void make_plan(const PackedAttnParams& p, const Cut& cut, Plan& plan, long long* sums) {
  const gdn_kv_dims& d = p.d;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, cta = int(blockIdx.x);
  const int each = (d.B + kTileThreads - 1) / kTileThreads;
  const int b0 = tid * each < d.B ? tid * each : d.B, b1 = b0 + each < d.B ? b0 + each : d.B;
  bool bad = tid == 0 && (p.cu[0] != 0 || p.cu[d.B] > p.n_tokens), empty = false;
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    bad |= p.cu[b] > p.cu[b + 1];
    const SeqRows s = load_sequence(p, b, cta == 0);
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
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kTileThreads / 32; ++i) {
    before += i < warp ? sums[i] : 0;
    all += sums[i];
  }
  before += x - mine;
  if (bad) all = 0;
  Plan q;
  q.head_tiles = all, q.tiles = all * d.Hkv;
  q.ctas = int(q.tiles < kCtas ? q.tiles : kCtas);
  q.empty = empty && !bad;
  q.b = q.h = 0, q.into = 0;
  if (tid == 0 && bad && cta == 0) atomicOr(p.err, kDevErrSeqlens);
  if (cta >= q.ctas) {
    if (tid == 0) plan = q;
  } else {
    const long long first = q.begin(cta);
    q.h = int(first / q.head_tiles);
    long long y = first - q.h * q.head_tiles;
    if (y >= before && y < before + mine) {  // (one thread)
      y -= before;
      for (int b = b0; b < b1; ++b) {
        const SeqRows s = load_sequence(p, b, false);
        const long long t = s.tiles(cut, s.blocks(cut));
        if (y < t) {
          q.b = b, q.into = y;
          break;
        }
        y -= t;
      }
      plan = q;
    }
  }
  __syncthreads();
}

// Outputs of rows without keys, whole blocks of them: 0 and -inf.
__device__ __noinline__ void write_empty(const PackedAttnParams& p, const Cut& cut) {
  const gdn_kv_dims& d = p.d;
  for (int b = int(blockIdx.x); b < d.B; b += kCtas) {
    const SeqRows s = load_sequence(p, b, false);
    const long long rows = (long long)s.without_keys(cut) * d.Hq, first = (long long)s.lo * d.Hq;
    uint4* const out = reinterpret_cast<uint4*>(p.out + first * d.D);
    for (long long k = threadIdx.x; k < rows * (d.D / 8); k += kTileThreads) out[k] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse)
      for (long long k = threadIdx.x; k < rows; k += kTileThreads) p.lse[first + k] = -INFINITY;
  }
}

// ---------------------------------------------------------------- segments
struct Seg {
  int tok0, rows;               // packed tokens, rows of the block
  int h;                        // kv head
  int pair;                     // they fill more than one row tile: both streams take every tile of keys
  int slot, keys, lim;          // as in BlockRec
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

// Walks a CTA's stretch segment by segment (a converged warp).  Lane i knows sequence from + i.
struct SegWalk {
  const PackedAttnParams& p;
  const PackedWs& w;
  const Cut& cut;
  const Plan& plan;
  const int cta, lane, G;
  long long begin, x, end;
  int h, b, k, t_in;  // the item at hand: kv head, sequence, block; its tiles before x
  int from;
  SeqRows mine;
  __device__ __forceinline__ SeqRows sequence(int i) {
    if (i < from || i >= from + 32) {
      from = i;
      const int at = i + lane < p.d.B ? i + lane : p.d.B - 1;
      mine = load_sequence(p, at, false);
    }
    const int l = i - from;
    SeqRows s;
    s.lo = __shfl_sync(0xffffffffu, mine.lo, l), s.n = __shfl_sync(0xffffffffu, mine.n, l);
    s.len = __shfl_sync(0xffffffffu, mine.len, l), s.pre_slot = __shfl_sync(0xffffffffu, mine.pre_slot, l);
    s.pre_keys = __shfl_sync(0xffffffffu, mine.pre_keys, l);
    return s;
  }
  __device__ __forceinline__ SegWalk(const PackedAttnParams& p_, const PackedWs& w_, const Cut& cut_, const Plan& plan_, int lane_)
      : p(p_), w(w_), cut(cut_), plan(plan_), cta(int(blockIdx.x)), lane(lane_), G(p_.d.Hq / p_.d.Hkv) {
    begin = x = end = 0;
    h = b = k = t_in = 0;
    from = -64;
    if (lane == 0) w.join[cta].rows = 0;
    if (cta >= plan.ctas) return;
    begin = x = plan.begin(cta), end = plan.begin(cta + 1);
    h = plan.h, b = plan.b;
    const SeqRows s = sequence(b);
    int n = s.blocks(cut);  // the last block with at most `into` tiles before it, 32 at a time
    while (n > 1) {
      const int step = (n + 31) / 32, i = lane * step;
      const uint32_t at_or_before = __ballot_sync(0xffffffffu, i < n && s.tiles(cut, k + i) <= plan.into);
      const int j = 31 - __clz(int(at_or_before));
      k += j * step;
      n = n - j * step < step ? n - j * step : step;
    }
    t_in = int(plan.into - s.tiles(cut, k));
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
      const int pre = s.pre_tiles(), keys = s.keys(cut, k), tiles = pre + (keys + kTileKeys - 1) / kTileKeys;
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
      const int second = x == begin ? 0 : 1;  // (of the CTA's pieces: one that its stretch begins with, one that it ends with)
      g.part = g.t0 == 0 && g.t1 == tiles ? -1 : (2 * cta + second) * kBlockRows;
      if (g.t0 == 0 && g.t1 < tiles && lane == 0)
        w.join[cta] = JoinRec{g.tok0, g.rows, h, cta, plan.cta_of(x + tiles - 1), g.part};
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
  // queries, (D, query head, token): boxes of G heads x the tokens of a row tile, and x a few tokens
  CUtensorMap qt, qs;
};
constexpr int kFewToks = 4;

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
  __shared__ float2 merge_ml[kTileRows];           // maximum (log2 units) and sum of a row, one stream's and then the other's
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - smem_addr(smem_raw));
  const TileBars bars = tile_bars<NS>(reinterpret_cast<uint64_t*>(smem + L::OFF_BAR));
  Seg* const segs = reinterpret_cast<Seg*>(smem + L::OFF_SEG);
  const int tid = int(threadIdx.x), warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const gdn_kv_dims& d = p.d;
  const int G = d.Hq / d.Hkv, tile_toks = cut.tile_toks, tile_rows = tile_toks * G;

  if (tid == 0) {
    init_tile_bars<NS>(bars);
    mbar_init(&merge_bar, 2 * kGroupThreads);
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
  make_plan(p, cut, plan, reinterpret_cast<long long*>(merge_ml));
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
    tensor_warp<D, F16>(warp - 9, lane, tmem, base, p.scale < 0.f, segs, bars, turns, wait_warp);
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax: stream s, one row per thread
    const int s = warp >> 2, r = tid & 127;
    const uint32_t lane_sel = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + tmem_s(s) + lane_sel, to = tmem + tmem_o(s) + lane_sel;
    const float c = fmaxf(fabsf(p.scale) * kLog2e, 1e-30f);  // (0 is as good as 1e-30)
    uint32_t n = 0, ns = 0;          // tiles of the CTA, tiles of this stream
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
      const uint32_t n0 = n;
      n += uint32_t(seg.t1 - seg.t0);
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
        if (!wait_warp(bars.s_ready + s, ns & 1)) {
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
          }, m, l);
        }
        first = false;
        if (left < kTileKeys && (left & 15)) {
          // values behind the last token of its unit may be anything: zero them, for 0 x NaN is NaN
          const uint32_t use = 2 * (n0 + uint32_t(t - seg.t0)) + 1, slot = use % NS;
          if (!wait_warp(bars.full + slot, (use / NS) & 1)) {
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
        mbar_arrive(bars.p_ready + s);
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
        const uint32_t to_other = tmem + tmem_o(s ^ 1) + lane_sel;
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
            for (int j = 0; j < 32; ++j) o[j] *= inv;
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
    SegWalk walk(p, w, cut, plan, lane);
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
          const bool few = seg.rows <= kFewToks * G && kFewToks < tile_toks;
          if (lane == 0) mbar_arrive_expect_tx(bars.q_ready + s, uint32_t((few ? kFewToks : tile_toks) * G) * D * 2);
          __syncwarp();
          if (lane < D / 64)
            tma_load3(base + L::OFF_Q + s * L::BYTES + lane * L::HALF, few ? &maps.qs : &maps.qt, lane * 64, seg.h * G,
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

// ---------------------------------------------------------------- join
// kJoinChunks CTAs for each CTA of the tile kernel, if a cut item begins in its stretch: a warp takes a row at a time,
// its pieces' log-sum-exps and, on their way with them, the first pieces' sums.
template <int D, bool F16>
__global__ void __launch_bounds__(32 * kJoinWarps) packed_join_kernel(const __grid_constant__ PackedAttnParams p, const __grid_constant__ PackedWs w) {
  constexpr int N = D / 32, U = 4;
  pdl_launch_dependents();
  pdl_wait();
  const gdn_kv_dims& d = p.d;
  const JoinRec rec = w.join[blockIdx.x % kCtas];
  const int G = d.Hq / d.Hkv, lane = threadIdx.x & 31;
  const int parts = rec.rows > 0 ? rec.c1 - rec.c0 + 1 : 0;
  for (int r = int(blockIdx.x / kCtas) * kJoinWarps + int(threadIdx.x >> 5); r < rec.rows; r += kJoinWarps * kJoinChunks) {
    // piece j's row: the first CTA's piece, then the one that each stretch begins with
    auto at = [&](int j) { return (j == 0 ? rec.part0 : 2 * (rec.c0 + j) * kBlockRows) + r; };
    float acc[N], v[U][N];
    auto load = [&](int j0, int end) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + u < end) {
          const float* o = w.o + (long long)at(j0 + u) * D + lane * N;
          if (N == 4)
            *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(o);
          else
            *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(o);
        }
    };
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    float M = -INFINITY, W = 0.f;
    for (int j0 = 0; j0 < parts; j0 += 32) {
      const int n = parts - j0 < 32 ? parts - j0 : 32;
      const float e = lane < n ? w.lse[at(j0 + lane)] : -INFINITY;
      load(j0, j0 + n);
      float mx = e;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float Mn = fmaxf(M, mx), f = M == -INFINITY ? 0.f : exp2f(M - Mn);
      const float wt = e == -INFINITY ? 0.f : exp2f(e - (Mn == -INFINITY ? 0.f : Mn));  // (NaN stays NaN)
      M = Mn;
      W = W * f + warp_sum(wt);
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] *= f;
      for (int i0 = 0; i0 < n; i0 += U) {
        if (i0 > 0) load(j0 + i0, j0 + n);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float wj = __shfl_sync(0xffffffffu, wt, (i0 + u) & 31);
          if (i0 + u < n && wj != 0.f)
#pragma unroll
            for (int k = 0; k < N; ++k) acc[k] += wj * v[u][k];
        }
      }
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] *= inv;
    const int tok = r / G;
    const long long row = (long long)(rec.tok0 + tok) * d.Hq + rec.h * G + (r - tok * G);
    uint32_t* const o = reinterpret_cast<uint32_t*>(p.out + row * D) + lane * (N / 2);
    if (N == 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(pack2<F16>(acc[0], acc[1]), pack2<F16>(acc[N - 2], acc[N - 1]));
    else
      *o = pack2<F16>(acc[0], acc[1]);
    if (p.lse && lane == 0) p.lse[row] = W == 0.f ? -INFINITY : (M + log2f(W)) * kLn2;
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
  return launch_dependent(packed_join_kernel<D, F16>, unsigned(kCtas * kJoinChunks), 32 * kJoinWarps, 0, stream, p, w);
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
  map(&maps.many[0], p.k_cache, 5, cd, cs, bb);
  map(&maps.many[1], p.v_cache, 5, cd, cs, bb);
  const cuuint64_t qd[3] = {cuuint64_t(d.D), cuuint64_t(d.Hq), cuuint64_t(p.n_tokens)};
  const cuuint64_t qst[2] = {2ull * d.D, 2ull * d.q_token_stride};
  const cuuint32_t bt[3] = {64, cuuint32_t(G), cuuint32_t(toks)}, bs[3] = {64, cuuint32_t(G), cuuint32_t(toks < kFewToks ? toks : kFewToks)};
  map(&maps.qt, p.q, 3, qd, qst, bt);
  map(&maps.qs, p.q, 3, qd, qst, bs);
  if (!ok) return cudaErrorInvalidValue;
  const PackedWs w = carve_packed(p.ws, d, nullptr);
  Cut cut{toks, 2 * toks, 0, p.causal};
  while ((cut.toks << cut.period_log) % kTileKeys) ++cut.period_log;
  if (d.D == 128) return d.dtype ? launch<128, true>(p, w, cut, box, maps, stream) : launch<128, false>(p, w, cut, box, maps, stream);
  return d.dtype ? launch<64, true>(p, w, cut, box, maps, stream) : launch<64, false>(p, w, cut, box, maps, stream);
}

}  // namespace gdn
