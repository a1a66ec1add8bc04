// Upkeep of the paged key/value cache: commit of accepted window tokens, fork / drop / reorder of
// sequences, compaction of the pool (contracts in include/gdn_kv.h).
//
// Each call is two launches.  The first plans: its CTA 0 (512 threads) walks lengths and
// reference counts and writes, into the workspace, which pages go where; its other CTAs copy the
// tables that are not updated in place.  It changes no input, so a call may work in place.  The
// second moves the data (all layers, keys and values) and then edits tables, lengths and
// reference counts from the plan.
//
// Bound: the move is a copy, 2 bytes of HBM traffic per byte moved; the plan reads 4 bytes per
// page of the pool and is a few dependent trips to L2 long.  A move takes 16 tokens of one layer
// at a time, keys and values together, 16 bytes a thread and piece, four or eight loads in
// flight a thread before its first store.  Pieces are found without a division (by multiplication, or
// straight on where a page's tokens lie one behind the other): with two divisions a piece the
// copy was bound by instructions, 5.1 of 6.8 TB/s over 1.65 GB.
#include "gdn_common.cuh"
#include "kv_kernels.h"

namespace gdn {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 16;  // tokens of one layer moved by one CTA at a time

struct CommitRec {  // plan of one sequence of a commit
  int32_t n;       // tokens kept
  int32_t len;     // tokens before
  int32_t first;   // its first new page's rank in the free list
  int32_t have;    // pages before
  uint64_t nodes;  // tree: the path's window nodes, 4 bits each, the root's first
  int32_t pad[2];
};

struct Move {  // one page's copy (fork, compact)
  int32_t from, to, tokens, pad;
};

// Workspace: header, the move list, the free pages, one int per page and two per slot, and last the
// records of a commit's sequences: fork and compact neither need them nor read B.
struct PagesWs {
  int32_t* head;      // [0] moves in the list, [1] live pages
  Move* move;         // [max(n_slots, n_pages)] fork, compact
  int32_t* ids;       // [n_pages] free pages in order
  int32_t* map;       // [n_pages] compact: new number of each page from n_live on (-1: it is free)
  int32_t* first;     // [n_slots] fork: lowest taker
  int32_t* made;      // [n_slots] fork: the slot's copied page (-1 none, -2 failed)
  CommitRec* rec;     // [B] commit
};

__host__ __device__ inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

__host__ __device__ inline PagesWs carve_pages(void* base, const gdn_kv_dims& d, size_t* total) {
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t o = 0;
  const size_t pages = size_t(d.n_pages), slots = size_t(d.n_slots), moves = pages > slots ? pages : slots;
  PagesWs w;
  w.head = reinterpret_cast<int32_t*>(p + o), o += 256;
  w.move = reinterpret_cast<Move*>(p + o), o += up256(sizeof(Move) * moves);
  w.ids = reinterpret_cast<int32_t*>(p + o), o += up256(4 * pages);
  w.map = reinterpret_cast<int32_t*>(p + o), o += up256(4 * pages);
  w.first = reinterpret_cast<int32_t*>(p + o), o += up256(4 * slots);
  w.made = reinterpret_cast<int32_t*>(p + o), o += up256(4 * slots);
  w.rec = reinterpret_cast<CommitRec*>(p + o);
  if (total) *total = o;
  return w;
}

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Exclusive prefix sum of v over the CTA (kPlanThreads threads) and the CTA's total.
__device__ __forceinline__ int block_scan(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the sums of the call before have been read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int s = lane < kPlanThreads / 32 ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return x - v + (warp > 0 ? before : 0);
}

// The lowest `want` free pages, in order, into ids; returns how many there are (at most want).
__device__ int list_free(const int32_t* ref, int n_pages, int want, int32_t* ids, int* sums) {
  int found = 0;
  for (int at = 0; at < n_pages && found < want; at += 4 * kPlanThreads) {
    const int p0 = at + 4 * int(threadIdx.x);
    int mask = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (p0 + q < n_pages && ref[p0 + q] == 0) mask |= 1 << q;
    int total;
    int r = found + block_scan(__popc(mask), sums, total);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if ((mask >> q & 1) && r < want) ids[r++] = p0 + q;
    found += total;
  }
  return found < want ? found : want;
}

// dst <- src, n ints, by the CTAs `cta` of `ctas` (a no-op in place).
__device__ void copy_ints(int32_t* dst, const int32_t* src, long long n, int cta, int ctas) {
  if (dst == src) return;
  for (long long i = (long long)cta * blockDim.x + threadIdx.x; i < n; i += (long long)ctas * blockDim.x) dst[i] = src[i];
}

__device__ __forceinline__ int pages_of(int len, int page_size) { return int((unsigned(len) + unsigned(page_size) - 1u) / unsigned(page_size)); }

// A slot's length, 0 (and a status bit) when it is negative or beyond the table's columns.
__device__ __forceinline__ int checked_len(int len, const gdn_kv_dims& d, uint32_t* err) {
  if (len < 0 || (long long)len > (long long)d.max_pages * d.page_size) {
    atomicOr(err, GDN_DEVERR_KV_LEN);
    return 0;
  }
  return len;
}

__device__ __forceinline__ uint4 load_piece(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Keys and values of `n` 16-byte pieces by the whole CTA; from(i) and to(i) are a piece's places (in
// elements, the same in keys and values).
// U pieces of each at a time a thread (4 for pages; 2 for the few rows of a commit, whose CTAs are more
// than the card holds at once: 26 us, 28 with 4, at 256 sequences and 12 layers).
template <int U, typename From, typename To>
__device__ __forceinline__ void move_pieces(uint16_t* k_dst, uint16_t* v_dst, const uint16_t* k_src, const uint16_t* v_src, int n,
                                            From from, To to) {
  for (int i0 = threadIdx.x; i0 < n; i0 += U * kMoveThreads) {
    uint4 k[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMoveThreads;
      if (i < n) {
        const long long o = from(i);
        k[u] = load_piece(k_src + o);
        v[u] = load_piece(v_src + o);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kMoveThreads;
      if (i < n) {
        const long long o = to(i);
        *reinterpret_cast<uint4*>(k_dst + o) = k[u];
        *reinterpret_cast<uint4*>(v_dst + o) = v[u];
      }
    }
  }
}

// Splits a piece of [token][head][D / 8] into its three indices; by_heads = ceil(2^32 / Hkv), exact
// for the at most 16 x 4096 (token, head) pairs of a move.
struct Piece {
  int t, h, e;
};
__device__ __forceinline__ Piece split_piece(int i, int d8_shift, int Hkv, uint32_t by_heads) {
  const int th = i >> d8_shift, t = Hkv == 1 ? th : int(__umulhi(uint32_t(th), by_heads));
  return Piece{t, th - t * Hkv, i - (th << d8_shift)};
}

// ---------------------------------------------------------------- commit
__global__ void __launch_bounds__(kPlanThreads) kv_commit_plan_kernel(const __grid_constant__ PagesParams p, const __grid_constant__ PagesWs w) {
  __shared__ int sums[32];
  grid_launch_dependents();
  grid_wait();
  const gdn_kv_dims& d = p.d;
  if (blockIdx.x > 0) {
    const int cta = int(blockIdx.x) - 1, ctas = int(gridDim.x) - 1;
    copy_ints(p.table_out, p.table_in, (long long)d.n_slots * d.max_pages, cta, ctas);
    copy_ints(p.len_out, p.len_in, d.n_slots, cta, ctas);
    copy_ints(p.ref_out, p.ref_in, d.n_pages, cta, ctas);
    return;
  }
  int wanted = 0;
  for (int b0 = 0; b0 < d.B; b0 += kPlanThreads) {
    const int b = b0 + int(threadIdx.x);
    int need = 0;
    CommitRec r{};
    if (b < d.B) {
      const int slot = d.slot0 + b;
      const int len = checked_len(p.len_in[slot], d, p.err);
      int n = p.accept[b];
      if (n < 0 || n > d.K) {
        atomicOr(p.err, GDN_DEVERR_ACCEPT_RANGE);
        n = 0;
      }
      uint64_t nodes = 0;
      if (p.parent && n > 0) {
        int up[kKvWinMax];  // (read together: one after the other they would be a trip to memory each)
#pragma unroll
        for (int t = 0; t < kKvWinMax; ++t) up[t] = t < n ? p.parent[(long long)b * d.K + t] : -1;
        uint32_t path = 1u << (n - 1);
        int count = 0;
#pragma unroll
        for (int t = kKvWinMax - 1; t >= 0; --t)
          if (path >> t & 1) {
            if (up[t] < -1 || up[t] >= t)
              atomicOr(p.err, GDN_DEVERR_TREE_PARENT);
            else if (up[t] >= 0)
              path |= 1u << up[t];
            nodes = nodes << 4 | uint64_t(t);  // (leaf first, so that the root ends lowest)
            ++count;
          }
        n = count;
      }
      const int have = pages_of(len, d.page_size);
      if (n > 0 && len % d.page_size != 0) {  // the page that still has room is this slot's own
        const int last = p.table_in[(long long)slot * d.max_pages + have - 1];
        if (last < 0 || last >= d.n_pages) {
          atomicOr(p.err, GDN_DEVERR_KV_PAGE);
          n = 0;
        } else if (p.ref_in[last] != 1) {
          atomicOr(p.err, GDN_DEVERR_KV_SHARED);
          n = 0;
        }
      }
      if ((long long)len + n > (long long)d.max_pages * d.page_size) {
        atomicOr(p.err, GDN_DEVERR_KV_FULL);
        n = 0;
      }
      need = n > 0 ? pages_of(len + n, d.page_size) - have : 0;
      r.n = n;
      r.len = len;
      r.have = have;
      r.nodes = nodes;
    }
    int total;
    r.first = wanted + block_scan(need, sums, total);
    if (b < d.B) w.rec[b] = r;
    wanted += total;
  }
  const int found = list_free(p.ref_in, d.n_pages, wanted < d.n_pages ? wanted : d.n_pages, w.ids, sums);
  if (found < wanted) {
    for (int b = int(threadIdx.x); b < d.B; b += kPlanThreads) {  // (each thread reads back its own records)
      CommitRec r = w.rec[b];
      const int need = r.n > 0 ? pages_of(r.len + r.n, d.page_size) - r.have : 0;
      if (need > 0 && r.first + need > found) {
        atomicOr(p.err, GDN_DEVERR_KV_FULL);
        w.rec[b].n = 0;
      }
    }
  }
}

// One CTA per (sequence, 16 tokens, layer).
__global__ void __launch_bounds__(kMoveThreads) kv_commit_move_kernel(const __grid_constant__ PagesParams p, const PagesWs w, int tiles,
                                                                      uint32_t by_heads) {
  grid_launch_dependents();
  grid_wait();
  const gdn_kv_dims& d = p.d;
  const int d8_shift = d.D == 128 ? 4 : 3;
  const int layer = int(blockIdx.x % unsigned(d.n_layers)), unit = int(blockIdx.x / unsigned(d.n_layers));
  const int tile = unit % tiles, b = unit / tiles;
  const CommitRec r = w.rec[b];
  const int t0 = tile * kMoveTokens;
  if (r.n <= t0) return;
  const int tokens = r.n - t0 < kMoveTokens ? r.n - t0 : kMoveTokens;
  const int slot = d.slot0 + b;
  const int32_t* row = p.table_in + (long long)slot * d.max_pages;
  // the tokens lie in the page of the first, from `in` on, and the one behind it
  const int at = r.len + t0, col = at / d.page_size, in = at - col * d.page_size;
  auto page_at = [&](int c) { return c < r.have ? row[c] : w.ids[r.first + c - r.have]; };
  const int page0 = page_at(col), page1 = in + tokens > d.page_size ? page_at(col + 1) : page0;
  const long long layer_at = layer * d.cache_layer_stride;
  const long long from = layer * d.win_layer_stride + (long long)b * d.K * d.win_token_stride;
  const int D = d.D;
  move_pieces<2>(
      p.k_cache, p.v_cache, p.k_win + from, p.v_win + from, tokens * d.Hkv << d8_shift,
      [&](int i) {
        const Piece q = split_piece(i, d8_shift, d.Hkv, by_heads);
        const int node = p.parent ? int(r.nodes >> (4 * q.t) & 15) : t0 + q.t;
        return node * d.win_token_stride + q.h * D + 8 * q.e;
      },
      [&](int i) {
        const Piece q = split_piece(i, d8_shift, d.Hkv, by_heads);
        const int pos = in + q.t;
        const bool behind = pos >= d.page_size;
        return layer_at + (behind ? page1 : page0) * d.cache_page_stride + (behind ? pos - d.page_size : pos) * d.cache_token_stride +
               q.h * d.cache_head_stride + 8 * q.e;
      });
  if (tile == 0 && layer == 0) {
    const int want = pages_of(r.len + r.n, d.page_size);
    int32_t* out = p.table_out + (long long)slot * d.max_pages;
    for (int c = r.have + int(threadIdx.x); c < want; c += kMoveThreads) {
      const int page = w.ids[r.first + c - r.have];
      out[c] = page;
      p.ref_out[page] = 1;
    }
    if (threadIdx.x == 0) p.len_out[slot] = r.len + r.n;
  }
}

// ---------------------------------------------------------------- fork
__global__ void __launch_bounds__(kPlanThreads) kv_fork_plan_kernel(const __grid_constant__ PagesParams p, const __grid_constant__ PagesWs w) {
  __shared__ int sums[32];
  grid_launch_dependents();
  grid_wait();
  const gdn_kv_dims& d = p.d;
  if (blockIdx.x > 0) {
    const int cta = int(blockIdx.x) - 1, ctas = int(gridDim.x) - 1;
    copy_ints(p.ref_out, p.ref_in, d.n_pages, cta, ctas);
    const long long entries = (long long)d.n_slots * d.max_pages;
    for (long long e = (long long)cta * kPlanThreads + threadIdx.x; e < entries; e += (long long)ctas * kPlanThreads) {
      const int i = int(e / d.max_pages), c = int(e - (long long)i * d.max_pages);
      int s = p.src[i];
      if (s < 0 || s >= d.n_slots) s = -1;
      p.table_out[e] = s < 0 ? -1 : p.table_in[(long long)s * d.max_pages + c];
    }
    return;
  }
  // lowest taker of each slot (in shared memory as far as that goes; the move reads it again)
  __shared__ int first_here[kPlanThreads];
  const bool here = d.n_slots <= kPlanThreads;
  int* const first = here ? first_here : w.first;
  for (int i = int(threadIdx.x); i < d.n_slots; i += kPlanThreads) first[i] = d.n_slots;
  __syncthreads();
  for (int i = int(threadIdx.x); i < d.n_slots; i += kPlanThreads) {
    const int s = p.src[i];
    if (s >= 0 && s < d.n_slots) atomicMin(&first[s], i);
  }
  __syncthreads();
  if (here && int(threadIdx.x) < d.n_slots) w.first[threadIdx.x] = first[threadIdx.x];
  int copies = 0;
  for (int pass = 0; pass < 2; ++pass) {  // count the copies; then hand out pages
    int found = 0;
    if (pass == 1) {
      found = list_free(p.ref_in, d.n_pages, copies < d.n_pages ? copies : d.n_pages, w.ids, sums);
      copies = 0;
      __syncthreads();  // the list is complete
    }
    for (int i0 = 0; i0 < d.n_slots; i0 += kPlanThreads) {
      const int i = i0 + int(threadIdx.x);
      int copy = 0, s = -1, len = 0;
      if (i < d.n_slots) {
        s = p.src[i];
        if (s < -1 || s >= d.n_slots) {
          atomicOr(p.err, GDN_DEVERR_KV_SLOT);
          s = -1;
        }
        if (s >= 0) {
          len = checked_len(p.len_in[s], d, p.err);
          copy = (len % d.page_size != 0 && first[s] != i) ? 1 : 0;
        }
      }
      int total;
      const int rank = copies + block_scan(copy, sums, total);
      if (pass == 1 && i < d.n_slots) {
        int made = -1;
        if (copy) {
          if (rank < found) {
            const int from = p.table_in[(long long)s * d.max_pages + len / d.page_size];
            const bool ok = from >= 0 && from < d.n_pages;
            if (!ok) atomicOr(p.err, GDN_DEVERR_KV_PAGE);
            made = w.ids[rank];
            w.move[rank] = Move{ok ? from : made, made, ok ? len % d.page_size : 0, 0};
          } else {
            atomicOr(p.err, GDN_DEVERR_KV_FULL);
            made = -2;
          }
        }
        w.made[i] = made;
      }
      copies += total;
    }
    if (pass == 1 && threadIdx.x == 0) w.head[0] = copies < found ? copies : found;
  }
}

// Reference count of page `id`, by `delta` (atomic: several slots may hold it).
__device__ __forceinline__ void add_ref(int32_t* ref, int id, int delta, const gdn_kv_dims& d, uint32_t* err) {
  if (id < 0 || id >= d.n_pages)
    atomicOr(err, GDN_DEVERR_KV_PAGE);
  else
    atomicAdd(&ref[id], delta);
}

// Copies the listed pages' filled tokens, all layers, keys and values.
__device__ __forceinline__ void move_pages(const PagesParams& p, const PagesWs& w, uint32_t by_heads) {
  const gdn_kv_dims& d = p.d;
  const int d8_shift = d.D == 128 ? 4 : 3;
  const unsigned tiles = unsigned(d.page_size + kMoveTokens - 1) / kMoveTokens, per_page = tiles * unsigned(d.n_layers);
  const bool straight = d.cache_head_stride == d.D && d.cache_token_stride == (long long)d.Hkv * d.D;
  const long long units = (long long)w.head[0] * per_page;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long page = u / per_page;
    const unsigned in_page = unsigned(u - page * per_page);
    const int layer = int(in_page / tiles), t0 = int(in_page % tiles) * kMoveTokens;
    const Move m = w.move[page];
    const int tokens = m.tokens - t0 < kMoveTokens ? m.tokens - t0 : kMoveTokens;
    if (tokens <= 0) continue;
    const long long base = layer * d.cache_layer_stride + t0 * d.cache_token_stride;
    const long long to = base + m.to * d.cache_page_stride, from = base + m.from * d.cache_page_stride;
    const int n = tokens * d.Hkv << d8_shift;
    if (straight) {
      auto at = [](int i) { return 8ll * i; };
      move_pieces<4>(p.k_cache + to, p.v_cache + to, p.k_cache + from, p.v_cache + from, n, at, at);
    } else {
      auto at = [&](int i) {
        const Piece q = split_piece(i, d8_shift, d.Hkv, by_heads);
        return q.t * d.cache_token_stride + q.h * d.cache_head_stride + 8 * q.e;
      };
      move_pieces<4>(p.k_cache + to, p.v_cache + to, p.k_cache + from, p.v_cache + from, n, at, at);
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) kv_fork_move_kernel(const __grid_constant__ PagesParams p, const __grid_constant__ PagesWs w, uint32_t by_heads) {
  grid_launch_dependents();
  grid_wait();
  const gdn_kv_dims& d = p.d;
  move_pages(p, w, by_heads);
  // (books last, from the other end: the CTAs with the fewest moves first)
  for (int i = int(gridDim.x - 1 - blockIdx.x); i < d.n_slots; i += int(gridDim.x)) {
    // as an old slot: a sequence that nobody took gives its pages back
    if (w.first[i] == d.n_slots) {
      int len = p.len_in[i];
      if (len < 0 || (long long)len > (long long)d.max_pages * d.page_size) len = 0;
      const int held = pages_of(len, d.page_size);
      for (int c = int(threadIdx.x); c < held; c += kMoveThreads)
        add_ref(p.ref_out, p.table_in[(long long)i * d.max_pages + c], -1, d, p.err);
    }
    // as a new slot: takers after the first add a reference to every page they share
    int s = p.src[i];
    if (s < 0 || s >= d.n_slots) s = -1;
    int len = s < 0 ? 0 : p.len_in[s];
    if (len < 0 || (long long)len > (long long)d.max_pages * d.page_size) len = 0;
    const int made = w.made[i];
    int32_t* row = p.table_out + (long long)i * d.max_pages;
    if (made == -2) {
      for (int c = int(threadIdx.x); c < d.max_pages; c += kMoveThreads) row[c] = -1;
      len = 0;
    } else if (s >= 0 && w.first[s] != i) {
      const int full = len / d.page_size;
      for (int c = int(threadIdx.x); c < full; c += kMoveThreads)
        add_ref(p.ref_out, p.table_in[(long long)s * d.max_pages + c], 1, d, p.err);
      if (made >= 0 && threadIdx.x == 0) {
        row[full] = made;
        add_ref(p.ref_out, made, 1, d, p.err);
      }
    }
    if (threadIdx.x == 0) p.len_out[i] = len;
  }
}

// ---------------------------------------------------------------- compact
__global__ void __launch_bounds__(kPlanThreads) kv_compact_plan_kernel(const __grid_constant__ PagesParams p, const __grid_constant__ PagesWs w) {
  __shared__ int sums[32];
  grid_launch_dependents();
  grid_wait();
  const gdn_kv_dims& d = p.d;
  if (blockIdx.x > 0) {
    copy_ints(p.ref_out, p.ref_in, d.n_pages, int(blockIdx.x) - 1, int(gridDim.x) - 1);
    return;
  }
  int mine = 0;
#pragma unroll 4
  for (int i = int(threadIdx.x); i < d.n_pages; i += kPlanThreads) mine += p.ref_in[i] > 0;
  int live;
  block_scan(mine, sums, live);
  // holes below `live` and live pages from there on: as many of one as of the other
  for (int side = 0; side < 2; ++side) {
    const int lo = side ? live : 0, hi = side ? d.n_pages : live;
    int count = 0;
    for (int at = lo; at < hi; at += 4 * kPlanThreads) {
      const int i0 = at + 4 * int(threadIdx.x);
      int take = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i0 + q < hi && (p.ref_in[i0 + q] > 0) == (side == 1)) take |= 1 << q;
      int total;
      int r = count + block_scan(__popc(take), sums, total);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + q;
        if (i >= hi) continue;
        const bool taken = take >> q & 1;
        if (side == 0) {
          if (taken) w.ids[r++] = i;
        } else {
          const int to = taken ? w.ids[r++] : -1;
          w.map[i] = to;
          if (taken) w.move[r - 1] = Move{i, to, d.page_size, 0};
        }
      }
      count += total;
    }
    __syncthreads();
    if (threadIdx.x == 0) w.head[0] = count, w.head[1] = live;
  }
}

__global__ void __launch_bounds__(kMoveThreads) kv_compact_move_kernel(const __grid_constant__ PagesParams p, const __grid_constant__ PagesWs w, uint32_t by_heads) {
  grid_launch_dependents();
  grid_wait();
  const gdn_kv_dims& d = p.d;
  const int live = w.head[1], moves = w.head[0];
  const long long at = (long long)blockIdx.x * kMoveThreads + threadIdx.x, step = (long long)gridDim.x * kMoveThreads;
  if (at == 0) p.n_live[0] = live;
  for (long long r = at; r < moves; r += step) {  // (one thread per pair: reads, then writes, in place too)
    const Move m = w.move[r];
    const int held = p.ref_in[m.from];
    p.ref_out[m.to] = held;
    p.ref_out[m.from] = 0;
  }
  for (int s = int(blockIdx.x); s < d.n_slots; s += int(gridDim.x)) {
    const int held = pages_of(checked_len(p.len_in[s], d, p.err), d.page_size);
    const int32_t* in = p.table_in + (long long)s * d.max_pages;
    int32_t* out = p.table_out + (long long)s * d.max_pages;
    for (int c = int(threadIdx.x); c < d.max_pages; c += kMoveThreads) {
      int page = in[c];
      if (c < held) {
        if (page < 0 || page >= d.n_pages)
          atomicOr(p.err, GDN_DEVERR_KV_PAGE);
        else if (page >= live && w.map[page] >= 0)
          page = w.map[page];
      }
      out[c] = page;
    }
  }
  move_pages(p, w, by_heads);
}

template <typename... Args>
cudaError_t launch_pdl(void (*kernel)(Args...), int grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

uint32_t by_heads(const gdn_kv_dims& d) { return uint32_t(((1ull << 32) + d.Hkv - 1) / d.Hkv); }  // (unused for one head)

// CTAs of a move over `units` pieces of pages: no more than there are pieces, nor than 40 to an SM,
// twenty times what runs at once - those that start later fill the gaps of those that end earlier
// (compaction of 1.66 GB: 268 us with 8 to an SM, 260 with 40, 271 with 160; fork of a population
// 45.5, 40.6, 43.5).
int move_grid(long long units) { return int(units < 1 ? 1 : (units < 152 * 40 ? units : 152 * 40)); }

// CTA 0 plans; one more CTA for each 16K ints of tables to copy.
int plan_grid(long long ints) { return 1 + int(ints < 1 ? 1 : (ints + 16383) / 16384 > 64 ? 64 : (ints + 16383) / 16384); }

}  // namespace

size_t pages_workspace_bytes(const gdn_kv_dims& d, int sequences) {
  size_t n = 0;
  carve_pages(nullptr, d, &n);
  return n + up256(sizeof(CommitRec) * size_t(sequences));
}

cudaError_t launch_commit(const PagesParams& p, cudaStream_t stream) {
  const gdn_kv_dims& d = p.d;
  const PagesWs w = carve_pages(p.ws, d, nullptr);
  const int tiles = (d.K + kMoveTokens - 1) / kMoveTokens;
  cudaError_t e = launch_pdl(kv_commit_plan_kernel, plan_grid((long long)d.n_slots * d.max_pages + d.n_pages),
                             kPlanThreads, stream, p, w);
  if (e != cudaSuccess) return e;
  const long long units = (long long)d.B * tiles * d.n_layers;
  if (units == 0) return cudaSuccess;
  return launch_pdl(kv_commit_move_kernel, int(units), kMoveThreads, stream, p, w, tiles, by_heads(d));
}

cudaError_t launch_fork(const PagesParams& p, cudaStream_t stream) {
  const gdn_kv_dims& d = p.d;
  const PagesWs w = carve_pages(p.ws, d, nullptr);
  cudaError_t e = launch_pdl(kv_fork_plan_kernel, plan_grid((long long)d.n_slots * d.max_pages + d.n_pages),
                             kPlanThreads, stream, p, w);
  if (e != cudaSuccess) return e;
  const long long units = (long long)d.n_slots * d.n_layers * (d.page_size / kMoveTokens);
  return launch_pdl(kv_fork_move_kernel, move_grid(units), kMoveThreads, stream, p, w, by_heads(d));
}

cudaError_t launch_compact(const PagesParams& p, cudaStream_t stream) {
  const gdn_kv_dims& d = p.d;
  const PagesWs w = carve_pages(p.ws, d, nullptr);
  cudaError_t e = launch_pdl(kv_compact_plan_kernel, plan_grid(d.n_pages), kPlanThreads, stream, p, w);
  if (e != cudaSuccess) return e;
  const long long units = (long long)d.n_pages * d.n_layers * (d.page_size / kMoveTokens);
  return launch_pdl(kv_compact_move_kernel, move_grid(units), kMoveThreads, stream, p, w, by_heads(d));
}

}  // namespace gdn
