/*
 * gdn_kv.h - C ABI of the paged key/value cache: the softmax-attention layers' half of a
 * speculative-decoding round on GB300 (sm_103a), next to the Gated DeltaNet half in gdn.h.
 *
 * A hybrid model interleaves GDN layers with softmax-attention layers.  In one round of B
 * sequences, each with a window of K drafted tokens,
 *   gdn_attn_verify  attends the window to the cache: a prefix that sequences share (read and
 *                    multiplied once for all of them), each sequence's own tokens, and the
 *                    window's own ancestors (a chain, or a token tree as in gdn_verify_tree);
 *   gdn_kv_commit    moves the accepted tokens' keys and values of all layers into pages;
 *   gdn_kv_fork      forks, drops and reorders sequences, sharing pages by reference count;
 *   gdn_kv_compact   moves the live pages to the lowest page numbers.
 * The window's keys and values stay outside the pages until they are accepted, so a rejected
 * draft needs no rollback here.
 *
 * The cache: k_cache and v_cache hold n_pages pages of page_size tokens for each of n_layers
 * layers.  Element (layer, page, token, head, i) is at
 *   layer * cache_layer_stride + page * cache_page_stride + token * cache_token_stride
 *   + head * cache_head_stride + i
 * in both, so [page][token][head][D] and [page][head][token][D] orders, and keys and values
 * interleaved in one buffer, are all described by the strides.  Where a call writes them, the two may
 * have no element in common (GDN_ERR_ALIAS).  A slot is one sequence (or one
 * shared prefix): row s of page_table [n_slots, max_pages] int32 lists its pages in order, and
 * seq_len[s] int32 counts its tokens; it owns ceil(seq_len / page_size) pages, and the rest of
 * the row is not read.  ref[p] int32 counts the slots that hold page p (plus whatever the
 * caller pins); a page with ref 0 is free.  Only whole pages are ever shared between slots, so
 * a page that still has room belongs to one slot.
 *
 * Conventions are those of gdn.h: the caller owns every buffer, calls are asynchronous on
 * `stream`, every argument is validated on the host before anything is enqueued, what only the
 * device can see (lengths, page numbers, parents) is checked there and reported by
 * gdn_device_status with the bits below.  Cache, window, q and out are bf16 or f16 (dtype) and
 * 16-byte aligned, int32 arrays 4-byte aligned, the workspace 256-byte aligned.  Outputs may not
 * overlap inputs or each other unless a call says so.
 */
#ifndef GDN_KV_GB300_H
#define GDN_KV_GB300_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the per-device status word (gdn_device_status). */
#define GDN_DEVERR_KV_LEN 32u      /* a seq_len was negative or beyond the table's columns; the slot was read as empty */
#define GDN_DEVERR_KV_PAGE 64u     /* a page number was outside 0..n_pages-1; results that read it are invalid */
#define GDN_DEVERR_KV_SLOT 128u    /* a slot index (prefix_of, src) was outside -1..n_slots-1; it was read as -1 */
#define GDN_DEVERR_KV_FULL 256u    /* no free page, or no column, was left; that sequence was not changed */
#define GDN_DEVERR_KV_SHARED 512u  /* commit found the partial last page held more than once; that sequence was not changed */
#define GDN_DEVERR_KV_WINDOW 1024u /* a win_len was outside 0..K and was clamped */

typedef struct {
  int32_t B;          /* sequences in the batch: slots slot0 .. slot0 + B - 1 */
  int32_t K;          /* window tokens, 1..16 (gdn_kv_commit of chains: 1..1048576) */
  int32_t Hq;         /* query heads, a multiple of Hkv, at most 128 Hkv (query head h reads kv head h / (Hq/Hkv)) */
  int32_t Hkv;        /* key/value heads */
  int32_t D;          /* head dim, 64 or 128 */
  int32_t page_size;  /* tokens per page, a multiple of 16, 16..1024 */
  int32_t n_pages;    /* pages in the pool */
  int32_t max_pages;  /* columns of the page table */
  int32_t n_slots;    /* rows of the page table */
  int32_t slot0;      /* the batch's first slot */
  int32_t n_layers;   /* layers in the cache */
  int32_t dtype;      /* 0: bf16, 1: f16 */
  int64_t cache_layer_stride, cache_page_stride, cache_token_stride, cache_head_stride; /* elements, multiples of 8 */
  int64_t q_token_stride;   /* elements between q rows [Hq * D] of consecutive tokens (b-major), a multiple of 8 */
  int64_t win_token_stride; /* the same for k_win / v_win rows [Hkv * D] */
  int64_t win_layer_stride; /* elements between layers of k_win / v_win (gdn_kv_commit) */
} gdn_kv_dims;

/*
 * Attention of the windows over the cache, one layer.  Row (b, t, h) attends to
 *   - all seq_len[p] tokens of slot p = prefix_of[b], if prefix_of is not NULL and p >= 0;
 *   - all seq_len[slot0 + b] tokens of its own slot;
 *   - window tokens j < win_len[b] with j == t or j an ancestor of t (parent NULL: j <= t)
 * and gets, with s_j = scale * q . k_j over those,
 *   lse = log sum_j exp(s_j),  out = sum_j exp(s_j - lse) v_j.
 *   layer      0..n_layers-1
 *   q          [B, K, Hq, D] (tokens q_token_stride apart); k_win, v_win [B, K, Hkv, D]
 *              (tokens win_token_stride apart)
 *   prefix_of  [B] int32 or NULL.  Consecutive sequences with the same prefix share one pass over
 *              it; equal prefixes apart from each other give the same results in more passes.
 *   win_len    [B] int32 or NULL (= K): tokens t >= win_len[b] are padding; their out is 0 and
 *              their lse -inf, and what q, k_win and v_win hold there (NaN included) reaches no
 *              other row
 *   parent     [B, K] int32 or NULL: parent[b][t] in -1..t-1, as in gdn_verify_tree; not read at padding
 *              tokens
 *   scale      finite
 *   out        [B, K, Hq, D] contiguous, dtype; lse [B, K, Hq] f32 or NULL
 *   workspace  at least gdn_attn_workspace_size() bytes, no initialisation needed, dead after
 *              the call
 * Scores, softmax statistics and sums are f32; the probabilities are rounded to dtype for the
 * product with the values (some of them twice, where a row's running maximum rises by more than
 * 2^8 within a tile of 128 keys: they then hold less than that row's new largest).  What the cache holds beyond a slot's tokens reaches no output; a
 * value that is not finite at a token that any row of the same window sees may reach every row
 * of that window.  Results do not depend on the order in which CTAs run.
 */
gdn_status gdn_attn_verify(const gdn_kv_dims* dims, int32_t layer, const void* q, const void* k_win,
                           const void* v_win, const void* k_cache, const void* v_cache, const int32_t* page_table,
                           const int32_t* seq_len, const int32_t* prefix_of, const int32_t* win_len,
                           const int32_t* parent, float scale, void* out, float* lse, void* workspace,
                           uint64_t workspace_bytes, gdn_stream_t stream);

/* Bytes of workspace gdn_attn_verify needs for `dims` (any lengths). */
gdn_status gdn_attn_workspace_size(const gdn_kv_dims* dims, uint64_t* bytes);

/*
 * Commit: sequence b keeps n_b tokens of its window, for all layers, at positions seq_len ..
 * seq_len + n_b - 1 of slot slot0 + b.
 *   accept_len  [B] int32, 0..K: without parent the first accept_len tokens; with parent
 *               (K <= 16) the path from the root to node accept_len - 1 (the convention of
 *               gdn_rollback after gdn_verify_tree).  Out of range: nothing is kept and
 *               GDN_DEVERR_ACCEPT_RANGE is set.
 *   k_win,v_win [n_layers, B, K, Hkv, D] (strides in dims)
 *   table_in/out [n_slots, max_pages], len_in/out [n_slots], ref_in/out [n_pages]: each out may
 *               be its in (in place).  Slots outside the batch are copied.
 * The pages that sequence b needs beyond its last one are the lowest free ones, handed out in
 * the order of b; they get ref 1.  With F free pages, sequence b gets its pages if the pages
 * wanted by sequences 0..b are at most F; otherwise it is left unchanged (GDN_DEVERR_KV_FULL), as
 * it is when its row has too few columns (it then wants no pages).  A partial last page with
 * ref != 1 leaves the sequence unchanged (GDN_DEVERR_KV_SHARED).
 */
gdn_status gdn_kv_commit(const gdn_kv_dims* dims, const int32_t* accept_len, const int32_t* parent,
                         const void* k_win, const void* v_win, void* k_cache, void* v_cache,
                         const int32_t* table_in, int32_t* table_out, const int32_t* len_in, int32_t* len_out,
                         const int32_t* ref_in, int32_t* ref_out, void* workspace, uint64_t workspace_bytes,
                         gdn_stream_t stream);

/*
 * Fork, drop and reorder: slot i of the outputs takes the sequence that slot src[i] of the inputs
 * holds (-1: slot i becomes empty).  A sequence that no slot takes is freed.  Full pages are
 * shared by all takers; a partial last page stays with the lowest taker, and every other taker
 * gets a copy of its filled tokens (all layers) in a page that is free in ref_in, the lowest free
 * pages going to the lowest slots.  Slots for which no free page is left become empty
 * (GDN_DEVERR_KV_FULL).  Row i of table_out is row src[i] of table_in but for the copied page
 * (-1 throughout for an empty slot).
 *   src [n_slots] int32; table_out and len_out may not overlap table_in and len_in; ref_out may
 *   be ref_in.  dims: B, K, Hq, slot0 and the q and window strides are not read.
 */
gdn_status gdn_kv_fork(const gdn_kv_dims* dims, const int32_t* src, void* k_cache, void* v_cache,
                       const int32_t* table_in, int32_t* table_out, const int32_t* len_in, int32_t* len_out,
                       const int32_t* ref_in, int32_t* ref_out, void* workspace, uint64_t workspace_bytes,
                       gdn_stream_t stream);

/*
 * Compact: with n pages live (ref > 0), the live pages numbered n and up move, lowest first, to
 * the free pages below n, lowest first, in all layers; the tables and ref follow, and *n_live
 * becomes n.  Pages 0..n-1 are then the live ones.  table_out may be table_in, ref_out ref_in.
 * A page that is live by a count that only the caller raised, with no table that names it, moves
 * like the others, and no output says where to.
 * dims: B, K, Hq, slot0 and the q and window strides are not read.
 */
gdn_status gdn_kv_compact(const gdn_kv_dims* dims, void* k_cache, void* v_cache, const int32_t* table_in,
                          int32_t* table_out, const int32_t* seq_len, const int32_t* ref_in, int32_t* ref_out,
                          int32_t* n_live, void* workspace, uint64_t workspace_bytes, gdn_stream_t stream);

/*
 * Bytes of workspace for `dims` that serve gdn_kv_commit, gdn_kv_fork and gdn_kv_compact alike.  The
 * last two do not read B: what B = 0 gives is enough for them.
 */
gdn_status gdn_kv_workspace_size(const gdn_kv_dims* dims, uint64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* GDN_KV_GB300_H */
