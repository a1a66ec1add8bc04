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
 * Around that, what comes before a window's attention, and prompts:
 *   gdn_attn_rope    norms and rotates the window's queries and keys as they come from the projection;
 *   gdn_kv_reserve   takes the pages for new tokens of each sequence, once for all layers;
 *   gdn_kv_append    brings one layer's packed tokens into place: queries and keys normed and rotated,
 *                    keys and values written to the reserved pages;
 *   gdn_attn_prefill attends packed queries to the pages, causally (prompts, chunks of prompts, single
 *                    tokens) or to all of a slot (cross attention to states of another length).
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
#define GDN_DEVERR_KV_LEN 32u      /* a seq_len was negative or beyond the table's columns; the slot was read as empty (also as said at a call) */
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
 * Bytes of workspace for `dims` that serve gdn_kv_commit, gdn_kv_reserve, gdn_kv_fork and gdn_kv_compact
 * alike.  The last two do not read B: what B = 0 gives is enough for them.
 */
gdn_status gdn_kv_workspace_size(const gdn_kv_dims* dims, uint64_t* bytes);

/*
 * Norm and rotation of the heads of queries and keys, and the strides of the rows they come from.
 * With a weight w [D] the head is first divided by its root mean square,
 *   x_i <- x_i (weight_offset + w_i) / sqrt(mean_j x_j^2 + eps),
 * then the pairs (a, b) of its first rot_dim elements are turned: with the angle phi of the pair at
 * the token's position,
 *   (a, b) <- magnitude * (a cos phi - b sin phi, b cos phi + a sin phi).
 * All of it is computed in f32 and rounded to dtype once.  The rest of the head is normed only.
 * Angles are exact for far positions: turns[i] is the i-th pair's angle of one token as a 64-bit
 * fraction of a turn (gdn_rope_turns), so that position x turns mod 2^64 is the angle.  Frequencies
 * scaled for long contexts are a matter of that table.
 */
typedef struct {
  int32_t rot_dim;       /* a multiple of 16, 0..D */
  int32_t interleaved;   /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2 i, 2 i + 1); i = 0 .. rot_dim / 2 - 1 */
  float magnitude;       /* of the rotated elements (1 unless long contexts rescale it); finite */
  float eps;             /* of the norms; finite, >= 0 */
  float weight_offset;   /* added to the norms' weights (0, or 1 where they are kept as differences from 1); finite */
  int32_t reserved;      /* 0 */
  int64_t q_token_stride, q_head_stride;   /* elements between tokens and heads of the q that is read, multiples of 8 */
  int64_t kv_token_stride, kv_head_stride; /* the same for k and v */
} gdn_rope;

/*
 * turns[i] (host, [n]) of radians[i] (host, [n]): the angle of a pair from one token to the next, such as
 * base^(-2 i / rot_dim), as a fraction of a turn times 2^64, rounded.  radians: finite, |radians| < 2^32.
 */
gdn_status gdn_rope_turns(const double* radians, int32_t n, uint64_t* turns);

/*
 * Norms and rotation of verify windows: queries and keys of B windows of K tokens from the projection to
 * where gdn_attn_verify and gdn_kv_commit read them.  Window token t of sequence b is at position
 *   seq_len[prefix_of[b]] (with a prefix) + seq_len[slot0 + b] + the number of its ancestors in the window
 * (a chain: t), or at positions[b][t].
 *   turns      [rot_dim / 2] uint64, 8-byte aligned (NULL if rot_dim is 0)
 *   q_weight, k_weight  [D] f32, 16-byte aligned, or NULL (no norm)
 *   q, k, v    [B, K, heads, D] with the strides in rope; any of them may be NULL together with its output
 *   seq_len    [n_slots] (NULL with positions); prefix_of, win_len [B], parent [B, K] or NULL as in
 *              gdn_attn_verify; positions [B, K] int32 or NULL (then prefix_of and parent are not read)
 *   q_out      [B, K, Hq, D], tokens q_token_stride apart; k_win, v_win [B, K, Hkv, D], tokens win_token_stride
 *              apart (strides in dims).  v_win is v.  Each may be its input where that has the same token
 *              stride and heads D apart (in place), and parts of rows of one buffer may be rewritten
 *              beside one another.
 * Padding tokens (t >= win_len[b]) become 0.  The cache's fields of dims are checked and, but for the number of
 * slots and the longest slot, not used.
 */
gdn_status gdn_attn_rope(const gdn_kv_dims* dims, const gdn_rope* rope, const uint64_t* turns, const float* q_weight,
                         const float* k_weight, const void* q, const void* k, const void* v, const int32_t* seq_len,
                         const int32_t* prefix_of, const int32_t* win_len, const int32_t* parent,
                         const int32_t* positions, void* q_out, void* k_win, void* v_win, gdn_stream_t stream);

/*
 * Reserve: slot slot0 + b grows by n_new[b] tokens (0..2^30), whose pages are taken and whose elements
 * are left as they are: a layer's gdn_kv_append fills them.  Pages, order, in-place use and failures are those of
 * gdn_kv_commit: a sequence that gets no pages (GDN_DEVERR_KV_FULL), whose last page is shared
 * (GDN_DEVERR_KV_SHARED) or whose n_new is out of range (GDN_DEVERR_KV_LEN) is left unchanged.
 * dims: K, Hq and the strides are checked as by gdn_kv_fork; the workspace is gdn_kv_workspace_size's.
 *
 * Which sequences were left unchanged is known on the device alone, and the last tokens of such a slot are not the
 * ones that were to follow.  gdn_kv_reserve_marked notes them for the calls that come after it, the _marked ones:
 *   refused    [n_slots] int32, or NULL: entry slot0 + b becomes -1 if the sequence got its tokens (or n_new[b] is 0),
 *              else the slot's length.  The other slots' entries are left as they are; -1 to begin with.
 * A slot whose length is still its entry of refused has not grown since.
 */
gdn_status gdn_kv_reserve(const gdn_kv_dims* dims, const int32_t* n_new, const int32_t* table_in, int32_t* table_out,
                          const int32_t* len_in, int32_t* len_out, const int32_t* ref_in, int32_t* ref_out,
                          void* workspace, uint64_t workspace_bytes, gdn_stream_t stream);
gdn_status gdn_kv_reserve_marked(const gdn_kv_dims* dims, const int32_t* n_new, const int32_t* table_in, int32_t* table_out,
                                 const int32_t* len_in, int32_t* len_out, const int32_t* ref_in, int32_t* ref_out,
                                 int32_t* refused, void* workspace, uint64_t workspace_bytes, gdn_stream_t stream);

/*
 * Append: one layer's packed new tokens.  Tokens cu_seqlens[b] .. cu_seqlens[b+1] - 1 are the last ones of
 * slot slot0 + b, whose seq_len counts them already (gdn_kv_reserve); token j of n is at its position
 * seq_len - n + j, and at that plus the prefix's tokens for the rotation (or at positions[token]).
 *   n_tokens   0 <= n_tokens < 2^31: rows of q, k, v
 *   cu_seqlens [B + 1] int32: 0 = c_0 <= ... <= c_B <= n_tokens, else GDN_DEVERR_SEQLENS is set and what the
 *              slots' last tokens hold is undefined.  Rows behind c_B reach no output, and none is written for them.
 *   q, q_out   [n_tokens, Hq, D] (strides in rope; q_token_stride in dims), or both NULL
 *   k, v       [n_tokens, Hkv, D] (strides in rope)
 *   k_cache, v_cache  written, as described above; q_out may be q as in gdn_attn_rope
 * A sequence with more tokens than its slot holds is not written (GDN_DEVERR_KV_LEN), nor are keys and values of
 * a token on a page outside the pool (GDN_DEVERR_KV_PAGE).  dims: K and win_token_stride are not read.
 * gdn_kv_append takes the slots' last tokens as they are: the caller knows that each sequence has got its room, or it
 * overwrites tokens that are cached, also for the sequences that share their pages.  gdn_kv_append_marked does not
 * rely on it: a sequence whose slot's length is refused[slot0 + b] is not written, q_out neither (GDN_DEVERR_KV_LEN).
 */
gdn_status gdn_kv_append(const gdn_kv_dims* dims, int32_t layer, const gdn_rope* rope, const uint64_t* turns,
                         const float* q_weight, const float* k_weight, int64_t n_tokens, const int32_t* cu_seqlens,
                         const void* q, const void* k, const void* v, const int32_t* positions, void* k_cache,
                         void* v_cache, const int32_t* page_table, const int32_t* seq_len, const int32_t* prefix_of,
                         void* q_out, gdn_stream_t stream);
gdn_status gdn_kv_append_marked(const gdn_kv_dims* dims, int32_t layer, const gdn_rope* rope, const uint64_t* turns,
                                const float* q_weight, const float* k_weight, int64_t n_tokens,
                                const int32_t* cu_seqlens, const void* q, const void* k, const void* v,
                                const int32_t* positions, void* k_cache, void* v_cache, const int32_t* page_table,
                                const int32_t* seq_len, const int32_t* refused, const int32_t* prefix_of, void* q_out,
                                gdn_stream_t stream);

/*
 * Attention of packed queries over the cache, one layer.  Row (token j of the n of sequence b, h) attends to
 *   - all seq_len[p] tokens of slot p = prefix_of[b], if prefix_of is not NULL and p >= 0;
 *   - causal != 0: the first seq_len[slot0 + b] - n + j + 1 tokens of its own slot (the row's own token is the
 *     last of them; fewer than one: none);
 *   - causal == 0: all seq_len[slot0 + b] tokens of its own slot (cross attention: the slot holds an encoder's
 *     states, and the queries of sequences that share a slot may be packed as one sequence's);
 * out and lse as in gdn_attn_verify; a row without keys gets out 0 and lse -inf.
 *   n_tokens, cu_seqlens  as in gdn_kv_append; where cu_seqlens is wrong nothing is written.  Rows of out and lse
 *              behind c_B are left as they are.
 *   q          [n_tokens, Hq, D], tokens q_token_stride apart
 *   out        [n_tokens, Hq, D] contiguous, dtype; lse [n_tokens, Hq] f32 or NULL
 *   workspace  at least gdn_attn_prefill_workspace_size() bytes, no initialisation needed, dead after the call
 *              (calls that may run at once, on two streams or in two graphs, need one each)
 * Rounding as in gdn_attn_verify.  What the cache holds beyond a slot's tokens reaches no output; a value
 * that is not finite at a token of a slot may reach every row with keys of the sequences that read the slot.
 * Results do not depend on the order in which CTAs run.  dims: K and win_token_stride are not read.
 * gdn_attn_prefill_marked, where causal != 0: rows of a sequence whose slot's length is refused[slot0 + b] see nothing,
 * not its prefix either, and get out 0 and lse -inf (GDN_DEVERR_KV_LEN).
 */
gdn_status gdn_attn_prefill(const gdn_kv_dims* dims, int32_t layer, int64_t n_tokens, const int32_t* cu_seqlens,
                            const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                            const int32_t* seq_len, const int32_t* prefix_of, int32_t causal, float scale, void* out,
                            float* lse, void* workspace, uint64_t workspace_bytes, gdn_stream_t stream);
gdn_status gdn_attn_prefill_marked(const gdn_kv_dims* dims, int32_t layer, int64_t n_tokens,
                                   const int32_t* cu_seqlens, const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* page_table, const int32_t* seq_len, const int32_t* refused,
                                   const int32_t* prefix_of, int32_t causal, float scale, void* out, float* lse,
                                   void* workspace, uint64_t workspace_bytes, gdn_stream_t stream);

/* Bytes of workspace gdn_attn_prefill needs for `dims` and n_tokens rows (any lengths). */
gdn_status gdn_attn_prefill_workspace_size(const gdn_kv_dims* dims, int64_t n_tokens, uint64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* GDN_KV_GB300_H */
