// Internal launch interface of the paged key/value cache (kv_api.cu) and its kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/gdn_kv.h"

namespace gdn {

constexpr int kKvWinMax = 16;  // longest window of the attention call and of a token tree

// ---- attention of the windows over the cache (gdn_attn_verify)
struct AttnParams {
  gdn_kv_dims d;
  int layer;
  const void* q;
  const void* k_win;
  const void* v_win;
  const void* k_cache;
  const void* v_cache;
  const int32_t* table;      // [n_slots, max_pages]
  const int32_t* seq_len;    // [n_slots]
  const int32_t* prefix_of;  // [B] or null
  const int32_t* win_len;    // [B] or null
  const int32_t* parent;     // [B, K] or null
  float scale;
  void* out;   // [B, K, Hq, D]
  float* lse;  // [B, K, Hq] or null
  void* ws;
  uint32_t* err;
  int tile_toks, tile_rows;  // tokens and rows (tokens x query heads per kv head) of a row tile; set by launch_attn
  uint32_t page_inv;         // of page_column (kv_index.h); set by launch_attn
};

size_t attn_workspace_bytes(const gdn_kv_dims& d);
cudaError_t launch_attn(const AttnParams& p, cudaStream_t stream);

// ---- pages (gdn_kv_commit, gdn_kv_fork, gdn_kv_compact)
struct PagesParams {
  gdn_kv_dims d;
  const int32_t* accept;     // commit, reserve: [B]
  const int32_t* parent;     // commit: [B, K] or null
  const int32_t* src;        // fork: [n_slots]
  const uint16_t* k_win;     // commit: [n_layers, B, K, Hkv, D]
  const uint16_t* v_win;
  uint16_t* k_cache;
  uint16_t* v_cache;
  const int32_t* table_in;
  int32_t* table_out;
  const int32_t* len_in;
  int32_t* len_out;
  const int32_t* ref_in;
  int32_t* ref_out;
  int32_t* refused;          // reserve: [n_slots] or null
  int32_t* n_live;           // compact
  void* ws;
  uint32_t* err;
};

// ---- norms and rotation of windows (gdn_attn_rope) and of packed tokens on their way to pages (gdn_kv_append)
struct RopeParams {
  gdn_kv_dims d;
  gdn_rope r;
  const uint64_t* turns;
  const float* q_weight;
  const float* k_weight;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  uint16_t* k_out;           // window, or the layer's pages
  uint16_t* v_out;
  const int32_t* seq_len;
  const int32_t* prefix_of;
  const int32_t* positions;
  const int32_t* win_len;    // windows
  const int32_t* parent;
  const int32_t* cu;         // packed tokens
  const int32_t* table;
  const int32_t* refused;    // [n_slots] or null
  uint32_t* err;
  int32_t n_tokens;
  int32_t hq, hk, hv;        // heads of each kind that the call handles
};

cudaError_t launch_rope_window(const RopeParams& p, cudaStream_t stream);
cudaError_t launch_append(const RopeParams& p, cudaStream_t stream);

// ---- attention of packed queries (gdn_attn_prefill)
struct PackedAttnParams {
  gdn_kv_dims d;
  int32_t n_tokens;
  const int32_t* cu;         // [B + 1]
  const uint16_t* q;
  const uint16_t* k_cache;   // of the layer
  const uint16_t* v_cache;
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* prefix_of;
  const int32_t* refused;    // [n_slots] or null
  int32_t causal;
  float scale;
  uint16_t* out;
  float* lse;
  void* ws;
  uint32_t* err;
};

size_t packed_attn_workspace_bytes(const gdn_kv_dims& d, int64_t n_tokens);
cudaError_t launch_packed_attn(const PackedAttnParams& p, cudaStream_t stream);

size_t pages_workspace_bytes(const gdn_kv_dims& d, int sequences);  // (those of a commit; else 0)
cudaError_t launch_commit(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_reserve(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_fork(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_compact(const PagesParams& p, cudaStream_t stream);

// This device's status word (gdn_api.cu); records and returns a status on failure.
gdn_status device_status_word(uint32_t** out);
// Clears this thread's gdn_last_error() text and returns GDN_OK.
gdn_status report_ok();
gdn_status report_error(gdn_status s, const char* msg);

}  // namespace gdn
