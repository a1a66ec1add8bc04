// C ABI of the paged key/value cache: host-side validation, launches, error reporting
// (include/gdn_kv.h).  As in gdn_api.cu, every argument is checked before anything is enqueued.
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kv_kernels.h"

namespace {

gdn_status fail(gdn_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return gdn::report_error(s, buf);
}

constexpr int kMaxBatch = 65535;
enum Use { kAttn, kCommit, kPool, kSlots, kRope, kPacked };  // (kSlots: a batch of slots; kPacked: of queries, too)

gdn_status check_dims(const gdn_kv_dims* d, Use use, bool tree) {
  if (!d) return fail(GDN_ERR_INVALID_ARG, "dims is NULL");
  if (d->Hkv < 1 || d->Hkv > 4096) return fail(GDN_ERR_INVALID_ARG, "Hkv=%d outside 1..4096", d->Hkv);
  if (d->D != 64 && d->D != 128) return fail(GDN_ERR_UNSUPPORTED, "D=%d (64 or 128)", d->D);
  if (d->page_size < 16 || d->page_size > 1024 || d->page_size % 16)
    return fail(GDN_ERR_UNSUPPORTED, "page_size=%d (a multiple of 16, 16..1024)", d->page_size);
  if (d->n_pages < 1 || d->n_pages > (1 << 28)) return fail(GDN_ERR_INVALID_ARG, "n_pages=%d outside 1..2^28", d->n_pages);
  if (d->n_slots < 1 || d->n_slots > (1 << 24)) return fail(GDN_ERR_INVALID_ARG, "n_slots=%d outside 1..2^24", d->n_slots);
  if (d->max_pages < 1 || (long long)d->max_pages * d->page_size > (1LL << 30))
    return fail(GDN_ERR_INVALID_ARG, "max_pages=%d (>= 1, at most 2^30 tokens)", d->max_pages);
  if (d->n_layers < 1 || d->n_layers > 65535) return fail(GDN_ERR_INVALID_ARG, "n_layers=%d outside 1..65535", d->n_layers);
  if (d->dtype != 0 && d->dtype != 1) return fail(GDN_ERR_INVALID_ARG, "dtype=%d (0: bf16, 1: f16)", d->dtype);
  const int64_t cs[4] = {d->cache_layer_stride, d->cache_page_stride, d->cache_token_stride, d->cache_head_stride};
  const char* cn[4] = {"layer", "page", "token", "head"};
  const int cn_n[4] = {d->n_layers, d->n_pages, d->page_size, d->Hkv};  // (the stride of a single entry is not used)
  for (int i = 0; i < 4; ++i)
    if (cn_n[i] > 1 && (cs[i] < d->D || cs[i] % 8 || cs[i] >= (1LL << 36)))
      return fail(GDN_ERR_INVALID_ARG, "cache_%s_stride=%lld (a multiple of 8, at least D)", cn[i], (long long)cs[i]);
  if (use == kPool) return GDN_OK;
  if (d->B < 0 || d->B > kMaxBatch) return fail(GDN_ERR_INVALID_ARG, "B=%d outside 0..%d", d->B, kMaxBatch);
  if (d->slot0 < 0 || (long long)d->slot0 + d->B > d->n_slots)
    return fail(GDN_ERR_INVALID_ARG, "slots %d..%d outside the table's %d", d->slot0, d->slot0 + d->B - 1, d->n_slots);
  if (use == kSlots) return GDN_OK;
  const int kmax = use == kAttn || use == kRope || tree ? gdn::kKvWinMax : 1 << 20;
  if (use != kPacked && (d->K < 1 || d->K > kmax)) return fail(GDN_ERR_UNSUPPORTED, "K=%d outside 1..%d", d->K, kmax);
  if (use == kPacked) {
  } else if (d->win_token_stride < (int64_t)d->Hkv * d->D || d->win_token_stride % 8 || d->win_token_stride >= (1LL << 36))
    return fail(GDN_ERR_INVALID_ARG, "win_token_stride=%lld (a multiple of 8, at least Hkv * D)", (long long)d->win_token_stride);
  if (use != kCommit) {
    if (d->Hq < 1 || d->Hq > 65536 || d->Hq % d->Hkv)
      return fail(d->Hq < 1 ? GDN_ERR_INVALID_ARG : GDN_ERR_UNSUPPORTED, "Hq=%d (a multiple of Hkv=%d)", d->Hq, d->Hkv);
    if (d->Hq / d->Hkv > 128) return fail(GDN_ERR_UNSUPPORTED, "Hq/Hkv=%d (at most 128)", d->Hq / d->Hkv);
    if (d->q_token_stride < (int64_t)d->Hq * d->D || d->q_token_stride % 8 || d->q_token_stride >= (1LL << 36))
      return fail(GDN_ERR_INVALID_ARG, "q_token_stride=%lld (a multiple of 8, at least Hq * D)", (long long)d->q_token_stride);
    if (use != kPacked && (long long)d->B * d->K * d->Hq > (1LL << 30)) return fail(GDN_ERR_UNSUPPORTED, "more than 2^30 rows");
  } else {
    if (d->n_layers > 1 && (d->win_layer_stride % 8 || d->win_layer_stride < (int64_t)d->Hkv * d->D ||
                            d->win_layer_stride >= (1LL << 40)))
      return fail(GDN_ERR_INVALID_ARG, "win_layer_stride=%lld (a multiple of 8, at least Hkv * D)", (long long)d->win_layer_stride);
    if ((long long)d->B * (d->K / 16 + 2) * d->n_layers > (1LL << 30)) return fail(GDN_ERR_UNSUPPORTED, "B * K * n_layers too large");
  }
  return GDN_OK;
}

struct Buf {
  const char* name;
  const void* p;
  unsigned long long bytes;
  int align;
  bool output, optional;
  const char* may_be;  // the input that this output may be
};

// A cache's dimensions, the largest stride first.
struct CacheDim {
  int64_t stride, n;
};
void sorted_dims(const gdn_kv_dims& d, CacheDim (&m)[4]) {
  m[0] = {d.cache_layer_stride, d.n_layers}, m[1] = {d.cache_page_stride, d.n_pages};
  m[2] = {d.cache_token_stride, d.page_size}, m[3] = {d.cache_head_stride, d.Hkv};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (m[j].stride > m[i].stride) {
        const CacheDim t = m[i];
        m[i] = m[j];
        m[j] = t;
      }
}

// Whether two caches of these dimensions, `delta` elements apart, share an element: whether delta is a
// sum of differences of indices times strides, and of places in a row.  Where the strides do not fold
// (check_cache_strides) what the smaller ones can add is less than a stride, so that only the two
// multiples next to delta come into question.
bool share_element(const CacheDim* m, int left, int64_t D, int64_t delta) {
  if (left == 0) return delta > -D && delta < D;
  if (m->n == 1) return share_element(m + 1, left - 1, D, delta);
  const int64_t q = delta / m->stride - (delta % m->stride < 0 ? 1 : 0);
  for (int64_t i = q; i <= q + 1; ++i)
    if (i > -m->n && i < m->n && share_element(m + 1, left - 1, D, delta - i * m->stride)) return true;
  return false;
}

// k_cache and v_cache may lie interleaved in one buffer
const char* const kInterleaved = "interleaved";
// tensors of rows, which check_rows looks at
const char* const kAmongRows = "rows";

// Null pointers, alignment, and overlaps of outputs with anything else.
gdn_status check_bufs(const gdn_kv_dims& d, const Buf* b, int n) {
  for (int i = 0; i < n; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(b[i].p);
    if (!a && !b[i].optional) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", b[i].name);
    if (a % unsigned(b[i].align)) return fail(GDN_ERR_INVALID_ARG, "%s is not %d-byte aligned", b[i].name, b[i].align);
  }
  for (int i = 0; i < n; ++i) {
    if (!b[i].output || !b[i].p) continue;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(b[i].p), hi = lo + b[i].bytes;
    for (int j = 0; j < n; ++j) {
      if (i == j || !b[j].p || (b[j].output && j < i)) continue;
      const uintptr_t lo2 = reinterpret_cast<uintptr_t>(b[j].p), hi2 = lo2 + b[j].bytes;
      if (lo >= hi2 || lo2 >= hi) continue;
      if (lo == lo2 && b[i].may_be == b[j].name) continue;
      if (b[i].may_be == kInterleaved && b[j].may_be == kInterleaved) {
        CacheDim m[4];
        sorted_dims(d, m);
        if (!share_element(m, 4, d.D, (int64_t(lo2) - int64_t(lo)) / 2)) continue;
      }
      if (b[i].may_be == kAmongRows && b[j].may_be == kAmongRows) continue;  // (check_rows)
      return fail(GDN_ERR_ALIAS, "%s overlaps %s", b[i].name, b[j].name);
    }
  }
  return GDN_OK;
}

// The rows [tokens][heads][D] of a tensor: tokens `step` elements apart, heads within them.
struct Rows {
  const char* name;
  const void* p;
  long long n, step, head_step, heads;
  bool output;
  const char* may_be;
  long long width(int D) const { return (heads - 1) * head_step + D; }
};

// Overlaps of outputs with the other tensors of rows.  Rows of one step may lie beside one another in the
// rows of one buffer, and an output may be its input where both have the same places.
gdn_status check_rows(const Rows* t, int n, int D) {
  for (int i = 0; i < n; ++i)
    if (t[i].p && t[i].step > 0 && t[i].n > (1LL << 58) / t[i].step) return fail(GDN_ERR_INVALID_ARG, "%s is too large", t[i].name);
  for (int i = 0; i < n; ++i) {
    if (!t[i].p || !t[i].output) continue;
    for (int j = 0; j < n; ++j) {
      if (i == j || !t[j].p || (t[j].output && j < i)) continue;
      const int64_t lo = int64_t(reinterpret_cast<uintptr_t>(t[i].p)), lo2 = int64_t(reinterpret_cast<uintptr_t>(t[j].p));
      const int64_t w = 2 * t[i].width(D), w2 = 2 * t[j].width(D);
      if (lo >= lo2 + 2 * (t[j].n - 1) * t[j].step + w2 || lo2 >= lo + 2 * (t[i].n - 1) * t[i].step + w) continue;
      const bool same_step = t[i].step == t[j].step || (t[i].n == 1 && t[j].n == 1);
      if (lo == lo2 && t[i].may_be == t[j].name && same_step && (t[i].head_step == t[j].head_step || t[i].heads == 1)) continue;
      if (t[i].step == t[j].step && t[i].step > 0) {
        const int64_t step = 2 * t[i].step, off = ((lo2 - lo) % step + step) % step;  // where row j begins in a row of i
        if (off >= w && off + w2 <= step) continue;
      }
      return fail(GDN_ERR_ALIAS, "%s overlaps %s", t[i].name, t[j].name);
    }
  }
  return GDN_OK;
}

// A norm's and rotation's description, and what belongs to it.
gdn_status check_rope(const gdn_rope* r, const gdn_kv_dims& d, const uint64_t* turns, const float* q_weight, const float* k_weight) {
  if (!r) return fail(GDN_ERR_INVALID_ARG, "rope is NULL");
  if (r->rot_dim < 0 || r->rot_dim > d.D) return fail(GDN_ERR_INVALID_ARG, "rot_dim=%d outside 0..%d", r->rot_dim, d.D);
  if (r->rot_dim % 16) return fail(GDN_ERR_UNSUPPORTED, "rot_dim=%d (a multiple of 16)", r->rot_dim);
  if (r->interleaved != 0 && r->interleaved != 1) return fail(GDN_ERR_INVALID_ARG, "interleaved=%d (0 or 1)", r->interleaved);
  if (r->reserved != 0) return fail(GDN_ERR_INVALID_ARG, "reserved=%d (0)", r->reserved);
  if (!std::isfinite(r->magnitude)) return fail(GDN_ERR_INVALID_ARG, "magnitude not finite");
  if (!std::isfinite(r->weight_offset)) return fail(GDN_ERR_INVALID_ARG, "weight_offset not finite");
  if (!std::isfinite(r->eps) || r->eps < 0.f) return fail(GDN_ERR_INVALID_ARG, "eps not finite or negative");
  const int64_t st[4] = {r->q_token_stride, r->q_head_stride, r->kv_token_stride, r->kv_head_stride};
  const char* const names[4] = {"q_token", "q_head", "kv_token", "kv_head"};
  for (int i = 0; i < 4; ++i)
    if (st[i] < 0 || st[i] % 8 || st[i] >= (1LL << 36))
      return fail(GDN_ERR_INVALID_ARG, "%s_stride=%lld (a multiple of 8, not negative)", names[i], (long long)st[i]);
  if (!turns && r->rot_dim > 0) return fail(GDN_ERR_INVALID_ARG, "turns is NULL");
  if (reinterpret_cast<uintptr_t>(turns) & 7u) return fail(GDN_ERR_INVALID_ARG, "turns is not 8-byte aligned");
  if (reinterpret_cast<uintptr_t>(q_weight) & 15u) return fail(GDN_ERR_INVALID_ARG, "q_weight is not 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(k_weight) & 15u) return fail(GDN_ERR_INVALID_ARG, "k_weight is not 16-byte aligned");
  return GDN_OK;
}

// The dims with the strides of single entries set to what a dense cache would have, so that
// nothing below needs to ask.
gdn_kv_dims normal(const gdn_kv_dims& in) {
  gdn_kv_dims d = in;
  if (d.Hkv == 1) d.cache_head_stride = d.D;
  if (d.n_pages == 1) d.cache_page_stride = d.D;
  if (d.n_layers == 1) d.cache_layer_stride = d.D, d.win_layer_stride = d.D;
  return d;
}

// Bytes from a cache pointer to the end of its last element.
unsigned long long cache_bytes(const gdn_kv_dims& d) {
  return 2ull * (unsigned long long)((d.n_layers - 1) * d.cache_layer_stride + (d.n_pages - 1) * d.cache_page_stride +
                                     (d.page_size - 1) * d.cache_token_stride + (d.Hkv - 1) * d.cache_head_stride + d.D);
}

// The index space of a strided buffer must not fold onto itself: sorted by stride, each dimension
// has to start at or beyond the extent of those below it.  (Reads would be harmless, but pages are
// written too.)
gdn_status check_cache_strides(const gdn_kv_dims& d) {
  CacheDim m[4];
  sorted_dims(d, m);
  int64_t extent = d.D;
  for (int i = 3; i >= 0; --i) {
    if (m[i].n == 1) continue;
    if (m[i].stride < extent) return fail(GDN_ERR_INVALID_ARG, "cache strides make elements overlap");
    if (m[i].n > (INT64_MAX / 4) / m[i].stride) return fail(GDN_ERR_INVALID_ARG, "cache too large");
    extent += (m[i].n - 1) * m[i].stride;
  }
  return GDN_OK;
}

#define GDN_RETURN_IF(e)              \
  do {                                \
    const gdn_status s_ = (e);        \
    if (s_ != GDN_OK) return s_;      \
  } while (0)

// Bytes from a rows' pointer to the end of its last element.
unsigned long long rows_bytes(const Rows& t, int D) {
  return t.p ? 2ull * (unsigned long long)((t.n - 1) * t.step + t.width(D)) : 0;
}

// A tensor of rows among the other buffers; check_rows looks at the rows among themselves.
Buf rows_buf(const Rows& t, int D) { return Buf{t.name, t.p, rows_bytes(t, D), 16, t.output, true, kAmongRows}; }

gdn::PagesParams pool_params(const gdn_kv_dims& d, void* k_cache, void* v_cache, const int32_t* table_in,
                             int32_t* table_out, const int32_t* ref_in, int32_t* ref_out, void* workspace) {
  gdn::PagesParams p{};
  p.d = d;
  p.k_cache = static_cast<uint16_t*>(k_cache);
  p.v_cache = static_cast<uint16_t*>(v_cache);
  p.table_in = table_in;
  p.table_out = table_out;
  p.ref_in = ref_in;
  p.ref_out = ref_out;
  p.ws = workspace;
  return p;
}

// The checks that the three pool calls share; fills in the status word.
gdn_status check_pool(gdn::PagesParams& p, const Buf* bufs, int n, uint64_t workspace_bytes) {
  GDN_RETURN_IF(check_cache_strides(p.d));
  const unsigned long long need = bufs[n - 1].bytes;  // (the last buffer is the workspace)
  if (workspace_bytes < need)
    return fail(GDN_ERR_INVALID_ARG, "workspace has %llu bytes, %llu needed", (unsigned long long)workspace_bytes, need);
  GDN_RETURN_IF(check_bufs(p.d, bufs, n));
  return gdn::device_status_word(&p.err);
}

}  // namespace

extern "C" {

gdn_status gdn_attn_workspace_size(const gdn_kv_dims* dims, uint64_t* bytes) {
  GDN_RETURN_IF(check_dims(dims, kAttn, false));
  if (!bytes) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = gdn::attn_workspace_bytes(*dims);
  return gdn::report_ok();
}

gdn_status gdn_attn_verify(const gdn_kv_dims* dims, int32_t layer, const void* q, const void* k_win,
                           const void* v_win, const void* k_cache, const void* v_cache, const int32_t* page_table,
                           const int32_t* seq_len, const int32_t* prefix_of, const int32_t* win_len,
                           const int32_t* parent, float scale, void* out, float* lse, void* workspace,
                           uint64_t workspace_bytes, gdn_stream_t stream) {
  GDN_RETURN_IF(check_dims(dims, kAttn, false));
  const gdn_kv_dims d = normal(*dims);
  GDN_RETURN_IF(check_cache_strides(d));
  if (layer < 0 || layer >= d.n_layers) return fail(GDN_ERR_INVALID_ARG, "layer=%d outside 0..%d", layer, d.n_layers - 1);
  if (!std::isfinite(scale)) return fail(GDN_ERR_INVALID_ARG, "scale not finite");
  if (d.B == 0) return gdn::report_ok();
  const unsigned long long rows = (unsigned long long)d.B * d.K, BK = rows - 1;
  const unsigned long long need = gdn::attn_workspace_bytes(d);
  if (workspace_bytes < need) return fail(GDN_ERR_INVALID_ARG, "workspace has %llu bytes, %llu needed", (unsigned long long)workspace_bytes, need);
  const Buf bufs[] = {
      {"q", q, 2 * (BK * d.q_token_stride + (unsigned long long)d.Hq * d.D), 16, false, false, nullptr},
      {"k_win", k_win, 2 * (BK * d.win_token_stride + (unsigned long long)d.Hkv * d.D), 16, false, false, nullptr},
      {"v_win", v_win, 2 * (BK * d.win_token_stride + (unsigned long long)d.Hkv * d.D), 16, false, false, nullptr},
      {"k_cache", k_cache, cache_bytes(d), 16, false, false, nullptr},
      {"v_cache", v_cache, cache_bytes(d), 16, false, false, nullptr},
      {"page_table", page_table, 4ull * d.n_slots * d.max_pages, 4, false, false, nullptr},
      {"seq_len", seq_len, 4ull * d.n_slots, 4, false, false, nullptr},
      {"prefix_of", prefix_of, 4ull * d.B, 4, false, true, nullptr},
      {"win_len", win_len, 4ull * d.B, 4, false, true, nullptr},
      {"parent", parent, 4ull * rows, 4, false, true, nullptr},
      {"out", out, 2ull * rows * d.Hq * d.D, 16, true, false, nullptr},
      {"lse", lse, 4ull * rows * d.Hq, 4, true, true, nullptr},
      {"workspace", workspace, need, 256, true, false, nullptr},
  };
  GDN_RETURN_IF(check_bufs(d, bufs, int(sizeof bufs / sizeof bufs[0])));
  uint32_t* err = nullptr;
  GDN_RETURN_IF(gdn::device_status_word(&err));
  const gdn::AttnParams p{d, layer, q, k_win, v_win, k_cache, v_cache, page_table, seq_len, prefix_of, win_len, parent,
                          scale, out, lse, workspace, err, 0, 0, 0};
  const cudaError_t e = gdn::launch_attn(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
  return gdn::report_ok();
}

gdn_status gdn_kv_workspace_size(const gdn_kv_dims* dims, uint64_t* bytes) {
  GDN_RETURN_IF(check_dims(dims, kPool, false));
  if (!bytes) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
  // (a batch that commit refuses takes no room)
  *bytes = gdn::pages_workspace_bytes(*dims, dims->B < 0 || dims->B > kMaxBatch ? 0 : dims->B);
  return gdn::report_ok();
}

gdn_status gdn_kv_commit(const gdn_kv_dims* dims, const int32_t* accept_len, const int32_t* parent,
                         const void* k_win, const void* v_win, void* k_cache, void* v_cache,
                         const int32_t* table_in, int32_t* table_out, const int32_t* len_in, int32_t* len_out,
                         const int32_t* ref_in, int32_t* ref_out, void* workspace, uint64_t workspace_bytes,
                         gdn_stream_t stream) {
  GDN_RETURN_IF(check_dims(dims, kCommit, parent != nullptr));
  const gdn_kv_dims d = normal(*dims);
  const unsigned long long BK = (unsigned long long)d.B * d.K;
  const bool none = d.B == 0;
  const unsigned long long win = none ? 0
                                      : 2 * ((d.n_layers - 1) * (unsigned long long)d.win_layer_stride +
                                             (BK - 1) * d.win_token_stride + (unsigned long long)d.Hkv * d.D);
  const Buf bufs[] = {
      {"accept_len", accept_len, 4ull * d.B, 4, false, none, nullptr},
      {"parent", parent, 4 * BK, 4, false, true, nullptr},
      {"k_win", k_win, win, 16, false, none, nullptr},
      {"v_win", v_win, win, 16, false, none, nullptr},
      {"table_in", table_in, 4ull * d.n_slots * d.max_pages, 4, false, false, nullptr},
      {"len_in", len_in, 4ull * d.n_slots, 4, false, false, nullptr},
      {"ref_in", ref_in, 4ull * d.n_pages, 4, false, false, nullptr},
      {"k_cache", k_cache, cache_bytes(d), 16, true, false, kInterleaved},
      {"v_cache", v_cache, cache_bytes(d), 16, true, false, kInterleaved},
      {"table_out", table_out, 4ull * d.n_slots * d.max_pages, 4, true, false, bufs[4].name},
      {"len_out", len_out, 4ull * d.n_slots, 4, true, false, bufs[5].name},
      {"ref_out", ref_out, 4ull * d.n_pages, 4, true, false, bufs[6].name},
      {"workspace", workspace, gdn::pages_workspace_bytes(d, d.B), 256, true, false, nullptr},
  };
  gdn::PagesParams p = pool_params(d, k_cache, v_cache, table_in, table_out, ref_in, ref_out, workspace);
  GDN_RETURN_IF(check_pool(p, bufs, int(sizeof bufs / sizeof bufs[0]), workspace_bytes));
  p.accept = accept_len;
  p.parent = parent;
  p.k_win = static_cast<const uint16_t*>(k_win);
  p.v_win = static_cast<const uint16_t*>(v_win);
  p.len_in = len_in;
  p.len_out = len_out;
  const cudaError_t e = gdn::launch_commit(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "commit launch: %s", cudaGetErrorString(e));
  return gdn::report_ok();
}

gdn_status gdn_kv_reserve_marked(const gdn_kv_dims* dims, const int32_t* n_new, const int32_t* table_in, int32_t* table_out,
                                 const int32_t* len_in, int32_t* len_out, const int32_t* ref_in, int32_t* ref_out,
                                 int32_t* refused, void* workspace, uint64_t workspace_bytes, gdn_stream_t stream) {
  GDN_RETURN_IF(check_dims(dims, kSlots, false));
  const gdn_kv_dims d = normal(*dims);
  const Buf bufs[] = {
      {"n_new", n_new, 4ull * d.B, 4, false, d.B == 0, nullptr},
      {"table_in", table_in, 4ull * d.n_slots * d.max_pages, 4, false, false, nullptr},
      {"len_in", len_in, 4ull * d.n_slots, 4, false, false, nullptr},
      {"ref_in", ref_in, 4ull * d.n_pages, 4, false, false, nullptr},
      {"table_out", table_out, 4ull * d.n_slots * d.max_pages, 4, true, false, bufs[1].name},
      {"len_out", len_out, 4ull * d.n_slots, 4, true, false, bufs[2].name},
      {"ref_out", ref_out, 4ull * d.n_pages, 4, true, false, bufs[3].name},
      {"refused", refused, 4ull * d.n_slots, 4, true, true, nullptr},
      {"workspace", workspace, gdn::pages_workspace_bytes(d, d.B), 256, true, false, nullptr},
  };
  gdn::PagesParams p = pool_params(d, nullptr, nullptr, table_in, table_out, ref_in, ref_out, workspace);
  GDN_RETURN_IF(check_pool(p, bufs, int(sizeof bufs / sizeof bufs[0]), workspace_bytes));
  p.accept = n_new;
  p.len_in = len_in;
  p.len_out = len_out;
  p.refused = refused;
  const cudaError_t e = gdn::launch_reserve(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "reserve launch: %s", cudaGetErrorString(e));
  return gdn::report_ok();
}

gdn_status gdn_kv_reserve(const gdn_kv_dims* dims, const int32_t* n_new, const int32_t* table_in, int32_t* table_out,
                          const int32_t* len_in, int32_t* len_out, const int32_t* ref_in, int32_t* ref_out,
                          void* workspace, uint64_t workspace_bytes, gdn_stream_t stream) {
  return gdn_kv_reserve_marked(dims, n_new, table_in, table_out, len_in, len_out, ref_in, ref_out, nullptr, workspace,
                               workspace_bytes, stream);
}

gdn_status gdn_kv_fork(const gdn_kv_dims* dims, const int32_t* src, void* k_cache, void* v_cache,
                       const int32_t* table_in, int32_t* table_out, const int32_t* len_in, int32_t* len_out,
                       const int32_t* ref_in, int32_t* ref_out, void* workspace, uint64_t workspace_bytes,
                       gdn_stream_t stream) {
  GDN_RETURN_IF(check_dims(dims, kPool, false));
  const gdn_kv_dims d = normal(*dims);
  const Buf bufs[] = {
      {"src", src, 4ull * d.n_slots, 4, false, false, nullptr},
      {"table_in", table_in, 4ull * d.n_slots * d.max_pages, 4, false, false, nullptr},
      {"len_in", len_in, 4ull * d.n_slots, 4, false, false, nullptr},
      {"ref_in", ref_in, 4ull * d.n_pages, 4, false, false, nullptr},
      {"k_cache", k_cache, cache_bytes(d), 16, true, false, kInterleaved},
      {"v_cache", v_cache, cache_bytes(d), 16, true, false, kInterleaved},
      {"table_out", table_out, 4ull * d.n_slots * d.max_pages, 4, true, false, nullptr},
      {"len_out", len_out, 4ull * d.n_slots, 4, true, false, nullptr},
      {"ref_out", ref_out, 4ull * d.n_pages, 4, true, false, bufs[3].name},
      {"workspace", workspace, gdn::pages_workspace_bytes(d, 0), 256, true, false, nullptr},
  };
  gdn::PagesParams p = pool_params(d, k_cache, v_cache, table_in, table_out, ref_in, ref_out, workspace);
  GDN_RETURN_IF(check_pool(p, bufs, int(sizeof bufs / sizeof bufs[0]), workspace_bytes));
  p.src = src;
  p.len_in = len_in;
  p.len_out = len_out;
  const cudaError_t e = gdn::launch_fork(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "fork launch: %s", cudaGetErrorString(e));
  return gdn::report_ok();
}

gdn_status gdn_kv_compact(const gdn_kv_dims* dims, void* k_cache, void* v_cache, const int32_t* table_in,
                          int32_t* table_out, const int32_t* seq_len, const int32_t* ref_in, int32_t* ref_out,
                          int32_t* n_live, void* workspace, uint64_t workspace_bytes, gdn_stream_t stream) {
  GDN_RETURN_IF(check_dims(dims, kPool, false));
  const gdn_kv_dims d = normal(*dims);
  const Buf bufs[] = {
      {"table_in", table_in, 4ull * d.n_slots * d.max_pages, 4, false, false, nullptr},
      {"seq_len", seq_len, 4ull * d.n_slots, 4, false, false, nullptr},
      {"ref_in", ref_in, 4ull * d.n_pages, 4, false, false, nullptr},
      {"k_cache", k_cache, cache_bytes(d), 16, true, false, kInterleaved},
      {"v_cache", v_cache, cache_bytes(d), 16, true, false, kInterleaved},
      {"table_out", table_out, 4ull * d.n_slots * d.max_pages, 4, true, false, bufs[0].name},
      {"ref_out", ref_out, 4ull * d.n_pages, 4, true, false, bufs[2].name},
      {"n_live", n_live, 4, 4, true, false, nullptr},
      {"workspace", workspace, gdn::pages_workspace_bytes(d, 0), 256, true, false, nullptr},
  };
  gdn::PagesParams p = pool_params(d, k_cache, v_cache, table_in, table_out, ref_in, ref_out, workspace);
  GDN_RETURN_IF(check_pool(p, bufs, int(sizeof bufs / sizeof bufs[0]), workspace_bytes));
  p.len_in = seq_len;
  p.n_live = n_live;
  const cudaError_t e = gdn::launch_compact(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "compact launch: %s", cudaGetErrorString(e));
  return gdn::report_ok();
}

gdn_status gdn_rope_turns(const double* radians, int32_t n, uint64_t* turns) {
  if (n < 0) return fail(GDN_ERR_INVALID_ARG, "n=%d is negative", n);
  if (n > 0 && (!radians || !turns)) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", radians ? "turns" : "radians");
  for (int i = 0; i < n; ++i)
    if (!(std::fabs(radians[i]) < 4294967296.0)) return fail(GDN_ERR_INVALID_ARG, "radians[%d] not finite or too large", i);
  for (int i = 0; i < n; ++i) {
    // 1 / 2 pi in two parts, and the product's rounding error: a turn's fraction to 2^-64 and beyond what
    // radians[i] itself is known to
    const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
    const double x = std::fabs(radians[i]), whole = x * hi, rest = std::fma(x, hi, -whole) + x * lo;
    const double f = whole - std::floor(whole);                        // (exact)
    const double up = std::floor(std::ldexp(f, 32)), low = std::ldexp(f, 32) - up;  // (exact)
    const double part = std::ldexp(low, 32) + std::ldexp(rest, 64);
    const uint64_t turn = (uint64_t(up) << 32) + uint64_t(int64_t(std::llrint(part)));
    turns[i] = radians[i] < 0.0 ? 0 - turn : turn;
  }
  return gdn::report_ok();
}

gdn_status gdn_attn_rope(const gdn_kv_dims* dims, const gdn_rope* rope, const uint64_t* turns, const float* q_weight,
                         const float* k_weight, const void* q, const void* k, const void* v, const int32_t* seq_len,
                         const int32_t* prefix_of, const int32_t* win_len, const int32_t* parent,
                         const int32_t* positions, void* q_out, void* k_win, void* v_win, gdn_stream_t stream) {
  GDN_RETURN_IF(check_dims(dims, kRope, false));
  const gdn_kv_dims d = normal(*dims);
  GDN_RETURN_IF(check_rope(rope, d, turns, q_weight, k_weight));
  if (!q != !q_out || !k != !k_win || !v != !v_win)
    return fail(GDN_ERR_INVALID_ARG, "%s without its %s", !q != !q_out ? "q" : !k != !k_win ? "k" : "v",
                (q && !q_out) || (k && !k_win) || (v && !v_win) ? "output" : "input");
  if (d.B == 0 || (!q && !k && !v)) return gdn::report_ok();
  const long long n = (long long)d.B * d.K, ks = rope->kv_token_stride, kh = rope->kv_head_stride;
  const Rows rows[] = {
      {"q", q, n, rope->q_token_stride, rope->q_head_stride, d.Hq, false, nullptr},
      {"k", k, n, ks, kh, d.Hkv, false, nullptr},
      {"v", v, n, ks, kh, d.Hkv, false, nullptr},
      {"q_out", q_out, n, d.q_token_stride, d.D, d.Hq, true, rows[0].name},
      {"k_win", k_win, n, d.win_token_stride, d.D, d.Hkv, true, rows[1].name},
      {"v_win", v_win, n, d.win_token_stride, d.D, d.Hkv, true, rows[2].name},
  };
  const unsigned long long pairs = 4ull * rope->rot_dim, row = 4ull * d.D;
  const Buf bufs[] = {
      rows_buf(rows[0], d.D), rows_buf(rows[1], d.D), rows_buf(rows[2], d.D), rows_buf(rows[3], d.D), rows_buf(rows[4], d.D), rows_buf(rows[5], d.D),
      {"turns", turns, pairs, 8, false, true, nullptr},
      {"q_weight", q_weight, row, 16, false, true, nullptr},
      {"k_weight", k_weight, row, 16, false, true, nullptr},
      {"seq_len", seq_len, 4ull * d.n_slots, 4, false, positions != nullptr, nullptr},
      {"prefix_of", prefix_of, 4ull * d.B, 4, false, true, nullptr},
      {"win_len", win_len, 4ull * d.B, 4, false, true, nullptr},
      {"parent", parent, 4ull * n, 4, false, true, nullptr},
      {"positions", positions, 4ull * n, 4, false, true, nullptr},
  };
  GDN_RETURN_IF(check_rows(rows, 6, d.D));
  GDN_RETURN_IF(check_bufs(d, bufs, int(sizeof bufs / sizeof bufs[0])));
  gdn::RopeParams p{};
  GDN_RETURN_IF(gdn::device_status_word(&p.err));
  p.d = d, p.r = *rope, p.turns = turns, p.q_weight = q_weight, p.k_weight = k_weight;
  p.q = static_cast<const uint16_t*>(q), p.k = static_cast<const uint16_t*>(k), p.v = static_cast<const uint16_t*>(v);
  p.q_out = static_cast<uint16_t*>(q_out), p.k_out = static_cast<uint16_t*>(k_win), p.v_out = static_cast<uint16_t*>(v_win);
  p.seq_len = seq_len, p.prefix_of = prefix_of, p.positions = positions, p.win_len = win_len, p.parent = parent;
  p.n_tokens = int32_t(n), p.hq = q ? d.Hq : 0, p.hk = k ? d.Hkv : 0, p.hv = v ? d.Hkv : 0;
  const cudaError_t e = gdn::launch_rope_window(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "rotation launch: %s", cudaGetErrorString(e));
  return gdn::report_ok();
}

gdn_status gdn_kv_append_marked(const gdn_kv_dims* dims, int32_t layer, const gdn_rope* rope, const uint64_t* turns,
                                const float* q_weight, const float* k_weight, int64_t n_tokens,
                                const int32_t* cu_seqlens, const void* q, const void* k, const void* v,
                                const int32_t* positions, void* k_cache, void* v_cache, const int32_t* page_table,
                                const int32_t* seq_len, const int32_t* refused, const int32_t* prefix_of, void* q_out,
                                gdn_stream_t stream) {
  GDN_RETURN_IF(check_dims(dims, kPacked, false));
  const gdn_kv_dims d = normal(*dims);
  GDN_RETURN_IF(check_cache_strides(d));
  GDN_RETURN_IF(check_rope(rope, d, turns, q_weight, k_weight));
  if (layer < 0 || layer >= d.n_layers) return fail(GDN_ERR_INVALID_ARG, "layer=%d outside 0..%d", layer, d.n_layers - 1);
  if (n_tokens < 0 || n_tokens >= (1LL << 31)) return fail(GDN_ERR_INVALID_ARG, "n_tokens=%lld outside 0..2^31-1", (long long)n_tokens);
  if (!q != !q_out) return fail(GDN_ERR_INVALID_ARG, "q without its %s", q ? "output" : "input");
  if (d.B == 0 || n_tokens == 0) return gdn::report_ok();
  const long long n = n_tokens, ks = rope->kv_token_stride, kh = rope->kv_head_stride;
  const Rows rows[] = {
      {"q", q, n, rope->q_token_stride, rope->q_head_stride, d.Hq, false, nullptr},
      {"k", k, n, ks, kh, d.Hkv, false, nullptr},
      {"v", v, n, ks, kh, d.Hkv, false, nullptr},
      {"q_out", q_out, n, d.q_token_stride, d.D, d.Hq, true, rows[0].name},
  };
  if (!k || !v) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", k ? "v" : "k");
  const unsigned long long pairs = 4ull * rope->rot_dim, row = 4ull * d.D;
  const Buf bufs[] = {
      rows_buf(rows[0], d.D), rows_buf(rows[1], d.D), rows_buf(rows[2], d.D), rows_buf(rows[3], d.D),
      {"turns", turns, pairs, 8, false, true, nullptr},
      {"q_weight", q_weight, row, 16, false, true, nullptr},
      {"k_weight", k_weight, row, 16, false, true, nullptr},
      {"cu_seqlens", cu_seqlens, 4ull * (d.B + 1), 4, false, false, nullptr},
      {"page_table", page_table, 4ull * d.n_slots * d.max_pages, 4, false, false, nullptr},
      {"seq_len", seq_len, 4ull * d.n_slots, 4, false, false, nullptr},
      {"refused", refused, 4ull * d.n_slots, 4, false, true, nullptr},
      {"prefix_of", prefix_of, 4ull * d.B, 4, false, true, nullptr},
      {"positions", positions, 4ull * n, 4, false, true, nullptr},
      {"k_cache", k_cache, cache_bytes(d), 16, true, false, kInterleaved},
      {"v_cache", v_cache, cache_bytes(d), 16, true, false, kInterleaved},
  };
  GDN_RETURN_IF(check_rows(rows, 4, d.D));
  GDN_RETURN_IF(check_bufs(d, bufs, int(sizeof bufs / sizeof bufs[0])));
  gdn::RopeParams p{};
  GDN_RETURN_IF(gdn::device_status_word(&p.err));
  p.d = d, p.r = *rope, p.turns = turns, p.q_weight = q_weight, p.k_weight = k_weight;
  p.q = static_cast<const uint16_t*>(q), p.k = static_cast<const uint16_t*>(k), p.v = static_cast<const uint16_t*>(v);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_cache) + layer * d.cache_layer_stride;
  p.v_out = static_cast<uint16_t*>(v_cache) + layer * d.cache_layer_stride;
  p.seq_len = seq_len, p.prefix_of = prefix_of, p.positions = positions, p.cu = cu_seqlens, p.table = page_table;
  p.refused = refused;
  p.n_tokens = int32_t(n), p.hq = q ? d.Hq : 0, p.hk = d.Hkv, p.hv = d.Hkv;
  const cudaError_t e = gdn::launch_append(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
  return gdn::report_ok();
}

gdn_status gdn_kv_append(const gdn_kv_dims* dims, int32_t layer, const gdn_rope* rope, const uint64_t* turns,
                         const float* q_weight, const float* k_weight, int64_t n_tokens, const int32_t* cu_seqlens,
                         const void* q, const void* k, const void* v, const int32_t* positions, void* k_cache,
                         void* v_cache, const int32_t* page_table, const int32_t* seq_len, const int32_t* prefix_of,
                         void* q_out, gdn_stream_t stream) {
  return gdn_kv_append_marked(dims, layer, rope, turns, q_weight, k_weight, n_tokens, cu_seqlens, q, k, v, positions,
                              k_cache, v_cache, page_table, seq_len, nullptr, prefix_of, q_out, stream);
}

gdn_status gdn_attn_prefill_workspace_size(const gdn_kv_dims* dims, int64_t n_tokens, uint64_t* bytes) {
  GDN_RETURN_IF(check_dims(dims, kPacked, false));
  if (n_tokens < 0 || n_tokens >= (1LL << 31)) return fail(GDN_ERR_INVALID_ARG, "n_tokens=%lld outside 0..2^31-1", (long long)n_tokens);
  if (!bytes) return fail(GDN_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = gdn::packed_attn_workspace_bytes(*dims, n_tokens);
  return gdn::report_ok();
}

gdn_status gdn_attn_prefill_marked(const gdn_kv_dims* dims, int32_t layer, int64_t n_tokens,
                                   const int32_t* cu_seqlens, const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* page_table, const int32_t* seq_len, const int32_t* refused,
                                   const int32_t* prefix_of, int32_t causal, float scale, void* out, float* lse,
                                   void* workspace, uint64_t workspace_bytes, gdn_stream_t stream) {
  GDN_RETURN_IF(check_dims(dims, kPacked, false));
  const gdn_kv_dims d = normal(*dims);
  GDN_RETURN_IF(check_cache_strides(d));
  if (layer < 0 || layer >= d.n_layers) return fail(GDN_ERR_INVALID_ARG, "layer=%d outside 0..%d", layer, d.n_layers - 1);
  if (n_tokens < 0 || n_tokens >= (1LL << 31)) return fail(GDN_ERR_INVALID_ARG, "n_tokens=%lld outside 0..2^31-1", (long long)n_tokens);
  if (n_tokens * d.Hq > (1LL << 33)) return fail(GDN_ERR_UNSUPPORTED, "more than 2^33 rows");
  if (n_tokens > (1LL << 58) / d.q_token_stride) return fail(GDN_ERR_INVALID_ARG, "q is too large");
  if (!std::isfinite(scale)) return fail(GDN_ERR_INVALID_ARG, "scale not finite");
  if (d.B == 0 || n_tokens == 0) return gdn::report_ok();
  const unsigned long long n = (unsigned long long)n_tokens, need = gdn::packed_attn_workspace_bytes(d, n_tokens);
  if (workspace_bytes < need) return fail(GDN_ERR_INVALID_ARG, "workspace has %llu bytes, %llu needed", (unsigned long long)workspace_bytes, need);
  const Buf bufs[] = {
      {"q", q, 2 * ((n - 1) * d.q_token_stride + (unsigned long long)d.Hq * d.D), 16, false, false, nullptr},
      {"k_cache", k_cache, cache_bytes(d), 16, false, false, nullptr},
      {"v_cache", v_cache, cache_bytes(d), 16, false, false, nullptr},
      {"cu_seqlens", cu_seqlens, 4ull * (d.B + 1), 4, false, false, nullptr},
      {"page_table", page_table, 4ull * d.n_slots * d.max_pages, 4, false, false, nullptr},
      {"seq_len", seq_len, 4ull * d.n_slots, 4, false, false, nullptr},
      {"refused", refused, 4ull * d.n_slots, 4, false, true, nullptr},
      {"prefix_of", prefix_of, 4ull * d.B, 4, false, true, nullptr},
      {"out", out, 2ull * n * d.Hq * d.D, 16, true, false, nullptr},
      {"lse", lse, 4ull * n * d.Hq, 4, true, true, nullptr},
      {"workspace", workspace, need, 256, true, false, nullptr},
  };
  GDN_RETURN_IF(check_bufs(d, bufs, int(sizeof bufs / sizeof bufs[0])));
  gdn::PackedAttnParams p{};
  GDN_RETURN_IF(gdn::device_status_word(&p.err));
  p.d = d, p.n_tokens = int32_t(n_tokens), p.cu = cu_seqlens;
  p.q = static_cast<const uint16_t*>(q);
  p.k_cache = static_cast<const uint16_t*>(k_cache) + layer * d.cache_layer_stride;
  p.v_cache = static_cast<const uint16_t*>(v_cache) + layer * d.cache_layer_stride;
  p.table = page_table, p.seq_len = seq_len, p.prefix_of = prefix_of, p.refused = refused, p.causal = causal != 0, p.scale = scale;
  p.out = static_cast<uint16_t*>(out), p.lse = lse, p.ws = workspace;
  const cudaError_t e = gdn::launch_packed_attn(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "prefill attention launch: %s", cudaGetErrorString(e));
  return gdn::report_ok();
}

gdn_status gdn_attn_prefill(const gdn_kv_dims* dims, int32_t layer, int64_t n_tokens, const int32_t* cu_seqlens,
                            const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                            const int32_t* seq_len, const int32_t* prefix_of, int32_t causal, float scale, void* out,
                            float* lse, void* workspace, uint64_t workspace_bytes, gdn_stream_t stream) {
  return gdn_attn_prefill_marked(dims, layer, n_tokens, cu_seqlens, q, k_cache, v_cache, page_table, seq_len, nullptr,
                                 prefix_of, causal, scale, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
