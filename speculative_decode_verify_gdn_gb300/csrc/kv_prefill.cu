// Attention of packed queries over the paged cache (gdn_attn_prefill; contract in include/gdn_kv.h).
//
// Mathematics: softmax over a row's keys in one pass with a running maximum m and sum l.  A warp per
// (token, query head); a lane holds D / 32 elements of the head.
#include "kv_device.cuh"

namespace gdn {

namespace {

constexpr int kRowWarps = 8;

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kRowWarps) prefill_rows_kernel(const __grid_constant__ PackedAttnParams p) {
  constexpr int N = D / 32;
  pdl_launch_dependents();
  pdl_wait();
  const gdn_kv_dims& d = p.d;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (row >= (long long)p.n_tokens * d.Hq) return;
  bool bad = p.cu[0] != 0 || p.cu[d.B] > p.n_tokens;
  for (int i = lane; i < d.B; i += 32) bad |= p.cu[i] > p.cu[i + 1];
  if (__any_sync(0xffffffffu, bad)) {
    atomicOr(p.err, kDevErrSeqlens);
    return;
  }
  const int token = int(row / d.Hq), h = int(row - (long long)token * d.Hq), kvh = h / (d.Hq / d.Hkv);
  const int b = find_sequence(p.cu, d.B, token, lane);
  const int lo = p.cu[b], hi = p.cu[b + 1];
  if (token >= hi) return;
  const int own = checked_slot_len(p.seq_len[d.slot0 + b], d, p.err);
  const int prefix = checked_prefix(p.prefix_of, b, d, p.err);
  float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const float2 x = unpack16<F16>(*reinterpret_cast<const uint32_t*>(p.q + token * d.q_token_stride + h * D + lane * N + j));
    q[j] = x.x * p.scale, q[j + 1] = x.y * p.scale, o[j] = o[j + 1] = 0.f;
  }
  for (int part = 0; part < 2; ++part) {
    const int slot = part ? d.slot0 + b : prefix;
    if (slot < 0) continue;
    long long n = part ? own : checked_slot_len(p.seq_len[slot], d, p.err);
    if (part && p.causal) n = (long long)own - (hi - lo) + (token - lo) + 1;
    for (int i = 0; i < n; ++i) {
      const int col = i / d.page_size, page = p.table[(long long)slot * d.max_pages + col];
      if (page < 0 || page >= d.n_pages) {
        atomicOr(p.err, GDN_DEVERR_KV_PAGE);
        continue;
      }
      const long long at = page * d.cache_page_stride + (i - col * d.page_size) * d.cache_token_stride + kvh * d.cache_head_stride + lane * N;
      float s = 0.f, v[N];
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const float2 k = unpack16<F16>(*reinterpret_cast<const uint32_t*>(p.k_cache + at + j));
        const float2 x = unpack16<F16>(*reinterpret_cast<const uint32_t*>(p.v_cache + at + j));
        s += q[j] * k.x + q[j + 1] * k.y;
        v[j] = x.x, v[j + 1] = x.y;
      }
      s = warp_sum(s);
      const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - mn), w = mn == -INFINITY ? 0.f : expf(s - mn);
      m = mn;
      l = l * f + w;
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = o[j] * f + w * v[j];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* const out = reinterpret_cast<uint32_t*>(p.out + ((long long)token * d.Hq + h) * D + lane * N);
#pragma unroll
  for (int j = 0; j < N; j += 2) out[j / 2] = pack16<F16>(o[j] * inv, o[j + 1] * inv);
  if (p.lse && lane == 0) p.lse[(long long)token * d.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t packed_attn_workspace_bytes(const gdn_kv_dims&, int64_t) { return 256; }

cudaError_t launch_packed_attn(const PackedAttnParams& p, cudaStream_t stream) {
  const unsigned grid = unsigned(((long long)p.n_tokens * p.d.Hq + kRowWarps - 1) / kRowWarps);
  auto kernel = p.d.D == 128 ? (p.d.dtype ? prefill_rows_kernel<128, true> : prefill_rows_kernel<128, false>)
                             : (p.d.dtype ? prefill_rows_kernel<64, true> : prefill_rows_kernel<64, false>);
  return launch_dependent(kernel, grid, 32 * kRowWarps, 0, stream, p);
}

}  // namespace gdn
