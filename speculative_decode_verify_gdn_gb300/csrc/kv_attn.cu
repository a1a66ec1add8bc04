// Attention of verify windows over the paged cache (contract in include/gdn_kv.h).
//
// One warp per row (sequence, window token, query head): the lanes hold the query, and the keys
// of the prefix, of the sequence and of the window pass one by one through an online softmax
// (running maximum and sum in f32).
#include <cuda_fp16.h>

#include "gdn_common.cuh"
#include "kv_kernels.h"

namespace gdn {

namespace {

constexpr int kRowWarps = 8;

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
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

template <int D, bool F16>
__global__ void __launch_bounds__(32 * kRowWarps) attn_row_kernel(const AttnParams p) {
  constexpr int N = D / 64;  // 32-bit words (pairs of elements) per lane
  const gdn_kv_dims& d = p.d;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (row >= (long long)d.B * d.K * d.Hq) return;
  const int h = int(row % d.Hq);
  const long long tok = row / d.Hq;
  const int t = int(tok % d.K), b = int(tok / d.K);
  const int kh = h / (d.Hq / d.Hkv);
  int win = p.win_len ? p.win_len[b] : d.K;
  if (win < 0 || win > d.K) {
    atomicOr(p.err, GDN_DEVERR_KV_WINDOW);
    win = win < 0 ? 0 : d.K;
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out) + row * (D / 2);
  if (t >= win) {
#pragma unroll
    for (int i = 0; i < N; ++i) out[32 * i + lane] = 0;
    if (p.lse && lane == 0) p.lse[row] = -INFINITY;
    return;
  }
  const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) + tok * d.q_token_stride + (long long)h * D);
  float2 qv[N], acc[N];
  const float c = p.scale * 1.44269504f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    qv[i] = unpack2<F16>(q[32 * i + lane]);
    qv[i].x *= c, qv[i].y *= c;
    acc[i] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  auto key = [&](const uint16_t* k, const uint16_t* v) {
    float s = 0.f;
    float2 vv[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 kk = unpack2<F16>(reinterpret_cast<const uint32_t*>(k)[32 * i + lane]);
      vv[i] = unpack2<F16>(reinterpret_cast<const uint32_t*>(v)[32 * i + lane]);
      s += qv[i].x * kk.x + qv[i].y * kk.y;
    }
    s = warp_sum(s);
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
    l = l * f + w;
    m = mn;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i].x = acc[i].x * f + w * vv[i].x, acc[i].y = acc[i].y * f + w * vv[i].y;
  };
  auto cached = [&](int slot) {
    const int n = slot_len(p, slot);
    const int32_t* pages = p.table + (long long)slot * d.max_pages;
    for (int at = 0; at < n; at += d.page_size) {
      const int page = pages[at / d.page_size];
      if (page < 0 || page >= d.n_pages) {
        atomicOr(p.err, GDN_DEVERR_KV_PAGE);
        continue;
      }
      const long long o = p.layer * d.cache_layer_stride + page * d.cache_page_stride + kh * d.cache_head_stride;
      const int in = n - at < d.page_size ? n - at : d.page_size;
      for (int i = 0; i < in; ++i)
        key(static_cast<const uint16_t*>(p.k_cache) + o + i * d.cache_token_stride,
            static_cast<const uint16_t*>(p.v_cache) + o + i * d.cache_token_stride);
    }
  };
  if (p.prefix_of) {
    const int s = p.prefix_of[b];
    if (s < -1 || s >= d.n_slots)
      atomicOr(p.err, GDN_DEVERR_KV_SLOT);
    else if (s >= 0)
      cached(s);
  }
  cached(d.slot0 + b);
  uint32_t seen = 0;
  if (p.parent) {
    for (int j = t; j >= 0;) {
      seen |= 1u << j;
      int up = p.parent[(long long)b * d.K + j];
      if (up < -1 || up >= j) {
        atomicOr(p.err, GDN_DEVERR_TREE_PARENT);
        up = -1;
      }
      j = up;
    }
  } else {
    seen = (2u << t) - 1u;
  }
  for (int j = 0; j < win; ++j)
    if (seen >> j & 1) {
      const long long o = ((long long)b * d.K + j) * d.win_token_stride + (long long)kh * D;
      key(static_cast<const uint16_t*>(p.k_win) + o, static_cast<const uint16_t*>(p.v_win) + o);
    }
  const float r = 1.f / l;  // a live row sees at least itself: l >= 1
#pragma unroll
  for (int i = 0; i < N; ++i) out[32 * i + lane] = pack2<F16>(acc[i].x * r, acc[i].y * r);
  if (p.lse && lane == 0) p.lse[row] = (m + log2f(l)) * 0.693147181f;
}

}  // namespace

size_t attn_workspace_bytes(const gdn_kv_dims&) { return 256; }

cudaError_t launch_attn(const AttnParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.d.B * p.d.K * p.d.Hq;
  const unsigned grid = unsigned((rows + kRowWarps - 1) / kRowWarps);
  if (p.d.D == 128) {
    if (p.d.dtype) attn_row_kernel<128, true><<<grid, 32 * kRowWarps, 0, stream>>>(p);
    else attn_row_kernel<128, false><<<grid, 32 * kRowWarps, 0, stream>>>(p);
  } else {
    if (p.d.dtype) attn_row_kernel<64, true><<<grid, 32 * kRowWarps, 0, stream>>>(p);
    else attn_row_kernel<64, false><<<grid, 32 * kRowWarps, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace gdn
