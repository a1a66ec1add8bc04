// Norms and rotation of the heads of queries and keys: of verify windows (gdn_attn_rope), and of packed
// tokens whose keys and values go to pages (gdn_kv_append).  Contracts in include/gdn_kv.h.
//
// Mathematics: a head x of D elements becomes y_i = x_i (c + w_i) / sqrt(mean x^2 + eps), and the pairs
// (a, b) of its first rot_dim elements (a cos - b sin, b cos + a sin) m.  The angle of a pair is
// position x turns in fractions of a turn, a 64-bit product modulo 2^64: exact to 2^-34 of a turn for
// every position below 2^30, where a 32-bit float of the angle is off by radians.  Its upper half, rounded
// to 32 bits, is turned into cosine and sine in f32 (half turns in [-1, 1): off by at most 2^-25).
//
// A CTA takes a few tokens with all their heads.  The first heads' loads go out at once; meanwhile a
// warp per token finds its sequence, position and place, and a thread per pair the token's cosines and
// sines, which all its heads share.  A head is D / 8 lanes, 8 elements each: where halves are paired, 4 of
// the first and the 4 that they pair with, so that no element has to change lanes.
//
// Bound: HBM, 2 bytes read and 2 written per element.
#include "kv_device.cuh"
#include "kv_index.h"

namespace gdn {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeToks = 4;   // tokens of a CTA, at most (a warp each looks them up)
constexpr int kRopeAhead = 4;  // heads that a group of lanes has in flight

struct Tok {
  long long at;  // packed: element of the token's first key (and value) in the layer's pages
  long long pos; // for the rotation (a slot and a prefix of 2^30 tokens each end at 2^31)
  int32_t live;  // windows: 0 is padding; packed: 0 is not written, 2 is q alone
};

// Position (and state) of window token `token`, by a converged warp.
__device__ __forceinline__ Tok window_token(const RopeParams& p, int token, int lane) {
  const gdn_kv_dims& d = p.d;
  const int b = token / d.K, t = token - b * d.K;
  Tok x{};
  int win = p.win_len ? p.win_len[b] : d.K;
  if (p.positions) {
    x.pos = p.positions[token];
  } else {
    const int slot = checked_prefix(p.prefix_of, b, d, p.err);
    x.pos = checked_slot_len(p.seq_len[d.slot0 + b], d, p.err);
    if (slot >= 0) x.pos += checked_slot_len(p.seq_len[slot], d, p.err);
  }
  if (win < 0 || win > d.K) {
    atomicOr(p.err, GDN_DEVERR_KV_WINDOW);
    win = win < 0 ? 0 : d.K;
  }
  x.live = t < win;
  if (p.positions) return x;
  if (!p.parent) {
    x.pos += t;
    return x;
  }
  // each lane holds a node's parent; four doublings reach every ancestor of 16 nodes
  int up = -1;
  if (lane < win) {
    up = p.parent[(long long)b * d.K + lane];
    if (up < -1 || up >= lane) {
      atomicOr(p.err, kDevErrTreeParent);
      up = -1;
    }
  }
  uint32_t path = 1u << lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __shfl_sync(0xffffffffu, path, up & 31);
    const int g = __shfl_sync(0xffffffffu, up, up & 31);
    if (up >= 0) path |= a, up = g;
  }
  x.pos += __popc(__shfl_sync(0xffffffffu, path, t)) - 1;
  return x;
}

// Position and place of packed token `token`, by a converged warp.
__device__ __forceinline__ Tok packed_token(const RopeParams& p, int token, int lane) {
  const gdn_kv_dims& d = p.d;
  Tok x{};
  const int b = find_sequence(p.cu, d.B, token, lane);
  const int lo = p.cu[b], hi = p.cu[b + 1];
  if (token < lo || token >= hi) return x;  // behind the last sequence (or bounds out of order)
  const int len = checked_slot_len(p.seq_len[d.slot0 + b], d, p.err);
  const int slot = checked_prefix(p.prefix_of, b, d, p.err);
  if ((long long)hi - lo > len) {
    atomicOr(p.err, GDN_DEVERR_KV_LEN);
    return x;
  }
  const int at = len - (hi - token), col = at / d.page_size;
  const int page = p.table[(long long)(d.slot0 + b) * d.max_pages + col];
  x.pos = at;
  if (slot >= 0) x.pos += checked_slot_len(p.seq_len[slot], d, p.err);
  if (p.positions) x.pos = p.positions[token];
  x.live = 1;
  if (page < 0 || page >= d.n_pages) {
    atomicOr(p.err, GDN_DEVERR_KV_PAGE);
    x.live = 2;
  }
  x.at = page * d.cache_page_stride + (at - col * d.page_size) * d.cache_token_stride;
  return x;
}

__device__ __forceinline__ uint2 load4(const uint16_t* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <int D, bool F16, bool PACKED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, const int toks, const uint32_t by_heads) {
  constexpr int LANES = D / 8, GROUPS = kRopeThreads / LANES, U = kRopeAhead;
  __shared__ Tok tok[kRopeToks];
  __shared__ __align__(16) float cs[kRopeToks][2][D / 2];
  __shared__ __align__(16) float weight[2][D];
  pdl_launch_dependents();
  pdl_wait();
  const gdn_kv_dims& d = p.d;
  const gdn_rope& r = p.r;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, l = tid % LANES, group = tid / LANES;
  const int tok0 = int(blockIdx.x) * toks, n = p.n_tokens - tok0 < toks ? p.n_tokens - tok0 : toks;
  const int H = p.hq + p.hk + p.hv, rows = n * H;
  const int half = r.rot_dim / 2;
  const bool turned = 8 * l < r.rot_dim;
  const int o0 = turned && !r.interleaved ? 4 * l : 8 * l, o1 = turned && !r.interleaved ? half + 4 * l : 8 * l + 4;

  struct Row {
    int t, h, kind;  // token of the CTA, head of its kind: 0 q, 1 k, 2 v
  };
  auto row_of = [&](int i) {
    Row x;
    x.t = by_heads ? int(__umulhi(uint32_t(i), by_heads)) : i / H;
    x.h = i - x.t * H;
    x.kind = x.h < p.hq ? 0 : x.h < p.hq + p.hk ? 1 : 2;
    x.h -= x.kind == 0 ? 0 : x.kind == 1 ? p.hq : p.hq + p.hk;
    return x;
  };
  uint2 a[U], b[U];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * GROUPS;
      a[u] = b[u] = make_uint2(0u, 0u);
      if (i < rows) {
        const Row x = row_of(i);
        const long long token = tok0 + x.t;
        const uint16_t* src = x.kind == 0 ? p.q + token * r.q_token_stride + x.h * r.q_head_stride
                                          : (x.kind == 1 ? p.k : p.v) + token * r.kv_token_stride + x.h * r.kv_head_stride;
        a[u] = load4(src + o0);
        b[u] = load4(src + o1);
      }
    }
  };
  load(group);

  if (warp < n) {
    const Tok x = PACKED ? packed_token(p, tok0 + warp, lane) : window_token(p, tok0 + warp, lane);
    if (lane == 0) tok[warp] = x;
  }
  if (p.q_weight)
    for (int i = tid; i < D; i += kRopeThreads) weight[0][i] = r.weight_offset + p.q_weight[i];
  if (p.k_weight)
    for (int i = tid; i < D; i += kRopeThreads) weight[1][i] = r.weight_offset + p.k_weight[i];
  if (PACKED && blockIdx.x == 0) {  // (a token's own bounds are checked where it is looked up)
    bool bad = tid == 0 && (p.cu[0] != 0 || p.cu[d.B] > p.n_tokens);
    for (int i = tid; i < d.B; i += kRopeThreads) bad |= p.cu[i] > p.cu[i + 1];
    if (bad) atomicOr(p.err, kDevErrSeqlens);
  }
  __syncthreads();
  for (int i = tid; i < n * (D / 2); i += kRopeThreads) {
    const int t = i / (D / 2), j = i % (D / 2);
    if (j < half) {
      const uint64_t turn = uint64_t(tok[t].pos) * p.turns[j];
      float s, c;
      sincospif(float(int32_t(uint32_t((turn + (1ull << 31)) >> 32))) * 0x1p-31f, &s, &c);
      cs[t][0][j] = c * r.magnitude;
      cs[t][1][j] = s * r.magnitude;
    }
  }
  __syncthreads();

  for (int base = group; base - group < rows; base += U * GROUPS) {
    if (base != group) load(base);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * GROUPS;
      const Row x = row_of(i < rows ? i : 0);
      const bool normed = x.kind == 0 ? p.q_weight != nullptr : x.kind == 1 && p.k_weight != nullptr;
      float v[8];
      {
        const float2 v0 = unpack16<F16>(a[u].x), v1 = unpack16<F16>(a[u].y), v2 = unpack16<F16>(b[u].x), v3 = unpack16<F16>(b[u].y);
        v[0] = v0.x, v[1] = v0.y, v[2] = v1.x, v[3] = v1.y, v[4] = v2.x, v[5] = v2.y, v[6] = v3.x, v[7] = v3.y;
      }
      if (p.q_weight || p.k_weight) {  // (the lanes of a warp may hold heads of different kinds: all sum)
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sq += v[j] * v[j];
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        if (normed) {
          const float inv = rsqrtf(sq * (1.f / D) + r.eps);
          const float4 w0 = *reinterpret_cast<const float4*>(&weight[x.kind][o0]), w1 = *reinterpret_cast<const float4*>(&weight[x.kind][o1]);
          v[0] *= inv * w0.x, v[1] *= inv * w0.y, v[2] *= inv * w0.z, v[3] *= inv * w0.w;
          v[4] *= inv * w1.x, v[5] *= inv * w1.y, v[6] *= inv * w1.z, v[7] *= inv * w1.w;
        }
      }
      if (i >= rows) continue;
      if (turned && x.kind < 2) {
        const float4 c = *reinterpret_cast<const float4*>(&cs[x.t][0][4 * l]), s = *reinterpret_cast<const float4*>(&cs[x.t][1][4 * l]);
        const float cj[4] = {c.x, c.y, c.z, c.w}, sj[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float &e0 = r.interleaved ? v[2 * j] : v[j], &e1 = r.interleaved ? v[2 * j + 1] : v[4 + j];
          const float y0 = e0 * cj[j] - e1 * sj[j], y1 = e1 * cj[j] + e0 * sj[j];
          e0 = y0, e1 = y1;
        }
      }
      uint2 out0 = a[u], out1 = b[u];  // (values are copied as they are)
      if (x.kind < 2 && (normed || turned)) {
        out0 = make_uint2(pack16<F16>(v[0], v[1]), pack16<F16>(v[2], v[3]));
        out1 = make_uint2(pack16<F16>(v[4], v[5]), pack16<F16>(v[6], v[7]));
      }
      const int live = tok[x.t].live;
      const long long token = tok0 + x.t;
      uint16_t* dst;
      if (PACKED) {
        if (live == 0 || (live == 2 && x.kind != 0)) continue;
        dst = x.kind == 0 ? p.q_out + token * d.q_token_stride + x.h * D
                          : (x.kind == 1 ? p.k_out : p.v_out) + tok[x.t].at + x.h * d.cache_head_stride;
      } else {
        if (!live) out0 = out1 = make_uint2(0u, 0u);
        dst = x.kind == 0 ? p.q_out + token * d.q_token_stride + x.h * D
                          : (x.kind == 1 ? p.k_out : p.v_out) + token * d.win_token_stride + x.h * D;
      }
      *reinterpret_cast<uint2*>(dst + o0) = out0;
      *reinterpret_cast<uint2*>(dst + o1) = out1;
    }
  }
}

template <bool PACKED>
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  const int toks = p.n_tokens <= 8 * 152 ? 1 : kRopeToks;
  const unsigned long long H = (unsigned long long)(p.hq + p.hk + p.hv);
  // ceil(2^32 / H): the quotient by H is exact while row x H < 2^32
  const uint32_t by_heads = H > 1 && H * H * toks < (1ull << 32) ? uint32_t(((1ull << 32) + H - 1) / H) : 0u;
  const unsigned grid = unsigned((p.n_tokens + toks - 1) / toks);
  auto kernel = p.d.D == 128 ? (p.d.dtype ? rope_kernel<128, true, PACKED> : rope_kernel<128, false, PACKED>)
                             : (p.d.dtype ? rope_kernel<64, true, PACKED> : rope_kernel<64, false, PACKED>);
  return launch_dependent(kernel, grid, kRopeThreads, 0, stream, p, toks, by_heads);
}

}  // namespace

cudaError_t launch_rope_window(const RopeParams& p, cudaStream_t stream) { return launch_rope<false>(p, stream); }
cudaError_t launch_append(const RopeParams& p, cudaStream_t stream) { return launch_rope<true>(p, stream); }

}  // namespace gdn
