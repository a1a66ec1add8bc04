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
// Bound: HBM, 2 bytes read and 2 written per element.  36864 ragged tokens to pages (Hq=32 Hkv=8 D=128, norms): 149 us,
// 6.1 TB/s (6.7 is a plain copy's); windows of 256 trees of 16 tokens, padded: 18.6 us for 77 MB, a single round of CTAs
// whose chain of lookups (lengths, prefix, tree), sines and heads is 10 us long; one token: 10.6 us, the host's.
// What carried it, in us of the 36864 tokens: a row of 16-lane groups with the coefficients worked out per head 271; packed
// arithmetic, heads in order within a kind 188; four heads in flight and 64 registers 162; CTAs of 128 threads 156;
// streaming stores 151; coefficients per token in shared memory 150.  Dropped: 16 elements a lane (spills, 165 and more);
// a load for each head that is done (reads and writes alternate in memory: 180).
#include "kv_device.cuh"
#include "kv_index.h"

namespace gdn {

namespace {

constexpr int kRopeThreads = 128;
// CTAs to an SM: windows 7 (72 registers, 24 to 28 bytes a thread spilled: 18.6 us, 21.3 with 8, at 256 trees of 16 tokens), packed
// tokens 8 (64 registers, 52 to 68 bytes spilled: 149.5 us, 152.7 with 7, at 36864 tokens).
constexpr int rope_ctas(bool packed) { return packed ? 8 : 7; }
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
  const int refused = p.refused ? p.refused[d.slot0 + b] : -1;
  const int len = checked_slot_len(p.seq_len[d.slot0 + b], d, p.err);
  const int slot = checked_prefix(p.prefix_of, b, d, p.err);
  // (a slot that is as long as when room for its tokens was refused: its last tokens are others)
  if ((long long)hi - lo > len || refused == len) {
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

// Eight elements of a head: a lane's four and the four that they pair with (INTER: pairs side by side).
struct Part {
  uint2 lo, hi;
};
__device__ __forceinline__ uint2 load4(const uint16_t* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// A token's transform of queries (0) and keys (1), as coefficients of the pairs (a, b) of a head:
// a <- a ca + b sb, b <- b cb + a sa, with the norm's weights and the magnitude in them.
template <int D>
struct Turn {
  float ca[D / 2], sb[D / 2], cb[D / 2], sa[D / 2];
};
// A lane's four pairs of them, two pairs to a float2.
struct Coefs {
  float2 ca[2], sb[2], cb[2], sa[2];
  template <int D>
  __device__ __forceinline__ Coefs(const Turn<D>& f, int first) {
    read(f.ca + first, ca), read(f.sb + first, sb), read(f.cb + first, cb), read(f.sa + first, sa);
  }
  static __device__ __forceinline__ void read(const float* p, float2 (&v)[2]) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = make_float2(x.x, x.y), v[1] = make_float2(x.z, x.w);
  }
};
__device__ __forceinline__ float rsqrt_fast(float x) {  // (to 2 units; a mean square below 2^-126 counts as 0)
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, bool F16, bool INTER>
__device__ __forceinline__ Part transform(const Part& x, const Coefs& f, bool turned, bool normed, float eps) {
  const float2 w0 = unpack2<F16>(x.lo.x), w1 = unpack2<F16>(x.lo.y), w2 = unpack2<F16>(x.hi.x), w3 = unpack2<F16>(x.hi.y);
  const float2 a[2] = {INTER ? make_float2(w0.x, w1.x) : w0, INTER ? make_float2(w2.x, w3.x) : w1};
  const float2 b[2] = {INTER ? make_float2(w0.y, w1.y) : w2, INTER ? make_float2(w2.y, w3.y) : w3};
  float2 y[2], z[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    y[j] = mul2(a[j], f.ca[j]), z[j] = mul2(b[j], f.cb[j]);
    if (turned) y[j] = fma2(b[j], f.sb[j], y[j]), z[j] = fma2(a[j], f.sa[j], z[j]);
  }
  if (normed) {
    float2 q = mul2(a[0], a[0]);
    q = fma2(a[1], a[1], q), q = fma2(b[0], b[0], q), q = fma2(b[1], b[1], q);
    float sq = q.x + q.y;
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const float inv = rsqrt_fast(sq * (1.f / D) + eps);
    const float2 inv2 = make_float2(inv, inv);
#pragma unroll
    for (int j = 0; j < 2; ++j) y[j] = mul2(y[j], inv2), z[j] = mul2(z[j], inv2);
  }
  if (INTER)
    return Part{make_uint2(pack2<F16>(y[0].x, z[0].x), pack2<F16>(y[0].y, z[0].y)), make_uint2(pack2<F16>(y[1].x, z[1].x), pack2<F16>(y[1].y, z[1].y))};
  return Part{make_uint2(pack2<F16>(y[0].x, y[0].y), pack2<F16>(y[1].x, y[1].y)), make_uint2(pack2<F16>(z[0].x, z[0].y), pack2<F16>(z[1].x, z[1].y))};
}

template <int D, bool F16, bool PACKED, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, rope_ctas(PACKED)) rope_kernel(const __grid_constant__ RopeParams p, const int toks) {
  constexpr int LANES = D / 8, GROUPS = kRopeThreads / LANES, U = kRopeAhead;
  __shared__ Tok tok[kRopeToks];
  __shared__ __align__(16) Turn<D> turn[kRopeToks][2];
  pdl_launch_dependents();
  pdl_wait();
  const gdn_kv_dims& d = p.d;
  const gdn_rope& r = p.r;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5, l = tid % LANES;
  const int tok0 = int(blockIdx.x) * toks, n = p.n_tokens - tok0 < toks ? p.n_tokens - tok0 : toks;
  // `per` groups of lanes share a token: heads g, g + per, ...
  const int per = GROUPS / toks, t = tid / LANES / per, g = tid / LANES % per;
  const bool there = t < n;
  const int half = r.rot_dim / 2;
  const bool turned = 8 * l < r.rot_dim;
  const int o0 = turned && !INTER ? 4 * l : 8 * l, o1 = turned && !INTER ? half + 4 * l : 8 * l + 4;
  const long long token = tok0 + (there ? t : 0);
  // what nobody reads is not fetched: windows' padding, and packed rows behind the last sequence (in a large call:
  // it costs the loads a trip to L2)
  bool fetch = there;
  if (!PACKED && p.win_len && there) fetch = int(token % d.K) < p.win_len[token / d.K];
  if (PACKED && toks > 1 && tok0 >= p.cu[d.B] && blockIdx.x > 0) return;

  auto load = [&](const uint16_t* src) { return Part{load4(src + o0), load4(src + o1)}; };
  const Part zero{make_uint2(0u, 0u), make_uint2(0u, 0u)};
  const uint16_t* q_src = p.q + token * r.q_token_stride + g * r.q_head_stride;
  const long long kv_at = token * r.kv_token_stride + g * r.kv_head_stride;
  const uint16_t *k_src = p.k + kv_at, *v_src = p.v + kv_at;
  const long long q_step = per * r.q_head_stride, kv_step = per * r.kv_head_stride;
  const int hq = there ? p.hq : 0, hk = there ? p.hk : 0, hv = there ? p.hv : 0;
  const int fq = fetch ? hq : 0, fk = fetch ? hk : 0, fv = fetch ? hv : 0;  // heads to fetch
  Part q[U], k = zero, v = zero;
  auto load_q = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u, q_src += q_step) q[u] = h + u * per < fq ? load(q_src) : zero;
  };
  load_q(g);
  if (g < fk) k = load(k_src);
  if (g < fv) v = load(v_src);

  // a thread's pair is the same in every token: its turns and weights are on their way, too
  static_assert(kRopeThreads % (D / 2) == 0 && kRopeThreads >= D / 2, "a thread's pair is the same in every token");
  const int pair = tid % (D / 2), pair_lane = pair / 4;
  const bool pair_turned = 8 * pair_lane < r.rot_dim;
  const int e0 = INTER ? 2 * pair : pair_turned ? pair : 4 * pair_lane + pair, e1 = INTER ? e0 + 1 : pair_turned ? half + pair : e0 + 4;
  const uint64_t step = pair_turned ? p.turns[pair] : 0;
  float w[2][2] = {{1.f, 1.f}, {1.f, 1.f}};
  if (p.q_weight) w[0][0] = p.q_weight[e0] + r.weight_offset, w[0][1] = p.q_weight[e1] + r.weight_offset;
  if (p.k_weight) w[1][0] = p.k_weight[e0] + r.weight_offset, w[1][1] = p.k_weight[e1] + r.weight_offset;
  if (warp < n) {
    const Tok x = PACKED ? packed_token(p, tok0 + warp, lane) : window_token(p, tok0 + warp, lane);
    if (lane == 0) tok[warp] = x;
  }
  if (PACKED && blockIdx.x == 0) {  // (a token's own bounds are checked where it is looked up)
    bool bad = tid == 0 && (p.cu[0] != 0 || p.cu[d.B] > p.n_tokens);
    for (int i = tid; i < d.B; i += kRopeThreads) bad |= p.cu[i] > p.cu[i + 1];
    if (bad) atomicOr(p.err, kDevErrSeqlens);
  }
  __syncthreads();
  for (int i = tid / (D / 2); i < n; i += kRopeThreads / (D / 2)) {
    float s = 0.f, c = 1.f;
    if (pair_turned) {
      const uint64_t angle = uint64_t(tok[i].pos) * step;
      sincospif(float(int32_t(uint32_t((angle + (1ull << 31)) >> 32))) * 0x1p-31f, &s, &c);
      c *= r.magnitude, s *= r.magnitude;
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      Turn<D>& f = turn[i][kind];
      f.ca[pair] = w[kind][0] * c, f.sb[pair] = -w[kind][1] * s, f.cb[pair] = w[kind][1] * c, f.sa[pair] = w[kind][0] * s;
    }
  }
  __syncthreads();

  const Tok here = tok[there ? t : 0];
  const Turn<D>* const mine = turn[there ? t : 0];
  const bool keep_q = PACKED ? here.live != 0 : true, keep_kv = PACKED ? here.live == 1 : true;
  const bool blank = !PACKED && !here.live;  // (padding)
  auto store = [&](uint16_t* dst, const Part& x) {
    __stcs(reinterpret_cast<uint2*>(dst + o0), blank ? zero.lo : x.lo);
    __stcs(reinterpret_cast<uint2*>(dst + o1), blank ? zero.lo : x.hi);
  };
  {  // (every lane of a warp runs the same number of rounds: heads are summed over lanes)
    const Coefs f(mine[0], 4 * l);
    uint16_t* q_dst = p.q_out + token * d.q_token_stride + g * D;
    for (int h0 = 0; h0 < p.hq; h0 += U * per) {
      if (h0 > 0) load_q(g + h0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * per;
        if (h >= p.hq) break;
        const Part y = transform<D, F16, INTER>(q[u], f, turned, p.q_weight != nullptr, r.eps);
        if (g + h < hq && keep_q) store(q_dst, y);
        q_dst += per * D;
      }
    }
  }
  {
    const Coefs f(mine[1], 4 * l);
    const long long to = PACKED ? here.at + g * d.cache_head_stride : token * d.win_token_stride + g * D;
    const long long to_step = PACKED ? per * d.cache_head_stride : per * D;
    uint16_t *k_dst = p.k_out + to, *v_dst = p.v_out + to;
    const int all = p.hk > p.hv ? p.hk : p.hv;
    for (int h0 = 0; h0 < all; h0 += per) {
      const int h = g + h0;
      const Part k_now = k, v_now = v;
      k_src += kv_step, v_src += kv_step;
      if (h + per < fk) k = load(k_src);
      if (h + per < fv) v = load(v_src);
      const Part y = transform<D, F16, INTER>(k_now, f, turned, p.k_weight != nullptr, r.eps);
      if (h < hk && keep_kv) store(k_dst, y);
      if (h < hv && keep_kv) store(v_dst, v_now);
      k_dst += to_step, v_dst += to_step;
    }
  }
}

template <bool PACKED>
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  // Tokens of a CTA: 1 while all CTAs are on the card at once, 2 up to three times as many tokens, then 4.  Us with 1, 2 and 4 in
  // a graph, windows of Hq=32 Hkv=8 and Hq=16 Hkv=2, D=128: 1024 tokens 5.5 8.0 10.8 and 4.6 5.1 6.1; 1072 7.2 8.3 9.4 and
  // 6.1 5.2 5.1; 2048 10.7 10.2 13.4 and 7.9 5.6 7.2; 2992 13.7 13.8 15.8 and 10.9 8.2 8.0; 4096 19.8 18.5 17.2 and 14.3 9.7 8.3.
  // Packed tokens: 1216 6.1 6.9 9.0 and 5.0 4.7 5.4; 2048 10.0 11.0 16.8 and 8.1 6.3 8.7; 3000 13.5 14.4 17.8 and 10.9 8.6 9.3;
  // 4096 19.3 19.1 19.4 and 14.1 9.9 9.6; 16384 69 70 71 and 50 36 33.
  const int wave = rope_ctas(PACKED) * 152, toks = p.n_tokens <= wave ? 1 : p.n_tokens <= 3 * wave ? 2 : kRopeToks;
  const unsigned grid = ctas_of(p.n_tokens, toks);
  const bool f16 = p.d.dtype != 0;
  auto kernel = [&]() -> void (*)(RopeParams, int) {
    if (p.d.D == 128)
      return p.r.interleaved ? (f16 ? rope_kernel<128, true, PACKED, true> : rope_kernel<128, false, PACKED, true>)
                             : (f16 ? rope_kernel<128, true, PACKED, false> : rope_kernel<128, false, PACKED, false>);
    return p.r.interleaved ? (f16 ? rope_kernel<64, true, PACKED, true> : rope_kernel<64, false, PACKED, true>)
                           : (f16 ? rope_kernel<64, true, PACKED, false> : rope_kernel<64, false, PACKED, false>);
  }();
  return launch_dependent(kernel, grid, kRopeThreads, 0, stream, p, toks);
}

}  // namespace

cudaError_t launch_rope_window(const RopeParams& p, cudaStream_t stream) { return launch_rope<false>(p, stream); }
cudaError_t launch_append(const RopeParams& p, cudaStream_t stream) { return launch_rope<true>(p, stream); }

}  // namespace gdn
