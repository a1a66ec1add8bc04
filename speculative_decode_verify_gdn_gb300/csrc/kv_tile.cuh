// What the attention kernels over the paged cache share: tiles of 128 keys against tiles of 128 rows, for two
// streams on one SM (kv_attn.cu describes the whole).
#pragma once

#include <cuda.h>

#include "kv_device.cuh"

namespace gdn {

constexpr int kCtas = 152;       // one per SM; no CTA waits for another, so any number is correct
constexpr int kTileKeys = 128;
constexpr int kTileRows = 128;   // rows of a stream's tile, whole tokens of G query heads: 128 / G * G are used
constexpr int kBlockRows = 256;  // rows of an item, at most
constexpr int kGroupThreads = 128;  // a softmax group: one thread per row of a stream
constexpr int kTileThreads = 3 * kGroupThreads;  // two softmax groups; producer, two tensor-core warps, scheduler
constexpr float kLn2 = 0.693147180559945f, kLog2e = 1.442695040888963f;
// A running maximum may lag behind by up to 8 powers of two before O is rescaled: probabilities
// stay below 2^8, far inside both 16-bit types, and keep their relative precision.
constexpr float kLag = 8.0f;
// Longest wait inside the tile kernel (kMaxLooks): looks of at most 4 us each (measured), 17 s in all.
constexpr uint32_t kMaxLooks = 1u << 22;
// The scheduler looks on for as long as a segment takes, every 220 ns: up to a slot of 2^30 tokens on one
// CTA, 7 s and for a pair of row tiles about twice that.  A CTA that is stuck is found by the other
// warps' waits, and the scheduler ends with them.
constexpr uint32_t kMaxTurnLooks = 1u << 14, kMaxIdle = 1u << 28;
constexpr int kSegRing = 4;  // segments between the scheduler and the other warps

__device__ __forceinline__ long long first_tile(long long c, long long tiles) { return c * tiles / kCtas; }
__device__ __forceinline__ int cta_of(long long x, long long tiles) {
  int c = int(float(x) * (float(kCtas) / float(tiles)));  // (within one of it)
  c = c < 0 ? 0 : c > kCtas - 1 ? kCtas - 1 : c;
  while (c > 0 && first_tile(c, tiles) > x) --c;
  while (c < kCtas - 1 && first_tile(c + 1, tiles) <= x) ++c;
  return c;
}

template <int D, typename Seg>
struct TileLayout {
  static constexpr int BYTES = kTileKeys * D * 2;  // a tile of keys, values or queries
  static constexpr int HALF = kTileKeys * 128;     // 64 of the D columns: 128 rows of 128 bytes
  static constexpr int STAGES = D == 128 ? 5 : 10;  // >= 5: two tiles of values wait while a third of keys is read
  static constexpr int OFF_Q = 0;                  // one per stream
  static constexpr int OFF_RING = 2 * BYTES;
  static constexpr int OFF_BAR = OFF_RING + STAGES * BYTES;
  static constexpr int NBAR = 2 * STAGES + 10 + 2 * kSegRing;
  static constexpr int OFF_SEG = OFF_BAR + NBAR * 8;  // segments on their way from the scheduler
  static constexpr int TOTAL = OFF_SEG + kSegRing * int(sizeof(Seg)) + 1024;  // 1024: the base is aligned by hand
};

// A box of tokens of one head, all D elements (two 64-column halves, 16 KB apart in the tile), by an
// elected lane of the converged warp.
template <int D>
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* m, int c1, int c2, int c3, int c4, uint32_t bar) {
  if (D == 128)
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%2, {%4, %6, %7, %8, %9}], [%3];\n\t"
        "@q cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%1], [%2, {%5, %6, %7, %8, %9}], [%3];\n\t}" ::"r"(dst),
        "r"(dst + kTileKeys * 128), "l"(m), "r"(bar), "r"(0), "r"(64), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];\n\t}" ::"r"(dst),
        "l"(m), "r"(bar), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Shared-memory descriptor of a 128-byte-swizzled operand: rows of 128 bytes, groups of 8 rows
// 1024 bytes apart (SBO); LBO is the step between 64-column halves of an MN-major operand and not
// used by a K-major one.
// Low word of a descriptor; the high word (SBO, version, layout) is the same for all of them.
__device__ __forceinline__ uint32_t swizzled_desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// S = Q K^T of a tile: steps of 16 of the D elements (32 bytes of a swizzled row, then the other
// 64-column half, H 16-byte units on).  The whole warp runs it and one elected lane issues: a
// branch to one lane would cost every step its operands' way into uniform registers.
template <int D>
__device__ __forceinline__ void umma_scores(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
#define GDN_STEP(off, acc)                                                                        \
  "add.u32 a, %1, " off ";\n\tadd.u32 b, %2, " off ";\n\tmov.b64 da, {a, %4};\n\tmov.b64 db, {b, %4};\n\t" \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, " acc ";\n\t"
#define GDN_HEAD "{\n\t.reg .pred q, t, f;\n\t.reg .b32 a, b;\n\t.reg .b64 da, db;\n\telect.sync _|q, 0xffffffff;\n\t" \
  "setp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 f, 0, 0;\n\t"
  if (D == 128)
    asm volatile(GDN_HEAD GDN_STEP("0", "f") GDN_STEP("2", "t") GDN_STEP("4", "t") GDN_STEP("6", "t") GDN_STEP("1024", "t")
                     GDN_STEP("1026", "t") GDN_STEP("1028", "t") GDN_STEP("1030", "t") "}" ::"r"(d_tmem),
                 "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kDescHi)
                 : "memory");
  else
    asm volatile(GDN_HEAD GDN_STEP("0", "f") GDN_STEP("2", "t") GDN_STEP("4", "t") GDN_STEP("6", "t") "}" ::"r"(d_tmem),
                 "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kDescHi)
                 : "memory");
#undef GDN_STEP
#undef GDN_HEAD
}

// O += P V (O = P V unless `more`): steps of 16 keys, 8 columns of P and 2048 bytes of values each;
// the first one, and the other seven of a whole tile.
__device__ __forceinline__ void umma_values_first(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t more) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(more), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void umma_values_rest(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc) {
#define GDN_STEP(acol, boff)                                                        \
  "add.u32 a, %1, " acol ";\n\tadd.u32 b, %2, " boff ";\n\tmov.b64 db, {b, %4};\n\t" \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, t;\n\t"
  asm volatile(
      "{\n\t.reg .pred q, t;\n\t.reg .b32 a, b;\n\t.reg .b64 db;\n\telect.sync _|q, 0xffffffff;\n\tsetp.eq.u32 t, 0, 0;\n\t"
      GDN_STEP("8", "128") GDN_STEP("16", "256") GDN_STEP("24", "384") GDN_STEP("32", "512") GDN_STEP("40", "640")
      GDN_STEP("48", "768") GDN_STEP("56", "896") "}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(kDescHi)
      : "memory");
#undef GDN_STEP
}

// The elected lane's arrival on `bar` once the products issued so far are done.
__device__ __forceinline__ void umma_commit_one(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
      : "memory");
}

// kind::f16 with A and B both f16 (F16) or bf16, f32 accumulator.
template <bool F16>
__device__ __forceinline__ uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 64 consecutive columns of this thread's tensor-memory lane, one load and one wait.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float* v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int q = 0; q < 64; ++q) v[q] = __uint_as_float(r[q]);
}

// 16 words to this thread's lane; tmem_st_wait() before anything relies on them.
__device__ __forceinline__ void tmem_st16_words(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 bytes (a sector) a thread.
__device__ __forceinline__ void store8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
               "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// A value that all lanes hold, in a form that the compiler knows to be the same in all of them (the
// tensor core's operands live in uniform registers).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint32_t uniform_from(uint32_t x, int lane) { return __shfl_sync(0xffffffffu, x, lane); }

// Maximum of 64 scores, in four chains of two values a step (NaN counts for nothing).
__device__ __forceinline__ float max64(const float (&x)[64]) {
  float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int j = 4; j < 60; j += 8)
#pragma unroll
    for (int q = 0; q < 4; ++q) m[q] = fmaxf(fmaxf(m[q], x[j + q]), x[j + 4 + q]);
#pragma unroll
  for (int q = 0; q < 4; ++q) m[q] = fmaxf(m[q], x[60 + q]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// 32 probabilities of this thread's row (16 words of tensor memory) times f, rounded to the type a second
// time: they belong to a tile's first half, whose second half holds a score whose weight is more than 2^kLag
// times the largest that the row knew of.
template <bool F16>
__device__ __forceinline__ void rescale_pairs(uint32_t taddr, float f) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 v = F16 ? __half22float2(*reinterpret_cast<const __half2*>(&r[j])) : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r[j]));
    r[j] = pack2<F16>(v.x * f, v.y * f);
  }
  tmem_st16_words(taddr, r);
}

// Tensor-memory columns: S of stream s (P over its first half once S has been read), then O.
constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t tmem_s(int s) { return 128u * uint32_t(s); }
__device__ __forceinline__ uint32_t tmem_o(int s) { return 256u + 128u * uint32_t(s); }

// A look at a barrier's phase, and one that sleeps until the phase is over, up to a time that the hardware sets (4 us; a
// time given with it wakes later: prompts of 4096..16384 tokens 3140 us with one, 3030 without).
__device__ __forceinline__ bool mbar_look(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_sleep(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The barriers of a CTA, behind its ring of tiles.
struct TileBars {
  uint64_t *full, *empty;               // [stages] a slot has landed; both streams are done with it
  uint64_t *q_ready, *s_ready, *p_ready, *o_done, *q_free;  // [2]
  uint64_t *seg_full, *seg_empty;       // [kSegRing]
};
template <int NS>
__device__ __forceinline__ TileBars tile_bars(uint64_t* bars) {
  uint64_t* const q = bars + 2 * NS;
  return TileBars{bars, bars + NS, q, q + 2, q + 4, q + 6, q + 8, q + 10, q + 10 + kSegRing};
}
template <int NS>
__device__ __forceinline__ void init_tile_bars(const TileBars& b, int tensor_warps) {  // one thread
  for (int i = 0; i < NS; ++i) {
    mbar_init(b.full + i, 1);
    mbar_init(b.empty + i, uint32_t(tensor_warps));  // an arrival each
  }
  for (int s = 0; s < 2; ++s) {
    mbar_init(b.q_ready + s, 1);
    mbar_init(b.q_free + s, 1);
    mbar_init(b.s_ready + s, 1);
    mbar_init(b.p_ready + s, kGroupThreads);
    mbar_init(b.o_done + s, 1);
  }
  for (int i = 0; i < kSegRing; ++i) {
    mbar_init(b.seg_full + i, 1);
    mbar_init(b.seg_empty + i, uint32_t(2 + tensor_warps + 2 * kGroupThreads / 32));  // every warp, the one that hands them on included
  }
}

// The tensor core's warp of stream s.
// A warp per stream, taking turns on the tiles they share: the O += P V of the stream's tile before
// and the S = Q K^T of its next go out in one go, 1024 cycles of the tensor core (16 products of
// 64), during which the other stream's softmax runs and the other warp does its waiting.  (Without
// turns the two streams' products interleave and take twice as long each; one warp for both leaves
// the tensor core idle while it waits.)  The whole warp walks the schedule, in uniform registers.
//
// Each of the two warps sees every tile land, in order, and releases each of its slots once - the
// stream that does not use a tile by a plain arrival.  A wait on a phase's parity is sound only
// within one phase of the barrier, and copies do not land in the order they were asked for:
// this way no slot can be filled again, or be a use behind, where either stream waits for it.
template <int D, bool F16, typename Seg, typename Wait>
__device__ __forceinline__ void tensor_warp(const int s, const int lane, const uint32_t tmem, const uint32_t base, const bool negative,
                                            const Seg* const segs, const TileBars& bars, volatile uint32_t* const turns, Wait wait_warp) {
  using L = TileLayout<D, Seg>;
  constexpr int NS = L::STAGES;
  uint64_t *const full = bars.full, *const empty = bars.empty, *const q_ready = bars.q_ready, *const s_ready = bars.s_ready,
           *const p_ready = bars.p_ready, *const o_done = bars.o_done, *const q_free = bars.q_free, *const seg_full = bars.seg_full,
           *const seg_empty = bars.seg_empty;
  const uint32_t tm = uniform(tmem), ts = tm + tmem_s(s), to = tm + tmem_o(s);
  const uint32_t q_desc = swizzled_desc_lo(base + L::OFF_Q + s * L::BYTES, 16);
  const uint32_t values_idesc = idesc_f16<F16>(kTileKeys, D) | (1u << 16);  // B (values) MN-major
  const uint32_t scores_idesc = negative ? 1u << 13 : 0u;              // a negative scale negates the queries
  uint32_t slot = 0, phase = 0;     // of a tile's keys; its values are in the slot behind
  uint32_t np = 0, nq = 0;          // P tiles, segments of this stream
  uint32_t theirs = 0, ours = 0;    // the other stream's turns ahead of this warp's next; this warp's
  // The tile whose O += P V is still to be issued.
  bool pending = false, p_first = false, p_last = false;
  uint32_t p_units = 0, p_slot = 0, p_phase = 0;
  bool ok = true;
  auto values = [&] {
    pending = false;
    tc_fence_after();
    const uint32_t db = swizzled_desc_lo(base + L::OFF_RING + p_slot * L::BYTES, L::HALF);
    umma_values_first(to, ts, db, values_idesc, p_first ? 0u : 1u);
    if (p_units == 8) {
      umma_values_rest(to, ts, db, values_idesc);
    } else {
#pragma unroll 1
      for (uint32_t u = 1; u < p_units; ++u) umma_values_first(to, ts + 8 * u, db + 128 * u, values_idesc, 1);
    }
    umma_commit_one(empty + p_slot);
    if (p_last) umma_commit_one(o_done + s);
  };
  for (uint32_t k = 0; ok; ++k) {
    const Seg& seg = segs[k % kSegRing];
    if (!wait_warp(seg_full + k % kSegRing, (k / kSegRing) & 1)) {
      ok = false;
      break;
    }
    const int t0 = int(uniform(uint32_t(seg.t0))), t1 = int(uniform(uint32_t(seg.t1)));
    const auto tiles = seg.tiles();
    const int parity = int(uniform(uint32_t(seg.parity)));
    const bool paired = uniform(seg.paired() ? 1u : 0u) != 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty + k % kSegRing);
    const bool end = t1 < 0;
    bool first = true;
#pragma unroll 1
    for (int t = t0; ok && (end || t < t1); ++t) {
      const uint32_t vslot = slot + 1 < NS ? slot + 1 : 0, vphase = slot + 1 < NS ? phase : phase ^ 1;
      const bool skip = !end && !paired && ((parity + t - t0) & 1) != s;  // the other stream's tile
      bool landed = false;
      // what has to be there before this warp's turn
      if (pending) {
        ok = wait_warp(full + p_slot, p_phase);
        landed = ok && !end && __all_sync(0xffffffffu, mbar_look(full + slot, phase) &&
                                                           (skip || !first || mbar_look(q_ready + s, nq & 1)));
        if (skip && landed && lane == 0) mbar_arrive(empty + slot);
        ok = ok && wait_warp(p_ready + s, np++ & 1);
      }
      if (skip) {
        // (tiles in alternation wait for memory: the values go at once, and their slot with them)
        if (ok && pending) values();
        ++theirs;
        if (!landed) {
          ok = ok && wait_warp(full + slot, phase);
          if (ok && lane == 0) mbar_arrive(empty + slot);
        }
        ok = ok && wait_warp(full + vslot, vphase);
        if (ok && lane == 0) mbar_arrive(empty + vslot);
        slot += 2, phase ^= slot >= NS ? 1u : 0u, slot -= slot >= NS ? NS : 0;
        continue;
      }
      if (!ok) break;
      if (paired && s == 1) ++theirs;
      // (turns are about time alone: nothing breaks should this look give up)
      for (uint32_t i = 0; paired && !end && i < kMaxTurnLooks && __any_sync(0xffffffffu, turns[s ^ 1] < theirs); ++i) {
      }
      if (pending) values();
      if (end) break;
      // S = Q K^T of this tile; a turn does not wait for keys that are late
      if (!landed) {
        if (lane == 0) turns[s] = ++ours;
        if (first) ok = wait_warp(q_ready + s, nq & 1);
        ok = ok && wait_warp(full + slot, phase);
        if (!ok) break;
      }
      tc_fence_after();
      const uint32_t units = uint32_t(tiles.units(t));
      const bool last = paired ? t == t1 - 1 : t1 - t <= 2;
      umma_scores<D>(ts, q_desc, swizzled_desc_lo(base + L::OFF_RING + slot * L::BYTES, 16),
                     idesc_f16<F16>(kTileKeys, int(16 * units)) | scores_idesc);
      if (landed && lane == 0) turns[s] = ++ours;
      umma_commit_one(s_ready + s);
      umma_commit_one(empty + slot);
      if (last) umma_commit_one(q_free + s);
      if (paired && s == 0) ++theirs;
      if (first) ++nq;
      pending = true, p_units = units, p_first = first, p_last = last, p_slot = vslot, p_phase = vphase;
      first = false;
      slot += 2, phase ^= slot >= NS ? 1u : 0u, slot -= slot >= NS ? NS : 0;
    }
    if (end) break;
  }
  if (!ok) {  // what is under way finishes before tensor memory is freed
    umma_commit_one(o_done + s);
    mbar_drain(o_done + s, 0);
    mbar_drain(o_done + s, 1);
  }
}

// A row's softmax over a tile: scores in tensor memory to probabilities there, with its running maximum m (unscaled)
// and sum l.  seen(q, g) is the mask of the keys from 64 q + 32 g on that the row sees, 32 of them, asked for where
// the tile is `masked`; a row that is not `live` never moves its maximum.
// settle() returns once O holds the tiles before.
template <int D, bool F16, typename Seen, typename Settle>
__device__ __forceinline__ void softmax_tile(const uint32_t ts, const uint32_t to, const float c, const bool live, const bool first,
                                             const bool masked, Seen seen, Settle settle, float& m, float& l) {
  // 64 scores at a time, in a loop (all 128 unrolled hold up the other warps' instruction fetches, 32
  // at a time wait longer for their loads).  The exponentials take the maximum that is known; only if
  // a row's next 64 lie more than kLag above it are O, its sum and the tile's P so far rescaled.
  // P goes over scores that have been read, rounded to the type of V: the product takes both of one 16-bit type, and a second
  // product for what the rounding drops would make its part of the tensor core's time twice as long.  Each weight is off
  // by half a step at most, the sum l is of the f32 weights: against float64 2.2e-3 of the output's norm in bf16 and 2.9e-4 in f16,
  // of which rounding the output alone is 1.7e-3 and 2.1e-4.
  float2 sum = make_float2(0.f, 0.f);
  const float2 c2 = make_float2(c, c);
#pragma unroll 1
  for (int q = 0; q < 2; ++q) {
    float x[64];
    tmem_ld64(ts + 64 * q, x);
    if (masked) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t see = seen(q, g);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[32 * g + j] = (see >> j) & 1u ? x[32 * g + j] : -INFINITY;
      }
    }
    const float mx = max64(x);
    const bool move = mx > m && !((mx - m) * c <= kLag) && live;  // (m = -inf: infinitely far)
    if (__any_sync(0xffffffffu, move)) {
      const float f = move ? exp2_fast((m - mx) * c) : 1.f;
      if (!first) {
        settle();
#pragma unroll 1
        for (int k2 = 0; k2 < D; k2 += 32) {
          float o[32];
          tmem_ld32(to + k2, o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] *= f;
          tmem_st32(to + k2, o);
        }
      }
      tmem_st_wait();
#pragma unroll 1
      for (int k2 = 0; k2 < 2 * q; ++k2) rescale_pairs<F16>(ts + 16 * k2, f);
      sum.x *= f, sum.y *= f, l *= f;
      if (move) m = mx;
    }
    const float mc = m == -INFINITY ? 0.f : m * c;
    const float2 mc2 = make_float2(-mc, -mc);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t pk[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 e = fma2(make_float2(x[32 * g + 2 * j], x[32 * g + 2 * j + 1]), c2, mc2);
        const float2 w2 = make_float2(exp2_fast(e.x), exp2_fast(e.y));
        sum = add2(sum, w2);
        pk[j] = pack2<F16>(w2.x, w2.y);
      }
      tmem_st16_words(ts + 32 * q + 16 * g, pk);
    }
  }
  l += sum.x + sum.y;
  tmem_st_wait();
}

// ---------------------------------------------------------------- launches
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (the library does not link against libcuda).
inline EncodeTiled encoder() {
  static const EncodeTiled f = [] {
    void* sym = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      sym = nullptr;
    return reinterpret_cast<EncodeTiled>(sym);
  }();
  return f;
}

}  // namespace gdn
