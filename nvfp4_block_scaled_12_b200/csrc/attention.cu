// Attention of a sequence over states of another length:
//     O = softmax(scale * Q K^T) V     over the first kv_lens[b] states
// on the sm_100a tensor cores, one pass over K and V with the running maximum
// and sum of the softmax.
//
// A work item is one K/V head of one batch entry and two tiles of up to 128
// query rows (slots 0 and 1) that share its K and V stream.  Query heads that
// share a K/V head are rows of one tile: row r is token r / group, head
// r % group, so K and V are read once per group.  Per 128-key tile and slot
//     S  = Q K^T       128 x 128 x DP  tcgen05.mma, Q and K from shared memory
//     P  = exp2(c S - c m)             softmax warps, S from and P to TMEM
//     O += P V         128 x DP x 128  tcgen05.mma, P from TMEM, V from shared
//                                      memory as a transposed operand
// with c = scale log2 e.
//
// TMEM: S | P0 | P1 | O0 | O1, 128 + 64 + 64 + 128 + 128 columns.  The two slots
// share one S: a softmax warp reads its row's scores into registers at once and
// hands S back, so the other slot's scores, and then its own next ones, are
// made while it works on these, and neither product is on its way from one
// tile to the next.  (With an S of its own per slot, P over it, a slot waited
// for both products every tile: 231 us for joint attention of 4608 tokens and
// 24 heads of 128, against 205 us.)
//
// Warps (12): 0-3 softmax of slot 0 (one row a thread), 4-7 of slot 1, 8 issues
// the scores' MMAs, 10 the products', 9 is the TMA producer (11 fills up their
// warpgroup, whose registers go to the softmax threads: a row's 128 scores stay
// in registers).  One issuer for both spent longer on its waits and commits
// than the tensor cores on its MMAs (249 us).  Shared memory: both Q tiles, a
// ring of K and V tiles, and a panel of O per slot on its way out.
//
// The reference m of a row is its first tile's maximum and moves only when a
// later tile's sum of P exceeds 2^15 (fp16 holds that, and a relative accuracy
// is all that matters below): then the tile is made again with its own maximum,
// and O is rescaled in TMEM.
// So only the first tile's maxima are ever taken; P of the others is made at
// once, and the sum, which is needed anyway, is the check.  S, the maximum, the
// sum and O are fp32; P is rounded to the type of V for the tensor cores (the
// sum takes it unrounded, so a row's error from this averages out over its keys).
//
// States from kv_lens[b] on contribute nothing whatever they hold: their
// scores are replaced, not added to, and in the last tile the V rows that the
// MMA reads beyond them (up to the next multiple of 16 keys) are zeroed in
// shared memory, since 0 * NaN is NaN.  Keys past the tensor arrive as zeros.
//
// What bounds it: the tensor cores' floor is 2048 clocks a step (two slots, two
// products), the exponentials' 2048 (16 a clock and SM); a step takes 3300.  The
// softmax warps are busy for 2560 to 2930 of them: those that share a scheduler
// with an MMA issuer are the slow ones.  Joint attention of 4608 tokens, 24 heads
// of 128: 200 to 205 us back to back = 1.27 to 1.31 PFLOP/s (0.79 of the measured
// bf16 burst; under the power cap 236); heads of 64: 179 us (113 are the exponentials' floor);
// 4096 queries over 512 and 382 states, 24 heads of 128: 57 us.  There a step takes
// 1.7 us and an item's two ends, which nothing covers, 2.3; and the 768 items in
// turns of 148 leave 28 CTAs a sixth one, 21 key tiles in all against 17 or 18: by
// these figures 49.5 us for the longest CTA and 42.8 for the average one, so about
// 7 us pass with four fifths of the SMs done.
// Measured and not kept: a share of the exponentials as a cubic on the FMA pipes
// (no gain at any share), two threads a row (a vote a tile: the same speed), an
// output warpgroup of its own (206 us), P handed over in halves.
//
// With fewer items than SMs the keys are split over the CTAs of a cluster, and
// where all queries of a K/V head fit one tile the two slots take its key tiles
// in turn: each part keeps its own m, sum and O, and they are joined through
// distributed shared memory in a fixed order (no workspace, no atomics, and the
// same result every time).
//
// Where, besides, those queries are at most 32 rows (kFew: one token, or a few),
// most of a tile would be rows of nothing, their exponentials the longest part
// of a step, and all the real ones on one warp of each slot.  Then the Q tile
// holds the rows four times, once per 32 lanes, and each warp of a slot takes
// the scores of 32 of the tile's 128 keys for its copy: P of the other keys
// stays zero, and every copy is a part of its own, with its own m, sum and O,
// joined within the CTA before the ranks join (a row that an infinite V turned
// into NaN that way is made once more, few_rows_again).  A tile then costs its two
// products, 0.57 us, instead of 1.05, and the ring has six stages for four.  One
// query over 16384, 14334, 12284 and 10239 states, 32 heads on 8 of 128: 41.5 us
// (218 MB: 5.3 TB/s); what is left is that the longest entry's CTAs end last (2 to 3
// us) and 6 us of start, join and end.  32 entries of 4096 states each: 84.7 us =
// 6.3 TB/s, 0.97 of a copy; short items pay their start and join (64 entries of 1024
// states, 16 heads of 64: 3.2 TB/s).  33 to 64 rows could have two copies; they have
// none.
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kAttMaxSplit = 8;  // the portable cluster size
constexpr int kAttTile = 128;  // query rows of a slot, keys of a tile
constexpr int kAttThreads = 384;  // three warpgroups: softmax of each slot, producer and MMA
constexpr uint32_t kPanelBytes = 128 * 128;  // 128 rows of 64 elements, 128-byte swizzle

// kDP: head width rounded up to 64 or 128 (the tensor maps zero-fill the rest).
// kFew: all queries of a K/V head are at most 32 rows (see the top).
template <int kDP, bool kFew>
struct ACfg {
  static constexpr int kPanels = kDP / 64;
  static constexpr uint32_t kTileBytes = kPanels * kPanelBytes;
  // (one Q tile and no panel of O on its way out leave the ring 64 KB more)
  static constexpr int kQTiles = kFew ? 1 : 2;
  static constexpr int kStages = kDP == 128 ? (kFew ? 6 : 4) : (kFew ? 11 : 8);
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffKv = kQTiles * kTileBytes;
  static constexpr uint32_t kOffOut = kOffKv + kStages * kTileBytes;  // a panel of O on its way out, per slot
  static constexpr uint32_t kOffBar = kOffOut + (kFew ? 0 : 2 * kPanelBytes);
  // kv_full, kv_empty per stage; q_full, q_empty, s_full, p_ready, pv_done, o_free,
  // o_written, drain per slot; s_free
  static constexpr uint32_t kNumBars = 2 * kStages + 16 + 1;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;  // + alignment slack
  // K/V split: a slot's fp32 partial rows (padded to spread them over the
  // banks) and its maxima and sums, in the idle ring and what follows it
  static constexpr uint32_t kPartStride = (kDP + 4) * 4;
  static constexpr uint32_t kPartSlot = 128 * kPartStride;
  static constexpr uint32_t kPartMl = 2 * kPartSlot;  // float2 (m, l) [2][128]
  static constexpr uint32_t kPartMlCta = kPartMl + 2 * 128 * 8;  // kFew: the CTA's (m, l) of a row [32]
  static_assert(kOffKv + kPartMlCta + 32 * 8 <= kOffBar, "the partial results fit");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(kSmemBytes > 233472 / 2, "one CTA per SM (all 512 TMEM columns are its own)");
};

// TMEM columns: one S for both slots, P and O of each.
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256;
constexpr uint32_t kSlotP = 64, kSlotO = 128;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed pairs of floats (the low half first) and their arithmetic.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Two values to the operand type, the first in the low half.
template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (kFp16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// kind::f16 instruction descriptor, M = 128: fp32 accumulator, A K-major, B
// K-major or (b_mn) with its N dimension contiguous.
template <bool kFp16>
__host__ __device__ constexpr uint32_t idesc_16(int n, bool b_mn) {
  return (1u << 4) | ((kFp16 ? 0u : 1u) << 7) | ((kFp16 ? 0u : 1u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// Shared-memory descriptor of a transposed operand: rows of 64 elements along
// N (128-byte swizzle), one per K; 8 rows are 1024 bytes apart, the next 64 of
// N a panel further.
__device__ __forceinline__ uint64_t sdesc_nmajor_sw128(uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kPanelBytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// The MMA warps run their loops as a whole and one elected lane (always the
// same) issues: the operands are then warp-uniform values in uniform registers.
// With the loop under `if (lane == 0)` every MMA moved its operands over first,
// and issuing them took longer than running them.

// D (TMEM) (+)= A (shared memory) * B (shared memory), 16-bit operands
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D (TMEM) (+)= A (TMEM, 16-bit pairs) * B (shared memory)
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* m, const void* src, int32_t x, int32_t y, int32_t z,
                                             int32_t w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Where a step's K and V and the next K are in a ring of S tiles that holds
// K, V, K, V, ..
template <int S>
struct RingPos {
  int stage = 0;  // this step's K
  uint32_t phase = 0u;
  __device__ __forceinline__ int v_stage() const { return stage + 1 < S ? stage + 1 : stage + 1 - S; }
  __device__ __forceinline__ uint32_t v_phase() const { return stage + 1 < S ? phase : phase ^ 1u; }
  __device__ __forceinline__ int k_stage() const { return stage + 2 < S ? stage + 2 : stage + 2 - S; }
  __device__ __forceinline__ uint32_t k_phase() const { return stage + 2 < S ? phase : phase ^ 1u; }
  __device__ __forceinline__ void next_step() {
    phase = k_phase();
    stage = k_stage();
  }
};

// Two 16-bit elements of a word, the low half first.
template <bool kFp16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (kFp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(bf16_lo(w), bf16_hi(w));
}

// One work item as every role sees it.
struct AttItem {
  int b, hk, tile0;    // batch entry, K/V head, first query tile
  int slots;           // 1 or 2 query tiles
  bool shared;         // both slots share the one tile and take its key tiles in turn
  int len;             // valid states of the batch entry
  int kt0, n;          // first key tile and key tiles of this CTA
};

__device__ __forceinline__ AttItem att_item(const AttentionParams& p, int item, int rank) {
  AttItem w;
  const int pair = item % p.pairs;
  const int bh = item / p.pairs;
  w.hk = bh % p.kv_heads;
  w.b = bh / p.kv_heads;
  w.tile0 = 2 * pair;
  w.slots = min(2, p.q_tiles - w.tile0);
  w.shared = p.join != 0 && p.q_tiles == 1;
  w.len = p.kv_lens != nullptr ? min(max(ld_after_wait(p.kv_lens + w.b), 0), p.kv_tokens) : p.kv_tokens;
  const unsigned tiles = (static_cast<unsigned>(w.len) + kAttTile - 1) / kAttTile;  // (at most 2^23)
  w.kt0 = 0;
  w.n = static_cast<int>(tiles);
  if (p.split > 1) {
    w.kt0 = static_cast<int>(tiles * rank / p.split);
    w.n = static_cast<int>(tiles * (rank + 1) / p.split) - w.kt0;
  }
  return w;
}

// kFew: rows of the CTA's joined parts (a bit each) once more where they hold NaN
// though their scores are numbers.  A copy of a row multiplies all keys of a tile,
// with probabilities of zero for the other copies' keys, and 0 * inf is NaN: for
// an infinite V that is the form's doing and not the definition's.  So the eight
// softmax warps take the CTA's keys in turn, each key with its own probability
// alone, and the columns that were NaN get their sum, in a fixed order: inf, or
// NaN where the definition has it too.  A way off the tensor cores: one query of
// 32 heads on 8 over 16384 states, four entries, takes 0.48 ms with an infinity in
// one state and 0.65 with one in every state, for 0.042.  Rows without an infinite
// or undefined V never come here; a function of its own, out of the way and with
// nothing of the kernel's passed in memory, costs them 0.3 us (inlined 0.7, with
// the item by reference 1.5).
template <int kDP, bool kFp16, typename C>
__device__ __noinline__ void few_rows_again(const AttentionParams& p, int item, int rank, unsigned rows, uint8_t* part) {
  constexpr int kWords = kDP / 64;  // of two elements: a lane's share of a row of V
  const AttItem w = att_item(p, item, rank);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int col = lane * 2 * kWords;
  const uint16_t* k = static_cast<const uint16_t*>(p.k) + w.b * p.k_batch + w.hk * p.k_head;
  const uint16_t* v = static_cast<const uint16_t*>(p.v) + w.b * p.v_batch + w.hk * p.v_head + col;
  const int end = min(w.len, (w.kt0 + w.n) * kAttTile);
  for (; rows != 0u; rows &= rows - 1u) {
    const int row = __ffs(static_cast<int>(rows)) - 1;
    const float mc = reinterpret_cast<const float2*>(part + C::kPartMlCta)[row].x * p.scale_log2;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + w.b * p.q_batch + (row / p.group) * p.q_token +
                        (w.hk * p.group + row % p.group) * p.q_head;
    float2 sum[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) sum[i] = make_float2(0.0f, 0.0f);
    // 32 keys a turn: a lane's own key's score, then the keys' V one after another
    for (int key0 = w.kt0 * kAttTile + warp * 32; key0 < end; key0 += 8 * 32) {
      float e = 0.0f;
      if (key0 + lane < end) {
        float s = 0.0f;
#pragma unroll 4
        for (int d = 0; d < p.D; d += 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(k + (key0 + lane) * p.k_token + d);
          const uint4 y = *reinterpret_cast<const uint4*>(q + d);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = unpack2<kFp16>(xw[i]), b = unpack2<kFp16>(yw[i]);
            s = fmaf(a.x, b.x, fmaf(a.y, b.y, s));
          }
        }
        e = exp2_approx(fmaf(s, p.scale_log2, -mc));
      }
      __syncwarp();
      const int n = min(32, end - key0);
#pragma unroll 8
      for (int t = 0; t < n; ++t) {
        const float et = __shfl_sync(0xffffffffu, e, t);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          float2 x = make_float2(0.0f, 0.0f);
          if (col < p.D) x = unpack2<kFp16>(reinterpret_cast<const uint32_t*>(v + (key0 + t) * p.v_token)[i]);
          sum[i].x = fmaf(et, x.x, sum[i].x);
          sum[i].y = fmaf(et, x.y, sum[i].y);
        }
      }
    }
    // (the joined row took the first part's place; the seven others of the row are read no more)
    auto part_of = [&](int t) { return reinterpret_cast<float2*>(part + (t * 32 + row) * C::kPartStride + col * 4); };
    if (warp > 0) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) part_of(warp)[i] = sum[i];
    }
    named_barrier_sync(2, 256);
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        float2 x = part_of(0)[i];
        for (int t = 1; t < 8; ++t) {
          sum[i].x += part_of(t)[i].x;
          sum[i].y += part_of(t)[i].y;
        }
        x.x = isnan(x.x) ? sum[i].x : x.x;
        x.y = isnan(x.y) ? sum[i].y : x.y;
        part_of(0)[i] = x;
      }
    }
  }
}

template <int kDP, bool kFp16, bool kFew>
__global__ void __launch_bounds__(kAttThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_o,
                     const __grid_constant__ AttentionParams p) {
  using C = ACfg<kDP, kFew>;
  constexpr float kMostSum = 0x1p15f;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* kv_empty = kv_full + S;
  uint64_t* q_full = kv_empty + S;  // and below: one per slot
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_ready = s_full + 2;
  uint64_t* pv_done = p_ready + 2;
  uint64_t* o_free = pv_done + 2;
  uint64_t* o_written = o_free + 2;
  uint64_t* drain = o_written + 2;
  uint64_t* s_free = drain + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  unsigned* again = reinterpret_cast<unsigned*>(smem + C::kOffMisc + 8);  // kFew: rows to make once more, a bit each
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = blockIdx.x / p.split;
  const int step = gridDim.x / p.split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);  // the slot's four softmax warps
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_free[i], 1);
      mbar_init(&o_written[i], 4);  // the slot's four softmax warps
      mbar_init(&drain[i], 1);
    }
    mbar_init(s_free, 4);  // the four softmax warps that read S
    *abort_flag = 0;
    *again = 0u;
    fence_mbar_init();
  }
  // rows of the Q tiles that no query fills (a group that does not divide 128;
  // kFew: of each of the tile's four copies of up to 32 rows)
  constexpr int kCopyRows = kFew ? 32 : 128;
  const int spare = (kCopyRows - p.tile_rows) * 8;  // 16-byte chunks of a copy's panel
  for (int t = threadIdx.x; t < C::kQTiles * C::kPanels * (128 / kCopyRows) * spare; t += kAttThreads) {
    const int copy = t / spare, at = t - copy * spare;
    *reinterpret_cast<uint4*>(smem + C::kOffQ + copy * (kCopyRows * 128) + p.tile_rows * 128 + at * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_async_smem();
  if (warp == 9 && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
    prefetch_tmap(&tmap_o);
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  unsigned fault = 0u;
  // The kernel is launched before the one in front of it has ended, and lets the
  // next one be: nothing up to here touched global memory.  (Call after call,
  // 4096 queries over 512 states 59.5 -> 57.1 us, one over 16384 46.5 -> 43.4.)
  launch_dependents();
  wait_for_previous_kernel();

  // every thread of the item's CTAs
  auto sync_cluster = [&]() {
    if (p.split > 1)
      cluster_sync();
    else
      named_barrier_sync(1, kAttThreads);
  };
  if (warp >= 8) {
    // (launched with 384 x 168 registers: 88 + 2 x 208 = 3 x 168)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
  }
  if (warp == 9) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      constexpr int kCopies = 128 / kCopyRows;
      const uint32_t q_bytes = C::kPanels * kCopies * static_cast<uint32_t>(p.tile_rows) * 128u;
      int64_t e = 0;             // ring entries issued
      uint32_t q_phase[2] = {0u, 0u};  // items whose tile went into the slot, mod 2
      bool q_used[2] = {false, false};
      auto load_q = [&](const AttItem& w, int i) {
        if (!mbar_wait(&q_empty[i], q_phase[i] ^ 1u, abort_flag)) return false;
        mbar_arrive_expect_tx(&q_full[i], q_bytes);
        for (int c = 0; c < C::kPanels * kCopies; ++c)
          tma_load_4d(smem + C::kOffQ + i * C::kTileBytes + c * (kCopyRows * 128), &tmap_q, &q_full[i],
                      (c / kCopies) * 64, w.hk * p.group, (w.tile0 + i) * p.tile_tokens, w.b * p.q_bmul);
        q_phase[i] ^= 1u;
        q_used[i] = true;
        return true;
      };
      auto load_kv = [&](const AttItem& w, const CUtensorMap* map, int kt, int bmul) {
        const int s = static_cast<int>(e % S);
        if (!mbar_wait(&kv_empty[s], (static_cast<uint32_t>(e / S) & 1u) ^ 1u, abort_flag)) return false;
        mbar_arrive_expect_tx(&kv_full[s], C::kTileBytes);
        for (int c = 0; c < C::kPanels; ++c)
          tma_load_4d(smem + C::kOffKv + s * C::kTileBytes + c * kPanelBytes, map, &kv_full[s], c * 64, w.hk,
                      kt * kAttTile, w.b * bmul);
        ++e;
        return true;
      };
      for (int item = first; item < p.items && fault == 0u; item += step) {
        const AttItem w = att_item(p, item, rank);
        for (int j = 0; j < w.n; ++j) {
          bool ok = j != 0 || load_q(w, 0);
          ok = ok && load_kv(w, &tmap_k, w.kt0 + j, p.k_bmul);
          if (j == 0 && w.slots == 2) ok = ok && load_q(w, 1);
          ok = ok && load_kv(w, &tmap_v, w.kt0 + j, p.v_bmul);
          if (!ok) {
            fault = kFaultProducerWait;
            break;
          }
        }
      }
      if (fault != 0u) *abort_flag = 1;
      // every copy issued has landed before the CTA may exit (in a normal run
      // the consumers have seen them all and these waits return at once)
      for (int64_t i = e - 1; i >= 0 && i >= e - S; --i)
        mbar_wait(&kv_full[i % S], static_cast<uint32_t>(i / S) & 1u, nullptr);
      for (int i = 0; i < 2; ++i)
        if (q_used[i]) mbar_wait(&q_full[i], q_phase[i] ^ 1u, nullptr);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ scores: S = Q_i K
    constexpr uint32_t idesc = idesc_16<kFp16>(kAttTile, false);
    RingPos<S> ring;  // of the present step's K
    uint32_t q_phase[2] = {0u, 0u}, s_phase = 1u;  // (nobody has S at the start)
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // of the whole warp
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      const bool ok = mbar_wait(bar, parity, abort_flag);
      return __all_sync(0xffffffffu, ok) != 0;
    };
    for (int item = first; item < p.items && fault == 0u; item += step) {
      const AttItem w = att_item(p, item, rank);
      for (int j = 0; j < w.n && fault == 0u; ++j, ring.next_step()) {
        const uint64_t kd = sdesc_kmajor_sw128(smem_u32(smem + C::kOffKv + ring.stage * C::kTileBytes));
        bool ok = wait(&kv_full[ring.stage], ring.phase);
        const int i0 = w.shared ? (j & 1) : 0, i1 = w.shared ? i0 + 1 : w.slots;
        for (int i = i0; i < i1 && ok; ++i) {
          const int qi = w.shared ? 0 : i;
          if (j == 0) {
            ok = wait(&q_full[qi], q_phase[qi]);
            q_phase[qi] ^= 1u;
          }
          ok = ok && wait(s_free, s_phase);  // the last S, the other slot's, has been read
          s_phase ^= 1u;
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = sdesc_kmajor_sw128(smem_u32(smem + C::kOffQ + qi * C::kTileBytes));
#pragma unroll
          for (int k = 0; k < kDP / 16; ++k) {
            const uint64_t off = static_cast<uint64_t>((k / 4) * (kPanelBytes >> 4) + (k % 4) * 2);
            mma_ss(tmem + kColS, qd + off, kd + off, idesc, k != 0 ? 1u : 0u);
          }
          tc_commit(&s_full[i]);
          if (j == w.n - 1) tc_commit(&q_empty[qi]);
          if (i == i1 - 1) tc_commit(&kv_empty[ring.stage]);
        }
        if (!ok) fault = kFaultMmaWait;
      }
    }
    if (fault != 0u) *abort_flag = 1;
    // every tcgen05 operation issued must complete before TMEM is released
    tc_commit(&drain[0]);
    if (!mbar_wait(&drain[0], 0u, nullptr)) fault |= kFaultDrainWait;
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ products: O_i (+)= P_i V
    constexpr uint32_t idesc = idesc_16<kFp16>(kDP, true);
    RingPos<S> ring;
    uint32_t p_phase[2] = {0u, 0u};
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      const bool ok = mbar_wait(bar, parity, abort_flag);
      return __all_sync(0xffffffffu, ok) != 0;
    };
    for (int item = first; item < p.items && fault == 0u; item += step) {
      const AttItem w = att_item(p, item, rank);
      for (int j = 0; j < w.n && fault == 0u; ++j, ring.next_step()) {
        const uint64_t vd = sdesc_nmajor_sw128(smem_u32(smem + C::kOffKv + ring.v_stage() * C::kTileBytes));
        const int k16 = min(kAttTile, w.len - (w.kt0 + j) * kAttTile + 15) / 16;  // 16-key steps with a valid key
        bool ok = wait(&kv_full[ring.v_stage()], ring.v_phase());
        const int i0 = w.shared ? (j & 1) : 0, i1 = w.shared ? i0 + 1 : w.slots;
        const bool adds = w.shared ? j > 1 : j > 0;  // not the slot's first product
        for (int i = i0; i < i1 && ok; ++i) {
          ok = wait(&p_ready[i], p_phase[i]);
          p_phase[i] ^= 1u;
          if (!ok) break;
          tc_fence_after();
          const uint32_t o = tmem + kColO + i * kSlotO, a = tmem + kColP + i * kSlotP;
          if (k16 == 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) mma_ts(o, a + k * 8, vd + k * (2048 >> 4), idesc, (adds || k != 0) ? 1u : 0u);
          } else {
            for (int k = 0; k < k16; ++k) mma_ts(o, a + k * 8, vd + k * (2048 >> 4), idesc, (adds || k != 0) ? 1u : 0u);
          }
          tc_commit(&pv_done[i]);
          if (i == i1 - 1) tc_commit(&kv_empty[ring.v_stage()]);
        }
        if (!ok) fault = kFaultMmaWait;
      }
    }
    if (fault != 0u) *abort_flag = 1;
    tc_commit(&drain[1]);
    if (!mbar_wait(&drain[1], 0u, nullptr)) fault |= kFaultDrainWait;
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
    // the row's reference and sum
    float m_ref = -INFINITY, l_sum = 0.0f;
    bool have = false;  // this thread's slot has a partial result in TMEM
    const int i = warp >> 2;  // slot
    const int row = (warp & 3) * 32 + lane;
    const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + kColS + t_lane, t_p = tmem + kColP + i * kSlotP + t_lane;
    const uint32_t t_o = tmem + kColO + i * kSlotO + t_lane;
    const float c = p.scale_log2;
    // this warp's keys of a tile (kFew: its copy of the rows takes a quarter)
    constexpr int kKeys = kFew ? 32 : 128;
    constexpr int kHalf = kFew ? 32 : 64;  // keys whose P is made at a time
    const int key0 = kFew ? (warp & 3) * 32 : 0;
    if constexpr (kFew) {  // P of the others' keys stays zero
      const uint32_t zero[16] = {};
#pragma unroll
      for (int k = 0; k < 64; k += 16) tmem_st_32x32b_x16(t_p + k, zero);
      tmem_st_wait();
    }
    uint32_t s_phase = 0u, pv_phase = 0u, o_phase = 0u;
    RingPos<S> ring;  // of this step's K
    auto all_lanes = [&](bool ok) {
      __syncwarp();
      return __all_sync(0xffffffffu, ok) != 0;
    };
    // a barrier wait of the whole warp (its first try by itself, as cheap as can be)
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      return all_lanes(mbar_wait(bar, parity, abort_flag));
    };
    for (int item = first; item < p.items && fault == 0u; item += step) {
      const AttItem w = att_item(p, item, rank);
      if (i >= w.slots && !w.shared) {
        for (int j = 0; j < w.n; ++j) ring.next_step();
        continue;
      }
      const int j0 = w.shared ? i : 0;  // this slot's first key tile
      m_ref = -INFINITY;
      l_sum = 0.0f;
      have = w.n > j0;
      for (int j = 0; j < w.n; ++j, ring.next_step()) {
        if (w.shared && (j & 1) != i) continue;
        const int valid = w.len - (w.kt0 + j) * kAttTile;  // keys of this tile (more than 128: all)
        if (!wait_all(&s_full[i], s_phase)) {
          fault = kFaultEpilogueWait;
          break;
        }
        s_phase ^= 1u;
        tc_fence_after();
        uint32_t r[kKeys];
        if constexpr (kFew) {
          tmem_ld_32x32b_x32(t_s + key0, r);
          tmem_ld_wait(r);
        } else {
          tmem_ld_32x32b_x64(t_s, r);
          tmem_ld_32x32b_x64(t_s + 64, r + 64);
          tmem_ld_wait_n<128>(r);
        }
        // S is in registers: the next scores, the other slot's, may come
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
        if (valid < kAttTile) {
#pragma unroll
          for (int k = 0; k < kKeys; ++k)
            if (key0 + k >= valid) r[k] = 0xFF800000u;  // -inf
          if ((i == 0 || w.shared) && (valid & 15) != 0) {
            // the V rows from the last valid state to the next multiple of 16
            // keys: zero, whatever they hold (0 * NaN would not be)
            if (!wait_all(&kv_full[ring.v_stage()], ring.v_phase())) {
              fault = kFaultEpilogueWait;
              break;
            }
            uint8_t* v = smem + C::kOffKv + ring.v_stage() * C::kTileBytes;
            const int chunks = (16 - (valid & 15)) * 8;  // 16-byte chunks of a panel's rows
            for (int t = row; t < chunks * C::kPanels; t += 128) {
              const int panel = t / chunks, at = t - panel * chunks;
              *reinterpret_cast<uint4*>(v + panel * kPanelBytes + valid * 128 + at * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
          }
        }
        auto row_max = [&]() {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < kKeys; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(r[k]));
          const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // A score that its scale takes out of fp32's range counts as that infinity:
          // -inf has a probability of zero, +inf makes the row NaN (with -c m infinite
          // every exponent would be, and P zero or infinite for finite scores)
          const float x = m * c;
          return fabsf(x) == INFINITY ? (x < 0.0f ? x : NAN) : m;
        };
        // P of the keys from kHalf h on with the present reference, two to a word
        uint32_t pk[kHalf / 2];
        auto make_p = [&](int h, float m) {
          const uint64_t c2 = f2_pack(c, c), mc2 = f2_pack(-m * c, -m * c);
          uint64_t sum[2] = {0u, 0u};
#pragma unroll
          for (int k = 0; k < kHalf / 2; ++k) {
            const uint64_t x =
                f2_fma(f2_pack(__uint_as_float(r[kHalf * h + 2 * k]), __uint_as_float(r[kHalf * h + 2 * k + 1])), c2, mc2);
            float a, b;
            f2_unpack(x, a, b);
            a = exp2_approx(a);
            b = exp2_approx(b);
            sum[k & 1] = f2_add(sum[k & 1], f2_pack(a, b));
            pk[k] = pack2<kFp16>(a, b);
          }
          float a, b;
          f2_unpack(f2_add(sum[0], sum[1]), a, b);
          return a + b;
        };
        auto store_p = [&](int h) {
#pragma unroll
          for (int k = 0; k < kHalf / 2; k += 16)
            tmem_st_32x32b_x16(t_p + key0 / 2 + (kHalf / 2) * h + k, *reinterpret_cast<const uint32_t(*)[16]>(pk + k));
        };
        // (a row without a finite score so far takes its next tile's maximum)
        if (j == j0 || m_ref == -INFINITY) m_ref = row_max();
        const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
        float tile_sum = make_p(0, m_use);
        if (j > j0) {
          // the last tile's product has read P (and O is complete up to it)
          if (!wait_all(&pv_done[i], pv_phase)) {
            fault = kFaultEpilogueWait;
            break;
          }
          pv_phase ^= 1u;
          tc_fence_after();
        }
        store_p(0);
        if constexpr (!kFew) tile_sum += make_p(1, m_use);
        if (j > j0) {
          const bool moves = tile_sum > kMostSum;
          if (__any_sync(0xffffffffu, moves)) {
            // rare: the tile's maximum becomes the reference, O and the sum so
            // far are scaled down to it, and P is made again
            const float m_new = moves ? row_max() : m_use;
            const float f = moves ? exp2_approx((m_use - m_new) * c) : 1.0f;
            if (moves) m_ref = m_new;
            l_sum *= f;
#pragma unroll 1
            for (int d = 0; d < kDP; d += 16) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(t_o + d, o);
              tmem_ld_wait_n<16>(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st_32x32b_x16(t_o + d, o);
            }
            tmem_st_wait();
            tile_sum = make_p(0, m_new);
            store_p(0);
            if constexpr (!kFew) tile_sum += make_p(1, m_new);
          }
        }
        if constexpr (!kFew) store_p(1);
        l_sum += tile_sum;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[i]);
      }
      if (fault != 0u) break;
      if (have) {
        if (!wait_all(&pv_done[i], pv_phase)) {
          fault = kFaultEpilogueWait;
          break;
        }
        pv_phase ^= 1u;
        tc_fence_after();
      }
      if (kFew || p.join) break;  // one item; joined below
      // ---- O / sum through shared memory, 64 columns at a time, to the output
      // (zeros where there are no states).  One row a thread straight to global
      // memory took 4200 clocks a tile: every store touched 32 lines.
      const float inv = have && l_sum != 0.0f ? 1.0f / l_sum : 0.0f;
      uint8_t* panel = smem + C::kOffOut + i * kPanelBytes;
#pragma unroll 1
      for (int d = 0; d < p.D; d += 64) {
        // (barriers with bounded waits between the slot's warps: after a
        // fault one of them may be gone)
        if (row == 0) {
          bulk_wait_read<0>();  // the last panel has left
          mbar_arrive(&o_free[i]);
        }
        if (!wait_all(&o_free[i], o_phase)) {
          fault = kFaultEpilogueWait;
          break;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[32];
          if (have) {
            tmem_ld_32x32b_x32(t_o + d + 32 * h, o);
            tmem_ld_wait(o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = pack2<kFp16>(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(panel + row * 128 + (((4 * h + k) ^ (row & 7)) * 16)) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_written[i]);
        if ((warp & 3) == 0) {
          if (!wait_all(&o_written[i], o_phase)) {
            fault = kFaultEpilogueWait;
            break;
          }
          if (lane == 0) {  // (rows past the queries and columns past the width are clipped)
            tma_store_4d(&tmap_o, panel, d, w.hk * p.group, (w.tile0 + i) * p.tile_tokens, w.b);
            bulk_commit();
          }
        }
        o_phase ^= 1u;
      }
      tc_fence_before();  // these reads of O come before the next item's P V
    }
    if (fault != 0u) *abort_flag = 1;
    if (row == 0) bulk_wait<0>();
    if (p.join) {
      // ------------------------------------------------------------ join of the key ranges
      // Every role of this CTA is done, so the ring is idle: each softmax thread
      // leaves its row's O (not normalised), reference and sum there.  Then the
      // cluster's threads share the item's rows: w_r = 2^(c (m_r - m)),
      // o = sum_r w_r O_r / sum_r w_r l_r, in the order of the ranks.
      tc_fence_before();
      named_barrier_sync(1, kAttThreads);
      tc_fence_after();
      uint8_t* part = smem + C::kOffKv;
      const AttItem w = att_item(p, first, rank);
      if (i < w.slots || w.shared) {
        *reinterpret_cast<float2*>(part + C::kPartMl + (i * 128 + row) * 8) = make_float2(m_ref, l_sum);
        uint8_t* dst = part + i * C::kPartSlot + row * C::kPartStride;
#pragma unroll 1
        for (int d = 0; d < kDP; d += 32) {
          uint32_t o[32];
          if (have) {
            tmem_ld_32x32b_x32(t_o + d, o);
            tmem_ld_wait(o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(dst + d * 4 + k * 16) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      if constexpr (kFew) {
        // the CTA's eight parts of a row (two slots, four copies) become one first
        named_barrier_sync(2, 256);
        float2* ml = reinterpret_cast<float2*>(part + C::kPartMl);
        bool any = false;
        const int queries = p.q_tokens * p.group;  // (the tile's rows behind them are nobody's)
        for (int u = threadIdx.x; u < queries * (kDP / 4); u += 256) {
          const int rr = u / (kDP / 4), g = u - rr * (kDP / 4);
          float m = -INFINITY;
#pragma unroll
          for (int t = 0; t < 8; ++t) m = fmaxf(m, ml[t * 32 + rr].x);
          float l = 0.0f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const float2 x = ml[t * 32 + rr];
            if (x.y == 0.0f) continue;  // no keys of its own
            const float f = exp2_approx((x.x - m) * c);
            const float4 a = *reinterpret_cast<const float4*>(part + (t * 32 + rr) * C::kPartStride + g * 16);
            l = fmaf(x.y, f, l);
            v.x = fmaf(a.x, f, v.x);
            v.y = fmaf(a.y, f, v.y);
            v.z = fmaf(a.z, f, v.z);
            v.w = fmaf(a.w, f, v.w);
          }
          // (in the place of the first part: only this thread reads these columns)
          *reinterpret_cast<float4*>(part + rr * C::kPartStride + g * 16) = v;
          if (g == 0) reinterpret_cast<float2*>(part + C::kPartMlCta)[rr] = make_float2(m, l);
          if (!isnan(l) && (isnan(v.x) || isnan(v.y) || isnan(v.z) || isnan(v.w))) {
            atomicOr(again, 1u << rr);
            any = true;
          }
        }
        __syncwarp();
        if (__builtin_expect(named_barrier_any(2, 256, any), 0))
          few_rows_again<kDP, kFp16, C>(p, first, rank, *again, part);
      }
      sync_cluster();
      if (*abort_flag == 0) {
        const int groups = p.D / 8;
        const int rows0 = min(p.tile_rows, (p.q_tokens - w.tile0 * p.tile_tokens) * p.group);
        const int rows1 = w.slots == 2 ? min(p.tile_rows, (p.q_tokens - (w.tile0 + 1) * p.tile_tokens) * p.group) : 0;
        for (int u = rank * 256 + threadIdx.x; u < (rows0 + rows1) * groups; u += p.split * 256) {
          const int rr = u / groups, g = u - rr * groups;
          const int i = rr >= rows0 ? 1 : 0;
          const int row = rr - (i ? rows0 : 0);
          // the row's parts: one per rank, or two where the slots shared the tile
          const int per_rank = w.shared && !kFew ? 2 : 1;
          auto part_at = [&](uint32_t base, uint32_t slot_bytes, int t) {
            const uint32_t a = base + (per_rank == 2 ? static_cast<uint32_t>(t & 1) * slot_bytes : 0u);
            return peer_smem(a, static_cast<uint32_t>(t / per_rank));
          };
          const uint32_t ml = smem_u32(part + (kFew ? C::kPartMlCta : C::kPartMl) + (i * 128 + row) * 8);
          const uint32_t src = smem_u32(part + i * C::kPartSlot + row * C::kPartStride + g * 32);
          float m = -INFINITY;
          for (int t = 0; t < p.split * per_rank; ++t) m = fmaxf(m, ld_shared_cluster_f2(part_at(ml, 128 * 8, t)).x);
          float l = 0.0f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int t = 0; t < p.split * per_rank; ++t) {
            const float2 x = ld_shared_cluster_f2(part_at(ml, 128 * 8, t));
            if (x.y == 0.0f) continue;  // no states in that range, or no finite score (a NaN's sum is NaN)
            const float f = exp2_approx((x.x - m) * p.scale_log2);
            l = fmaf(x.y, f, l);
            const uint32_t at = part_at(src, C::kPartSlot, t);
            const float4 a = ld_shared_cluster_f4(at), b = ld_shared_cluster_f4(at + 16);
            v[0] = fmaf(a.x, f, v[0]);
            v[1] = fmaf(a.y, f, v[1]);
            v[2] = fmaf(a.z, f, v[2]);
            v[3] = fmaf(a.w, f, v[3]);
            v[4] = fmaf(b.x, f, v[4]);
            v[5] = fmaf(b.y, f, v[5]);
            v[6] = fmaf(b.z, f, v[6]);
            v[7] = fmaf(b.w, f, v[7]);
          }
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          const int token = (w.tile0 + i) * p.tile_tokens + row / p.group;
          uint16_t* out = static_cast<uint16_t*>(p.out) + w.b * p.out_batch + static_cast<int64_t>(token) * p.out_token +
                          static_cast<int64_t>(w.hk * p.group + row % p.group) * p.out_head;
          *reinterpret_cast<uint4*>(out + g * 8) =
              make_uint4(pack2<kFp16>(v[0] * inv, v[1] * inv), pack2<kFp16>(v[2] * inv, v[3] * inv),
                         pack2<kFp16>(v[4] * inv, v[5] * inv), pack2<kFp16>(v[6] * inv, v[7] * inv));
        }
      }
    }
  }
  if (warp >= 8 && p.join) {  // the join's two barriers
    __syncwarp();
    tc_fence_before();
    named_barrier_sync(1, kAttThreads);
    sync_cluster();
  }
  if (fault != 0u && lane == 0 && p.fault != nullptr) atomicOr(p.fault, fault);
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_sync();  // nobody reads this CTA's shared memory any more
  tc_fence_after();
  if (warp == 8) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// Clusters of `split` CTAs that the device holds at once (0: it cannot).
template <int kDP, bool kFp16>
int resident_clusters(int split, const DeviceInfo& dev) {
  static std::atomic<int> cache[kMaxDevices][kAttMaxSplit + 1];  // the count plus one; the same for any two threads
  int n = cache[dev.device][split].load(std::memory_order_relaxed) - 1;
  if (n < 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kAttThreads, 1, 1);
    cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms / split * split), 1, 1);
    cfg.dynamicSmemBytes = ACfg<kDP, false>::kSmemBytes;  // (kFew's too fills an SM)
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, attention_kernel<kDP, kFp16, false>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    cache[dev.device][split].store(n + 1, std::memory_order_relaxed);
  }
  return n;
}

template <int kDP, bool kFp16, bool kFew>
cudaError_t launch_kernel(const AttentionMaps& m, const AttentionParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  using C = ACfg<kDP, kFew>;
  auto kernel = attention_kernel<kDP, kFp16, kFew>;
  static SmemLimit limit;
  cudaError_t err = limit.raise(kernel, C::kSmemBytes, dev.device);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kAttThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  if (p.items > INT32_MAX / p.split) return cudaErrorInvalidConfiguration;
  const int ctas = p.join ? p.items * p.split : (p.items < dev.num_sms ? p.items : dev.num_sms);
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  err = cudaLaunchKernelEx(&cfg, kernel, m.q, m.k, m.v, m.o, p);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

template <int kDP, bool kFp16>
cudaError_t launch(const AttentionMaps& m, AttentionParams p, cudaStream_t stream, const DeviceInfo& dev) {
  // (the occupancy query below needs the limit too)
  static SmemLimit limit;
  cudaError_t err = limit.raise(attention_kernel<kDP, kFp16, false>, ACfg<kDP, false>::kSmemBytes, dev.device);
  if (err != cudaSuccess) return err;
  // How an item is shared out, by its cost in key tiles of one slot: whole
  // items in turn, one CTA per SM (kTurnCost for an item's ends), or items with
  // CTAs of their own, in waves of the clusters that fit, each taking its share
  // of the key tiles (two at a time where the slots share the only query tile)
  // plus kJoinCost for the start and the join.
  constexpr int kTurnCost = 1, kJoinCost = 3;
  const int tiles = (p.kv_tokens + kAttTile - 1) / kAttTile;
  const int at_once = p.q_tiles == 1 ? 2 : 1;  // key tiles that a joined item's CTA has in work
  auto waves = [](int n, int fit) { return static_cast<int64_t>((n + fit - 1) / fit); };
  p.split = 1;
  p.join = 0;
  int64_t best = waves(p.items, dev.num_sms) * (tiles + kTurnCost);
  for (int split = at_once == 2 ? 1 : 2; split <= kAttMaxSplit && split * at_once <= tiles; ++split) {
    if (split > 1 && p.items > dev.num_sms / 2) break;
    const int fit = split > 1 ? resident_clusters<kDP, kFp16>(split, dev) : dev.num_sms;
    if (fit == 0) continue;
    const int64_t cost = waves(p.items, fit) * ((tiles + split * at_once - 1) / (split * at_once) + kJoinCost);
    if (cost < best) {
      best = cost;
      p.split = split;
      p.join = 1;
    }
  }
  if (p.join != 0 && p.q_tiles == 1 && p.tile_rows <= 32)
    return launch_kernel<kDP, kFp16, true>(m, p, stream, dev);
  return launch_kernel<kDP, kFp16, false>(m, p, stream, dev);
}

}  // namespace

cudaError_t launch_attention(const AttentionMaps& m, const AttentionParams& p, bool fp16, cudaStream_t stream,
                             const DeviceInfo& dev) {
  if (p.D <= 64) return fp16 ? launch<64, true>(m, p, stream, dev) : launch<64, false>(m, p, stream, dev);
  return fp16 ? launch<128, true>(m, p, stream, dev) : launch<128, false>(m, p, stream, dev);
}

}  // namespace nvfp4
