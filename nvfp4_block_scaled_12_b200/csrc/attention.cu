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
//     O += P V         128 x DP x 128  tcgen05.mma, P from TMEM (over S), V
//                                      from shared memory as a transposed operand
// with c = scale log2 e.  The two slots alternate: the tensor cores work on
// one while the softmax warps work on the other.
//
// The reference m of a row is its first tile's maximum and moves only when a
// later maximum exceeds it by 2^8 in P (P stays below 2^8, far inside the
// types' ranges, and the sums in fp32 keep their relative accuracy); only
// then is O rescaled in TMEM.  S, the maximum, the sum and O are fp32; P is
// rounded to the type of V for the tensor cores (the sum takes it unrounded,
// so a row's error from this averages out over its keys).
//
// States from kv_lens[b] on contribute nothing whatever they hold: their
// scores are replaced, not added to, and in the last tile the V rows that the
// MMA reads beyond them (up to the next multiple of 16 keys) are zeroed in
// shared memory, since 0 * NaN is NaN.  Keys past the tensor arrive as zeros.
//
// Warps (12): 0-3 softmax of slot 0 (one row a thread), 4-7 of slot 1, 8 MMA
// issuer, 9 TMA producer (10 and 11 fill up their warpgroup, whose registers go
// to the softmax threads: a row's 128 scores stay in registers).  TMEM: S0 | S1 | O0 | O1, 128 columns each.  Shared
// memory: both Q tiles and a ring of K and V tiles in their order of use.
//
// With fewer items than SMs the keys are split over the CTAs of a cluster:
// each keeps its own m, sum and O, which are joined through distributed shared
// memory in the order of the ranks (no workspace, no atomics, and the same
// result every time).
#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kAttTile = 128;  // query rows of a slot, keys of a tile
constexpr int kAttThreads = 384;  // three warpgroups: softmax of each slot, producer and MMA
constexpr uint32_t kPanelBytes = 128 * 128;  // 128 rows of 64 elements, 128-byte swizzle

// kDP: head width rounded up to 64 or 128 (the tensor maps zero-fill the rest).
template <int kDP>
struct ACfg {
  static constexpr int kPanels = kDP / 64;
  static constexpr uint32_t kTileBytes = kPanels * kPanelBytes;
  static constexpr int kStages = kDP == 128 ? 5 : 8;
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffKv = 2 * kTileBytes;
  static constexpr uint32_t kOffBar = kOffKv + kStages * kTileBytes;
  // kv_full, kv_empty per stage; q_full, q_empty, s_full, p_ready, o_full per slot; drain
  static constexpr uint32_t kNumBars = 2 * kStages + 10 + 1;
  static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;  // + alignment slack
  // K/V split: a slot's fp32 partial rows (padded to spread them over the
  // banks) and its maxima and sums, in the idle ring
  static constexpr uint32_t kPartStride = (kDP + 4) * 4;
  static constexpr uint32_t kPartSlot = 128 * kPartStride;
  static constexpr uint32_t kPartMl = 2 * kPartSlot;  // float2 (m, l) [2][128]
  static_assert(kPartMl + 2 * 128 * 8 <= kStages * kTileBytes, "the partial results fit the ring");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

constexpr uint32_t kColS = 0, kColO = 256;  // TMEM columns of slot 0; slot 1 is 128 further

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// D (TMEM) (+)= A (TMEM, 16-bit pairs) * B (shared memory)
__device__ __forceinline__ void tc_mma_16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
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

// One work item as every role sees it.
struct AttItem {
  int b, hk, tile0;    // batch entry, K/V head, first query tile
  int slots;           // 1 or 2 query tiles
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
  w.len = p.kv_lens != nullptr ? min(max(__ldg(p.kv_lens + w.b), 0), p.kv_tokens) : p.kv_tokens;
  const int tiles = (w.len + kAttTile - 1) / kAttTile;
  w.kt0 = static_cast<int>(static_cast<int64_t>(tiles) * rank / p.split);
  w.n = static_cast<int>(static_cast<int64_t>(tiles) * (rank + 1) / p.split) - w.kt0;
  return w;
}

template <int kDP, bool kFp16>
__global__ void __launch_bounds__(kAttThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ AttentionParams p) {
  using C = ACfg<kDP>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* kv_empty = kv_full + S;
  uint64_t* q_full = kv_empty + S;  // and below: one per slot
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_ready = s_full + 2;
  uint64_t* o_full = p_ready + 2;
  uint64_t* drain = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
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
      mbar_init(&o_full[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9 && lane == 0) {
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
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

  if (warp >= 8) {
    // (launched with 384 x 168 registers: 88 + 2 x 208 = 3 x 168)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
  }
  if (warp == 9) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t q_bytes = C::kPanels * static_cast<uint32_t>(p.tile_rows) * 128u;
      int64_t e = 0;             // ring entries issued
      uint32_t q_phase[2] = {0u, 0u};  // items whose tile went into the slot, mod 2
      bool q_used[2] = {false, false};
      auto load_q = [&](const AttItem& w, int i) {
        if (!mbar_wait(&q_empty[i], q_phase[i] ^ 1u, abort_flag)) return false;
        mbar_arrive_expect_tx(&q_full[i], q_bytes);
        for (int c = 0; c < C::kPanels; ++c)
          tma_load_4d(smem + C::kOffQ + i * C::kTileBytes + c * kPanelBytes, &tmap_q, &q_full[i], c * 64,
                      w.hk * p.group, (w.tile0 + i) * p.tile_tokens, w.b * p.q_bmul);
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
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_16<kFp16>(kAttTile, false);
      constexpr uint32_t idesc_pv = idesc_16<kFp16>(kDP, true);
      int64_t e = 0;  // ring entries consumed: K of step s is entry 2s, V is 2s + 1
      uint32_t q_phase[2] = {0u, 0u}, p_phase[2] = {0u, 0u};
      // the step whose P V is still to be issued
      struct {
        int slots = 0;
        int64_t v_entry = 0;
        uint32_t accumulate = 0;
        int k16 = 0;  // 16-key steps that hold a valid key
        bool last = false;
      } pend;
      auto wait_kv = [&](int64_t entry) {
        return mbar_wait(&kv_full[entry % S], static_cast<uint32_t>(entry / S) & 1u, abort_flag);
      };
      // O_i (+)= P_i V of the pending step
      auto issue_pv = [&](int i) {
        if (i >= pend.slots) return true;
        if (!mbar_wait(&p_ready[i], p_phase[i], abort_flag)) return false;
        p_phase[i] ^= 1u;
        if (i == 0 && !wait_kv(pend.v_entry)) return false;
        tc_fence_after();
        const uint64_t vd =
            sdesc_nmajor_sw128(smem_u32(smem + C::kOffKv + static_cast<uint32_t>(pend.v_entry % S) * C::kTileBytes));
        const uint32_t o = tmem + kColO + i * 128, a = tmem + kColS + i * 128;
        for (int k = 0; k < pend.k16; ++k)
          tc_mma_16_ts(o, a + k * 8, vd + k * (2048 >> 4), idesc_pv, (k != 0) ? 1u : pend.accumulate);
        if (pend.last) tc_commit(&o_full[i]);
        if (i == pend.slots - 1) tc_commit(&kv_empty[pend.v_entry % S]);
        return true;
      };
      for (int item = first; item < p.items && fault == 0u; item += step) {
        const AttItem w = att_item(p, item, rank);
        for (int j = 0; j < w.n; ++j) {
          bool ok = true;
          for (int i = 0; i < 2 && ok; ++i) {
            ok = issue_pv(i);
            if (!ok || i >= w.slots) continue;
            if (i == 0) ok = wait_kv(e);
            if (ok && j == 0) {
              ok = mbar_wait(&q_full[i], q_phase[i], abort_flag);
              q_phase[i] ^= 1u;
            }
            if (!ok) continue;
            tc_fence_after();
            const uint64_t qd = sdesc_kmajor_sw128(smem_u32(smem + C::kOffQ + i * C::kTileBytes));
            const uint64_t kd =
                sdesc_kmajor_sw128(smem_u32(smem + C::kOffKv + static_cast<uint32_t>(e % S) * C::kTileBytes));
#pragma unroll
            for (int k = 0; k < kDP / 16; ++k) {
              const uint64_t off = static_cast<uint64_t>((k / 4) * (kPanelBytes >> 4) + (k % 4) * 2);
              tc_mma_bf16(tmem + kColS + i * 128, qd + off, kd + off, idesc_qk, k != 0 ? 1u : 0u);
            }
            tc_commit(&s_full[i]);
            if (j == w.n - 1) tc_commit(&q_empty[i]);
            if (i == w.slots - 1) tc_commit(&kv_empty[e % S]);
          }
          if (!ok) {
            fault = kFaultMmaWait;
            break;
          }
          pend.slots = w.slots;
          pend.v_entry = e + 1;
          pend.accumulate = j != 0 ? 1u : 0u;
          pend.k16 = min(kAttTile, w.len - (w.kt0 + j) * kAttTile + 15) / 16;
          pend.last = j == w.n - 1;
          e += 2;
        }
      }
      if (fault == 0u && (!issue_pv(0) || !issue_pv(1))) fault = kFaultMmaWait;
      if (fault != 0u) *abort_flag = 1;
      // every tcgen05 operation issued must complete before TMEM is released
      tc_commit(drain);
      if (!mbar_wait(drain, 0u, nullptr)) fault |= kFaultDrainWait;
    }
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
    const uint32_t t_s = tmem + kColS + i * 128 + t_lane, t_o = tmem + kColO + i * 128 + t_lane;
    const float c = p.scale_log2;
    uint32_t s_phase = 0u, o_phase = 0u;
    int64_t steps = 0;  // key tiles so far (slot 0 sees every one of the CTA)
    auto all_lanes = [&](bool ok) {
      __syncwarp();
      return __all_sync(0xffffffffu, ok) != 0;
    };
    for (int item = first; item < p.items && fault == 0u; item += step) {
      const AttItem w = att_item(p, item, rank);
      if (i >= w.slots) continue;
      m_ref = -INFINITY;
      l_sum = 0.0f;
      have = w.n > 0;
      for (int j = 0; j < w.n; ++j, ++steps) {
        const int valid = w.len - (w.kt0 + j) * kAttTile;  // keys of this tile (more than 128: all)
        if (!all_lanes(mbar_wait(&s_full[i], s_phase, abort_flag))) {
          fault = kFaultEpilogueWait;
          break;
        }
        s_phase ^= 1u;
        tc_fence_after();
        uint32_t r[128];
        tmem_ld_32x32b_x64(t_s, r);
        tmem_ld_32x32b_x64(t_s + 64, r + 64);
        tmem_ld_wait_n<128>(r);
        if (valid < kAttTile) {
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (k >= valid) r[k] = 0xFF800000u;  // -inf
          if (i == 0 && (valid & 15) != 0) {
            // the V rows from the last valid state to the next multiple of 16
            // keys: zero, whatever they hold (0 * NaN would not be)
            const int64_t entry = 2 * steps + 1;
            const bool ok = mbar_wait(&kv_full[entry % S], static_cast<uint32_t>(entry / S) & 1u, abort_flag);
            if (!all_lanes(ok)) {
              fault = kFaultEpilogueWait;
              break;
            }
            uint8_t* v = smem + C::kOffKv + static_cast<uint32_t>(entry % S) * C::kTileBytes;
            const int chunks = (16 - (valid & 15)) * 8;  // 16-byte chunks of a panel's rows
            for (int t = row; t < chunks * C::kPanels; t += 128) {
              const int panel = t / chunks, at = t - panel * chunks;
              *reinterpret_cast<uint4*>(v + panel * kPanelBytes + valid * 128 + at * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(r[k]));
        const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (j == 0) {
          m_ref = m_tile;
        } else {
          const bool moves = (m_tile - m_ref) * c > 8.0f;
          if (__any_sync(0xffffffffu, moves)) {
            // (S of this tile is complete, and it was issued after the
            // previous tile's P V: nobody else touches O)
            const float f = moves ? exp2_approx((m_ref - m_tile) * c) : 1.0f;
            if (moves) m_ref = m_tile;
            l_sum *= f;
#pragma unroll 1
            for (int d = 0; d < kDP; d += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(t_o + d, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st_32x32b_x16(t_o + d, *reinterpret_cast<const uint32_t(*)[16]>(o));
              tmem_st_32x32b_x16(t_o + d + 16, *reinterpret_cast<const uint32_t(*)[16]>(o + 16));
            }
          }
        }
        const float mc = -m_ref * c;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int g = 0; g < 4; ++g) {  // 32 keys: 16 TMEM columns of P
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float a = exp2_approx(fmaf(__uint_as_float(r[g * 32 + 2 * k]), c, mc));
            const float b = exp2_approx(fmaf(__uint_as_float(r[g * 32 + 2 * k + 1]), c, mc));
            sum[(2 * k) & 3] += a;
            sum[(2 * k + 1) & 3] += b;
            pk[k] = pack2<kFp16>(a, b);
          }
          tmem_st_32x32b_x16(t_s + g * 16, pk);
        }
        l_sum += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[i]);
      }
      if (fault != 0u) break;
      if (w.n > 0) {
        if (!all_lanes(mbar_wait(&o_full[i], o_phase, abort_flag))) {
          fault = kFaultEpilogueWait;
          break;
        }
        o_phase ^= 1u;
        tc_fence_after();
      }
      if (p.split > 1) break;  // one item; joined below
      // ---- O / sum to the output row (zeros where there are no states)
      const int token = (w.tile0 + i) * p.tile_tokens + row / p.group;
      const bool write = row < p.tile_rows && token < p.q_tokens;
      const float inv = w.n > 0 ? 1.0f / l_sum : 0.0f;
      uint16_t* out = static_cast<uint16_t*>(p.out) + w.b * p.out_batch + static_cast<int64_t>(token) * p.out_token +
                      static_cast<int64_t>(w.hk * p.group + row % p.group) * p.out_head;
#pragma unroll 1
      for (int d = 0; d < p.D; d += 32) {
        uint32_t o[32];
        if (w.n > 0) {
          tmem_ld_32x32b_x32(t_o + d, o);
          tmem_ld_wait(o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (!write) continue;
        uint32_t y[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          y[k] = pack2<kFp16>(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (d + 8 * h < p.D)
            *reinterpret_cast<uint4*>(out + d + 8 * h) = make_uint4(y[4 * h], y[4 * h + 1], y[4 * h + 2], y[4 * h + 3]);
      }
      tc_fence_before();  // these reads of O come before the next item's P V
    }
    if (fault != 0u) *abort_flag = 1;
    if (p.split > 1) {
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
      if (i < w.slots) {
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
      cluster_sync();
      if (*abort_flag == 0) {
        const int groups = p.D / 8;
        const int rows0 = min(p.tile_rows, (p.q_tokens - w.tile0 * p.tile_tokens) * p.group);
        const int rows1 = w.slots == 2 ? min(p.tile_rows, (p.q_tokens - (w.tile0 + 1) * p.tile_tokens) * p.group) : 0;
        for (int u = rank * 256 + threadIdx.x; u < (rows0 + rows1) * groups; u += p.split * 256) {
          const int rr = u / groups, g = u - rr * groups;
          const int i = rr >= rows0 ? 1 : 0;
          const int row = rr - (i ? rows0 : 0);
          const uint32_t ml = smem_u32(part + C::kPartMl + (i * 128 + row) * 8);
          const uint32_t src = smem_u32(part + i * C::kPartSlot + row * C::kPartStride + g * 32);
          float m = -INFINITY;
          for (int s = 0; s < p.split; ++s) m = fmaxf(m, ld_shared_cluster_f2(peer_smem(ml, s)).x);
          float l = 0.0f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int s = 0; s < p.split; ++s) {
            const float2 x = ld_shared_cluster_f2(peer_smem(ml, s));
            if (x.x == -INFINITY) continue;  // no states in that range
            const float f = exp2_approx((x.x - m) * p.scale_log2);
            l = fmaf(x.y, f, l);
            const uint32_t at = peer_smem(src, s);
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
          const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
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
  if (warp >= 8 && p.split > 1) {  // the join's two barriers
    __syncwarp();
    tc_fence_before();
    named_barrier_sync(1, kAttThreads);
    cluster_sync();
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

template <int kDP, bool kFp16>
cudaError_t launch(const AttentionMaps& m, const AttentionParams& p, cudaStream_t stream, const DeviceInfo& dev) {
  using C = ACfg<kDP>;
  auto kernel = attention_kernel<kDP, kFp16>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kAttThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 1 : 0;
  // a split item has a cluster of its own; otherwise one CTA per SM takes items in turn
  const int ctas = p.split > 1 ? p.items * p.split : (p.items < dev.num_sms ? p.items : dev.num_sms);
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  err = cudaLaunchKernelEx(&cfg, kernel, m.q, m.k, m.v, p);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

}  // namespace

int attention_split(int64_t items, int64_t kv_tokens, int num_sms) {
  const int64_t tiles = (kv_tokens + kAttTile - 1) / kAttTile;
  int split = 1;
  while (split < 8 && split * 2 <= tiles && items * split * 2 <= num_sms) split *= 2;
  return split;
}

cudaError_t launch_attention(const AttentionMaps& m, const AttentionParams& p, bool fp16, cudaStream_t stream,
                             const DeviceInfo& dev) {
  if (p.D <= 64) return fp16 ? launch<64, true>(m, p, stream, dev) : launch<64, false>(m, p, stream, dev);
  return fp16 ? launch<128, true>(m, p, stream, dev) : launch<128, false>(m, p, stream, dev);
}

}  // namespace nvfp4
