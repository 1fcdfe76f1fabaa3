// Rotary positions with several axes (time, height, width) on query and key
// heads, optionally after the RMS norm of each head.
//
// A head's first R = sum(axis_dims) elements form R/2 pairs; pair i belongs to
// one axis and turns by pos[token, axis] * f_i with f_i = theta^(-2 i_a / d_a)
// (i_a counts the pair within its axis of d_a elements) or, with one ladder
// shared by all axes, theta^(-2 i / R).  Pairs are neighbours (2i, 2i+1) or
// halves (i, i + R/2); elements from R on pass through.
//
// The kernel is bound by memory: 2 bytes read and 2 written per element.  A
// group of 2^n >= D/8 lanes owns one token and up to 24 heads of it; a lane
// owns the same four pairs (eight elements) of every head, so the four sines
// and cosines are worked out once for all of them and a row's norm is a shuffle
// within the group.  Lanes load the next four heads before they use the last
// four, 16 bytes each (two 8-byte halves in the half layout), and four blocks
// fit an SM.  30940 tokens x 24 heads x 128: 59.9 us (380 MB: 6.3 TB/s, 0.97 of a
// copy).  4608 tokens x 48 heads x 128 (113 MB) over six sets of buffers, more than
// the L2 holds: 20.4 us (5.5 TB/s, 0.85), with the norms 22.5 (5.0 TB/s, 0.77);
// on one set of buffers, which the L2 mostly holds, 15.8 and 18.0.
//
// The angle is reduced in 64 bits: t = pos * (f_i / 2 pi) turns, of which only
// t - rint(t) goes on in 32 bits, so a position of a million costs no accuracy
// (in 32 bits its angle would be off by 0.03).  Its sine and cosine are the
// hardware's (within 2^-20.9 on [-pi, pi], far below the 16-bit rounding of the
// result; sincospif was a third of the instructions).  Sums of squares, the
// norm and the rotation are 32-bit; the result is rounded once.
#include <math.h>

#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kRopeThreads = 256;

// Two 16-bit elements of a word to floats and back, rounded to nearest.
template <bool kFp16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (kFp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (kFp16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  return pack_bf16x2(lo, hi);
}

// Eight elements of a row: 16 bytes at element `lo`, or 8 bytes there and 8 at `hi`.
__device__ __forceinline__ uint4 load_eight(const uint16_t* row, int lo, int hi, bool split) {
  if (!split) return *reinterpret_cast<const uint4*>(row + lo);
  const uint2 a = *reinterpret_cast<const uint2*>(row + lo), b = *reinterpret_cast<const uint2*>(row + hi);
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_eight(uint16_t* row, int lo, int hi, bool split, uint4 v) {
  if (!split) {
    *reinterpret_cast<uint4*>(row + lo) = v;
  } else {
    *reinterpret_cast<uint2*>(row + lo) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(row + hi) = make_uint2(v.z, v.w);
  }
}

template <bool kFp16, bool kInterleaved, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ double turns[kRopeMaxPairs];  // f_i / 2 pi
  for (int i = threadIdx.x; i < p.R / 2; i += kRopeThreads) turns[i] = p.turns[i];
  __syncthreads();
  // The kernel is launched before the one in front of it has ended, and lets the
  // next one be: nothing up to here touched global memory.  (Without it call
  // after call took 2.3 us more for the first of these, 2.9 for the second.)
  launch_dependents();
  wait_for_previous_kernel();
  const int lane = threadIdx.x & (p.group - 1);
  const int64_t u64 = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) / p.group;
  const bool live = u64 < p.units && lane * 8 < p.D;
  const int u = live ? static_cast<int>(u64) : 0;
  const int token = u / p.units_per_token;
  const int part = u - token * p.units_per_token;
  const int which = part >= p.parts0 ? 1 : 0;
  const RopeTensor& t = p.t[which];
  const int head0 = (part - (which ? p.parts0 : 0)) * t.heads_per_unit;
  const int nh = live ? min(t.heads_per_unit, t.heads - head0) : 0;
  const int b = token / p.L, l = token - b * p.L;

  // this lane's elements of every head
  const bool rotary = lane * 8 < p.R;
  const bool split = !kInterleaved && rotary;
  const int lo = split ? lane * 4 : lane * 8;
  const int hi = p.R / 2 + lane * 4;
  const uint16_t* in = static_cast<const uint16_t*>(t.in) + b * t.in_batch + l * t.in_token + head0 * t.in_head;
  uint16_t* out = static_cast<uint16_t*>(t.out) + b * t.out_batch + l * t.out_token + head0 * t.out_head;
  uint4 next[4];
  // (the pointers step from head to head with the norm, which is bound by its
  // instructions; without it, bound by memory, that took 62.9 us for 59.8)
  auto load_from = [&](int h0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (h0 + i < nh) next[i] = load_eight(kNorm ? in : in + (h0 + i) * t.in_head, lo, hi, split);
      if (kNorm) in += t.in_head;
    }
  };
  load_from(0);

  float cs[4], sn[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    cs[j] = 1.0f;
    sn[j] = 0.0f;
  }
  if (live && rotary) {
    const int64_t pos0 = static_cast<int64_t>(b) * p.pos_batch_stride + static_cast<int64_t>(l) * p.n_axes;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int pair = lane * 4 + j;
      int axis = 0;
#pragma unroll
      for (int a = 1; a < kRopeMaxAxes; ++a) axis += (a < p.n_axes && pair >= p.first_pair[a]) ? 1 : 0;
      const double pos = p.pos_float ? static_cast<double>(static_cast<const float*>(p.positions)[pos0 + axis])
                                     : static_cast<double>(static_cast<const int32_t*>(p.positions)[pos0 + axis]);
      const double turn = pos * turns[pair];
      __sincosf(6.2831853f * static_cast<float>(turn - rint(turn)), &sn[j], &cs[j]);
    }
  }
  // A pair (a, b) turns into (ca a - sb b, sa a + cb b): a norm's weights are part
  // of these, and its root is left for the head.
  const bool normed = kNorm && t.weight != nullptr;
  float ca[4], sb[4], sa[4], cb[4];
  if constexpr (kNorm) {
    float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (normed && live) {
      const uint4 x = load_eight(static_cast<const uint16_t*>(t.weight), lo, hi, split);
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = unpack2<kFp16>(xw[j]);
        w[2 * j] = v.x;
        w[2 * j + 1] = v.y;
      }
    }
    const bool apart = !kInterleaved && rotary;  // a pair's elements are four apart, not neighbours
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float wa = apart ? w[j] : w[2 * j], wb = apart ? w[j + 4] : w[2 * j + 1];
      ca[j] = cs[j] * wa;
      sb[j] = sn[j] * wb;
      sa[j] = sn[j] * wa;
      cb[j] = cs[j] * wb;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ca[j] = cb[j] = cs[j];
      sa[j] = sb[j] = sn[j];
    }
  }

  // every lane of a warp takes the same number of turns: the shuffles below need them all
  for (int h0 = 0; h0 < p.heads_per_unit; h0 += 4) {
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = next[i];
    load_from(h0 + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool use = h0 + i < nh;
      const uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 e = unpack2<kFp16>(xw[j]);
        v[2 * j] = e.x;
        v[2 * j + 1] = e.y;
      }
      if (kNorm) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
        ss = use ? ss : 0.0f;  // (lanes past the width take part with nothing)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (p.group > o) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (normed) {
          const float r = rsqrtf(ss * p.inv_d + p.eps);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= r;
        }
      }
      if (!kNorm && !use) continue;
      uint32_t y[4];
      if (kInterleaved || !rotary) {
        // (lanes that pass through have cosines of 1: times the weight, or as they are)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[j] = rotary  ? pack2<kFp16>(ca[j] * v[2 * j] - sb[j] * v[2 * j + 1], sa[j] * v[2 * j] + cb[j] * v[2 * j + 1])
                 : kNorm ? pack2<kFp16>(ca[j] * v[2 * j], cb[j] * v[2 * j + 1])
                         : pack2<kFp16>(v[2 * j], v[2 * j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          y[j] = pack2<kFp16>(ca[2 * j] * v[2 * j] - sb[2 * j] * v[2 * j + 4],
                              ca[2 * j + 1] * v[2 * j + 1] - sb[2 * j + 1] * v[2 * j + 5]);
          y[j + 2] = pack2<kFp16>(sa[2 * j] * v[2 * j] + cb[2 * j] * v[2 * j + 4],
                                  sa[2 * j + 1] * v[2 * j + 1] + cb[2 * j + 1] * v[2 * j + 5]);
        }
      }
      if (use)
        store_eight(kNorm ? out : out + (h0 + i) * t.out_head, lo, hi, split, make_uint4(y[0], y[1], y[2], y[3]));
      if (kNorm) out += t.out_head;
    }
  }
}

template <bool kFp16, bool kInterleaved, bool kNorm>
cudaError_t launch(const RopeParams& p, unsigned blocks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, rope_kernel<kFp16, kInterleaved, kNorm>, p);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <bool kFp16>
cudaError_t launch(const RopeParams& p, unsigned blocks, bool interleaved, bool norm, cudaStream_t stream) {
  if (interleaved) return norm ? launch<kFp16, true, true>(p, blocks, stream) : launch<kFp16, true, false>(p, blocks, stream);
  return norm ? launch<kFp16, false, true>(p, blocks, stream) : launch<kFp16, false, false>(p, blocks, stream);
}

}  // namespace

bool rope_plan(RopeParams* p, int64_t tokens, int num_sms, int64_t* blocks) {
  p->group = 1;
  while (p->group * 8 < p->D) p->group *= 2;
  p->inv_d = 1.0f / static_cast<float>(p->D);
  // Heads of one unit: up to 24 share their sines and cosines where that leaves
  // every SM two blocks' worth of units, fewer where the units would be too few
  // to keep the memory busy.  At most 24 / 12 / 6 / 3 heads, in us, call after call:
  //   48 heads x 4608 tokens with norms, in the L2    18.0 / 19.2 / 26.4 / 34.2
  //                                     beyond it     22.5 / 20.5 / 26.5 / 34.3
  //                          no norms,  in the L2     15.8 / 16.9 / 20.5 / 26.1
  //                                     beyond it     20.4 / 19.7 / 21.2 / 26.3
  //   24 heads x 30940 tokens, no norms               60.1 / 58.3 / 64.7 / 82.9
  // 24 is the best where the projection has just left Q and K in the L2, 12 (two
  // waves of half the work) by 1 to 2 us where everything comes from memory.
  for (int most = 24;; most /= 2) {
    int parts[2] = {0, 0};
    p->heads_per_unit = 0;
    for (int i = 0; i < 2; ++i) {
      RopeTensor& t = p->t[i];
      if (t.heads == 0) continue;
      parts[i] = (t.heads + most - 1) / most;
      t.heads_per_unit = (t.heads + parts[i] - 1) / parts[i];
      p->heads_per_unit = t.heads_per_unit > p->heads_per_unit ? t.heads_per_unit : p->heads_per_unit;
    }
    p->parts0 = parts[0];
    p->units_per_token = parts[0] + parts[1];
    p->units = tokens * p->units_per_token;
    if (most == 1 || p->units * p->group >= static_cast<int64_t>(num_sms) * 2 * kRopeThreads) break;
  }
  *blocks = (p->units * p->group + kRopeThreads - 1) / kRopeThreads;
  return p->units <= INT32_MAX && *blocks <= INT32_MAX;
}

cudaError_t launch_rope(const RopeParams& p, int64_t blocks, bool fp16, bool interleaved, bool norm,
                        cudaStream_t stream) {
  const unsigned n = static_cast<unsigned>(blocks);
  return fp16 ? launch<true>(p, n, interleaved, norm, stream) : launch<false>(p, n, interleaved, norm, stream);
}

}  // namespace nvfp4
