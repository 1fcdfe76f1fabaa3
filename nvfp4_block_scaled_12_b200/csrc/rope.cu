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
// group of 2^n >= D/8 lanes owns one token and up to `heads_per_unit` heads of
// it; a lane owns the same four pairs (eight elements) of every head, so the
// four sines and cosines are worked out once for all of them and a row's norm
// is a shuffle within the group.  Lanes load four heads before they use the
// first, 16 bytes each (two 8-byte halves in the half layout).
//
// The angle is reduced in 64 bits: t = pos * (f_i / 2 pi) turns, of which only
// t - rint(t) goes on to sincospif in 32 bits, so a position of a million
// costs no accuracy (in 32 bits its angle would be off by 0.03).  Sums of
// squares, the norm and the rotation are 32-bit; the result is rounded once.
#include <math.h>

#include "internal.h"

namespace nvfp4 {

namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }

// Eight elements of a row: 16 bytes at `lo`, or 8 bytes at `lo` and 8 at `hi`.
template <typename T>
struct alignas(16) Eight {
  T e[8];
};

template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* row, int lo, int hi, bool split) {
  union {
    uint4 u;
    uint2 h[2];
    Eight<T> e;
  } v;
  if (split) {
    v.h[0] = *reinterpret_cast<const uint2*>(row + lo);
    v.h[1] = *reinterpret_cast<const uint2*>(row + hi);
  } else {
    v.u = *reinterpret_cast<const uint4*>(row + lo);
  }
  return v.e;
}

template <typename T>
__device__ __forceinline__ void store_eight(T* row, int lo, int hi, bool split, const Eight<T>& x) {
  union {
    uint4 u;
    uint2 h[2];
    Eight<T> e;
  } v;
  v.e = x;
  if (split) {
    *reinterpret_cast<uint2*>(row + lo) = v.h[0];
    *reinterpret_cast<uint2*>(row + hi) = v.h[1];
  } else {
    *reinterpret_cast<uint4*>(row + lo) = v.u;
  }
}

template <typename T, bool kInterleaved, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ double turns[kRopeMaxPairs];  // f_i / 2 pi
  for (int i = threadIdx.x; i < p.R / 2; i += kRopeThreads) turns[i] = p.turns[i];
  __syncthreads();
  const int lane = threadIdx.x & (p.group - 1);
  const int64_t u64 = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) / p.group;
  const bool live = u64 < p.units && lane * 8 < p.D;
  const int u = live ? static_cast<int>(u64) : 0;
  const int token = u / p.units_per_token;
  const int part = u - token * p.units_per_token;
  const int which = part >= p.parts0 ? 1 : 0;
  const RopeTensor& t = p.t[which];
  const int head0 = (part - (which ? p.parts0 : 0)) * p.heads_per_unit;
  const int nh = min(p.heads_per_unit, t.heads - head0);
  const int b = token / p.L, l = token - b * p.L;

  // this lane's elements of every head
  const bool rotary = lane * 8 < p.R;
  const bool split = !kInterleaved && rotary;
  const int lo = split ? lane * 4 : lane * 8;
  const int hi = p.R / 2 + lane * 4;

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
      sincospif(2.0f * static_cast<float>(turn - rint(turn)), &sn[j], &cs[j]);
    }
  }
  float w[8];
  if (kNorm) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.0f;
    if (live && t.weight != nullptr) {
      const Eight<T> x = load_eight(static_cast<const T*>(t.weight), lo, hi, split);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = to_f32(x.e[j]);
    }
  }
  const T* in = static_cast<const T*>(t.in) + b * t.in_batch + l * t.in_token + head0 * t.in_head;
  T* out = static_cast<T*>(t.out) + b * t.out_batch + l * t.out_token + head0 * t.out_head;

  // every lane of a warp takes the same number of turns: the shuffles below need them all
  for (int h0 = 0; h0 < p.heads_per_unit; h0 += 4) {
    Eight<T> x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (live && h0 + i < nh) x[i] = load_eight(in + (h0 + i) * t.in_head, lo, hi, split);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool use = live && h0 + i < nh;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = use ? to_f32(x[i].e[j]) : 0.0f;
      if (kNorm) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
        for (int o = p.group >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (t.weight != nullptr) {
          const float r = rsqrtf(ss / static_cast<float>(p.D) + p.eps);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= r * w[j];
        }
      }
      if (!use) continue;
      Eight<T> y;
      if (rotary) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int ia = kInterleaved ? 2 * j : j, ib = kInterleaved ? 2 * j + 1 : j + 4;
          from_f32(v[ia] * cs[j] - v[ib] * sn[j], y.e[ia]);
          from_f32(v[ia] * sn[j] + v[ib] * cs[j], y.e[ib]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) from_f32(v[j], y.e[j]);
      }
      store_eight(out + (h0 + i) * t.out_head, lo, hi, split, y);
    }
  }
}

template <typename T>
cudaError_t launch(const RopeParams& p, unsigned blocks, bool interleaved, bool norm, cudaStream_t stream) {
  if (interleaved) {
    if (norm)
      rope_kernel<T, true, true><<<blocks, kRopeThreads, 0, stream>>>(p);
    else
      rope_kernel<T, true, false><<<blocks, kRopeThreads, 0, stream>>>(p);
  } else {
    if (norm)
      rope_kernel<T, false, true><<<blocks, kRopeThreads, 0, stream>>>(p);
    else
      rope_kernel<T, false, false><<<blocks, kRopeThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

bool rope_plan(RopeParams* p, int64_t tokens, int num_sms, int64_t* blocks) {
  p->group = 1;
  while (p->group * 8 < p->D) p->group *= 2;
  const int h0 = p->t[0].heads, h1 = p->t[1].heads;
  // Heads of one unit: eight share their sines and cosines when that leaves
  // every SM two blocks' worth of units, fewer where the units would be too
  // few to keep the memory busy.
  int hpu = 8;
  int64_t units = 0;
  for (;; hpu /= 2) {
    p->parts0 = (h0 + hpu - 1) / hpu;
    p->units_per_token = p->parts0 + (h1 + hpu - 1) / hpu;
    units = tokens * p->units_per_token;
    if (hpu == 1 || units * p->group >= static_cast<int64_t>(num_sms) * 2 * kRopeThreads) break;
  }
  p->heads_per_unit = hpu;
  p->units = units;
  *blocks = (units * p->group + kRopeThreads - 1) / kRopeThreads;
  return units <= INT32_MAX && *blocks <= INT32_MAX;
}

cudaError_t launch_rope(const RopeParams& p, int64_t blocks, bool fp16, bool interleaved, bool norm,
                        cudaStream_t stream) {
  const unsigned n = static_cast<unsigned>(blocks);
  return fp16 ? launch<__half>(p, n, interleaved, norm, stream) : launch<__nv_bfloat16>(p, n, interleaved, norm, stream);
}

}  // namespace nvfp4
