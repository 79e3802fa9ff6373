// The pointwise part of the gated linear recurrence, shared by its kernels:
//
//   a = exp(-rate sigmoid(r)) or sigmoid(r);  m = sqrt(1 - a^2) or 1 - a;  u = [sigmoid(i)] x
#ifndef SSMSCAN_GSCAN_KERNEL_H
#define SSMSCAN_GSCAN_KERNEL_H

#include "device.h"
#include "model.h"

namespace ssm {
namespace {

// sigmoid(v) and sigmoid(-v), each to a few ulp: with e = exp(-v) they are 1 / (1 + e)
// and e / (1 + e).  Where e is infinite the second is 1; a NaN stays one.
__device__ __forceinline__ void sigmoids(float v, float* pos, float* neg) {
  const float e = __builtin_amdgcn_exp2f(-v * kLog2e);
  const float p = __builtin_amdgcn_rcpf(1.0f + e);
  *pos = p;
  *neg = e > 8.0e37f ? 1.0f : e * p;
}

// 1 - exp(-w) for w >= 0 (and, by the same formulas, w < 0), given exp(-w) to an ulp.
// Below 1/2 the difference would lose what w is small by: there the series
// w (1 - w/2 (1 - w/3 (..))) up to w^8, whose next term is w^8 / 9! < 1.1e-8 of it.
__device__ __forceinline__ float one_minus_exp(float w, float e) {
  float s = __builtin_fmaf(w, -1.0f / 8.0f, 1.0f);
  s = __builtin_fmaf(w * s, -1.0f / 7.0f, 1.0f);
  s = __builtin_fmaf(w * s, -1.0f / 6.0f, 1.0f);
  s = __builtin_fmaf(w * s, -1.0f / 5.0f, 1.0f);
  s = __builtin_fmaf(w * s, -1.0f / 4.0f, 1.0f);
  s = __builtin_fmaf(w * s, -1.0f / 3.0f, 1.0f);
  s = __builtin_fmaf(w * s, -1.0f / 2.0f, 1.0f);
  return __builtin_fabsf(w) < 0.5f ? w * s : 1.0f - e;
}

struct Decay {
  float a;      // the decay
  float m;      // the input's coefficient
  float pos;    // sigmoid(r)
  float neg;    // sigmoid(-r)
};

template <bool RATE, bool LERP>
__device__ __forceinline__ Decay decay(float r, float rate) {
  Decay d;
  sigmoids(r, &d.pos, &d.neg);
  if constexpr (RATE) {
    const float y = rate * d.pos;
    d.a = __builtin_amdgcn_exp2f(-y * kLog2e);
    d.m = LERP ? one_minus_exp(y, d.a) : __builtin_amdgcn_sqrtf(one_minus_exp(2.0f * y, d.a * d.a));
  } else {
    d.a = d.pos;
    d.m = LERP ? d.neg : __builtin_amdgcn_sqrtf(d.neg * (1.0f + d.pos));
  }
  return d;
}

// dm/dlog a: of 1 - a, or of sqrt(1 - a^2), where a zero m has no derivative (0).
template <bool LERP>
__device__ __forceinline__ float decay_slope(const Decay& d) {
  if constexpr (LERP) return -d.a;
  return d.m == 0.0f ? 0.0f : -d.a * d.a * __builtin_amdgcn_rcpf(d.m);
}

}  // namespace
}  // namespace ssm

#endif  // SSMSCAN_GSCAN_KERNEL_H
