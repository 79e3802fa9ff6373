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

// ------------------------------------------------------------ the chain of tiles
//
// A workgroup holds a tile in registers: kSteps steps of each of its wavefronts, 64 CH
// channels.  Within it a step is h -> a h + b, so a tile is h -> P h + H with P and H
// its own, known once it is loaded.  What enters a tile is then joined without reading
// anything twice: tiles come in groups of kGsGroup; a tile publishes (P, H), waits for
// the state that enters its group and for the (P, H) of the group's tiles before it,
// and composes them in order; the group's last tile publishes the state that enters the
// next group.  Sums are composed in a fixed order, so the results do not depend on which
// workgroup runs when.
//
// Every wait ends: tiles are handed out by a counter, in the order of the chain, so what
// a tile waits for belongs to workgroups that are running already; publishing (P, H)
// waits for nothing, and the first group's state is there from the start.  (The count
// of polls is bounded all the same.)  A published word is one atomic store of all its
// bits, told from memory that is still to be written by a pattern that no result has.

constexpr uint32_t kUnwritten = 0xffffffffu;    // a NaN that no arithmetic returns
constexpr int kMostPolls = 1 << 22;

struct Chain {
  uint64_t* parts;       // [strips][tiles][channels] (P, H)
  uint32_t* states;      // [strips][groups][channels]: the state that enters a group
  uint32_t* next;        // tiles handed out
  int32_t tiles, groups, strips;
};

// (P, H) as one word; a NaN as the usual one.
__device__ __forceinline__ uint32_t word_of(float v) { return v == v ? __float_as_uint(v) : 0x7fc00000u; }
__device__ __forceinline__ void publish(uint64_t* at, float P, float H) {
  __hip_atomic_store(at, (uint64_t)word_of(P) | (uint64_t)word_of(H) << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint32_t* at, float h) {
  __hip_atomic_store(at, word_of(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What enters tile `tile` (counted along the chain) of a strip, for one wavefront's
// channels lane + 64 c; P and H are the tile's own.  Publishes them, and for the last of a
// group the next group's state.
template <int CH>
__device__ __forceinline__ void chain_enter(const Chain& c, int strip, int tile, const float (&P)[CH], const float (&H)[CH],
                                            float (&h)[CH]) {
  const int lane = threadIdx.x & 63;
  const int group = tile / kGsGroup, in = tile % kGsGroup;
  uint64_t* mine = c.parts + ((int64_t)strip * c.tiles + tile) * (64 * CH) + lane;
  uint32_t* state = c.states + ((int64_t)strip * c.groups + group) * (64 * CH) + lane;
  const bool last = in == kGsGroup - 1 || tile == c.tiles - 1;
  if (!last) {
#pragma unroll
    for (int k = 0; k < CH; ++k) publish(mine + 64 * k, P[k], H[k]);
  }
  uint32_t s[CH];
  uint64_t w[kGsGroup - 1][CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) s[k] = kUnwritten;
#pragma unroll
  for (int j = 0; j < kGsGroup - 1; ++j)
#pragma unroll
    for (int k = 0; k < CH; ++k) w[j][k] = ~0ull;
  for (int poll = 0; poll < kMostPolls; ++poll) {
    bool missing = false;
#pragma unroll
    for (int k = 0; k < CH; ++k) s[k] = __hip_atomic_load(state + 64 * k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int j = 0; j < kGsGroup - 1; ++j)
      if (j < in) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
          w[j][k] = __hip_atomic_load(mine + (j - in) * (64 * CH) + 64 * k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
#pragma unroll
    for (int k = 0; k < CH; ++k) missing |= s[k] == kUnwritten;
#pragma unroll
    for (int j = 0; j < kGsGroup - 1; ++j)
      if (j < in) {
#pragma unroll
        for (int k = 0; k < CH; ++k) missing |= (uint32_t)w[j][k] == kUnwritten;
      }
    if (!__any(missing)) break;
    __builtin_amdgcn_s_sleep(1);
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    h[k] = __uint_as_float(s[k]);
#pragma unroll
    for (int j = 0; j < kGsGroup - 1; ++j)
      if (j < in) h[k] = __builtin_fmaf(__uint_as_float((uint32_t)w[j][k]), h[k], __uint_as_float((uint32_t)(w[j][k] >> 32)));
  }
  if (last && tile + 1 < c.tiles) {
#pragma unroll
    for (int k = 0; k < CH; ++k) publish(state + 64 * CH + 64 * k, __builtin_fmaf(P[k], h[k], H[k]));
  }
}

// ------------------------------------------------------------------------ a tile

// A lane's CH neighbouring channels of a token as they lie in memory: one fp32 or bf16
// value, or two bf16 values in a word.
template <typename T, int CH>
__device__ __forceinline__ uint32_t load_raw(const void* p, int64_t token, int64_t row, uint32_t d) {
  const char* at = static_cast<const char*>(p) + token * row * (int64_t)sizeof(T);     // the same for all lanes
  const uint32_t off = d * (uint32_t)sizeof(T);
  if constexpr (sizeof(T) * CH == 4) return *reinterpret_cast<const uint32_t*>(at + off);
  else return *reinterpret_cast<const uint16_t*>(at + off);
}
template <typename T>
__device__ __forceinline__ float raw_value(uint32_t w, int k) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w);
  else return __uint_as_float(k ? w & 0xffff0000u : w << 16);
}
template <typename T, int CH>
__device__ __forceinline__ void store_raw(void* p, int64_t token, int64_t row, uint32_t d, const float (&v)[CH]) {
  char* at = static_cast<char*>(p) + token * row * (int64_t)sizeof(T) + d * (uint32_t)sizeof(T);
  if constexpr (sizeof(T) == 4) {
    if constexpr (CH == 2) *reinterpret_cast<float2*>(at) = make_float2(v[0], v[1]);
    else *reinterpret_cast<float*>(at) = v[0];
  } else {
    if constexpr (CH == 2) *reinterpret_cast<uint32_t*>(at) = pack_bf16x2(v[0], v[1]);
    else *reinterpret_cast<uint16_t*>(at) = f32_to_bf16_rne(v[0]);
  }
}

}  // namespace
}  // namespace ssm

#endif  // SSMSCAN_GSCAN_KERNEL_H
