// The pointwise part of the gated linear recurrence, shared by its kernels:
//
//   a = exp(-rate sigmoid(r)) or sigmoid(r);  m = sqrt(1 - a^2) or 1 - a;  u = [sigmoid(i)] x
#ifndef SSMSCAN_GSCAN_KERNEL_H
#define SSMSCAN_GSCAN_KERNEL_H

#include "device.h"
#include "gscan_plan.h"
#include "model.h"

namespace ssm {
namespace {

// exp(-v), from which sigmoid(v) = 1 / (1 + e) and sigmoid(-v) = e / (1 + e): each to a few
// ulp, and about half an ulp more for a unit of |v|, by which the argument's rounding moves e
// (by up to 8 half ulps at |v| = 10, 31 at 40, 62 at 80).  Where the second is needed, e is held at 8e37
// past fp32's range, whose reciprocal is still a normal number: the sigmoids are then 1.25e-38
// and 1.  A NaN stays one.
template <bool BOTH>
__device__ __forceinline__ float gate_exp(float v) {
  const float e = __builtin_amdgcn_exp2f(-v * kLog2e);
  return BOTH && e > 8.0e37f ? 8.0e37f : e;
}
__device__ __forceinline__ float gate_open(float e) { return __builtin_amdgcn_rcpf(1.0f + e); }

// 1 - exp(-w), given exp(-w) to an ulp, for w >= 0 or (SIGNED) of either sign.  Below 3/4
// the difference would lose what w is small by: there w times a polynomial of degree 5 in
// w, fitted to (1 - exp(-w)) / w over [0, 3/4] (off by at most 2.1e-8 of it, exact at 0);
// of the other sign it is -exp(-w) (1 - exp(w)).
template <bool SIGNED>
__device__ __forceinline__ float one_minus_exp(float w, float e) {
  const float v = SIGNED ? __builtin_fabsf(w) : w;
  float s = __builtin_fmaf(v, -0.00101896108f, 0.00804723334f);
  s = __builtin_fmaf(s, v, -0.0415632911f);
  s = __builtin_fmaf(s, v, 0.166650176f);
  s = __builtin_fmaf(s, v, -0.499999136f);
  s = w * __builtin_fmaf(s, v, 1.0f);
  if (SIGNED) s *= w < 0.0f ? e : 1.0f;
  asm volatile("" : "+v"(s));       // (computed, not branched around: a branch would part the steps)
  return v < 0.75f ? s : 1.0f - e;
}

// A step's decay and its input's coefficient, from e = exp(-r); rate2 = rate log2 e.
template <bool RATE, bool LERP>
__device__ __forceinline__ void decay(float e, float rate2, float* a, float* m) {
  const float pos = gate_open(e);
  if constexpr (RATE) {
    const float y = rate2 * pos;
    *a = __builtin_amdgcn_exp2f(-y);
    *m = LERP ? one_minus_exp<true>(y * kLn2, *a) : __builtin_amdgcn_sqrtf(one_minus_exp<false>(y * (2.0f * kLn2), *a * *a));
  } else {
    *a = pos;
    const float neg = e * pos;
    *m = LERP ? neg : __builtin_amdgcn_sqrtf(neg * (1.0f + pos));
  }
}

// dm/dlog a: of 1 - a, or of sqrt(1 - a^2), where a zero m has no derivative (0).
template <bool LERP>
__device__ __forceinline__ float decay_slope(float a, float m) {
  if constexpr (LERP) return -a;
  return m == 0.0f ? 0.0f : -a * a * __builtin_amdgcn_rcpf(m);
}

// p h + b, over steps whose decays' product is p.  GROW: decays may exceed 1, and p fp32's
// range, where a state of 0 stays 0 as in the steps themselves.
template <bool GROW>
__device__ __forceinline__ float onward(float p, float h, float b) {
  const float v = __builtin_fmaf(p, h, b);
  return GROW && h == 0.0f ? b : v;
}

// ------------------------------------------------------------ the chain of tiles
//
// A workgroup holds a tile in registers: some steps of each of its wavefronts, 64 CH
// channels.  Within it a step is h -> a h + b, so a tile is h -> P h + H with P and H
// its own, known once it is loaded.  What enters a tile is then joined without reading
// anything twice: tiles come in groups; a tile publishes (P, H), composes the (P, H) of
// the group's tiles before it in order, and waits for the state that enters its group;
// the group's last tile publishes the state that enters the next group.  Everything is
// composed in a fixed order, so the results do not depend on which workgroup runs when.
//
// Every wait ends: tiles are handed out by a counter, in the order of the chain, so what
// a tile waits for belongs to workgroups that are running already; publishing (P, H)
// waits for nothing, and the first group's state is there from the start.  (The count
// of polls is bounded all the same.)  A published word is one atomic store of all its
// bits, told from memory that is still to be written by a pattern that no result has.

constexpr uint32_t kUnwritten = 0xffffffffu;    // a NaN that no arithmetic returns
constexpr int kMostPolls = 1 << 22;
constexpr int kPartsAtOnce = 4;

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
template <bool GROW, int CH>
__device__ __forceinline__ void chain_enter(const Chain& c, int strip, int tile, const float (&P)[CH], const float (&H)[CH],
                                            float (&h)[CH]) {
  const int lane = threadIdx.x & 63;
  const int group = tile / c.group, in = tile % c.group;
  uint64_t* mine = c.parts + ((int64_t)strip * c.tiles + tile) * (64 * CH) + lane;
  uint32_t* state = c.states + ((int64_t)strip * c.groups + group) * (64 * CH) + lane;
  const bool last = in == c.group - 1 || tile == c.tiles - 1;
  if (!last) {
#pragma unroll
    for (int k = 0; k < CH; ++k) publish(mine + 64 * k, P[k], H[k]);
  }
  float gp[CH], gh[CH];      // of the group's tiles before this one
#pragma unroll
  for (int k = 0; k < CH; ++k) gp[k] = 1.0f, gh[k] = 0.0f;
  for (int j0 = 0; j0 < in; j0 += kPartsAtOnce) {
    uint64_t w[kPartsAtOnce][CH];
    for (int poll = 0; poll < kMostPolls; ++poll) {
      bool missing = false;
#pragma unroll
      for (int j = 0; j < kPartsAtOnce; ++j)
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          // (in the last round, the group's last one before this again)
          const int from = j0 + j < in ? j0 + j : in - 1;
          w[j][k] = __hip_atomic_load(mine + (from - in) * (64 * CH) + 64 * k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
      for (int j = 0; j < kPartsAtOnce; ++j)
#pragma unroll
        for (int k = 0; k < CH; ++k) missing |= (uint32_t)w[j][k] == kUnwritten;
      if (!__any(missing)) break;
      __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int j = 0; j < kPartsAtOnce; ++j)
      if (j0 + j < in) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const float p = __uint_as_float((uint32_t)w[j][k]);
          gp[k] *= p;
          gh[k] = onward<GROW>(p, gh[k], __uint_as_float((uint32_t)(w[j][k] >> 32)));
        }
      }
  }
  uint32_t s[CH];
  for (int poll = 0; poll < kMostPolls; ++poll) {
    bool missing = false;
#pragma unroll
    for (int k = 0; k < CH; ++k) s[k] = __hip_atomic_load(state + 64 * k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int k = 0; k < CH; ++k) missing |= s[k] == kUnwritten;
    if (!__any(missing)) break;
    __builtin_amdgcn_s_sleep(1);
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) h[k] = onward<GROW>(gp[k], __uint_as_float(s[k]), gh[k]);
  if (last && tile + 1 < c.tiles) {
#pragma unroll
    for (int k = 0; k < CH; ++k) publish(state + 64 * CH + 64 * k, onward<GROW>(P[k], h[k], H[k]));
  }
}

// ------------------------------------------------------------------------ a tile

// A tensor's rows from some token on, through a buffer descriptor: the row is a scalar
// offset and the lane's channels a vector one, so that an access costs no arithmetic, and
// what a lane whose offset is kNowhere reads is 0 and what it writes is dropped.  (Rows are
// at most 2^24 elements apart: 15 of them stay within the descriptor.)
constexpr uint32_t kNowhere = 0x80000000u;
struct Rows {
  __amdgpu_buffer_rsrc_t at;
  uint32_t row;       // bytes
  __device__ __forceinline__ Rows(const void* p, int64_t token, int64_t row_elems, int size) : row((uint32_t)row_elems * size) {
    // (the same for all lanes)
    char* first = const_cast<char*>(static_cast<const char*>(p)) + token * row_elems * size;
    const uint64_t bits = (uint64_t)(uintptr_t)first;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)bits), hi = __builtin_amdgcn_readfirstlane((uint32_t)(bits >> 32));
    at = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), 0, 0x7fffffff, 0x00020000);
  }
};

// A lane's CH neighbouring channels of a token as they lie in memory: one fp32 or bf16
// value, or two bf16 values in a word.
template <typename T, int CH>
__device__ __forceinline__ uint32_t load_raw(const Rows& r, int j, uint32_t d) {
  if constexpr (sizeof(T) * CH == 4) return __builtin_amdgcn_raw_buffer_load_b32(r.at, d, j * r.row, 0);
  else return __builtin_amdgcn_raw_buffer_load_b16(r.at, d, j * r.row, 0);
}
template <typename T>
__device__ __forceinline__ float raw_value(uint32_t w, int k) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w);
  else return __uint_as_float(k ? w & 0xffff0000u : w << 16);
}
// ... and CH values.
template <typename T, int CH>
__device__ __forceinline__ void load_values(const Rows& r, int j, uint32_t d, float (&v)[CH]) {
  if constexpr (sizeof(T) * CH == 8) {
    const auto w = __builtin_amdgcn_raw_buffer_load_b64(r.at, d, j * r.row, 0);
    v[0] = __uint_as_float(w[0]);
    v[1] = __uint_as_float(w[1]);
  } else {
    const uint32_t w = load_raw<T, CH>(r, j, d);
#pragma unroll
    for (int k = 0; k < CH; ++k) v[k] = raw_value<T>(w, k);
  }
}
// STREAM: past the caches.
template <bool STREAM, typename T, int CH>
__device__ __forceinline__ void store_raw(const Rows& r, int j, uint32_t d, const float (&v)[CH]) {
  constexpr int kAux = STREAM ? 2 : 0;      // non-temporal
  if constexpr (sizeof(T) == 4) {
    typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
    if constexpr (CH == 2)
      __builtin_amdgcn_raw_buffer_store_b64(u2_t{__float_as_uint(v[0]), __float_as_uint(v[1])}, r.at, d, j * r.row, kAux);
    else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), r.at, d, j * r.row, kAux);
  } else {
    if constexpr (CH == 2) __builtin_amdgcn_raw_buffer_store_b32(pack_bf16x2(v[0], v[1]), r.at, d, j * r.row, kAux);
    else __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16_rne(v[0]), r.at, d, j * r.row, kAux);
  }
}
}  // namespace
}  // namespace ssm

#endif  // SSMSCAN_GSCAN_KERNEL_H
