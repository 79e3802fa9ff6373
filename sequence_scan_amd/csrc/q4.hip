// gfx950 kernels of libssmscan: products of few rows with 4-bit weights,
//   out[m][n] = sum_k x[m][k] (code[n][k] - zero[n][g]) scale[n][g] + bias[n],
// g = k / group, and the quantisation of a weight matrix into that form.
//
// A decode step's projections read every weight for a handful of rows, so the
// codes' bytes bound them (half a byte per weight at the HBM rate), as long as
// decoding costs about one VALU operation per weight.  Codes become bf16 operands
// of v_mfma_f32_16x16x32_bf16 by bit placement: 0x4180 | code << 3 is 16 + code,
// exactly; two codes per shift and and-or.  The 16 and the zero point leave by
// the group's sum of x: sum x (16 + code) - (16 + zero) sum x, scaled and added
// in fp32.  Rows of x take the other operand's 16 rows; up to 16 cost what one
// does.  fp32 x enters as three bf16 terms, as rows of their own that the
// epilogue adds (all 24 bits).
//
// Codes go from HBM to registers, 16 bytes per lane: 32 codes of one row, so 16
// rows x 128 codes (a "piece") per load of a wavefront.  For groups below 128 the
// four lanes of a row exchange words (a 4 x 4 transpose by row swaps), which makes
// every product cover 32 consecutive codes, one group's; for groups of 128 the
// order does not matter and x is read in the same order instead.  A workgroup owns
// some columns of out and all of K; its wavefronts split K in pieces and are joined
// in order at the end (no atomics: a call gives the same bits every time).
//
// Three forms.  Up to 16 rows of x (its terms counted) every workgroup rounds,
// orders and sums x itself: all of it at once, where it fits (q4_fits_kernel), or in
// slabs (q4_slabs_kernel).  Above, that would cost each of them as much as its
// products, so a small kernel lays x out once (q4_rows_kernel) as the LDS images of
// all slabs, and the workgroups load them straight to LDS, a slab ahead, and the
// codes two slabs ahead (q4_wide_kernel).
//
// Measured, back to back: one row x 10576 x 2560 (13.5 MB of codes) 7.4 us, of which the
// launch and the wait for the first bytes are about half; 2 rows x 16384 x 16384 (134 MB)
// 37 us, 3.6 TB/s; 48 rows x 16384 x 8192 (67 MB) 30 us, 3 of them to lay out x.  There no one
// thing bounds it: of 34 us then, it took 23, 31 and 31 without its loads, its matrix
// products and its reads of x, since the 16 wavefronts that a CU holds meet at a barrier every slab.
#include <algorithm>

#include "block.h"
#include "lds_load.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;

// Eight codes as bf16 pairs of 16 + code, in the order (0, 4), (1, 5), (2, 6), (3, 7).
// The mask comes in a vector register (q4_mask): with that, and-or is one
// instruction, which takes one constant from elsewhere, not two.
__device__ __forceinline__ uint32_t q4_mask() {
  uint32_t mask = 0x00780078u;
  asm("" : "+v"(mask));
  return mask;
}
__device__ __forceinline__ bf16x8_t q4_decode(uint32_t w, uint32_t mask) {
  const uint32_t base = 0x41804180u;
  const u32x4_t t = {((w << 3) & mask) | base, ((w >> 1) & mask) | base, ((w >> 5) & mask) | base, ((w >> 9) & mask) | base};
  return __builtin_bit_cast(bf16x8_t, t);
}

// Word j of the row of 16 lanes i becomes word i of row j.
__device__ __forceinline__ u32x4_t q4_transpose(u32x4_t w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4_t{c[0], c[1], d[0], d[1]};
}

// A scale as it is stored, and its value: apart, so that the wait for the load
// falls where the value is used, a slab later.
__device__ __forceinline__ uint32_t q4_scale_bits(const Q4Args& a, int64_t at) {
  uint32_t bits;
  if (a.scale_bf16) bits = static_cast<const uint16_t*>(a.scales)[at];
  else bits = static_cast<const uint32_t*>(a.scales)[at];
  return bits;
}
__device__ __forceinline__ float q4_scale(const Q4Args& a, uint32_t bits) { return __uint_as_float(a.scale_bf16 ? bits << 16 : bits); }

// Rows of x that MT tiles of 16 hold: all of them in bf16, a third in fp32.
constexpr int q4_rows(int mt, bool xf32) { return xf32 ? 16 * mt / 3 : 16 * mt; }

// The codes' pair order of eight consecutive bf16.
__device__ __forceinline__ u32x4_t q4_pairs(u32x4_t p) {
  return u32x4_t{__builtin_amdgcn_perm(p[2], p[0], 0x05040100u), __builtin_amdgcn_perm(p[2], p[0], 0x07060302u),
                 __builtin_amdgcn_perm(p[3], p[1], 0x05040100u), __builtin_amdgcn_perm(p[3], p[1], 0x07060302u)};
}

// Eight values of x from element `at` on, as floats and (bf16) as they are.
template <bool XF32>
__device__ __forceinline__ void q4_x(const void* x, int64_t at, float* f, u32x4_t& p) {
  if constexpr (XF32) {
    const float4 v0 = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 v1 = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + 4);
    f[0] = v0.x; f[1] = v0.y; f[2] = v0.z; f[3] = v0.w;
    f[4] = v1.x; f[5] = v1.y; f[6] = v1.z; f[7] = v1.w;
  } else {
    p = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(p[e] << 16);
      f[2 * e + 1] = __uint_as_float(p[e] & 0xffff0000u);
    }
  }
}

// Eight values of a row of x: their sum over the group's lanes (a lane holds
// eight consecutive k), and per term the bf16 operand (f keeps the rest).
template <int GROUP>
__device__ __forceinline__ float q4_group_sum(const float* f) {
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum += f[e];
  sum += SSM_DPP(0.0f, sum, 0xB1, 0xf);                                // quad_perm [1,0,3,2]
  sum += SSM_DPP(0.0f, sum, 0x4E, 0xf);                                // quad_perm [2,3,0,1]
  if constexpr (GROUP >= 64) sum += SSM_DPP(0.0f, sum, 0x141, 0xf);    // row_half_mirror
  if constexpr (GROUP >= 128) sum += SSM_DPP(0.0f, sum, 0x140, 0xf);   // row_mirror
  return sum;
}
__device__ __forceinline__ u32x4_t q4_term(float* f) {
  u32x4_t p;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    p[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
    f[2 * e] -= __uint_as_float(p[e] << 16);
    f[2 * e + 1] -= __uint_as_float(p[e] & 0xffff0000u);
  }
  return q4_pairs(p);
}

// ------------------------------------------------ few rows, x in LDS at once
//
// All of x, its sums and the columns' scales are staged once (q4_fits says where), and
// the wavefronts then walk their pieces of K without a barrier, codes kAhead pieces
// ahead.
constexpr int kFitsBytes = 64 * 1024;
constexpr int kAhead = 4;

// LDS: x [live][pieces * 128 + 8], sums [pieces * 128 / GROUP][16], scales
// [..][16]; the join takes its place.
struct Q4Fit {
  int64_t x, sums, bytes;
};
inline __host__ __device__ Q4Fit q4_fit(int live, int k, int group) {
  Q4Fit f;
  const int64_t wide = (k + 127) / 128 * 128, groups = wide / group;
  f.x = (int64_t)live * (wide + 8) * 2;
  f.sums = f.x + groups * 16 * 4;
  f.bytes = f.sums + groups * 16 * 8;
  const int64_t join = (int64_t)kWaves * 16 * 17 * 4;
  if (f.bytes < join) f.bytes = join;
  return f;
}

template <int GROUP, bool XF32>
__global__ void __launch_bounds__(kThreads, 4) q4_fits_kernel(Q4Args a) {
  constexpr int kTerms = XF32 ? 3 : 1;
  extern __shared__ __attribute__((aligned(16))) char raw[];
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = l & 15, q = l >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int live = a.m * kTerms;                            // rows of LDS in use
  const int groups = a.k / GROUP;
  const int pieces = (a.k + 127) / 128;
  const int wide = pieces * 128, SX = wide + 8;
  const Q4Fit fit = q4_fit(live, a.k, GROUP);
  uint16_t* const sx = reinterpret_cast<uint16_t*>(raw);
  float* const ssum = reinterpret_cast<float*>(raw + fit.x);
  float2* const ssc = reinterpret_cast<float2*>(raw + fit.sums);

  // This lane's row of codes (a column of out); past n the last one again.  A
  // wavefront's pieces are w, w + 8, ..; past its last it loads the row's end
  // again.
  const int mine = (pieces - w + kWaves - 1) / kWaves;
  const uint8_t* const cw = a.codes + min(n0 + lr, (int64_t)a.n - 1) * (a.k / 2);
  u32x4_t code[kAhead];
  auto get_codes = [&](int i) SSM_INLINE {
    return *reinterpret_cast<const u32x4_t*>(cw + min((w + kWaves * i) * 128 + 32 * q, a.k - 32) / 2);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) code[i] = get_codes(i);

  // x, a vector of eight k per thread.  A row's vectors are a multiple of 16 (wide
  // is one of 128), so the lanes that share a group's sum are in one row of x.
  const int vecs = wide / 8;
  for (int v = tid; v < a.m * vecs; v += kThreads) {
    const int row = v / vecs, c = v % vecs;
    float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    u32x4_t p = {0u, 0u, 0u, 0u};
    if (8 * c < a.k) q4_x<XF32>(a.x, (int64_t)row * a.x_row + 8 * c, f, p);
    const float sum = q4_group_sum<GROUP>(f);
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
      const int to = t * a.m + row;
      *reinterpret_cast<u32x4_t*>(&sx[to * SX + 8 * c]) = XF32 ? q4_term(f) : q4_pairs(p);
      if (c % (GROUP / 8) == 0) ssum[c / (GROUP / 8) * 16 + to] = t == 0 ? sum : 0.0f;
    }
  }
  for (int e = tid; e < 16 * groups; e += kThreads) {
    const int c = e / groups, g = e % groups;
    const int64_t at = min(n0 + c, (int64_t)a.n - 1) * groups + g;
    ssc[g * 16 + c] = make_float2(q4_scale(a, q4_scale_bits(a, at)), (float)(16 + (a.zeros != nullptr ? a.zeros[at] : 8)));
  }
  for (int e = 16 * groups + tid; e < 16 * (wide / GROUP); e += kThreads) ssc[e] = make_float2(0.0f, 0.0f);   // past k
  block_sync();

  const uint32_t mask = q4_mask();
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint16_t* const xrow = sx + min(lr, live - 1) * SX;     // rows past the last repeat it
  for (int i0 = 0; i0 < mine; i0 += kAhead) {
#pragma unroll
    for (int ii = 0; ii < kAhead; ++ii) {
      const int i = i0 + ii;
      if (i >= mine) break;
      const u32x4_t c = GROUP < 128 ? q4_transpose(code[ii]) : code[ii];
      if (i + kAhead < mine) code[ii] = get_codes(i + kAhead);
      const int piece = w + kWaves * i;
      f32x4_t d;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        constexpr int kPer = GROUP / 32;       // products per group
        // product j's codes of lane row q: 32 j + 8 q + 0..7 of the piece (groups
        // of 128: 32 q + 8 j + 0..7)
        const bf16x8_t xo = *reinterpret_cast<const bf16x8_t*>(xrow + 128 * piece + (GROUP < 128 ? 32 * j + 8 * q : 32 * q + 8 * j));
        if (j % kPer == 0) d = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, q4_decode(c[j], mask), d, 0, 0, 0);
        if (j % kPer == kPer - 1) {
          const int g = (128 / GROUP) * piece + j / kPer;
          const f32x4_t xs = *reinterpret_cast<const f32x4_t*>(&ssum[g * 16 + 4 * q]);
          const float2 sc = ssc[g * 16 + lr];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(sc.x, __builtin_fmaf(-sc.y, xs[r], d[r]), acc[r]);
        }
      }
    }
  }
  block_sync();
  // Join the wavefronts' parts, in order, and the terms of x.
  float(*part)[16][17] = reinterpret_cast<float(*)[16][17]>(raw);
#pragma unroll
  for (int r = 0; r < 4; ++r) part[w][4 * q + r][lr] = acc[r];
  block_sync();
  for (int e = tid; e < a.m * 16; e += kThreads) {
    const int m = e / 16, c = e % 16;
    if (n0 + c >= a.n) continue;
    float y = 0.0f;
    for (int t = 0; t < kTerms; ++t)
#pragma unroll
      for (int k = 0; k < kWaves; ++k) y += part[k][t * a.m + m][c];
    if (a.bias != nullptr) y += a.bias[n0 + c];
    const int64_t at = (int64_t)m * a.n + n0 + c;
    if (a.out_bf16) Io<uint16_t>::store(a.out, at, y);
    else Io<float>::store(a.out, at, y);
  }
}

// ----------------------------------------------- up to 16 rows, x in slabs
//
// x's slab, its sums and the slab's scales go through LDS, loaded a slab ahead
// into registers, and codes two slabs ahead (each slab of a pair has registers of its
// own: to move a load's result is to wait for it); NH wavefronts share a piece, 32
// columns each.
template <int GROUP, int NH, bool XF32>
__global__ void __launch_bounds__(kThreads, 4) q4_slabs_kernel(Q4Args a) {
  constexpr int kTerms = XF32 ? 3 : 1;
  constexpr int KQ = kWaves / NH;            // 128-wide pieces of a slab
  constexpr int kSlab = 128 * KQ;
  constexpr int kCols = 32 * NH;
  constexpr int kVec = kSlab / 8;            // 16-byte vectors of an x row
  constexpr int SX = kSlab + 8;              // row stride of x in LDS
  constexpr int kG = kSlab / GROUP;          // groups of a slab
  constexpr int kRows = 16;
  constexpr int NX = (q4_rows(1, XF32) * kVec + kThreads - 1) / kThreads;   // x vectors per thread
  constexpr int NS = (kCols * kG + kThreads - 1) / kThreads;   // scales per thread
  struct Lds {
    uint16_t x[kRows * SX] __attribute__((aligned(16)));
    float sum[kG][kRows] __attribute__((aligned(16)));       // groups' sums of x
    float2 sc[kG][kCols];                                     // scale, 16 + zero
  };
  constexpr int kJoin = KQ * kRows * (kCols + 1) * 4;
  __shared__ __attribute__((aligned(16))) char raw[sizeof(Lds) > kJoin ? sizeof(Lds) : kJoin];
  Lds& s = *reinterpret_cast<Lds*>(raw);

  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nh = w % NH, kq = w / NH;
  const int lr = l & 15, q = l >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kCols;
  const int m0 = (int)blockIdx.y * a.rows_per;               // first row of x
  const int mrows = min(a.rows_per, a.m - m0);
  const int live = mrows * kTerms;                          // rows of LDS in use
  const int groups = a.k / GROUP;
  const int slabs = (a.k + kSlab - 1) / kSlab;
  const int64_t kb = a.k / 2;                                // bytes of a row of codes

  // This lane's two rows of codes (columns of out); past n the last one again.
  const uint8_t* cw[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) cw[t] = a.codes + min(n0 + 32 * nh + 16 * t + lr, (int64_t)a.n - 1) * kb;

  u32x4_t code[2][2], xv[NX][XF32 ? 2 : 1];
  uint32_t sv[NS];
  int zv[NS];
  auto get_codes = [&](int slab, u32x4_t* to) SSM_INLINE {
    const int64_t off = min(min(slab, slabs - 1) * kSlab + 128 * kq + 32 * q, a.k - 32) / 2;
#pragma unroll
    for (int t = 0; t < 2; ++t) to[t] = *reinterpret_cast<const u32x4_t*>(cw[t] + off);
  };
  auto issue = [&](int slab) SSM_INLINE {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int v = tid + kThreads * i;
      const int row = v / kVec, k = slab * kSlab + (v % kVec) * 8;
      // (past the row's end, its last vector again: staged as zero)
      const int64_t at = (int64_t)(m0 + min(row, mrows - 1)) * a.x_row + min(k, a.k - 8);
      if constexpr (XF32) {
        const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(a.x) + at);
        xv[i][0] = p[0];
        xv[i][1] = p[1];
      } else {
        xv[i][0] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.x) + at);
      }
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int e = tid + kThreads * i;
      const int c = min(e / kG, kCols - 1), g = min(slab * kG + e % kG, groups - 1);
      const int64_t at = min(n0 + c, (int64_t)a.n - 1) * groups + g;
      sv[i] = q4_scale_bits(a, at);
      zv[i] = a.zeros != nullptr ? a.zeros[at] : 8;
    }
  };
  auto stage = [&](int slab) SSM_INLINE {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int v = tid + kThreads * i;
      const int row = v / kVec, c = v % kVec;
      if (row < mrows) {     // whole wavefronts: a row is one or two of them
        if (slab * kSlab + c * 8 >= a.k) {
#pragma unroll
          for (int e = 0; e < (XF32 ? 2 : 1); ++e) xv[i][e] = u32x4_t{0u, 0u, 0u, 0u};
        }
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (XF32) {
            f[e] = __uint_as_float(xv[i][0][e]);
            f[4 + e] = __uint_as_float(xv[i][1][e]);
          } else {
            f[2 * e] = __uint_as_float(xv[i][0][e] << 16);
            f[2 * e + 1] = __uint_as_float(xv[i][0][e] & 0xffff0000u);
          }
        }
        const float sum = q4_group_sum<GROUP>(f);
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
          const int to = t * mrows + row;      // terms of one row lie mrows apart
          *reinterpret_cast<u32x4_t*>(&s.x[to * SX + c * 8]) = XF32 ? q4_term(f) : q4_pairs(xv[i][0]);
          if (c % (GROUP / 8) == 0) s.sum[c / (GROUP / 8)][to] = t == 0 ? sum : 0.0f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int e = tid + kThreads * i;
      if (e < kCols * kG) s.sc[e % kG][e / kG] = make_float2(q4_scale(a, sv[i]), (float)(16 + zv[i]));
    }
  };

  const uint32_t mask = q4_mask();
  f32x4_t acc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  if (slabs > 0) {
    issue(0);
#pragma unroll
    for (int i = 0; i < 2; ++i) get_codes(i, code[i]);
  }
  auto step = [&](int slab, auto half) SSM_INLINE {
    stage(slab);
    u32x4_t cur[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      cur[t] = GROUP < 128 ? q4_transpose(code[half][t]) : code[half][t];
      asm volatile("" : "+v"(cur[t]));     // (taken before the loads below are issued)
    }
    if (slab + 1 < slabs) issue(slab + 1);
    if (slab + 2 < slabs) get_codes(slab + 2, code[half]);
    block_sync();
    f32x4_t d[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      constexpr int kPer = GROUP / 32;       // products per group
      // product j's codes of lane row q: 32 j + 8 q + 0..7 of the piece (groups
      // of 128: 32 q + 8 j + 0..7)
      const int k = 128 * kq + (GROUP < 128 ? 32 * j + 8 * q : 32 * q + 8 * j);
      const bf16x8_t xo = *reinterpret_cast<const bf16x8_t*>(&s.x[min(lr, live - 1) * SX + k]);   // (rows past the last repeat it)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (j % kPer == 0) d[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, q4_decode(cur[t][j], mask), d[t], 0, 0, 0);
      }
      if (j % kPer == kPer - 1) {
        const int g = 128 * kq / GROUP + j / kPer;
        const f32x4_t xs = *reinterpret_cast<const f32x4_t*>(&s.sum[g][4 * q]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float2 sc = s.sc[g][32 * nh + 16 * t + lr];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_fmaf(sc.x, __builtin_fmaf(-sc.y, xs[r], d[t][r]), acc[t][r]);
        }
      }
    }
    block_sync();
  };
  for (int slab = 0; slab < slabs; slab += 2) {
    step(slab, std::integral_constant<int, 0>());
    if (slab + 1 < slabs) step(slab + 1, std::integral_constant<int, 1>());
  }

  // Join the wavefronts' parts, in order, and the terms of x.
  float(*part)[kRows][kCols + 1] = reinterpret_cast<float(*)[kRows][kCols + 1]>(raw);
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[kq][4 * q + r][32 * nh + 16 * t + lr] = acc[t][r];
  block_sync();
  for (int e = tid; e < mrows * kCols; e += kThreads) {
    const int m = e / kCols, c = e % kCols;
    if (n0 + c >= a.n) continue;
    float y = 0.0f;
    for (int t = 0; t < kTerms; ++t)
#pragma unroll
      for (int k = 0; k < KQ; ++k) y += part[k][t * mrows + m][c];
    if (a.bias != nullptr) y += a.bias[n0 + c];
    const int64_t at = (int64_t)(m0 + m) * a.n + n0 + c;
    if (a.out_bf16) Io<uint16_t>::store(a.out, at, y);
    else Io<float>::store(a.out, at, y);
  }
}

// ---------------------------------------------------------- more rows than 16

constexpr int kWideSlab = 512, kWideCols = 64, kWideSplit = 4;   // k, columns, pieces of a slab
constexpr int kWideThreads = 64 * kWideSplit * (kWideCols / 16);   // a wavefront per piece and 16 columns

// A slab's LDS image: `live` rows of 1024 bytes, 16-byte unit u of row r at
// position u ^ (r & 15) (then 16 rows' reads of one unit use all banks), and the
// groups' sums [kG][kRows], padded to 1024 bytes.
template <int MT, int GROUP>
struct Q4Image {
  static constexpr int kRows = 16 * MT;
  static constexpr int kG = kWideSlab / GROUP;
  static constexpr int kSums = (kG * kRows * 4 + 1023) / 1024;      // units of 1024 bytes
  static __host__ __device__ int64_t bytes(int live) { return (int64_t)(live + kSums) * 1024; }
};

// One vector of eight k per thread, a wavefront per row and slab: x's terms in the
// codes' order and the sums, zero past k.  grid: slabs, rows of x, blocks of rows.
template <int MT, int GROUP, bool XF32>
__global__ void __launch_bounds__(64) q4_rows_kernel(Q4Args a) {
  using I = Q4Image<MT, GROUP>;
  constexpr int kTerms = XF32 ? 3 : 1;
  const int l = threadIdx.x, slab = blockIdx.x, row = blockIdx.y;
  const int m0 = (int)blockIdx.z * a.rows_per;
  const int mrows = min(a.rows_per, a.m - m0);
  if (row >= mrows) return;
  const int64_t image = I::bytes(a.rows_per * kTerms);     // one size for all blocks
  char* to = a.image + ((int64_t)blockIdx.z * gridDim.x + slab) * image;
  const int live = mrows * kTerms;
  const int k = slab * kWideSlab + 8 * l;
  float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  u32x4_t p = {0u, 0u, 0u, 0u};
  if (k < a.k) q4_x<XF32>(a.x, (int64_t)(m0 + row) * a.x_row + k, f, p);
  const float sum = q4_group_sum<GROUP>(f);
  float* const sums = reinterpret_cast<float*>(to + (int64_t)live * 1024);
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    const int r = t * mrows + row;
    *reinterpret_cast<u32x4_t*>(to + (int64_t)r * 1024 + 16 * (l ^ (r & 15))) = XF32 ? q4_term(f) : q4_pairs(p);
    if (l % (GROUP / 8) == 0) sums[l / (GROUP / 8) * I::kRows + r] = t == 0 ? sum : 0.0f;
  }
}

template <int MT, int GROUP>
__global__ void __launch_bounds__(kWideThreads) q4_wide_kernel(Q4Args a) {
  using I = Q4Image<MT, GROUP>;
  constexpr int kRows = I::kRows, kG = I::kG;
  constexpr int NS = kWideCols * kG / kWideThreads;     // scales per thread
  static_assert(NS * kWideThreads == kWideCols * kG || kWideCols * kG < kWideThreads, "scales fill the workgroup");
  constexpr int kS = NS > 0 ? NS : 1;
  struct Lds {
    char x[2][(kRows + I::kSums) * 1024] __attribute__((aligned(1024)));
    float2 sc[2][kG][kWideCols];                    // scale, -(16 + zero) scale
  };
  constexpr int kJoin = kWideSplit * kRows * (kWideCols + 1) * 4;
  static_assert(sizeof(Lds) >= kJoin, "the join fits the slabs' place");
  __shared__ Lds s;

  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nt = w & 3, kq = w >> 2;     // 16-column tile, piece of the slab
  const int lr = l & 15, q = l >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kWideCols;
  const int m0 = (int)blockIdx.y * a.rows_per;
  const int mrows = min(a.rows_per, a.m - m0);
  const int live = mrows * a.terms;
  const int groups = a.k / GROUP;
  const int slabs = (a.k + kWideSlab - 1) / kWideSlab;
  const int64_t kb = a.k / 2;
  const int64_t image = I::bytes(a.rows_per * a.terms);
  const char* img = a.image + (int64_t)blockIdx.y * slabs * image;

  // Workgroups start at different slabs: at one time their rows' codes then lie at
  // different offsets, spread over the memory's channels.
  const int first = (int)blockIdx.x % slabs;
  auto slab_at = [&](int i) SSM_INLINE { return i + first < slabs ? i + first : i + first - slabs; };
  const uint8_t* const cw = a.codes + min(n0 + 16 * nt + lr, (int64_t)a.n - 1) * kb;
  auto get_codes = [&](int i) SSM_INLINE {
    const int slab = slab_at(min(i, slabs - 1));
    return *reinterpret_cast<const u32x4_t*>(cw + min(slab * kWideSlab + 128 * kq + 32 * q, a.k - 32) / 2);
  };
  const int units = live + I::kSums;
  auto load_image = [&](int i, int to) SSM_INLINE {
    const char* from = img + slab_at(i) * image;
    for (int u = w; u < units; u += kWideThreads / 64) load_lds(from + u * 1024, 16u * l, &s.x[to][u * 1024]);
  };
  const int sc_col = tid / kG, sc_g = tid % kG;     // (several per thread: kWideThreads / kG columns apart)
  uint32_t sv[kS];
  int zv[kS];
  auto get_scales = [&](int n) SSM_INLINE {
    const int slab = slab_at(n);
#pragma unroll
    for (int i = 0; i < kS; ++i) {
      const int64_t at = min(n0 + min(sc_col + i * (kWideThreads / kG), kWideCols - 1), (int64_t)a.n - 1) * groups +
                         min(slab * kG + sc_g, groups - 1);
      sv[i] = q4_scale_bits(a, at);
      zv[i] = a.zeros != nullptr ? a.zeros[at] : 8;
    }
  };
  auto put_scales = [&](int to) SSM_INLINE {
#pragma unroll
    for (int i = 0; i < kS; ++i) {
      const int c = sc_col + i * (kWideThreads / kG);
      const float sc = q4_scale(a, sv[i]);
      if (c < kWideCols) s.sc[to][sc_g][c] = make_float2(sc, -(float)(16 + zv[i]) * sc);
    }
  };

  const uint32_t mask = q4_mask();
  f32x4_t acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // This lane's operands of x in a slab: product j's, of row tile m, at
  // at[m] ^ 64 j' (j' = j, or for groups of 128 its place within the unit's bits);
  // rows past the last repeat it.
  uint32_t at[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = min(16 * m + lr, live - 1);
    at[m] = (uint32_t)(row * 1024 + 16 * ((16 * kq + (GROUP < 128 ? q : 4 * q)) ^ (row & 15)));
  }
  constexpr int kPiece = 128 / GROUP;                 // groups of a piece
  const uint32_t sum_at = (uint32_t)(live * 1024 + ((kq * kPiece + (q < kPiece ? q : 0)) * kRows + lr) * 4);
  constexpr uint32_t kHop = GROUP < 128 ? 64 : 16;

  u32x4_t code[2];
  load_image(0, 0);
  get_scales(0);
  put_scales(0);
#pragma unroll
  for (int i = 0; i < 2; ++i) code[i] = get_codes(i);
  loaded<2>();
  block_sync();
  auto step = [&](int slab, auto buffer) SSM_INLINE {
    constexpr int cur = decltype(buffer)::value;
    // This slab's codes are taken out of their loads before the next slab's loads
    // are issued, which the wait for them would otherwise include.
    u32x4_t c = GROUP < 128 ? q4_transpose(code[cur]) : code[cur];
    asm volatile("" : "+v"(c));
    const bool more = slab + 1 < slabs;
    if (more) {
      load_image(slab + 1, cur ^ 1);
      get_scales(slab + 1);
    }
    code[cur] = get_codes(slab + 2);
    const char* const tile = s.x[cur];
    // Four tiles in groups of 32: addresses are computed again in every slab, or they
    // would all be kept, past the registers that there are.
    if constexpr (MT * kG >= 64) {
#pragma unroll
      for (int m = 0; m < MT; ++m) asm volatile("" : "+v"(at[m]));
    }
    // What the codes' 16 and zero points add, taken off for the piece's groups at
    // once: -(16 + zero) scale times the groups' sums, an fp32 product of depth 4
    // (lane row q: group q, where there are so many).
    {
      const int g = kq * kPiece + (q < kPiece ? q : 0);
      const float off = s.sc[cur][g][16 * nt + lr].y;
      const float co = q < kPiece ? off : 0.0f;
      const float* const sums = reinterpret_cast<const float*>(tile + sum_at);
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(sums[16 * m], co, acc[m], 0, 0, 0);
    }
    f32x4_t d[MT];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      constexpr int kPer = GROUP / 32;
      const bf16x8_t wo = q4_decode(c[j], mask);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bf16x8_t xo = *reinterpret_cast<const bf16x8_t*>(tile + (at[m] ^ (kHop * j)));
        if (j % kPer == 0) d[m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        d[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo, wo, d[m], 0, 0, 0);
      }
      if (j % kPer == kPer - 1) {
        const float sc = s.sc[cur][kq * kPiece + j / kPer][16 * nt + lr].x;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][r] = __builtin_fmaf(sc, d[m][r], acc[m][r]);
      }
      if constexpr (MT > 2) __builtin_amdgcn_sched_barrier(0);   // (one product's operands at a time: 128 registers)
    }
    if (more) put_scales(cur ^ 1);
    loaded<1>();       // all but this slab's load of codes
    block_sync();
  };
  for (int slab = 0; slab < slabs; slab += 2) {
    step(slab, std::integral_constant<int, 0>());
    if (slab + 1 < slabs) step(slab + 1, std::integral_constant<int, 1>());
  }

  float(*part)[kRows][kWideCols + 1] = reinterpret_cast<float(*)[kRows][kWideCols + 1]>(&s);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[kq][16 * m + 4 * q + r][16 * nt + lr] = acc[m][r];
  block_sync();
  for (int e = tid; e < mrows * kWideCols; e += kWideThreads) {
    const int m = e / kWideCols, c = e % kWideCols;
    if (n0 + c >= a.n) continue;
    float y = 0.0f;
    for (int t = 0; t < a.terms; ++t)
#pragma unroll
      for (int k = 0; k < kWideSplit; ++k) y += part[k][t * mrows + m][c];
    if (a.bias != nullptr) y += a.bias[n0 + c];
    const int64_t at = (int64_t)(m0 + m) * a.n + n0 + c;
    if (a.out_bf16) Io<uint16_t>::store(a.out, at, y);
    else Io<float>::store(a.out, at, y);
  }
}

// One group per thread: scale = (max - min) / 15 over the group's values and 0,
// rounded to the scales' type; zero = the code of 0; codes to the nearest step.
template <typename Tw>
__global__ void __launch_bounds__(256) q4_quantize_kernel(const Tw* w, uint8_t* codes, void* scales, uint8_t* zeros, int64_t total,
                                                          int group, int scale_bf16) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const Tw* p = w + i * group;
  float lo = 0.0f, hi = 0.0f;
  for (int k = 0; k < group; ++k) {
    const float v = ld_in(p + k);
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
  float sc = (hi - lo) / 15.0f;
  if (scale_bf16) {
    const uint16_t b = f32_to_bf16_rne(sc);
    static_cast<uint16_t*>(scales)[i] = b;
    sc = bf16_to_f32(b);
  } else {
    static_cast<float*>(scales)[i] = sc;
  }
  const float z = sc > 0.0f ? fminf(rintf(-lo / sc), 15.0f) : 8.0f;
  zeros[i] = (uint8_t)z;
  uint8_t* out = codes + i * (group / 2);
  for (int k = 0; k < group; k += 2) {
    uint8_t c[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float v = sc > 0.0f ? rintf(ld_in(p + k + e) / sc) + z : z;
      c[e] = (uint8_t)fminf(fmaxf(v, 0.0f), 15.0f);
    }
    out[k / 2] = (uint8_t)(c[0] | (c[1] << 4));
  }
}

// 16-row tiles of x for a call of m rows, and rows of x per workgroup.
struct Q4Shape {
  int mt, rows_per, terms, slabs, blocks;
};
Q4Shape q4_shape(const Q4Args& a) {
  Q4Shape h{1, 0, a.x_bf16 ? 1 : 3, 0, 0};
  while (h.mt < 4 && q4_rows(h.mt, !a.x_bf16) < a.m) ++h.mt;
  h.rows_per = std::min(a.m, q4_rows(h.mt, !a.x_bf16));
  h.slabs = (a.k + kWideSlab - 1) / kWideSlab;
  h.blocks = (a.m + h.rows_per - 1) / h.rows_per;
  return h;
}

// Columns per workgroup of the form in slabs: 64 where that gives every CU a
// workgroup, else 32.
int q4_slab_cols(const Q4Args& a) { return (int64_t)a.n < 64ll * a.cus ? 32 : 64; }

// All of x in LDS, 16 columns per workgroup: for up to four rows (terms counted;
// each workgroup stages them all), where the workgroups of the form in slabs would
// leave a quarter of their last round of CUs idle or more.  Measured, all of x against
// slabs, one row (microseconds): 2560 x 5120 6.4, 7.3; 10576 x 2560 7.4, 8.4; 20480 x
// 5120 14.5, 17.6; but 8192 x 8192 13.4, 11.4; 16384 x 8192 20.5, 17.0; 65536 x 2560
// 24.5, 19.5.  10576 x 2560 by rows: 2 7.7, 8.4; 4 8.4, 8.8; 8 10.3, 9.2.
bool q4_fits(const Q4Shape& h, const Q4Args& a) {
  const int cols = q4_slab_cols(a);
  const int64_t wgs = ((int64_t)a.n + cols - 1) / cols, places = (wgs + a.cus - 1) / a.cus * a.cus;
  return a.k > 0 && a.m * h.terms <= 4 && 4 * wgs <= 3 * places && q4_fit(a.m * h.terms, a.k, a.group).bytes <= kFitsBytes;
}

template <int GROUP, bool XF32>
void launch_q4_x(const Q4Args& args, const Q4Shape& h, hipStream_t s) {
  Q4Args a = args;
  a.rows_per = h.rows_per;
  a.terms = h.terms;
  if (q4_fits(h, a)) {
    const dim3 grid((unsigned)((a.n + 15) / 16));
    hipLaunchKernelGGL((q4_fits_kernel<GROUP, XF32>), grid, dim3(kThreads), (uint32_t)q4_fit(a.m * h.terms, a.k, GROUP).bytes, s, a);
    return;
  }
  if (h.mt == 1 || a.k == 0) {
    const int nh = q4_slab_cols(a) / 32;
    if (h.mt > 1) a.rows_per = q4_rows(1, XF32);       // (k = 0: the bias alone)
    const dim3 grid((unsigned)((a.n + 32 * nh - 1) / (32 * nh)), (unsigned)((a.m + a.rows_per - 1) / a.rows_per));
    if (nh == 1) hipLaunchKernelGGL((q4_slabs_kernel<GROUP, 1, XF32>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((q4_slabs_kernel<GROUP, 2, XF32>), grid, dim3(kThreads), 0, s, a);
    return;
  }
  const dim3 rows((unsigned)h.slabs, (unsigned)h.rows_per, (unsigned)h.blocks);
  const dim3 grid((unsigned)((a.n + kWideCols - 1) / kWideCols), (unsigned)h.blocks);
  auto run = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    hipLaunchKernelGGL((q4_rows_kernel<MT, GROUP, XF32>), rows, dim3(64), 0, s, a);
    hipLaunchKernelGGL((q4_wide_kernel<MT, GROUP>), grid, dim3(kWideThreads), 0, s, a);
  };
  if (h.mt == 2) run(std::integral_constant<int, 2>());
  else if (h.mt == 3) run(std::integral_constant<int, 3>());
  else run(std::integral_constant<int, 4>());
}

template <int GROUP>
int64_t image_bytes(const Q4Shape& h) {
  const int64_t live = (int64_t)h.rows_per * h.terms;
  const int64_t one = h.mt == 2 ? Q4Image<2, GROUP>::bytes((int)live)
                      : h.mt == 3 ? Q4Image<3, GROUP>::bytes((int)live) : Q4Image<4, GROUP>::bytes((int)live);
  return one * h.slabs * h.blocks;
}

}  // namespace

int64_t q4_image_bytes(const Q4Args& a) {
  const Q4Shape h = q4_shape(a);
  if (h.mt == 1 || a.k == 0) return 0;
  return a.group == 32 ? image_bytes<32>(h) : a.group == 64 ? image_bytes<64>(h) : image_bytes<128>(h);
}

hipError_t launch_q4(const Q4Args& a, hipStream_t s) {
  const Q4Shape h = q4_shape(a);
  if (a.x_bf16) {
    if (a.group == 32) launch_q4_x<32, false>(a, h, s);
    else if (a.group == 64) launch_q4_x<64, false>(a, h, s);
    else launch_q4_x<128, false>(a, h, s);
  } else {
    if (a.group == 32) launch_q4_x<32, true>(a, h, s);
    else if (a.group == 64) launch_q4_x<64, true>(a, h, s);
    else launch_q4_x<128, true>(a, h, s);
  }
  return hipGetLastError();
}

hipError_t launch_q4_quantize(const void* w, bool w_bf16, uint8_t* codes, void* scales, bool scale_bf16, uint8_t* zeros,
                              int64_t groups, int group, hipStream_t s) {
  const dim3 grid((unsigned)((groups + 255) / 256));
  if (w_bf16)
    hipLaunchKernelGGL(q4_quantize_kernel<uint16_t>, grid, dim3(256), 0, s, static_cast<const uint16_t*>(w), codes, scales, zeros,
                       groups, group, scale_bf16 ? 1 : 0);
  else
    hipLaunchKernelGGL(q4_quantize_kernel<float>, grid, dim3(256), 0, s, static_cast<const float*>(w), codes, scales, zeros, groups,
                       group, scale_bf16 ? 1 : 0);
  return hipGetLastError();
}

}  // namespace ssm
