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
// A workgroup of eight wavefronts owns 32 NH columns of W and all of K.  It takes
// K in slabs; x's slab, the groups' sums and the slab's scales go through LDS,
// shared by the wavefronts, which split the slab into 128-wide pieces (and the
// columns in NH parts of 32).  Codes go from HBM to registers, 16 bytes per lane:
// 32 codes of one row, so 16 rows x 128 codes per load.  For groups below 128
// the four lanes of a row exchange words (a 4 x 4 transpose by row swaps), which
// makes every product cover 32 consecutive codes, one group's; for groups of
// 128 the order does not matter and x is read in the same order instead.  Loads
// of the next slab are issued before the current one's arithmetic.
#include <algorithm>

#include "block.h"
#include "device.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;

// Eight codes as bf16 pairs of 16 + code, in the order (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ bf16x8_t q4_decode(uint32_t w) {
  const uint32_t mask = 0x00780078u, base = 0x41804180u;
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

// Rows of x that MT tiles of 16 hold: all of them in bf16, a third in fp32.
constexpr int q4_rows(int mt, bool xf32) { return xf32 ? 16 * mt / 3 : 16 * mt; }

// MT: 16-row tiles of x (its terms counted as rows).
template <int MT, int GROUP, int NH, bool XF32>
__global__ void __launch_bounds__(kThreads, MT <= 2 ? 4 : 2) q4_kernel(Q4Args a) {
  constexpr int kTerms = XF32 ? 3 : 1;
  constexpr int KQ = kWaves / NH;            // 128-wide pieces of a slab
  constexpr int kSlab = 128 * KQ;
  constexpr int kCols = 32 * NH;
  constexpr int kVec = kSlab / 8;            // 16-byte vectors of an x row
  constexpr int SX = kSlab + 8;              // row stride of x in LDS
  constexpr int kG = kSlab / GROUP;          // groups of a slab
  constexpr int kRows = 16 * MT;
  constexpr int NX = (q4_rows(MT, XF32) * kVec + kThreads - 1) / kThreads;   // x vectors per thread
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

  u32x4_t code[2], xv[NX][XF32 ? 2 : 1];
  float sv[NS];
  int zv[NS];
  auto issue = [&](int slab) SSM_INLINE {
    const int k0 = slab * kSlab + 128 * kq + 32 * q;
    const int64_t off = min(k0, a.k - 32) / 2;
#pragma unroll
    for (int t = 0; t < 2; ++t) code[t] = *reinterpret_cast<const u32x4_t*>(cw[t] + off);
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int v = tid + kThreads * i;
      const int row = v / kVec, k = slab * kSlab + (v % kVec) * 8;
      const bool in = row < mrows && k < a.k;
      const int64_t at = in ? (int64_t)(m0 + row) * a.x_row + k : 0;
      if constexpr (XF32) {
        const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(a.x) + at);
        xv[i][0] = in ? p[0] : u32x4_t{0u, 0u, 0u, 0u};
        xv[i][1] = in ? p[1] : u32x4_t{0u, 0u, 0u, 0u};
      } else {
        xv[i][0] = in ? *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.x) + at) : u32x4_t{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int e = tid + kThreads * i;
      const int c = min(e / kG, kCols - 1), g = min(slab * kG + e % kG, groups - 1);
      const int64_t at = min(n0 + c, (int64_t)a.n - 1) * groups + g;
      sv[i] = a.scale_bf16 ? bf16_to_f32(static_cast<const uint16_t*>(a.scales)[at]) : static_cast<const float*>(a.scales)[at];
      zv[i] = a.zeros != nullptr ? a.zeros[at] : 8;
    }
  };
  auto stage = [&]() SSM_INLINE {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int v = tid + kThreads * i;
      const int row = v / kVec, c = v % kVec;
      if (row < mrows) {     // whole wavefronts: a row is one or two of them
        float f[8], sum = 0.0f;
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
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += f[e];
        sum += SSM_DPP(0.0f, sum, 0xB1, 0xf);                                // quad_perm [1,0,3,2]
        sum += SSM_DPP(0.0f, sum, 0x4E, 0xf);                                // quad_perm [2,3,0,1]
        if constexpr (GROUP >= 64) sum += SSM_DPP(0.0f, sum, 0x141, 0xf);    // row_half_mirror
        if constexpr (GROUP >= 128) sum += SSM_DPP(0.0f, sum, 0x140, 0xf);   // row_mirror
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
          u32x4_t p;
          if constexpr (XF32) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
              f[2 * e] -= __uint_as_float(p[e] << 16);
              f[2 * e + 1] -= __uint_as_float(p[e] & 0xffff0000u);
            }
          } else {
            p = xv[i][0];
          }
          // the codes' pair order
          const u32x4_t o = {__builtin_amdgcn_perm(p[2], p[0], 0x05040100u), __builtin_amdgcn_perm(p[2], p[0], 0x07060302u),
                             __builtin_amdgcn_perm(p[3], p[1], 0x05040100u), __builtin_amdgcn_perm(p[3], p[1], 0x07060302u)};
          const int to = t * mrows + row;      // terms of one row lie mrows apart
          *reinterpret_cast<u32x4_t*>(&s.x[to * SX + c * 8]) = o;
          if (c % (GROUP / 8) == 0) s.sum[c / (GROUP / 8)][to] = t == 0 ? sum : 0.0f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int e = tid + kThreads * i;
      if (e < kCols * kG) s.sc[e % kG][e / kG] = make_float2(sv[i], (float)(16 + zv[i]));
    }
  };

  f32x4_t acc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < 2; ++t) acc[m][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  if (slabs > 0) issue(0);
  for (int slab = 0; slab < slabs; ++slab) {
    stage();
    u32x4_t cur[2] = {code[0], code[1]};
    if (slab + 1 < slabs) issue(slab + 1);
    block_sync();
    if constexpr (GROUP < 128) {
#pragma unroll
      for (int t = 0; t < 2; ++t) cur[t] = q4_transpose(cur[t]);
    }
    f32x4_t d[MT][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      constexpr int kPer = GROUP / 32;       // products per group
      // product j's codes of lane row q: 32 j + 8 q + 0..7 of the piece (groups
      // of 128: 32 q + 8 j + 0..7)
      const int k = 128 * kq + (GROUP < 128 ? 32 * j + 8 * q : 32 * q + 8 * j);
      bf16x8_t xo[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = min(16 * m + lr, live - 1);     // rows past the last repeat it
        xo[m] = *reinterpret_cast<const bf16x8_t*>(&s.x[row * SX + k]);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const bf16x8_t wo = q4_decode(cur[t][j]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (j % kPer == 0) d[m][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          d[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xo[m], wo, d[m][t], 0, 0, 0);
        }
      }
      if (j % kPer == kPer - 1) {
        const int g = 128 * kq / GROUP + j / kPer;
        float2 sc[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) sc[t] = s.sc[g][32 * nh + 16 * t + lr];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const f32x4_t xs = *reinterpret_cast<const f32x4_t*>(&s.sum[g][16 * m + 4 * q]);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[m][t][r] = __builtin_fmaf(sc[t].x, __builtin_fmaf(-sc[t].y, xs[r], d[m][t][r]), acc[m][t][r]);
        }
      }
    }
    block_sync();
  }

  // Join the wavefronts' parts, in order, and the terms of x.
  float(*part)[kRows][kCols + 1] = reinterpret_cast<float(*)[kRows][kCols + 1]>(raw);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[kq][16 * m + 4 * q + r][32 * nh + 16 * t + lr] = acc[m][t][r];
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

template <int GROUP, bool XF32>
void launch_q4_g(const Q4Args& a, int mt, int nh, dim3 grid, hipStream_t s) {
  if (mt == 1 && nh == 1) hipLaunchKernelGGL((q4_kernel<1, GROUP, 1, XF32>), grid, dim3(kThreads), 0, s, a);
  else if (mt == 1) hipLaunchKernelGGL((q4_kernel<1, GROUP, 2, XF32>), grid, dim3(kThreads), 0, s, a);
  else if (mt == 2) hipLaunchKernelGGL((q4_kernel<2, GROUP, 2, XF32>), grid, dim3(kThreads), 0, s, a);
  else if (mt == 3) hipLaunchKernelGGL((q4_kernel<3, GROUP, 2, XF32>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((q4_kernel<4, GROUP, 2, XF32>), grid, dim3(kThreads), 0, s, a);
}

template <bool XF32>
void launch_q4_x(const Q4Args& args, hipStream_t s) {
  Q4Args a = args;
  int mt = 1;
  while (mt < 4 && q4_rows(mt, XF32) < a.m) ++mt;
  a.rows_per = q4_rows(mt, XF32);
  // 64 columns per workgroup where that gives every CU one, or where several
  // tiles of x have to be shared by as many columns as possible; else 32
  const int nh = mt == 1 && (int64_t)a.n < 64ll * a.cus ? 1 : 2;
  const dim3 grid((unsigned)((a.n + 32 * nh - 1) / (32 * nh)), (unsigned)((a.m + a.rows_per - 1) / a.rows_per));
  if (a.group == 32) launch_q4_g<32, XF32>(a, mt, nh, grid, s);
  else if (a.group == 64) launch_q4_g<64, XF32>(a, mt, nh, grid, s);
  else launch_q4_g<128, XF32>(a, mt, nh, grid, s);
}

}  // namespace

hipError_t launch_q4(const Q4Args& a, hipStream_t s) {
  if (a.x_bf16) launch_q4_x<false>(a, s);
  else launch_q4_x<true>(a, s);
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
