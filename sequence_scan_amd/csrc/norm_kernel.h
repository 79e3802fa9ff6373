// The norm kernels' template, instantiated by norm_add.hip and norm_gate.hip.
//
// A norm runs over `width` consecutive channels of one row.  All of them are
// held in registers, eight per lane and step, so that every tensor is read and
// written once:
//   forward:  r (= alpha res + scale x, or x, or x silu(z)) -> m, v in fp32
//             -> n = (r - m) / sqrt(v + eps) -> n w + b (silu(z)) -> out
//   backward: with u = dy w, one round of sums S1 = sum (r - m)^2 and
//             S2 = sum u (r - m) gives both 1 / std and mean(u n):
//             dr = (u - [mean u] - (r - m) S2 / (W std^2)) / std
// Memory is what bounds it: a few operations per element against 4 to 20 bytes.
// Measured (PyTorch's copy of 1 GiB runs at 5.2 TB/s, the library's streaming probe at
// 6.5): add norm of 16384 x 2560, bf16 into an fp32 residual, 96 us, 5.3 TB/s, its
// backward with all three column sums 142 + 5 us, 5.2 TB/s; gated norm of 16384 x 5120
// 103 us, 4.9 TB/s; the backward over 80 heads of 64 162 + 4 us, 5.1 TB/s.  One row of 2560
// takes 2.2 us, a launch's own time.
//
// Two layouts.  Up to 512 channels, T lanes of a wavefront (8, 16, 32 or 64)
// hold one norm, and the sums stay within the wavefront (DPP and the row
// swaps); up to 1024, a whole wavefront does, with two steps per lane.  A
// wavefront then covers 64 / T norms: neighbouring groups of one row first,
// which are contiguous in memory, rows after that.  Above 1024, a workgroup of
// up to 16 wavefronts holds one norm and joins its wavefronts' sums in LDS.
// Workgroups walk the rows with the stride of the grid, 8 (backward: 4, whose column
// sums are a row of workspace each) of four wavefronts per CU.
//
// Widths need not be multiples of eight: the last active lane's eight channels
// end at the width and overlap its neighbour's; the repeated ones are left out
// of the sums and the stores.  Widths below eight take one predicated lane
// (TINY).  gfx950 reads and writes 16 bytes at any
// element-aligned address, so rows and groups may start anywhere.
#ifndef SSMSCAN_NORM_KERNEL_H
#define SSMSCAN_NORM_KERNEL_H

#include "block.h"
#include "device.h"

namespace ssm {
namespace {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Eight consecutive elements at any element-aligned address, as fp32.
__device__ __forceinline__ void get8(const float* p, float* o) {
  const u32x4_any a = *reinterpret_cast<const u32x4_any*>(p);
  const u32x4_any b = *reinterpret_cast<const u32x4_any*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = __uint_as_float(a[i]);
    o[4 + i] = __uint_as_float(b[i]);
  }
}
__device__ __forceinline__ void get8(const uint16_t* p, float* o) {
  const u32x4_any a = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(a[i] << 16);
    o[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void put8(float* p, const float* v) {
  u32x4_any a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __float_as_uint(v[i]);
    b[i] = __float_as_uint(v[4 + i]);
  }
  *reinterpret_cast<u32x4_any*>(p) = a;
  *reinterpret_cast<u32x4_any*>(p + 4) = b;
}
__device__ __forceinline__ void put8(uint16_t* p, const float* v) {
  u32x4_any a;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<u32x4_any*>(p) = a;
}

// Eight elements as they are, and their values: apart, for loads a row ahead.
template <typename T>
struct Raw8 {
  u32x4_any q[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = *reinterpret_cast<const u32x4_any*>(p + 4 * i);
  }
  __device__ __forceinline__ void values(float* o) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) o[i] = __uint_as_float(q[i / 4][i % 4]);
      else o[i] = __uint_as_float((i & 1) ? q[0][i / 2] & 0xffff0000u : q[0][i / 2] << 16);
    }
  }
};

// Up to eight elements (TINY: the first n, the rest 0).
template <bool TINY, typename T>
__device__ __forceinline__ void get(const T* p, int n, float* o) {
  if constexpr (!TINY) {
    get8(p, o);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = j < n ? ld_in(p + j) : 0.0f;
  }
}
// The lane's own ones of eight: without the first dup, which its neighbour stores.
template <bool TINY, typename T>
__device__ __forceinline__ void put(T* p, int n, int dup, const float* v) {
  if (!TINY && dup == 0) {
    put8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= dup && j < n) st_in(p + j, v[j]);
  }
}
template <bool TINY>
__device__ __forceinline__ void put_as(bool bf16, void* p, int64_t i, int n, int dup, const float* v) {
  if (bf16) put<TINY>(static_cast<uint16_t*>(p) + i, n, dup, v);
  else put<TINY>(static_cast<float*>(p) + i, n, dup, v);
}
template <bool TINY>
__device__ __forceinline__ void get_as(bool bf16, const void* p, int64_t i, int n, float* v) {
  if (bf16) get<TINY>(static_cast<const uint16_t*>(p) + i, n, v);
  else get<TINY>(static_cast<const float*>(p) + i, n, v);
}

// The sum over aligned groups of T lanes, in every lane of the group.  All
// lanes of a group are active together.
template <int T>
__device__ __forceinline__ float lanes_sum(float v) {
  v += SSM_DPP(0.0f, v, 0xB1, 0xf);                            // quad_perm [1,0,3,2]
  v += SSM_DPP(0.0f, v, 0x4E, 0xf);                            // quad_perm [2,3,0,1]
  v += SSM_DPP(0.0f, v, 0x141, 0xf);                           // row_half_mirror
  if constexpr (T >= 16) v += SSM_DPP(0.0f, v, 0x140, 0xf);    // row_mirror
  if constexpr (T >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (T >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// 1 / sqrt(v).  The instruction takes values below the smallest normal number as zero,
// and a row's mean square may lie there where eps does (below 1.2e-38).
__device__ __forceinline__ float norm_rsqrt(float v) {
  const bool small = v < 0x1p-100f;
  const float r = __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v);
  return small ? r * 0x1p32f : r;
}

constexpr int kNormWaves = 4;    // wavefronts per workgroup of the wavefront layout

// Where a lane works.  T > 0: the wavefront layout; T == 0: the workgroup
// layout.
template <int T, int NV, bool TINY>
struct NormPlace {
  int e0[NV];      // first channel of step v, within the group
  int dup[NV];     // leading channels of it that another lane also holds (8: none are this lane's)
  bool on[NV];     // the lane holds channels in step v
  int g;           // group
  bool glive;      // g exists
  int64_t row0;    // first row of the wavefront (T > 0) or workgroup
  int rslot;       // row offset of the lane
  int64_t step;
  __device__ explicit NormPlace(const NormArgs& a, int gs) {
    int lane;
    if constexpr (T > 0) {
      const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      const int rs = 64 / T / gs;
      lane = l % T;
      const int gw = blockIdx.y * gs + (l / T) % gs;
      glive = gw < a.groups;
      g = min(gw, a.groups - 1);
      rslot = l / (T * gs);
      row0 = ((int64_t)blockIdx.x * kNormWaves + w) * rs;
      step = (int64_t)gridDim.x * kNormWaves * rs;
    } else {
      lane = threadIdx.x;
      g = blockIdx.y;
      glive = true;
      rslot = 0;
      row0 = blockIdx.x;
      step = gridDim.x;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = 8 * (lane + v * (T > 0 ? T : (int)blockDim.x));
      on[v] = e < a.width;
      e0[v] = TINY ? 0 : min(e, a.width - 8);
      dup[v] = on[v] ? e - e0[v] : 8;
    }
  }
  // Channel j of step v is this lane's (n: the width, where it is below eight).
  __device__ __forceinline__ bool own(int v, int j, int n) const {
    return j >= dup[v] && (!TINY || j < n);
  }
};

// Sums of M values over the norm's lanes, in every one of them.
template <int T, int M>
struct NormSum {
  int par = 0;
  __device__ __forceinline__ void operator()(float* v) {
    if constexpr (T > 0) {
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] = lanes_sum<T>(v[m]);
    } else {
      // two sets of slots in turn: a wavefront can be one round ahead of the
      // slowest reader, never two
      __shared__ float slots[2][M][16];
      const int w = threadIdx.x >> 6, nw = blockDim.x >> 6;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        v[m] = lanes_sum<64>(v[m]);
        if ((threadIdx.x & 63) == 0) slots[par][m][w] = v[m];
      }
      block_sync();
#pragma unroll
      for (int m = 0; m < M; ++m) {
        float s = 0.0f;
        for (int i = 0; i < nw; ++i) s += slots[par][m][i];
        v[m] = s;
      }
      par ^= 1;
    }
  }
};

constexpr int kModeAdd = 0, kModeGate = 1, kModeGateLast = 2;   // gate before or after the norm

// Forward.  Tx: type of x and z; Tr: type of the residual stream (add).
template <int MODE, typename Tx, typename Tr, int T, int NV, bool TINY>
__global__ void __launch_bounds__(T > 0 ? 64 * kNormWaves : 1024) norm_fwd_kernel(NormArgs a, int gs) {
  const NormPlace<T, NV, TINY> at(a, gs);
  NormSum<T, 1> total;
  const bool ragged = TINY || (a.width & 7) != 0;
  const float inv_w = 1.0f / (float)a.width;
  const int64_t wide = (int64_t)a.groups * a.width;
  const int64_t gbase = (int64_t)at.g * a.width;
  const Tx* x = static_cast<const Tx*>(a.x) + gbase;
  const Tx* z = static_cast<const Tx*>(a.z);
  if (MODE != kModeAdd && z != nullptr) z += gbase;
  const Tr* res = static_cast<const Tr*>(a.res);
  const float* bias = a.bias ? a.bias + gbase : nullptr;
  const int n = TINY ? a.width : 8;
  float w[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[v][j] = 1.0f;
    if (a.w != nullptr) get<TINY>(a.w + gbase + at.e0[v], n, w[v]);
  }
  // In the workgroup layout a row's loads are issued a row ahead: its wavefronts wait
  // for each other in every row, and would all wait for memory after that (gated norm
  // of 16384 x 5120: 114 us without, 103 with; the add norm, which stores twice as
  // much as it loads ahead, has gained little or lost: 65536 x 1280 182, 194).
  constexpr bool kAhead = T == 0 && MODE != kModeAdd;
  Raw8<Tx> nx, nz;
  auto fetch = [&](int64_t row) SSM_INLINE {
    nx.load(x + row * a.x_stride + at.e0[0]);
    if (z != nullptr) nz.load(z + row * a.z_stride + at.e0[0]);
  };
  if constexpr (kAhead)
    if (at.row0 < a.rows) fetch(at.row0);
  for (int64_t base = at.row0; base < a.rows; base += at.step) {
    const int64_t row = min(base + at.rslot, a.rows - 1);
    const bool live = T == 0 || (base + at.rslot < a.rows && at.glive);
    // every load of the row first
    float r[NV][8], gate[NV][8], xv[NV][8], zr[NV][8];
    if constexpr (kAhead) {
      static_assert(NV == 1, "one step per lane");
      nx.values(xv[0]);
      if (z != nullptr) nz.values(zr[0]);
      if (base + at.step < a.rows) fetch(base + at.step);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        get<TINY>(x + row * a.x_stride + at.e0[v], n, xv[v]);
        if constexpr (MODE != kModeAdd)
          if (z != nullptr) get<TINY>(z + row * a.z_stride + at.e0[v], n, zr[v]);
      }
      if constexpr (MODE == kModeAdd) {
        if (res != nullptr) {
#pragma unroll
          for (int v = 0; v < NV; ++v) get<TINY>(res + row * wide + at.e0[v], n, r[v]);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (MODE == kModeAdd) {
        if (a.scale != nullptr) {
          float sc[8];
          get<TINY>(a.scale + at.e0[v], n, sc);
#pragma unroll
          for (int j = 0; j < 8; ++j) xv[v][j] *= sc[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[v][j] = res != nullptr ? __builtin_fmaf(a.alpha, r[v][j], xv[v][j]) : xv[v][j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          gate[v][j] = z != nullptr ? silu_f(zr[v][j]) : 1.0f;
          r[v][j] = MODE == kModeGate ? xv[v][j] * gate[v][j] : xv[v][j];
        }
      }
    }
    float mean = 0.0f;
    if (a.center) {
      float m[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) m[0] += at.own(v, j, n) ? r[v][j] : 0.0f;
      total(m);
      mean = m[0] * inv_w;
    }
    float sq[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float t = 0.0f;
      if (ragged) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float k = at.own(v, j, n) ? r[v][j] - mean : 0.0f;
          t = __builtin_fmaf(k, k, t);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float k = r[v][j] - mean;
          t = __builtin_fmaf(k, k, t);
        }
      }
      sq[0] += at.on[v] ? t : 0.0f;
    }
    total(sq);
    const float rstd = norm_rsqrt(__builtin_fmaf(sq[0], inv_w, a.eps));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t at0 = row * wide + gbase + at.e0[v];
      if constexpr (MODE == kModeAdd) {
        if (a.res_out != nullptr && live && at.on[v]) put<TINY>(static_cast<Tr*>(a.res_out) + at0, n, at.dup[v], r[v]);
      }
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = (r[v][j] - mean) * rstd * w[v][j];
      if (bias != nullptr) {
        float bv[8];
        get<TINY>(bias + at.e0[v], n, bv);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] += bv[j];
      }
      if constexpr (MODE == kModeGateLast) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= gate[v][j];
      }
      if (live && at.on[v]) put_as<TINY>(a.out_bf16, a.out, at0, n, at.dup[v], y);
    }
  }
}

// Backward.  Add: Tx is the type of dout, Tr of the residual stream; gate: Tx is
// the type of x and z, Tr of dout.  Column sums stay in registers over the
// workgroup's rows and leave as one row of a.part.
template <int MODE, typename Tx, typename Tr, int T, int NV, bool TINY>
__global__ void __launch_bounds__(T > 0 ? 64 * kNormWaves : 1024) norm_bwd_kernel(NormArgs a, int gs) {
  const NormPlace<T, NV, TINY> at(a, gs);
  NormSum<T, 2> total;
  const bool ragged = TINY || (a.width & 7) != 0;
  const float inv_w = 1.0f / (float)a.width;
  const int64_t wide = (int64_t)a.groups * a.width;
  const int64_t gbase = (int64_t)at.g * a.width;
  using Td = typename std::conditional<MODE == kModeAdd, Tx, Tr>::type;
  const Td* dout = static_cast<const Td*>(a.dout) + gbase;
  const Tx* x = static_cast<const Tx*>(a.x);
  const Tx* z = static_cast<const Tx*>(a.z);
  if constexpr (MODE != kModeAdd) {
    x += gbase;
    if (z != nullptr) z += gbase;
  }
  const float* bias = a.bias ? a.bias + gbase : nullptr;
  const int n = TINY ? a.width : 8;
  float w[NV][8], cw[NV][8], cb[NV][8], cs[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[v][j] = 1.0f;
      cw[v][j] = cb[v][j] = cs[v][j] = 0.0f;
    }
    if (a.w != nullptr) get<TINY>(a.w + gbase + at.e0[v], n, w[v]);
  }
  // (as in the forward: gated 16384 x 5120 184 us without, 167 with; the add norm's
  // three column sums leave too few registers, 16384 x 2560 131, 172)
  constexpr bool kAhead = T == 0 && MODE != kModeAdd;
  Raw8<Td> nd;
  Raw8<Tx> nx, nz;
  auto fetch = [&](int64_t row) SSM_INLINE {
    nd.load(dout + row * wide + at.e0[0]);
    nx.load(x + row * a.x_stride + at.e0[0]);
    if (z != nullptr) nz.load(z + row * a.z_stride + at.e0[0]);
  };
  if constexpr (kAhead)
    if (at.row0 < a.rows) fetch(at.row0);
  for (int64_t base = at.row0; base < a.rows; base += at.step) {
    const int64_t row = min(base + at.rslot, a.rows - 1);
    const bool live = T == 0 || (base + at.rslot < a.rows && at.glive);
    float x_[NV][8], dy_[NV][8], gate[NV][8], slope[NV][8];
    if constexpr (kAhead) {
      static_assert(NV == 1, "one step per lane");
      nd.values(dy_[0]);
      nx.values(x_[0]);
      if (z != nullptr) nz.values(gate[0]);
      if (base + at.step < a.rows) fetch(base + at.step);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        get<TINY>(dout + row * wide + at.e0[v], n, dy_[v]);
        if constexpr (MODE == kModeAdd) {
          get<TINY>(static_cast<const Tr*>(a.res) + row * wide + at.e0[v], n, x_[v]);
        } else {
          get<TINY>(x + row * a.x_stride + at.e0[v], n, x_[v]);
          if (z != nullptr) get<TINY>(z + row * a.z_stride + at.e0[v], n, gate[v]);
        }
      }
    }
    if constexpr (MODE != kModeAdd) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (z != nullptr) {
            const float sg = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-gate[v][j] * kLog2e));
            gate[v][j] *= sg;                                            // silu
            slope[v][j] = __builtin_fmaf(gate[v][j], 1.0f - sg, sg);     // its derivative
          } else {
            gate[v][j] = 1.0f;
            slope[v][j] = 0.0f;
          }
        }
    }
    // the normed value, and the gradient at the norm's output
    auto rv = [&](int v, int j) SSM_INLINE { return MODE == kModeGate ? x_[v][j] * gate[v][j] : x_[v][j]; };
    auto dv = [&](int v, int j) SSM_INLINE { return MODE == kModeGateLast ? dy_[v][j] * gate[v][j] : dy_[v][j]; };
    float mu = 0.0f, mean = 0.0f;
    if (a.center) {
      float m[2] = {0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m[0] += at.own(v, j, n) ? rv(v, j) : 0.0f;
          m[1] += at.own(v, j, n) ? dv(v, j) * w[v][j] : 0.0f;
        }
      total(m);
      mean = m[0] * inv_w;
      mu = m[1] * inv_w;
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float t0 = 0.0f, t1 = 0.0f;
      if (ragged) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float k = at.own(v, j, n) ? rv(v, j) - mean : 0.0f;
          t0 = __builtin_fmaf(k, k, t0);
          t1 = __builtin_fmaf(k, at.own(v, j, n) ? dv(v, j) * w[v][j] : 0.0f, t1);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float k = rv(v, j) - mean;
          t0 = __builtin_fmaf(k, k, t0);
          t1 = __builtin_fmaf(k, dv(v, j) * w[v][j], t1);
        }
      }
      s[0] += at.on[v] ? t0 : 0.0f;
      s[1] += at.on[v] ? t1 : 0.0f;
    }
    total(s);
    const float rstd = norm_rsqrt(__builtin_fmaf(s[0], inv_w, a.eps));
    const float c = rstd * (rstd * s[1] * inv_w);     // (the square alone could overflow)
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float d[8], y[8];   // dr; the normed row
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float k = rv(v, j) - mean;
        y[j] = k * rstd;
        d[j] = rstd * (dv(v, j) * w[v][j] - mu - k * c);
      }
      if (live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          cw[v][j] = __builtin_fmaf(dv(v, j), y[j], cw[v][j]);
          cb[v][j] += dv(v, j);
        }
      }
      const int64_t at0 = row * wide + gbase + at.e0[v];
      if constexpr (MODE == kModeAdd) {
        if (a.dres != nullptr) {
          float dr[8];
          get<TINY>(static_cast<const Tr*>(a.dres) + at0, n, dr);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += dr[j];
        }
        if (a.sums == 3) {
          float xv[8];
          get_as<TINY>(a.x_bf16, a.x, row * a.x_stride + at.e0[v], n, xv);
          if (live) {
#pragma unroll
            for (int j = 0; j < 8; ++j) cs[v][j] = __builtin_fmaf(xv[j], d[j], cs[v][j]);
          }
        }
        if (a.res_out != nullptr) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = a.alpha * d[j];
          if (live && at.on[v]) put<TINY>(static_cast<Tr*>(a.res_out) + at0, n, at.dup[v], o);
        }
        if (a.out != nullptr) {
          if (a.scale != nullptr) {
            float sc[8];
            get<TINY>(a.scale + at.e0[v], n, sc);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] *= sc[j];
          }
          if (live && at.on[v]) put_as<TINY>(a.x_bf16, a.out, at0, n, at.dup[v], d);
        }
      } else {
        float dz[8];
        if constexpr (MODE == kModeGateLast) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] *= w[v][j];
          if (bias != nullptr) {
            float bv[8];
            get<TINY>(bias + at.e0[v], n, bv);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += bv[j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) dz[j] = dy_[v][j] * y[j] * slope[v][j];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dz[j] = d[j] * x_[v][j] * slope[v][j];
            d[j] *= gate[v][j];
          }
        }
        if (live && at.on[v]) {
          put<TINY>(static_cast<Tx*>(a.out) + at0, n, at.dup[v], d);
          if (z != nullptr) put<TINY>(static_cast<Tx*>(a.dz) + at0, n, at.dup[v], dz);
        }
      }
    }
  }
  if (a.part == nullptr) return;
  // One row of column sums per workgroup.  In the wavefront layout the row
  // slots of a wavefront (lanes T * gs apart) and then the wavefronts are added.
  float* part = a.part + (int64_t)blockIdx.x * a.sums * wide + gbase;
  if constexpr (T == 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (at.on[v]) {
        put<TINY>(part + at.e0[v], n, at.dup[v], cw[v]);
        put<TINY>(part + wide + at.e0[v], n, at.dup[v], cb[v]);
        if (a.sums == 3) put<TINY>(part + 2 * wide + at.e0[v], n, at.dup[v], cs[v]);
      }
  } else {
    __shared__ float slots[kNormWaves][64][8 * NV + 1];
    const int l = threadIdx.x & 63, wv = threadIdx.x >> 6;
    auto join = [&](float (&c)[NV][8], int k) SSM_INLINE {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) slots[wv][l][8 * v + j] = c[v][j];
      block_sync();
      if (wv == 0 && l < T * gs && at.glive) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (at.on[v]) {
            float t[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float sum = 0.0f;
              for (int q = 0; q < kNormWaves; ++q)
                for (int m = l; m < 64; m += T * gs) sum += slots[q][m][8 * v + j];
              t[j] = sum;
            }
            put<TINY>(part + k * wide + at.e0[v], n, at.dup[v], t);
          }
      }
      block_sync();
    };
    join(cw, 0);
    join(cb, 1);
    if (a.sums == 3) join(cs, 2);
  }
}

// ------------------------------------------------------------------- launches

// The layout by width alone: T lanes per norm up to 512 channels (and two steps
// per lane up to 1024), a workgroup of ceil(width / 512) wavefronts above.
struct NormShape {
  int t;        // lanes per norm, 0: the workgroup layout
  int nv;
  int threads;
  int gs;       // groups side by side in a wavefront
  dim3 grid;
};

inline NormShape norm_shape(const NormArgs& a, int per_cu) {
  NormShape s{};
  const int n8 = (a.width + 7) / 8;
  s.t = n8 <= 8 ? 8 : n8 <= 16 ? 16 : n8 <= 32 ? 32 : n8 <= 128 ? 64 : 0;
  s.gs = 1;
  if (s.t > 0) {
    s.nv = n8 <= 64 ? 1 : 2;
    s.threads = 64 * kNormWaves;
    while (2 * s.gs * s.t <= 64 && s.gs < a.groups) s.gs *= 2;
    const int rows_per = kNormWaves * (64 / s.t / s.gs);
    const int gy = (a.groups + s.gs - 1) / s.gs;
    const int64_t most = std::max<int64_t>(1, (int64_t)a.cus * per_cu / gy);
    s.grid = dim3((unsigned)std::max<int64_t>(1, std::min({(a.rows + rows_per - 1) / rows_per, most, (int64_t)kNormMaxBlocks})),
                  (unsigned)gy);
  } else {
    s.nv = 1;
    const int waves = (n8 + 63) / 64;
    s.threads = 64 * waves;
    const int64_t most = std::max<int64_t>(1, (int64_t)a.cus * std::max(1, per_cu * kNormWaves / waves) / a.groups);
    s.grid = dim3((unsigned)std::max<int64_t>(1, std::min({a.rows, most, (int64_t)kNormMaxBlocks})), (unsigned)a.groups);
  }
  return s;
}

#define SSM_NORM_LAUNCH(T, NV, TINY)                                                                              \
  hipLaunchKernelGGL((KERN<MODE, Tx, Tr, T, NV, TINY>), sh.grid, dim3((unsigned)sh.threads), 0, s, a, sh.gs)
#define SSM_NORM_DISPATCH()                                   \
  do {                                                        \
    if (a.width < 8) SSM_NORM_LAUNCH(8, 1, true);             \
    else if (sh.t == 8) SSM_NORM_LAUNCH(8, 1, false);         \
    else if (sh.t == 16) SSM_NORM_LAUNCH(16, 1, false);       \
    else if (sh.t == 32) SSM_NORM_LAUNCH(32, 1, false);       \
    else if (sh.t == 64 && sh.nv == 1) SSM_NORM_LAUNCH(64, 1, false); \
    else if (sh.t == 64) SSM_NORM_LAUNCH(64, 2, false);       \
    else SSM_NORM_LAUNCH(0, 1, false);                        \
  } while (0)

constexpr int kNormFwdPerCu = 8, kNormBwdPerCu = 4;   // workgroups of four wavefronts per CU that walk the rows

template <int MODE, typename Tx, typename Tr>
void launch_norm_fwd_t(const NormArgs& a, hipStream_t s) {
#define KERN norm_fwd_kernel
  const NormShape sh = norm_shape(a, kNormFwdPerCu);
  SSM_NORM_DISPATCH();
#undef KERN
}
template <int MODE, typename Tx, typename Tr>
void launch_norm_bwd_t(const NormArgs& a, hipStream_t s) {
#define KERN norm_bwd_kernel
  const NormShape sh = norm_shape(a, kNormBwdPerCu);
  SSM_NORM_DISPATCH();
#undef KERN
}

}  // namespace
}  // namespace ssm

#endif  // SSMSCAN_NORM_KERNEL_H
