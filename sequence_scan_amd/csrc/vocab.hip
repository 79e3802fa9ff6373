// gfx950 kernels of libssmscan: cross entropy and distillation against a large
// vocabulary.  Everything large is one kind of product, C = A B^T of two bf16 matrices
// whose rows run along the contracted dimension, on bf16 matrix cores with fp32 sums;
// what differs is what becomes of a tile of C in the registers.
#include <algorithm>

#include "device.h"
#include "model.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float acc4_t __attribute__((ext_vector_type(4)));

constexpr int kK = 64;            // contracted elements in a stage: rows of 128 bytes
constexpr int kTile = kVocabTile;   // rows and columns of a workgroup's tile of C

// A bf16 matrix whose rows run along the contracted dimension.
struct Side {
  const uint16_t* p;
  int64_t ld;       // elements between rows
  int32_t rows;
};

// A wavefront's load of 64 x 16 bytes straight to LDS through a buffer descriptor:
// lane l's go to `to` + 16 l, and a lane whose offset lies past the buffer's end
// leaves zeros.
__device__ __forceinline__ void load_lds16(i32x4_t buffer, uint32_t off, uint32_t to) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(off), "s"(buffer)
      : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)static_cast<const char*>(p);
}

// The descriptor of `rows` rows from row r0 on: reads past the last row's end give 0.
__device__ __forceinline__ i32x4_t buffer_of(const Side& m, int64_t r0, int rows, int k) {
  const uint64_t base = (uint64_t)(uintptr_t)(m.p + r0 * m.ld);
  const int64_t left = m.rows - r0 < rows ? m.rows - r0 : rows;
  const uint32_t bytes = left > 0 ? (uint32_t)(((left - 1) * m.ld + k) * 2) : 0;
  i32x4_t d;
  d.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
  d.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xffff);
  d.z = __builtin_amdgcn_readfirstlane((int)bytes);
  d.w = 0x00020000;     // raw, 32-bit elements
  return d;
}

// A workgroup of 2 x 4 wavefronts computes a 256 x 256 tile of C, a wavefront 128 x 64
// of it.  A stage holds 64 contracted elements of the tile's 256 + 256 rows (64 KB), of
// which there are two: one is multiplied while the other arrives.
//
// In LDS a row's eight 16-byte pieces are permuted: piece c of row r is at place
// c ^ ((r >> 1) & 7).  A matrix operand takes one piece of each of 16 rows, which then
// meet all 64 banks once.
struct Stages {
  alignas(1024) char a[2][kTile * kK * 2];
  alignas(1024) char b[2][kTile * kK * 2];
};

// acc[mi][ni][i]: C[wm * 128 + mi * 16 + (lane & 15)][wn * 64 + ni * 16 + 4 * (lane >> 4) + i].
typedef acc4_t Acc[8][4];

__device__ __forceinline__ void multiply(const Side& A, const Side& B, int64_t m0, int64_t n0, int k, Stages& s, Acc acc) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const i32x4_t ba = buffer_of(A, m0, kTile, k), bb = buffer_of(B, n0, kTile, k);
  // a wavefront loads rows wave * 32 .. + 31 of either side, eight at a time
  const int row = wave * 32 + (lane >> 3);
  const int c = (lane & 7) ^ ((lane >> 4) & 3);         // of rows 0..7 of 16; rows 8..15 differ in bit 2
  uint32_t oa[4], ob[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t piece = (uint32_t)(c ^ ((j & 1) << 2)) * 16;
    oa[j] = (uint32_t)((row + j * 8) * A.ld * 2) + piece;
    ob[j] = (uint32_t)((row + j * 8) * B.ld * 2) + piece;
  }
  const uint32_t la = lds_address(s.a[0]) + wave * 4096, lb = lds_address(s.b[0]) + wave * 4096;
  constexpr uint32_t kStage = kTile * kK * 2;
  auto load = [&](int k0, int stage) SSM_INLINE {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int piece = k0 + (c ^ ((j & 1) << 2)) * 8;
      const uint32_t past = piece < k ? 0 : 0x80000000u;      // (descriptors end below 2^31)
      load_lds16(ba, (oa[j] + k0 * 2) | past, la + stage * kStage + j * 1024);
      load_lds16(bb, (ob[j] + k0 * 2) | past, lb + stage * kStage + j * 1024);
    }
  };
#pragma unroll
  for (int mi = 0; mi < 8; ++mi)
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) acc[mi][ni] = acc4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int at = (lane & 15) * 128 + (((lane >> 4) ^ ((lane & 15) >> 1)) & 7) * 16;
  load(0, 0);
  const int stages = (k + kK - 1) / kK;
  for (int t = 0; t < stages; ++t) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    block_sync();
    if (t + 1 < stages) load((t + 1) * kK, (t + 1) & 1);
    const char* pa = s.a[t & 1] + wm * 128 * 128;
    const char* pb = s.b[t & 1] + wn * 64 * 128;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      bf16x8_t fa[8], fb[4];
#pragma unroll
      for (int ni = 0; ni < 4; ++ni) fb[ni] = *reinterpret_cast<const bf16x8_t*>(pb + ni * 2048 + (at ^ (kk * 64)));
#pragma unroll
      for (int mi = 0; mi < 8; ++mi) fa[mi] = *reinterpret_cast<const bf16x8_t*>(pa + mi * 2048 + (at ^ (kk * 64)));
#pragma unroll
      for (int mi = 0; mi < 8; ++mi)
#pragma unroll
        for (int ni = 0; ni < 4; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[ni], fa[mi], acc[mi][ni], 0, 0, 0);
    }
  }
}

// The tile of C that a workgroup computes.  Workgroups go round the eight XCDs, whose
// L2s are their own: each XCD gets a run of tiles, in groups of eight rows of tiles that
// go through the columns together, so that the 32 tiles under way read 8 + 4 panels.
__device__ __forceinline__ void tile_place(int tiles_m, int tiles_n, int* m, int* n) {
  const int total = tiles_m * tiles_n, id = blockIdx.x;
  const int each = total >> 3, rest = total & 7, xcd = id & 7;
  const int t = xcd * each + (xcd < rest ? xcd : rest) + (id >> 3);
  const int group = t / (8 * tiles_n), first = group * 8;
  const int high = tiles_m - first < 8 ? tiles_m - first : 8;
  const int in = t - first * tiles_n;
  *m = first + in % high;
  *n = in / high;
}

// ----------------------------------------------------------------- the forward

// For every 256 columns a row's maximum and sum of exponentials (base 2), and the
// target's logit where it lies in them.
template <bool ONE>
__global__ void __launch_bounds__(512, 2) vocab_stats_kernel(VocabArgs a, float2* __restrict__ stats, float* __restrict__ picked,
                                                             int tiles_m, int tiles_n) {
  __shared__ Stages s;
  int tm, tn;
  tile_place(tiles_m, tiles_n, &tm, &tn);
  const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;
  Acc acc;
  multiply(Side{a.x, a.x_row, a.rows}, Side{a.w, a.w_row, a.vocab}, m0, n0, a.width, s, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave >> 2, wn = wave & 3;
  const int n = wn * 64 + 4 * (lane >> 4);          // + ni * 16 + i
  const int columns = (int)(a.vocab - n0 < kTile ? a.vocab - n0 : kTile);
  block_sync();
  float2* part = reinterpret_cast<float2*>(s.a[0]);      // [4][256]
#pragma unroll
  for (int mi = 0; mi < 8; ++mi) {
    const int m = wm * 128 + mi * 16 + (lane & 15);
    float top = -__builtin_inff();
#pragma unroll
    for (int ni = 0; ni < 4; ++ni)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float z = n + ni * 16 + i < columns ? acc[mi][ni][i] * a.scale : -__builtin_inff();
        acc[mi][ni][i] = z;
        top = __builtin_fmaxf(top, z);
      }
    if constexpr (ONE) {
      if (m0 + m < a.rows) {
        const int64_t d = a.index[m0 + m] - n0 - n;
        if (d >= 0 && d < 64 && (d & 12) == 0) {
          float z = 0.0f;
#pragma unroll
          for (int ni = 0; ni < 4; ++ni)
#pragma unroll
            for (int i = 0; i < 4; ++i) z = d == ni * 16 + i ? acc[mi][ni][i] : z;
          if (n0 + n + d < a.vocab) picked[m0 + m] = z;
        }
      }
    }
    top = __builtin_fmaxf(top, __shfl_xor(top, 16));
    top = __builtin_fmaxf(top, __shfl_xor(top, 32));
    const float top2 = top == -__builtin_inff() ? 0.0f : top * kLog2e;
    float sum = 0.0f;
#pragma unroll
    for (int ni = 0; ni < 4; ++ni)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[mi][ni][i], kLog2e, -top2));
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (lane < 16) part[wn * 256 + m] = make_float2(top2, sum);
  }
  block_sync();
  const int m = threadIdx.x;
  if (m < kTile && m0 + m < a.rows) {
    float2 r = part[m];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float2 o = part[w * 256 + m];
      if (w * 64 < columns) {
        const float top = __builtin_fmaxf(r.x, o.x);
        r.y = r.y * __builtin_amdgcn_exp2f(r.x - top) + o.y * __builtin_amdgcn_exp2f(o.x - top);
        r.x = top;
      }
    }
    stats[(int64_t)tn * a.rows + m0 + m] = r;
  }
}

// The logits at a row's indices, one wavefront for each.
__global__ void __launch_bounds__(256) vocab_pick_kernel(VocabArgs a) {
  const int64_t e = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (e >= (int64_t)a.rows * a.top) return;
  const int64_t v = a.index[e];
  float z = 0.0f;
  if (v >= 0 && v < a.vocab) {
    const uint16_t* x = a.x + e / a.top * a.x_row;
    const uint16_t* w = a.w + v * a.w_row;
    for (int k = lane * 8; k < a.width; k += 512) {
      float xv[8], wv[8];
      Vec16<uint16_t>::unpack(*reinterpret_cast<const uint4*>(x + k), xv);
      Vec16<uint16_t>::unpack(*reinterpret_cast<const uint4*>(w + k), wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) z = __builtin_fmaf(xv[i], wv[i], z);
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) z += __shfl_xor(z, o);
    z *= a.scale;
  }
  if (lane == 0) a.logits[e] = z;
}

// What one row's indices and teacher logits say, over a wavefront: whether the row
// counts (an index that is in the vocabulary and not without weight), whether an index
// lies past the vocabulary, and the softmax of the teacher's.
struct Teacher {
  bool counts, past;
  float top2, sum;      // of the teacher's logits over the temperature, in base 2
};
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const float w = __shfl_xor(v, o);
    v = v != v ? v : (w != w ? w : __builtin_fmaxf(v, w));     // (a NaN stays)
  }
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ Teacher teacher_of(const VocabArgs& a, int64_t row, int lane) {
  const float t2 = kLog2e / a.temperature;
  Teacher t;
  float top = -__builtin_inff();
  bool past = false;
  for (int k = lane; k < a.top; k += 64) {
    const int64_t v = a.index[row * a.top + k];
    past |= v >= a.vocab;
    if (v >= 0) {
      const float l = a.teacher[row * a.top + k] * t2;
      top = top != top ? top : (l != l ? l : __builtin_fmaxf(top, l));
    }
  }
  t.top2 = wave_max(top);
  t.past = __any(past);
  t.counts = !t.past && t.top2 != -__builtin_inff();
  float sum = 0.0f;
  for (int k = lane; k < a.top; k += 64)
    if (a.index[row * a.top + k] >= 0) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(a.teacher[row * a.top + k], t2, -t.top2));
  t.sum = wave_sum(sum);
  return t;
}

// A row's log sum of exponentials from its pieces', and its loss: a wavefront a row.
template <bool ONE>
__global__ void __launch_bounds__(256) vocab_loss_kernel(VocabArgs a, const float2* __restrict__ stats,
                                                         const float* __restrict__ picked, int tiles_n) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= a.rows) return;
  float top = -__builtin_inff();
  for (int n = lane; n < tiles_n; n += 64) {
    const float v = stats[(int64_t)n * a.rows + row].x;
    top = top != top ? top : (v != v ? v : __builtin_fmaxf(top, v));
  }
  top = wave_max(top);
  float sum = 0.0f;
  for (int n = lane; n < tiles_n; n += 64) {
    const float2 v = stats[(int64_t)n * a.rows + row];
    sum = __builtin_fmaf(v.y, __builtin_amdgcn_exp2f(v.x - top), sum);
  }
  sum = wave_sum(sum);
  // top is the largest logit in base 2, of which ln 2 gives back its value to an ulp
  const float lse = __builtin_fmaf(top, kLn2, __builtin_amdgcn_logf(sum) * kLn2);
  float loss = 0.0f;
  if constexpr (ONE) {
    const int64_t v = a.index[row];
    if (v >= a.vocab) loss = __builtin_nanf("");
    else if (v >= 0) loss = (lse - picked[row]) + a.z_loss * lse * lse;
  } else {
    const Teacher t = teacher_of(a, row, lane);
    if (t.past) loss = __builtin_nanf("");
    else if (t.counts) {
      const float t2 = kLog2e / a.temperature;
      const float logsum = __builtin_amdgcn_logf(t.sum);
      for (int k = lane; k < a.top; k += 64) {
        const float l2 = __builtin_fmaf(a.teacher[row * a.top + k], t2, -t.top2) - logsum;     // log2 q
        const float q = __builtin_amdgcn_exp2f(l2);
        if (a.index[row * a.top + k] >= 0 && q != 0.0f)
          loss = __builtin_fmaf(q, __builtin_fmaf(l2, kLn2, lse - a.logits[row * a.top + k]), loss);
      }
      loss = wave_sum(loss) * a.temperature * a.temperature;
    }
  }
  if (lane == 0) {
    a.lse[row] = lse;
    a.loss[row] = loss;
  }
}

// ---------------------------------------------------------------- the gradients

// What a row's dz is formed from: dz = soft exp2(z log2 e - lse2) less hard q at its
// indices.  soft = hard = 0 for a row that takes no part.
struct RowGrad {
  float lse2, soft, hard;
  int32_t target;       // cross entropy: its column, or -1
};

template <bool ONE>
__global__ void __launch_bounds__(256) vocab_rows_kernel(VocabArgs a, RowGrad* __restrict__ rows) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= a.rows) return;
  RowGrad g{0.0f, 0.0f, 0.0f, -1};
  const float lse = a.lse_in[row];
  if constexpr (ONE) {
    const int64_t v = a.index[row];
    if (v >= 0 && v < a.vocab) {
      const float d = a.dloss[row] * a.scale;
      g = RowGrad{lse * kLog2e, d * __builtin_fmaf(2.0f * a.z_loss, lse, 1.0f), d, (int32_t)v};
    }
  } else {
    // (a.scale is over the temperature: its square leaves one of them)
    const float d = a.dloss[row] * a.temperature * a.temperature * a.scale;
    if (teacher_of(a, row, lane).counts) g = RowGrad{lse * kLog2e, d, d, -1};
    else g.target = -2;
  }
  if constexpr (ONE) {
    if (g.target < 0) g.target = -2;
  }
  if (lane == 0) rows[row] = g;
}

// dst[c][r] = src[r][c] for r below `rows` and c below `cols`, 0 for r from there to
// dst_rows (its padded length), and for the rows that take no part.
__global__ void __launch_bounds__(256) vocab_transpose_kernel(const uint16_t* __restrict__ src, int64_t src_ld, int rows, int cols,
                                                              uint16_t* __restrict__ dst, int64_t dst_ld,
                                                              const RowGrad* __restrict__ takes) {
  __shared__ uint16_t t[64][66];
  const int r0 = blockIdx.x * 64, c0 = blockIdx.y * 64;
  const int i = threadIdx.x & 63, j = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int r = r0 + j + k * 4, c = c0 + i;
    const bool in = r < rows && c < cols && (!takes || takes[r].target != -2);
    t[j + k * 4][i] = in ? src[(int64_t)r * src_ld + c] : 0;
  }
  block_sync();
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int c = c0 + j + k * 4, r = r0 + i;
    if (c < cols && r < dst_ld) dst[(int64_t)c * dst_ld + r] = t[i][j + k * 4];
  }
}

// dz of a piece of the vocabulary from the logits, computed once more, as [rows, ldz]
// and as [columns, ldt] (each padded with zeros).
__global__ void __launch_bounds__(512, 2) vocab_dz_kernel(VocabArgs a, const RowGrad* __restrict__ rows, int64_t v0, int columns,
                                                          uint16_t* __restrict__ dz, int64_t ldz, uint16_t* __restrict__ dzt,
                                                          int64_t ldt, int tiles_m, int tiles_n) {
  __shared__ Stages s;
  int tm, tn;
  tile_place(tiles_m, tiles_n, &tm, &tn);
  const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;
  Acc acc;
  multiply(Side{a.x, a.x_row, a.rows}, Side{a.w + v0 * a.w_row, a.w_row, columns}, m0, n0, a.width, s, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave >> 2, wn = wave & 3;
  const float s2 = a.scale * kLog2e;
#pragma unroll
  for (int mi = 0; mi < 8; ++mi) {
    const int64_t m = m0 + wm * 128 + mi * 16 + (lane & 15);
    RowGrad g{0.0f, 0.0f, 0.0f, -2};
    if (m < a.rows) g = rows[m];
    const int64_t target = g.target < 0 ? -1 : g.target - v0;
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) {
      const int64_t n = n0 + wn * 64 + ni * 16 + 4 * (lane >> 4);
      float d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = g.soft * __builtin_amdgcn_exp2f(__builtin_fmaf(acc[mi][ni][i], s2, -g.lse2));
        d[i] = g.target == -2 || n + i >= columns ? 0.0f : p - (n + i == target ? g.hard : 0.0f);
      }
      const uint32_t lo = pack_bf16x2(d[0], d[1]), hi = pack_bf16x2(d[2], d[3]);
      if (m < a.rows && n < ldz) *reinterpret_cast<uint2*>(dz + m * ldz + n) = make_uint2(lo, hi);
      if (m < ldt) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < columns) dzt[(n + i) * ldt + m] = (uint16_t)((i < 2 ? lo : hi) >> ((i & 1) * 16));
      }
    }
  }
}

// Distillation: dz at the teacher's indices, formed from the stored logits in place of
// the rounded softmax.
__global__ void __launch_bounds__(256) vocab_fix_kernel(VocabArgs a, const RowGrad* __restrict__ rows, int64_t v0, int columns,
                                                        uint16_t* __restrict__ dz, int64_t ldz, uint16_t* __restrict__ dzt, int64_t ldt) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= a.rows) return;
  const RowGrad g = rows[row];
  if (g.target == -2) return;
  const Teacher t = teacher_of(a, row, lane);
  const float t2 = kLog2e / a.temperature, by = 1.0f / t.sum;
  const int64_t at = row * a.top;
  for (int k = lane; k < a.top; k += 64) {
    const int64_t n = a.index[at + k] - v0;
    if (n < 0 || n >= columns) continue;
    float q = 0.0f;
    for (int j = 0; j < a.top; ++j)
      if (a.index[at + j] == a.index[at + k]) q += __builtin_amdgcn_exp2f(__builtin_fmaf(a.teacher[at + j], t2, -t.top2));
    const float p = g.soft * __builtin_amdgcn_exp2f(__builtin_fmaf(a.logits_in[at + k], kLog2e, -g.lse2));
    const uint16_t d = f32_to_bf16_rne(p - g.hard * q * by);
    dz[row * ldz + n] = d;
    dzt[n * ldt + row] = d;
  }
}

// out (or sum) = [sum +] A B^T: a piece's part of dx, and dweight.
__global__ void __launch_bounds__(512, 2) vocab_product_kernel(Side A, Side B, int k, float* __restrict__ sum, bool first, bool last,
                                                               uint16_t* __restrict__ out, int64_t ld, int tiles_m, int tiles_n) {
  __shared__ Stages s;
  int tm, tn;
  tile_place(tiles_m, tiles_n, &tm, &tn);
  const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;
  Acc acc;
  multiply(A, B, m0, n0, k, s, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave >> 2, wn = wave & 3;
#pragma unroll
  for (int mi = 0; mi < 8; ++mi) {
    const int64_t m = m0 + wm * 128 + mi * 16 + (lane & 15);
    if (m >= A.rows) continue;
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) {
      const int64_t n = n0 + wn * 64 + ni * 16 + 4 * (lane >> 4);
      if (n >= B.rows) continue;
      float4 v = make_float4(acc[mi][ni][0], acc[mi][ni][1], acc[mi][ni][2], acc[mi][ni][3]);
      if (!first) {
        const float4 o = *reinterpret_cast<const float4*>(sum + m * ld + n);
        v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
      }
      if (last) *reinterpret_cast<uint2*>(out + m * ld + n) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      else *reinterpret_cast<float4*>(sum + m * ld + n) = v;
    }
  }
}

int64_t tiles(int64_t n) { return (n + kTile - 1) / kTile; }
int64_t padded(int64_t n) { return (n + kK - 1) / kK * kK; }

// Consecutive parts of the workspace.
struct Parts {
  int64_t bytes = 0;
  int64_t add(int64_t n) {
    const int64_t at = bytes;
    bytes += (n + 255) / 256 * 256;
    return at;
  }
};

struct FwdParts : Parts {
  int64_t stats, picked;
  explicit FwdParts(const VocabArgs& a) {
    stats = add(tiles(a.vocab) * a.rows * 8);
    picked = add(a.teacher ? 0 : (int64_t)a.rows * 4);
  }
};

struct BwdParts : Parts {
  int64_t rows, xt, wt, dz, dzt, sum;
  int64_t piece, ldz, ldt;
  explicit BwdParts(const VocabArgs& a) {
    piece = std::min(vocab_piece(a), (int64_t)a.vocab);
    ldz = padded(piece);
    ldt = padded(a.rows);
    rows = add((int64_t)a.rows * (int64_t)sizeof(RowGrad));
    xt = add(a.dw ? a.width * ldt * 2 : 0);
    wt = add(a.dx ? a.width * ldz * 2 : 0);
    dz = add(a.rows * ldz * 2);
    dzt = add(piece * ldt * 2);
    sum = add(a.dx && piece < a.vocab ? (int64_t)a.rows * a.width * 4 : 0);
  }
};

unsigned fours(int64_t n) { return (unsigned)((n + 3) / 4); }

}  // namespace

int64_t vocab_piece(const VocabArgs& a) {
  // (past kVocabMaxLd columns a tile of the transposed weights would not fit a descriptor)
  const int64_t each = std::min<int64_t>(kVocabMaxLd, kVocabPieceBytes / 2 / std::max(1, a.rows));
  return std::max<int64_t>(kTile, each / kTile * kTile);
}

int64_t vocab_fwd_bytes(const VocabArgs& a) { return FwdParts(a).bytes; }
int64_t vocab_bwd_bytes(const VocabArgs& a) { return BwdParts(a).bytes; }

hipError_t launch_vocab_fwd(const VocabArgs& a, hipStream_t s) {
  const FwdParts at(a);
  float2* stats = reinterpret_cast<float2*>(a.work + at.stats);
  float* picked = reinterpret_cast<float*>(a.work + at.picked);
  const int tm = (int)tiles(a.rows), tn = (int)tiles(a.vocab);
  const bool one = a.teacher == nullptr;
  auto k = one ? vocab_stats_kernel<true> : vocab_stats_kernel<false>;
  hipLaunchKernelGGL(k, dim3((unsigned)(tm * tn)), dim3(512), 0, s, a, stats, picked, tm, tn);
  if (!one)
    hipLaunchKernelGGL(vocab_pick_kernel, dim3(fours((int64_t)a.rows * a.top)), dim3(256), 0, s, a);
  auto l = one ? vocab_loss_kernel<true> : vocab_loss_kernel<false>;
  hipLaunchKernelGGL(l, dim3(fours(a.rows)), dim3(256), 0, s, a, stats, picked, tn);
  return hipGetLastError();
}

hipError_t launch_vocab_bwd(const VocabArgs& a, hipStream_t s) {
  const BwdParts at(a);
  RowGrad* rows = reinterpret_cast<RowGrad*>(a.work + at.rows);
  uint16_t* xt = reinterpret_cast<uint16_t*>(a.work + at.xt);
  uint16_t* wt = reinterpret_cast<uint16_t*>(a.work + at.wt);
  uint16_t* dz = reinterpret_cast<uint16_t*>(a.work + at.dz);
  uint16_t* dzt = reinterpret_cast<uint16_t*>(a.work + at.dzt);
  float* sum = reinterpret_cast<float*>(a.work + at.sum);
  const bool one = a.teacher == nullptr;
  auto rk = one ? vocab_rows_kernel<true> : vocab_rows_kernel<false>;
  hipLaunchKernelGGL(rk, dim3(fours(a.rows)), dim3(256), 0, s, a, rows);
  const unsigned wide = (unsigned)((a.width + 63) / 64);
  if (a.dw)
    hipLaunchKernelGGL(vocab_transpose_kernel, dim3((unsigned)(at.ldt / 64), wide), dim3(256), 0, s, a.x, a.x_row, a.rows, a.width,
                       xt, at.ldt, rows);
  const int tm = (int)tiles(a.rows), td = (int)tiles(a.width);
  for (int64_t v0 = 0; v0 < a.vocab; v0 += at.piece) {
    const int columns = (int)std::min<int64_t>(at.piece, a.vocab - v0);
    const int64_t ldz = padded(columns);
    const int tn = (int)tiles(columns);
    hipLaunchKernelGGL(vocab_dz_kernel, dim3((unsigned)(tm * tn)), dim3(512), 0, s, a, rows, v0, columns, dz, ldz, dzt, at.ldt,
                       tm, tn);
    if (!one) hipLaunchKernelGGL(vocab_fix_kernel, dim3(fours(a.rows)), dim3(256), 0, s, a, rows, v0, columns, dz, ldz, dzt, at.ldt);
    if (a.dx) {
      hipLaunchKernelGGL(vocab_transpose_kernel, dim3((unsigned)(ldz / 64), wide), dim3(256), 0, s, a.w + v0 * a.w_row, a.w_row,
                         columns, a.width, wt, ldz, (const RowGrad*)nullptr);
      hipLaunchKernelGGL(vocab_product_kernel, dim3((unsigned)(tm * td)), dim3(512), 0, s, Side{dz, ldz, a.rows},
                         Side{wt, ldz, a.width}, (int)ldz, sum, v0 == 0, v0 + columns == a.vocab, a.dx, (int64_t)a.width, tm, td);
    }
    if (a.dw)
      hipLaunchKernelGGL(vocab_product_kernel, dim3((unsigned)(tn * td)), dim3(512), 0, s, Side{dzt, at.ldt, columns},
                         Side{xt, at.ldt, a.width}, (int)at.ldt, sum, true, true, a.dw + v0 * a.width, (int64_t)a.width, tn, td);
  }
  return hipGetLastError();
}

}  // namespace ssm
