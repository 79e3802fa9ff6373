// The chunk walk of linear attention, shared by the forward and the backward
// (linattn.hip, linattn_bwd.hip).
//
// With cumulative log decays c_i inside a chunk, one walk computes, for rows A,
// sources B and values X of any meaning,
//   out_i = sum_{j <= i} exp(c_i - c_j) (A_i . B_j) X_j + exp(c_i) A_i S
//   S    <- exp(c_end) S + sum_j exp(c_end - c_j) B_j X_j^T
// or, walking back in time (REV), the same with j >= i, the decays
// exp(c_j - c_i), exp(c_end - c_i), exp(c_j), and S arriving from the right.
// Every product of the operator and of its gradients has this form:
//   out: (A, B, X) = (q, k, v)           dq: (dout, v, k)
//   dk, back in time: (v, dout, q)       dv, back in time: (k, q, dout)
//
// Per chunk, on v_mfma_f32_16x16x32_bf16 with fp32 accumulation:
//   G = A B^T;  W = G o decay;  Y = diag(row) A S^T + W X;  S^T += B^T diag(src) X
// A, B and X are bf16 inputs, exact as operands.  Computed operands are fp32 and
// enter as sums of bf16 terms (v's rounding, the rest's rounding, ...): W and the
// state in the readout as two, 2^-18 of the value off, which out's own rounding
// hides; the scaled X of the state update as three, all its bits, since states
// are kept and handed on in fp32.  The readout takes three terms too where the
// decay's gradient comes of it, which adds up differences of such sums.
//
// A workgroup of four wavefronts owns 64 value columns of one (batch row, head)
// and walks its chunks of kLaQ steps; wavefront w holds columns 16 w .. 16 w + 15
// of S^T for the whole sequence in accumulator registers, whose layout is, up to a
// fixed permutation of the contracted index, the operand layout that the readout
// needs.  G and Y are formed transposed (the products' operands swapped): a lane
// then holds one step and four consecutive columns, one wide access to W and out.  Tiles are staged in LDS as they lie in memory; operands contracted over
// time are read with the transposing ds_read_b64_tr_b16.
#ifndef SSMSCAN_LINATTN_KERNEL_H
#define SSMSCAN_LINATTN_KERNEL_H

#include "block.h"
#include "device.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ bf16x8_t la_op(const uint16_t* p) { return *reinterpret_cast<const bf16x8_t*>(p); }

__device__ __forceinline__ bf16x8_t la_op2(const uint16_t* p0, const uint16_t* p1) {
  const bf16x4_t a = *reinterpret_cast<const bf16x4_t*>(p0);
  const bf16x4_t b = *reinterpret_cast<const bf16x4_t*>(p1);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Transposing read: within 16 lanes, lane i gets element i % 4 of the 8-byte
// pieces addressed by lanes 4 e + i / 4, e = 0..3.
__device__ __forceinline__ i16x4_t la_tr(const uint16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(p));
}

// Rows r0 .. r0 + 7 of column c0 + (lane % 16) of a row-major tile.
__device__ __forceinline__ bf16x8_t la_col8(const uint16_t* tile, int stride, int r0, int c0, int l) {
  const int k = l & 15;
  const uint16_t* a0 = tile + (r0 + (k >> 2)) * stride + c0 + 4 * (k & 3);
  const i16x4_t lo = la_tr(a0);
  const i16x4_t hi = la_tr(a0 + 4 * stride);
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ f32x4_t la_mfma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Two fp32 values as sums of N pairs of bf16 terms: a value's rounding, the
// rest's rounding, ...; the first value in the low half.  The rest v - bf16(v) is
// exact in fp32; the two-term dot product forms it in one instruction, from the
// packed pair (a half that is not finite spoils its neighbour's too: they are of
// one value column, which is lost then anyway).
template <int N>
struct LaSplit {
  uint32_t t[N];
};
template <int N>
__device__ __forceinline__ LaSplit<N> la_split(float v0, float v1) {
  LaSplit<N> r;
  // (-1, 0) and (0, -1), kept in registers: as an instruction's own constant, -1.0
  // does not mean the packed pair that the compiler takes it for
  uint32_t first = 0x0000bf80u, second = 0xbf800000u;
  asm("" : "+s"(first), "+s"(second));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    r.t[i] = pack_bf16x2(v0, v1);
    if (i + 1 < N) {
      const bf16x2_t p = __builtin_bit_cast(bf16x2_t, r.t[i]);
      v0 = __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2_t, first), v0, false);
      v1 = __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2_t, second), v1, false);
    }
  }
  return r;
}

// Prefix sums over a wavefront in 64 bits (row shifts, then the rows' totals).
template <int CTRL, int ROWS>
__device__ __forceinline__ double la_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ double la_prefix(double v) {
  v += la_dpp<0x111, 0xf>(v);   // row_shr:1
  v += la_dpp<0x112, 0xf>(v);   // row_shr:2
  v += la_dpp<0x114, 0xf>(v);   // row_shr:4
  v += la_dpp<0x118, 0xf>(v);   // row_shr:8
  v += la_dpp<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
  v += la_dpp<0x143, 0xc>(v);   // row_bcast:31 into rows 2 and 3
  return v;
}

// The sum over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ float la_row_sum(float v) {
  v += SSM_DPP(0.0f, v, 0xB1, 0xf);    // quad_perm [1,0,3,2]
  v += SSM_DPP(0.0f, v, 0x4E, 0xf);    // quad_perm [2,3,0,1]
  v += SSM_DPP(0.0f, v, 0x141, 0xf);   // row_half_mirror
  v += SSM_DPP(0.0f, v, 0x140, 0xf);   // row_mirror
  return v;
}

// The sum over the four rows of 16 lanes, in all of them.
__device__ __forceinline__ float la_rows_sum(float v) {
  const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(t[0]) + __uint_as_float(t[1]);
  const auto u = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(u[0]) + __uint_as_float(u[1]);
}

// Whether the 8-column vector `vec` of a row lies within `dim` columns.
__device__ __forceinline__ bool la_in(int vec, int dim) { return vec * 8 < dim; }

constexpr int kWalkOut = 0;     // the products alone
constexpr int kWalkState = 1;   // no rows and no output: the state at the end of the time chunk
constexpr int kWalkDq = 2;      // with the decay gradient's parts of dq: Z = q
constexpr int kWalkDk = 3;      // ... of dk: Z = k

// LDS of one walk (C: contracted columns, 64 or 128).  What both phases of a
// chunk read is held twice, so that the next chunk is staged while the current
// one's second phase runs.
template <int C, int KIND>
struct LaTile {
  static constexpr int SA = C + 8, SB = C + 16, SX = 64 + 16, SZ = 64 + 8, SW = kLaQ + 8;
  static constexpr bool kZ = KIND == kWalkDq || KIND == kWalkDk;
  static constexpr int kBlk = kLaQ / 16;
  uint16_t B[2][kLaQ * SB] __attribute__((aligned(16)));
  uint16_t X[2][kLaQ * SX] __attribute__((aligned(16)));
  uint16_t A[KIND == kWalkState ? 8 : kLaQ * SA] __attribute__((aligned(16)));
  uint16_t Z[kZ ? kLaQ * SZ : 8] __attribute__((aligned(16)));
  uint16_t W[2][KIND == kWalkState ? 8 : kLaQ * SW] __attribute__((aligned(16)));   // hi, lo
  float cum[2][kLaQ] __attribute__((aligned(16)));   // log2 decay summed from the chunk's first step, inclusive
  float low[2][kLaQ] __attribute__((aligned(16)));   // what it lacks of the 64-bit sum
  float row[2][kLaQ];                                // factor of A S^T
  float src[2][kLaQ] __attribute__((aligned(16)));   // factor of X in the state update
  float end[2];                                      // exp(c_end)
  int bad[2];                                        // the chunk's X holds a value that is not finite
  int badstep[2][64];                                // column's first (REV: last) such step
  float dot[kZ ? 4 : 1][kLaQ];                       // per wavefront: Z . (diag(row) A S^T)
  float rs[KIND == kWalkDq ? kBlk : 1][kLaQ];        // row sums of M by column block
  float cs[KIND == kWalkDq ? kBlk : 1][kLaQ] __attribute__((aligned(16)));   // column sums of M by row block
};

// One walk.  `h`, `b`: head and batch row; `x0`: first value column of the
// slice; `kt`: time chunk.
template <int C, int KIND, bool REV>
__device__ __forceinline__ void la_walk(const LaWalk& a, LaTile<C, KIND>& s, int b, int h, int slice, int kt) {
  using T = LaTile<C, KIND>;
  constexpr int NT = C / 16;                  // 16 x 16 state tiles per wavefront
  constexpr int NB = kLaQ / 16;               // 16-step blocks per chunk
  static_assert(NB == 2, "the products over a chunk's steps are one instruction deep");
  constexpr int NR = kLaQ * C / 8 / 256;      // 16-byte vectors of A and B per thread and chunk
  constexpr int NX = kLaQ * 64 / 8 / 256;     // ... of X and Z
  constexpr bool kOut = KIND != kWalkState;
  constexpr bool kZ = T::kZ;
  constexpr int kTerms = kZ ? 3 : 2;          // bf16 terms of the state in the readout
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = l & 15, q = l >> 4;
  const int x0 = slice * 64;
  const int K = a.n_chunks;
  const int64_t t_begin = (int64_t)kt * a.chunk_len;
  const int64_t L = min(a.chunk_len, a.seqlen - t_begin);
  auto base = [&](const LaOperand& o, int col) SSM_INLINE {
    return o.p + ((int64_t)b * a.seqlen + t_begin) * o.row + (int64_t)(h / o.share) * o.head + col;
  };
  const uint16_t* Ab = kOut ? base(a.A, 0) : nullptr;
  const uint16_t* Bb = base(a.B, 0);
  const uint16_t* Xb = base(a.X, x0);
  const uint16_t* Zb = kZ ? base(a.Z, x0) : nullptr;
  const float* gb = a.decay + (int64_t)b * a.decay_b + t_begin * a.decay_t + h;
  const int xdim = min(64, a.xdim - x0);      // value columns of this slice that exist
  const int p = 16 * w + lr;                  // this lane's value column in the slice

  // Rows of 16-byte vectors; rows past the sequence's last step re-read that step
  // (their X, Z and decay are then zero), columns past the tensor's width read its
  // first vector and are not staged (zero in LDS from the start).  Addresses are
  // a chunk's base, uniform across the workgroup, plus a 32-bit byte offset: one
  // chunk of any tensor spans less than 2^31 bytes (checked on the host).
  struct Bank {
    u32x4_t A[kOut ? NR : 1], B[NR], X[NX], Z[kZ ? NX : 1];
  };
  Bank bank;
  struct Offsets {
    uint32_t A[kOut ? NR : 1], B[NR], X[NX], Z[kZ ? NX : 1];
  };
  auto offsets = [&](int nt) SSM_INLINE {
    Offsets o;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int v = tid + 256 * r;
      const uint32_t row = (uint32_t)min(v / (C / 8), nt - 1), c16 = la_in(v % (C / 8), a.cdim) ? v % (C / 8) * 16u : 0u;
      if constexpr (kOut) o.A[r] = row * ((uint32_t)a.A.row * 2u) + c16;
      o.B[r] = row * ((uint32_t)a.B.row * 2u) + c16;
    }
#pragma unroll
    for (int r = 0; r < NX; ++r) {
      const int v = tid + 256 * r;
      const uint32_t row = (uint32_t)min(v >> 3, nt - 1), c16 = la_in(v & 7, xdim) ? (v & 7) * 16u : 0u;
      o.X[r] = row * ((uint32_t)a.X.row * 2u) + c16;
      if constexpr (kZ) o.Z[r] = row * ((uint32_t)a.Z.row * 2u) + c16;
    }
    return o;
  };
  auto load = [&](int64_t t0, const Offsets& o) SSM_INLINE {
    auto at = [&](const uint16_t* p, const LaOperand& t, uint32_t off) SSM_INLINE {
      return *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(p + t0 * t.row) + off);
    };
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if constexpr (kOut) bank.A[r] = at(Ab, a.A, o.A[r]);
      bank.B[r] = at(Bb, a.B, o.B[r]);
    }
#pragma unroll
    for (int r = 0; r < NX; ++r) {
      bank.X[r] = at(Xb, a.X, o.X[r]);
      if constexpr (kZ) bank.Z[r] = at(Zb, a.Z, o.Z[r]);
    }
  };
  const Offsets whole = offsets(kLaQ);
  auto issue = [&](int64_t t0, int nt) SSM_INLINE {
    if (nt == kLaQ) load(t0, whole);
    else load(t0, offsets(nt));
  };

  auto stage = [&](int nt, int to) SSM_INLINE {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int v = tid + 256 * r;
      const int row = v / (C / 8), c8 = v % (C / 8);
      if (la_in(c8, a.cdim)) {
        if constexpr (kOut) *reinterpret_cast<u32x4_t*>(&s.A[row * T::SA + c8 * 8]) = bank.A[r];
        *reinterpret_cast<u32x4_t*>(&s.B[to][row * T::SB + c8 * 8]) = bank.B[r];
      }
    }
#pragma unroll
    for (int r = 0; r < NX; ++r) {
      const int v = tid + 256 * r;
      const int row = v >> 3, c8 = v & 7;
      if (!la_in(c8, xdim)) continue;
      u32x4_t x = bank.X[r];
      if (nt < kLaQ && row >= nt) {
        x = u32x4_t{0u, 0u, 0u, 0u};
        if constexpr (kZ) bank.Z[r] = x;   // M's rows past the end
      }
      // W is zero where j comes after i, and zero times a value that is not
      // finite is not zero: such values of X are taken out here and put back
      // into the rows and the state that they reach (poison, below)
      auto mag = [&](int e) SSM_INLINE { return __builtin_bit_cast(u16x2_t, x[e] & 0x7fff7fffu); };
      const uint32_t top = __builtin_bit_cast(
          uint32_t, __builtin_elementwise_max(__builtin_elementwise_max(mag(0), mag(1)), __builtin_elementwise_max(mag(2), mag(3))));
      if (((top + 0x00800080u) & 0x80008000u) != 0u) {   // an exponent of all ones
        s.bad[to] = 1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t half = (e & 1) ? 0xffff0000u : 0x0000ffffu;
          if ((x[e >> 1] & half & 0x7f807f80u) == (half & 0x7f807f80u)) {
            if (REV) atomicMax(&s.badstep[to][c8 * 8 + e], row);
            else atomicMin(&s.badstep[to][c8 * 8 + e], row);
            x[e >> 1] &= ~half;
          }
        }
      }
      *reinterpret_cast<u32x4_t*>(&s.X[to][row * T::SX + c8 * 8]) = x;
      if constexpr (kZ) *reinterpret_cast<u32x4_t*>(&s.Z[row * T::SZ + c8 * 8]) = bank.Z[r];
    }
  };

  // The last wavefront sums the decays, a chunk ahead.
  float g = 0.0f;      // this lane's step
  float csum = 0.0f;   // log2 decay of the whole time chunk
  auto get_decay = [&](int64_t t0, int nt) SSM_INLINE { g = gb[(t0 + min(l, nt - 1)) * a.decay_t]; };
  auto sum_decay = [&](int nt, int to) SSM_INLINE {
    // exp2 of anything below -150 is 0 in fp32: decays are held above -160, so
    // that a decay of minus infinity (forget everything) leaves the differences
    // of sums finite.  Sums are held as two floats (from 64 bits): W needs
    // their differences, which one float would give to 2^-24 of the sums only.
    const float one = g * kLog2e;
    const double c = la_prefix(l < nt ? (double)(one < -160.0f ? -160.0f : one) : 0.0);
    const uint64_t cb = __builtin_bit_cast(uint64_t, c);
    const uint32_t e0 = __builtin_amdgcn_readlane((uint32_t)cb, kLaQ - 1);
    const uint32_t e1 = __builtin_amdgcn_readlane((uint32_t)(cb >> 32), kLaQ - 1);
    const double c_end = __builtin_bit_cast(double, (uint64_t)e0 | ((uint64_t)e1 << 32));
    csum += (float)c_end;
    if (l < kLaQ) {
      const float hi = (float)c, rest = (float)(c_end - c);
      s.cum[to][l] = hi;
      s.low[to][l] = (float)(c - (double)hi);
      s.row[to][l] = __builtin_amdgcn_exp2f(REV ? rest : hi) * a.row_scale;
      s.src[to][l] = __builtin_amdgcn_exp2f(REV ? hi : rest) * a.src_scale;
    }
    if (l == 0) s.end[to] = __builtin_amdgcn_exp2f((float)c_end);
  };

  // S^T: tile t holds contracted columns [16 t, 16 t + 16) x this wavefront's 16
  // value columns; register r of a lane is S^T[16 t + 4 q + r][p].  Stored
  // states are [dv][dk], so a walk whose values are k or q reads them
  // transposed (element strides st_x, st_c).
  const int64_t per = (int64_t)a.xdim * a.cdim;
  const int edge = REV ? K - 1 : 0;
  const float* src = kt == edge ? (a.first != nullptr ? a.first + ((int64_t)b * a.nheads + h) * per : nullptr)
                    : KIND == kWalkState ? nullptr
                    : a.chunk_states + ((int64_t)(b * K + (REV ? kt + 1 : kt - 1)) * a.nheads + h) * per;
  // (cdim is a multiple of 8, so four consecutive columns are in or out together)
  const uint32_t sx = (uint32_t)(x0 + p) * (uint32_t)a.st_x;
  f32x4_t accS[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    accS[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const int c = 16 * t + 4 * q;
    if (src != nullptr && p < xdim && c < a.cdim) {
      if (a.st_c == 1) {
        accS[t] = *reinterpret_cast<const f32x4_t*>(src + sx + c);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) accS[t][r] = src[sx + (uint32_t)(c + r) * (uint32_t)a.st_c];
      }
    }
  }

  if (tid < 128) s.badstep[tid >> 6][tid & 63] = REV ? -1 : kLaQ;
  if (tid < 2) s.bad[tid] = 0;
  // columns past the tensors' widths are never staged
  if (a.cdim < C || xdim < 64) {
    for (int e = tid; e < 2 * kLaQ * T::SB; e += 256) s.B[0][e] = 0;
    for (int e = tid; e < 2 * kLaQ * T::SX; e += 256) s.X[0][e] = 0;
    if constexpr (kOut)
      for (int e = tid; e < kLaQ * T::SA; e += 256) s.A[e] = 0;
    if constexpr (kZ)
      for (int e = tid; e < kLaQ * T::SZ; e += 256) s.Z[e] = 0;
  }
  if constexpr (kOut) {
    // W's block beyond the triangle
    for (int e = tid; e < 2 * 256; e += 256) {
      const int k = e >> 8, i = (e >> 4) & 15, j = e & 15;
      s.W[k][(i + (REV ? 16 : 0)) * T::SW + j + (REV ? 0 : 16)] = 0;
    }
  }
  block_sync();

  const int64_t chunks = (L + kLaQ - 1) / kLaQ;
  auto start_of = [&](int64_t ch) SSM_INLINE { return (REV ? chunks - 1 - ch : ch) * kLaQ; };
  auto steps_of = [&](int64_t ch) SSM_INLINE { return (int)min((int64_t)kLaQ, L - start_of(ch)); };
  issue(start_of(0), steps_of(0));
  if (w == 3) {
    get_decay(start_of(0), steps_of(0));
    sum_decay(steps_of(0), 0);
    if (chunks > 1) get_decay(start_of(1), steps_of(1));
  }
  stage(steps_of(0), 0);
  if (chunks > 1) issue(start_of(1), steps_of(1));
  block_sync();
  for (int64_t ch = 0; ch < chunks; ++ch) {
    const int64_t t0 = start_of(ch);
    const int nt = steps_of(ch);
    const int cur = (int)(ch & 1);
    const bool more = ch + 1 < chunks;
    if (w == 3 && more) {
      sum_decay(steps_of(ch + 1), cur ^ 1);
      if (ch + 2 < chunks) get_decay(start_of(ch + 2), steps_of(ch + 2));
    }
    const uint16_t* const tB = s.B[cur];
    const uint16_t* const tX = s.X[cur];

    f32x4_t accY[kOut ? NB : 1];
    if constexpr (kOut) {
      // Phase 1.  The triangle's three 16 x 16 tiles of G, one each for the first
      // three wavefronts (the last one sums decays), transposed: lane (q, lr)
      // holds row i = 16 ib + lr, columns j = 16 jb + 4 q + r.
      const int ib = REV ? (w == 2 ? 1 : 0) : (w == 0 ? 0 : 1);
      const int jb = REV ? (w == 0 ? 0 : 1) : (w == 2 ? 1 : 0);
      const int i = 16 * ib + lr, j0 = 16 * jb + 4 * q;
      if (w < 3) {
        f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < C / 32; ++m)
          acc = la_mfma(la_op(&tB[(16 * jb + lr) * T::SB + 32 * m + 8 * q]), la_op(&s.A[i * T::SA + 32 * m + 8 * q]), acc);
        const float ci = s.cum[cur][i], li = s.low[cur][i];
        const f32x4_t cj = *reinterpret_cast<const f32x4_t*>(&s.cum[cur][j0]);
        const f32x4_t lj = *reinterpret_cast<const f32x4_t*>(&s.low[cur][j0]);
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float d = __builtin_amdgcn_exp2f(REV ? cj[r] - ci + (lj[r] - li) : ci - cj[r] + (li - lj[r])) * a.w_scale;
          v[r] = (REV ? j0 + r >= i : j0 + r <= i) ? acc[r] * d : 0.0f;
        }
        const LaSplit<2> s0 = la_split<2>(v[0], v[1]), s1 = la_split<2>(v[2], v[3]);
        *reinterpret_cast<uint2*>(&s.W[0][i * T::SW + j0]) = make_uint2(s0.t[0], s1.t[0]);
        *reinterpret_cast<uint2*>(&s.W[1][i * T::SW + j0]) = make_uint2(s0.t[1], s1.t[1]);
        if constexpr (KIND == kWalkDq) {
          // M = W o (q k^T) below the diagonal, over this slice's columns of q
          // and k: its row and column sums, in fp32 from exact products
          f32x4_t pk = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int m = 0; m < 2; ++m)
            pk = la_mfma(la_op(&tX[(16 * jb + lr) * T::SX + 32 * m + 8 * q]), la_op(&s.Z[i * T::SZ + 32 * m + 8 * q]), pk);
          float rowsum = 0.0f;
          f32x4_t colsum;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float m = j0 + r < i ? v[r] * pk[r] : 0.0f;
            rowsum += m;
            colsum[r] = la_row_sum(m);
          }
          rowsum = la_rows_sum(rowsum);
          if (q == 0) s.rs[jb][i] = rowsum;
          if (lr == 0) *reinterpret_cast<f32x4_t*>(&s.cs[ib][j0]) = colsum;
        }
      }
      // The entering state as operands of the readout: tiles 2 m and 2 m + 1 give
      // the eight k slots of product m (columns 32 m + 4 q + 0..3 and
      // 32 m + 16 + 4 q + 0..3), and A is read in the same order.
#pragma unroll
      for (int n = 0; n < NB; ++n) accY[n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m = 0; m < C / 32; ++m) {
        u32x4_t t[kTerms];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const f32x4_t& tile = accS[2 * m + r / 2];
          const LaSplit<kTerms> sp = la_split<kTerms>(tile[2 * (r & 1)], tile[2 * (r & 1) + 1]);
#pragma unroll
          for (int e = 0; e < kTerms; ++e) t[e][r] = sp.t[e];
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const uint16_t* arow = &s.A[(16 * n + lr) * T::SA + 32 * m + 4 * q];
          const bf16x8_t av = la_op2(arow, arow + 16);
#pragma unroll
          for (int e = 0; e < kTerms; ++e) accY[n] = la_mfma(__builtin_bit_cast(bf16x8_t, t[e]), av, accY[n]);
        }
      }
      float rowf[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) rowf[n] = s.row[cur][16 * n + lr];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) accY[n][r] *= rowf[n];
      if constexpr (kZ) {
        // Z . readout over this wavefront's 16 columns
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const uint2 z = *reinterpret_cast<const uint2*>(&s.Z[(16 * n + lr) * T::SZ + 16 * w + 4 * q]);
          float d = accY[n][0] * __uint_as_float(z.x << 16);
          d = __builtin_fmaf(accY[n][1], __uint_as_float(z.x & 0xffff0000u), d);
          d = __builtin_fmaf(accY[n][2], __uint_as_float(z.y << 16), d);
          d = __builtin_fmaf(accY[n][3], __uint_as_float(z.y & 0xffff0000u), d);
          d = la_rows_sum(d);
          if (q == 0) s.dot[w][16 * n + lr] = d;
        }
      }
      block_sync();
    }

    // Phase 2: Y += W X, stored; the state moves past the chunk, and the next
    // chunk is staged (A and Z, which only phase 1 reads, in place).
    const bool poison = s.bad[cur] != 0;
    const int bad_at = s.badstep[cur][p];
    const float e_end = s.end[cur];
    const bf16x8_t xo = la_col8(tX, T::SX, 8 * q, 16 * w, l);   // X[8 q .. 8 q + 7][p]
    const f32x4_t f0 = *reinterpret_cast<const f32x4_t*>(&s.src[cur][8 * q]);
    const f32x4_t f1 = *reinterpret_cast<const f32x4_t*>(&s.src[cur][8 * q + 4]);
    bf16x8_t xs[3];
    {
      const u32x4_t xw = __builtin_bit_cast(u32x4_t, xo);
      u32x4_t t[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float g0 = e < 2 ? f0[2 * e] : f1[2 * e - 4], g1 = e < 2 ? f0[2 * e + 1] : f1[2 * e - 3];
        const LaSplit<3> sp = la_split<3>(__uint_as_float(xw[e] << 16) * g0, __uint_as_float(xw[e] & 0xffff0000u) * g1);
#pragma unroll
        for (int k = 0; k < 3; ++k) t[k][e] = sp.t[k];
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) xs[k] = __builtin_bit_cast(bf16x8_t, t[k]);
    }
    if constexpr (kOut) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int n = 0; n < NB; ++n)
          accY[n] = la_mfma(xo, la_op(&s.W[e][(16 * n + lr) * T::SW + 8 * q]), accY[n]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) accS[t][r] *= e_end;
      const bf16x8_t bt = la_col8(tB, T::SB, 8 * q, 16 * t, l);
#pragma unroll
      for (int k = 0; k < 3; ++k) accS[t] = la_mfma(bt, xs[k], accS[t]);
    }
    if (poison && (REV ? bad_at >= 0 : bad_at < kLaQ)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) accS[t][r] = __builtin_nanf("");
    }
    // The next chunk is staged before this one's stores are issued: loads and
    // stores complete in order, and waiting for the loads must not mean waiting
    // for younger stores.
    if (more) stage(steps_of(ch + 1), cur ^ 1);
    if constexpr (kOut) {
      if (poison) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = s.badstep[cur][16 * w + 4 * q + r];
#pragma unroll
          for (int ib = 0; ib < NB; ++ib)
            if (REV ? 16 * ib + lr <= at : 16 * ib + lr >= at) accY[ib][r] = __builtin_nanf("");
        }
      }
      // four consecutive columns of step 16 ib + lr (xdim is a multiple of 8)
      const int64_t o0 = (((int64_t)b * a.seqlen + t_begin + t0) * a.nheads + h) * a.xdim + x0;
      const int py = 16 * w + 4 * q;
      if (py < xdim) {
        auto store = [&](auto type) SSM_INLINE {
          using To = decltype(type);
          char* const base = reinterpret_cast<char*>(static_cast<To*>(a.out) + o0);
          const uint32_t rowb = (uint32_t)a.nheads * (uint32_t)a.xdim * (uint32_t)sizeof(To);
          const uint32_t at = (uint32_t)lr * rowb + (uint32_t)py * (uint32_t)sizeof(To);
#pragma unroll
          for (int ib = 0; ib < NB; ++ib)
            if (nt == kLaQ || 16 * ib + lr < nt) {
              const float y[4] = {accY[ib][0], accY[ib][1], accY[ib][2], accY[ib][3]};
              store_row<To, 4>(reinterpret_cast<To*>(base + (at + 16u * (uint32_t)ib * rowb)), y);
            }
        };
        if (a.out_bf16) store(uint16_t{});
        else store(float{});
      }
      if constexpr (kZ) {
        if (tid < nt) {
          float d = s.dot[0][tid] + s.dot[1][tid] + s.dot[2][tid] + s.dot[3][tid];
          if constexpr (KIND == kWalkDq) {
            float m = 0.0f;
            for (int k = 0; k <= tid >> 4; ++k) m += s.rs[k][tid];
            for (int k = tid >> 4; k < NB; ++k) m -= s.cs[k][tid];
            d += m;
          }
          if (poison) d = __builtin_nanf("");
          a.part[(((int64_t)slice * a.batch + b) * a.nheads + h) * a.seqlen + t_begin + t0 + tid] = d;
        }
      }
    }
    if (ch + 2 < chunks) issue(start_of(ch + 2), steps_of(ch + 2));
    block_sync();
    if (poison) {
      if (tid < 64) s.badstep[cur][tid] = REV ? -1 : kLaQ;
      if (tid == 0) s.bad[cur] = 0;
      block_sync();
    }
  }

  const int far = REV ? 0 : K - 1;
  float* dst = KIND == kWalkState ? a.chunk_out + ((int64_t)(b * K + kt) * a.nheads + h) * per
              : kt == far && a.last != nullptr ? a.last + ((int64_t)b * a.nheads + h) * per : nullptr;
  if (dst != nullptr && p < xdim) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = 16 * t + 4 * q;
      if (c >= a.cdim) continue;
      if (a.st_c == 1) {
        *reinterpret_cast<f32x4_t*>(dst + sx + c) = accS[t];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) dst[sx + (uint32_t)(c + r) * (uint32_t)a.st_c] = accS[t][r];
      }
    }
  }
  if (KIND == kWalkState && slice == 0 && w == 3 && l == 0) a.chunk_decay[(int64_t)(b * K + kt) * a.nheads + h] = csum;
}

// Heads and slots (value slices, or slices of several walks) of a flat grid:
// workgroups go to the eight XCDs in turn, so the slots of one head, which read
// the same rows, are numbered eight apart.
__device__ __forceinline__ void la_place(int f, int heads, int slots, int* bh, int* slot) {
  const int full = heads / 8 * 8 * slots;
  if (f < full) {
    *slot = f / 8 % slots;
    *bh = f / (8 * slots) * 8 + f % 8;
  } else {
    *slot = (f - full) % slots;
    *bh = heads / 8 * 8 + (f - full) / slots;
  }
}

}  // namespace
}  // namespace ssm

#endif  // SSMSCAN_LINATTN_KERNEL_H
