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
// A, B and X are bf16 inputs, exact as operands; W, the scaled X and the state
// are fp32 and enter as two bf16 operands, hi = bf16(v) and lo = bf16(v - hi).
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

struct LaSplit {
  uint32_t hi, lo;
};
__device__ __forceinline__ LaSplit la_split(float v0, float v1) {
  const uint32_t hi = pack_bf16x2(v0, v1);
  return {hi, pack_bf16x2(v0 - __uint_as_float(hi << 16), v1 - __uint_as_float(hi & 0xffff0000u))};
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

// LDS of one walk (C: contracted columns, 64 or 128).
template <int C, int KIND>
struct LaTile {
  static constexpr int SA = C + 8, SB = C + 16, SP = 64 + 8, SW = kLaQ + 8;
  static constexpr bool kZ = KIND == kWalkDq || KIND == kWalkDk;
  static constexpr int kBlk = kLaQ / 16;
  uint16_t B[kLaQ * SB] __attribute__((aligned(16)));
  uint16_t X[kLaQ * SP] __attribute__((aligned(16)));
  uint16_t A[KIND == kWalkState ? 8 : kLaQ * SA] __attribute__((aligned(16)));
  uint16_t Z[kZ ? kLaQ * SP : 8] __attribute__((aligned(16)));
  uint16_t W[2][KIND == kWalkState ? 8 : kLaQ * SW] __attribute__((aligned(16)));   // hi, lo
  float cum[kLaQ] __attribute__((aligned(16)));   // cumulative log2 decay from the chunk's first step, inclusive
  float row[kLaQ];          // factor of A S^T
  float src[kLaQ] __attribute__((aligned(16)));   // factor of X in the state update
  float end;                // exp(c_end)
  int bad;                  // the chunk's X holds a value that is not finite
  int badstep[64];          // column's first (REV: last) such step
  float dot[kZ ? 4 : 1][kLaQ];                              // per wavefront: Z . (diag(row) A S^T)
  float rs[KIND == kWalkDq ? kBlk : 1][kLaQ];               // row sums of M by column block
  float cs[KIND == kWalkDq ? kBlk : 1][kLaQ] __attribute__((aligned(16)));               // column sums of M by row block
};

// One walk.  `h`, `b`: head and batch row; `x0`: first value column of the
// slice; `kt`: time chunk.
template <int C, int KIND, bool REV>
__device__ __forceinline__ void la_walk(const LaWalk& a, LaTile<C, KIND>& s, int b, int h, int slice, int kt) {
  using T = LaTile<C, KIND>;
  constexpr int NT = C / 16;                  // 16 x 16 state tiles per wavefront
  constexpr int NB = kLaQ / 16;               // 16-step blocks per chunk
  constexpr int NR = kLaQ * C / 8 / 256;      // 16-byte vectors of A and B per thread and chunk
  constexpr int NX = kLaQ * 64 / 8 / 256;     // ... of X and Z
  constexpr bool kOut = KIND != kWalkState;
  constexpr bool kZ = T::kZ;
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

  // Rows of 16-byte vectors; rows past the chunk's last step re-read that step
  // (their X and decay are then zero), columns past the tensor's width read its
  // first vector and count as zero.
  struct Bank {
    u32x4_t A[kOut ? NR : 1], B[NR], X[NX], Z[kZ ? NX : 1];
    float g;
  };
  Bank bank;
  // Addresses are a chunk's base, uniform across the workgroup, plus a 32-bit
  // byte offset: one chunk of any tensor spans less than 2^31 bytes (checked on
  // the host).
  auto issue = [&](int64_t t0, int nt) SSM_INLINE {
    auto at = [&](const uint16_t* p, const LaOperand& o, uint32_t off) SSM_INLINE {
      return *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(p + t0 * o.row) + off);
    };
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int v = tid + 256 * r;
      const uint32_t row = (uint32_t)min(v / (C / 8), nt - 1), c16 = la_in(v % (C / 8), a.cdim) ? v % (C / 8) * 16u : 0u;
      if constexpr (kOut) bank.A[r] = at(Ab, a.A, row * ((uint32_t)a.A.row * 2u) + c16);
      bank.B[r] = at(Bb, a.B, row * ((uint32_t)a.B.row * 2u) + c16);
    }
#pragma unroll
    for (int r = 0; r < NX; ++r) {
      const int v = tid + 256 * r;
      const uint32_t row = (uint32_t)min(v >> 3, nt - 1), c16 = la_in(v & 7, xdim) ? (v & 7) * 16u : 0u;
      bank.X[r] = at(Xb, a.X, row * ((uint32_t)a.X.row * 2u) + c16);
      if constexpr (kZ) bank.Z[r] = at(Zb, a.Z, row * ((uint32_t)a.Z.row * 2u) + c16);
    }
    if (tid < kLaQ) bank.g = gb[(t0 + min(tid, nt - 1)) * a.decay_t];
  };

  constexpr u32x4_t kZero = {0u, 0u, 0u, 0u};
  float csum = 0.0f;   // wavefront 0: log2 decay of the whole time chunk
  auto stage = [&](int nt) SSM_INLINE {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int v = tid + 256 * r;
      const int row = v / (C / 8), c8 = v % (C / 8);
      const bool in = la_in(c8, a.cdim);
      if constexpr (kOut) *reinterpret_cast<u32x4_t*>(&s.A[row * T::SA + c8 * 8]) = in ? bank.A[r] : kZero;
      *reinterpret_cast<u32x4_t*>(&s.B[row * T::SB + c8 * 8]) = in ? bank.B[r] : kZero;
    }
#pragma unroll
    for (int r = 0; r < NX; ++r) {
      const int v = tid + 256 * r;
      const int row = v >> 3, c8 = v & 7;
      const bool in = row < nt && la_in(c8, xdim);
      u32x4_t x = in ? bank.X[r] : kZero;
      // W is zero where j comes after i, and zero times a value that is not
      // finite is not zero: such values of X are taken out here and put back
      // into the rows and the state that they reach (poison, below)
      u32x4_t t;
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = ((x[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
      if ((t[0] | t[1] | t[2] | t[3]) != 0u) {
        s.bad = 1;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((t[e >> 1] >> (16 * (e & 1))) & 0x8000u) {
            if (REV) atomicMax(&s.badstep[c8 * 8 + e], row);
            else atomicMin(&s.badstep[c8 * 8 + e], row);
            x[e >> 1] &= (e & 1) ? 0x0000ffffu : 0xffff0000u;
          }
      }
      *reinterpret_cast<u32x4_t*>(&s.X[row * T::SP + c8 * 8]) = x;
      if constexpr (kZ) *reinterpret_cast<u32x4_t*>(&s.Z[row * T::SP + c8 * 8]) = in ? bank.Z[r] : kZero;
    }
    if (w == 0) {
      // exp2 of anything below -150 is 0 in fp32: decays are held above -160,
      // so that a decay of minus infinity (forget everything) leaves the
      // differences of sums finite
      float c = l < nt ? bank.g * kLog2e : 0.0f;
      c = c < -160.0f ? -160.0f : c;
      float one = 1.0f;
      affine_wave_scan(one, c);   // (1, c) pairs compose to prefix sums of c
      const float c_end = readlane_f(c, kLaQ - 1);
      csum += c_end;
      if (l < kLaQ) {
        s.cum[l] = c;
        s.row[l] = __builtin_amdgcn_exp2f(REV ? c_end - c : c) * a.row_scale;
        s.src[l] = __builtin_amdgcn_exp2f(REV ? c : c_end - c) * a.src_scale;
      }
      if (l == 0) s.end = __builtin_amdgcn_exp2f(c_end);
    }
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
  bool has_state = src != nullptr;

  if (tid < 64) s.badstep[tid] = REV ? -1 : kLaQ;
  if (tid == 0) s.bad = 0;
  if constexpr (kOut) {
    // W's 16 x 16 blocks that the 32-wide products read beyond the triangle
    for (int e = tid; e < 2 * (NB / 2) * 256; e += 256) {
      const int k = e & 1, blk = (e >> 1) / 256, i = (e >> 1) % 256 / 16, j = (e >> 1) % 16;
      const int bi = REV ? 2 * blk + 1 : 2 * blk, bj = REV ? 2 * blk : 2 * blk + 1;
      s.W[k][(16 * bi + i) * T::SW + 16 * bj + j] = 0;
    }
  }
  block_sync();

  const int64_t chunks = (L + kLaQ - 1) / kLaQ;
  auto start_of = [&](int64_t ch) SSM_INLINE { return (REV ? chunks - 1 - ch : ch) * kLaQ; };
  auto steps_of = [&](int64_t ch) SSM_INLINE { return (int)min((int64_t)kLaQ, L - start_of(ch)); };
  issue(start_of(0), steps_of(0));
  for (int64_t ch = 0; ch < chunks; ++ch) {
    const int64_t t0 = start_of(ch);
    const int nt = steps_of(ch);
    stage(nt);
    if (ch + 1 < chunks) issue(start_of(ch + 1), steps_of(ch + 1));
    block_sync();

    f32x4_t accY[kOut ? NB : 1];
    if constexpr (kOut) {
      // Phase 1: the triangle's 16 x 16 tiles of G, decayed into W, by turns.
      int turn = 0;
#pragma unroll
      for (int ib = 0; ib < NB; ++ib)
#pragma unroll
        for (int jb = 0; jb < NB; ++jb) {
          if (REV ? jb < ib : jb > ib) continue;
          if ((turn++ & 3) != w) continue;
          // transposed: lane (q, lr) holds row i = 16 ib + lr, columns
          // j = 16 jb + 4 q + r
          f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int m = 0; m < C / 32; ++m)
            acc = la_mfma(la_op(&s.B[(16 * jb + lr) * T::SB + 32 * m + 8 * q]),
                          la_op(&s.A[(16 * ib + lr) * T::SA + 32 * m + 8 * q]), acc);
          const int i = 16 * ib + lr, j0 = 16 * jb + 4 * q;
          const float ci = s.cum[i];
          const f32x4_t cj = *reinterpret_cast<const f32x4_t*>(&s.cum[j0]);
          float v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float d = __builtin_amdgcn_exp2f(REV ? cj[r] - ci : ci - cj[r]) * a.w_scale;
            v[r] = (ib != jb || (REV ? j0 + r >= i : j0 + r <= i)) ? acc[r] * d : 0.0f;
          }
          const LaSplit s0 = la_split(v[0], v[1]), s1 = la_split(v[2], v[3]);
          *reinterpret_cast<uint2*>(&s.W[0][i * T::SW + j0]) = make_uint2(s0.hi, s1.hi);
          *reinterpret_cast<uint2*>(&s.W[1][i * T::SW + j0]) = make_uint2(s0.lo, s1.lo);
          if constexpr (KIND == kWalkDq) {
            // M = W o (q k^T) below the diagonal, over this slice's columns of
            // q and k: its row and column sums, in fp32 from exact products
            f32x4_t pk = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < 2; ++m)
              pk = la_mfma(la_op(&s.X[(16 * jb + lr) * T::SP + 32 * m + 8 * q]),
                           la_op(&s.Z[(16 * ib + lr) * T::SP + 32 * m + 8 * q]), pk);
            float rowsum = 0.0f;
            f32x4_t colsum;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float m = (ib != jb || j0 + r < i) ? v[r] * pk[r] : 0.0f;
              rowsum += m;
              colsum[r] = la_row_sum(m);
            }
            rowsum = la_rows_sum(rowsum);
            if (q == 0) s.rs[jb][i] = rowsum;
            if (lr == 0) *reinterpret_cast<f32x4_t*>(&s.cs[ib][j0]) = colsum;
          }
        }
      // The entering state's readout: tiles 2 m and 2 m + 1 give the eight k
      // slots of product m (columns 32 m + 4 q + 0..3 and 32 m + 16 + 4 q +
      // 0..3), and A is read in the same order.
#pragma unroll
      for (int ib = 0; ib < NB; ++ib) accY[ib] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (has_state) {
#pragma unroll
        for (int m = 0; m < C / 32; ++m) {
          u32x4_t hw, lw;
#pragma unroll
          for (int r = 0; r < 4; r += 2) {
            const LaSplit s0 = la_split(accS[2 * m][r], accS[2 * m][r + 1]);
            const LaSplit s1 = la_split(accS[2 * m + 1][r], accS[2 * m + 1][r + 1]);
            hw[r / 2] = s0.hi;
            lw[r / 2] = s0.lo;
            hw[2 + r / 2] = s1.hi;
            lw[2 + r / 2] = s1.lo;
          }
          const bf16x8_t shi = __builtin_bit_cast(bf16x8_t, hw);
          const bf16x8_t slo = __builtin_bit_cast(bf16x8_t, lw);
#pragma unroll
          for (int ib = 0; ib < NB; ++ib) {
            const uint16_t* arow = &s.A[(16 * ib + lr) * T::SA + 32 * m + 4 * q];
            const bf16x8_t av = la_op2(arow, arow + 16);
            accY[ib] = la_mfma(shi, av, accY[ib]);
            accY[ib] = la_mfma(slo, av, accY[ib]);
          }
        }
#pragma unroll
        for (int ib = 0; ib < NB; ++ib) {
          const float f = s.row[16 * ib + lr];
#pragma unroll
          for (int r = 0; r < 4; ++r) accY[ib][r] *= f;
        }
      }
      if constexpr (kZ) {
        // Z . readout over this wavefront's 16 columns
#pragma unroll
        for (int ib = 0; ib < NB; ++ib) {
          const uint2 z = *reinterpret_cast<const uint2*>(&s.Z[(16 * ib + lr) * T::SP + 16 * w + 4 * q]);
          float d = accY[ib][0] * __uint_as_float(z.x << 16);
          d = __builtin_fmaf(accY[ib][1], __uint_as_float(z.x & 0xffff0000u), d);
          d = __builtin_fmaf(accY[ib][2], __uint_as_float(z.y << 16), d);
          d = __builtin_fmaf(accY[ib][3], __uint_as_float(z.y & 0xffff0000u), d);
          d = la_rows_sum(d);
          if (q == 0) s.dot[w][16 * ib + lr] = d;
        }
      }
      block_sync();
    }

    // Phase 2: Y += W X, stored; the state moves past the chunk.
    const bool poison = s.bad != 0;
    const int bad_at = poison ? s.badstep[p] : 0;
    bf16x8_t xo[NB / 2];
#pragma unroll
    for (int kk = 0; kk < NB / 2; ++kk) xo[kk] = la_col8(s.X, T::SP, 32 * kk + 8 * q, 16 * w, l);
    if constexpr (kOut) {
#pragma unroll
      for (int ib = 0; ib < NB; ++ib)
#pragma unroll
        for (int kk = 0; kk < NB / 2; ++kk) {
          if (REV ? kk < ib / 2 : kk > ib / 2) continue;
          accY[ib] = la_mfma(xo[kk], la_op(&s.W[0][(16 * ib + lr) * T::SW + 32 * kk + 8 * q]), accY[ib]);
          accY[ib] = la_mfma(xo[kk], la_op(&s.W[1][(16 * ib + lr) * T::SW + 32 * kk + 8 * q]), accY[ib]);
        }
      if (poison) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = s.badstep[16 * w + 4 * q + r];
#pragma unroll
          for (int ib = 0; ib < NB; ++ib)
            if (REV ? 16 * ib + lr <= at : 16 * ib + lr >= at) accY[ib][r] = __builtin_nanf("");
        }
      }
      // four consecutive columns of step 16 ib + lr (xdim is a multiple of 8)
      const int64_t o0 = ((((int64_t)b * a.seqlen + t_begin + t0) * a.nheads + h) * a.xdim + x0);
      const int py = 16 * w + 4 * q;
      const uint32_t orow = (uint32_t)a.nheads * (uint32_t)a.xdim;
      if (py < xdim) {
#pragma unroll
        for (int ib = 0; ib < NB; ++ib) {
          const int i = 16 * ib + lr;
          if (i < nt) {
            const float y[4] = {accY[ib][0], accY[ib][1], accY[ib][2], accY[ib][3]};
            const uint32_t off = (uint32_t)i * orow + (uint32_t)py;
            if (a.out_bf16) store_row<uint16_t, 4>(static_cast<uint16_t*>(a.out) + o0 + off, y);
            else store_row<float, 4>(static_cast<float*>(a.out) + o0 + off, y);
          }
        }
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
    {
      bf16x8_t xh[NB / 2], xl[NB / 2];
#pragma unroll
      for (int kk = 0; kk < NB / 2; ++kk) {
        const float* f = &s.src[32 * kk + 8 * q];
        const u32x4_t xw = __builtin_bit_cast(u32x4_t, xo[kk]);
        u32x4_t hv, lv;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const LaSplit sp = la_split(__uint_as_float(xw[e] << 16) * f[2 * e], __uint_as_float(xw[e] & 0xffff0000u) * f[2 * e + 1]);
          hv[e] = sp.hi;
          lv[e] = sp.lo;
        }
        xh[kk] = __builtin_bit_cast(bf16x8_t, hv);
        xl[kk] = __builtin_bit_cast(bf16x8_t, lv);
      }
      const float e_end = s.end;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4_t acc = accS[t];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] *= e_end;
#pragma unroll
        for (int kk = 0; kk < NB / 2; ++kk) {
          const bf16x8_t bt = la_col8(s.B, T::SB, 32 * kk + 8 * q, 16 * t, l);
          acc = la_mfma(bt, xh[kk], acc);
          acc = la_mfma(bt, xl[kk], acc);
        }
        if (poison && (REV ? bad_at >= 0 : bad_at < kLaQ)) {
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] = __builtin_nanf("");
        }
        accS[t] = acc;
      }
    }
    has_state = true;
    block_sync();
    if (poison) {
      if (tid < 64) s.badstep[tid] = REV ? -1 : kLaQ;
      if (tid == 0) s.bad = 0;
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
  if (KIND == kWalkState && slice == 0 && tid == 0) a.chunk_decay[(int64_t)(b * K + kt) * a.nheads + h] = csum;
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
