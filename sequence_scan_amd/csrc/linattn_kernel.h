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
// A, B and X are bf16 inputs, exact as operands.  Computed operands (W, the state in
// the readout, the scaled X of the state update) are fp32 and enter as sums of three
// bf16 terms (v's rounding, the rest's rounding, and its rest's), all their bits: outputs
// may be fp32, and are then within fp32's own roundings of the exact sums.
//
// A workgroup of four wavefronts owns 64 value columns of one (batch row, head)
// and walks its chunks of kLaQ steps; wavefront w holds columns 16 w .. 16 w + 15
// of S^T for the whole sequence in accumulator registers, whose layout is, up to a
// fixed permutation of the contracted index, the operand layout that the readout
// needs.  G and Y are formed transposed (the products' operands swapped): a lane
// then holds one step and four consecutive columns, one wide access to W and to the output's rows.  Tiles are staged in LDS as
// they lie in memory; operands contracted over time are read with the transposing
// ds_read_b64_tr_b16.
//
// Chunks of 32 steps: chunks of 64 halve the work on the state (its rounding for the
// readout and its scaling, two fifths of a wavefront's vector instructions here), but
// hold twice the LDS, so two workgroups per CU in place of three.
//
// What bounds it: prompts of 8 x 2048, 40 heads of 128 x 128, take 232 us, 3.0 TB/s of
// the bytes that they have to move (135 us at a copy's rate).  Of 226 us, before W and the
// readout's state had their third term, they took 174 without loads and 197 without
// stores: a chunk's chain of products, roundings and
// two barriers is what its three wavefronts per SIMD wait for, and memory overlaps it
// only in part.  The third terms, 10 of a chunk's 58 products and an eighth of its vector
// instructions, cost 205 -> 232 us here and 420 -> 434 us in the gradients; without them
// fp32 outputs were off by 2.0e-6 to 2.5e-6 of their norm, with them by 1.3e-7.
#ifndef SSMSCAN_LINATTN_KERNEL_H
#define SSMSCAN_LINATTN_KERNEL_H

#include <type_traits>

#include "block.h"
#include "lds_load.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// Tiles of bf16 in LDS, W bytes per row, in units of 16 bytes.  They are filled by
// loads that go straight to LDS, 1024 consecutive bytes per wavefront, so rows
// cannot be padded; instead unit u of row r lies at position u ^ f(r).  A cycle
// serves 64 banks, 16 units: the eight rows of half a wavefront's transposing read
// (r, r + 1 .. r + 3, r + 8 .. r + 11, two neighbouring units each) and the 16 rows
// of its 8-byte reads (one unit) then lie in different banks.  (Reads of 16 bytes
// from 16 rows take two cycles in place of one with the wider tiles.)
template <int W>
__device__ __forceinline__ uint32_t la_flip(int row) {
  const uint32_t b0 = row & 1, b1 = (row >> 1) & 1, b2 = (row >> 2) & 1, b3 = (row >> 3) & 1;
  if constexpr (W == 256) return 16u * (b2 | b0 << 1 | b1 << 2 | b3 << 3);
  else if constexpr (W == 128) return 16u * (b2 | b1 << 1 | b3 << 2);
  else return 16u * (b2 | (b2 ^ b3) << 1);     // 64
}

template <int W>
struct LaRows {
  char* p;
  // (The position's bits flip independently, so that with a constant part of it the
  // address is one xor or an immediate offset away.)
  __device__ __forceinline__ char* at(int row, int byte) const { return p + row * W + ((uint32_t)byte ^ la_flip<W>(row)); }
  // Eight columns from 8 u.
  __device__ __forceinline__ bf16x8_t op(int row, int u) const { return *reinterpret_cast<const bf16x8_t*>(at(row, 16 * u)); }
  // Columns c .. c + 3 and c + 16 .. c + 19 (c a multiple of 4).
  __device__ __forceinline__ bf16x8_t op2(int row, int c) const {
    const bf16x4_t a = *reinterpret_cast<const bf16x4_t*>(at(row, 2 * c));
    const bf16x4_t b = *reinterpret_cast<const bf16x4_t*>(at(row, 2 * c + 32));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ __forceinline__ uint2 four(int row, int c) const { return *reinterpret_cast<const uint2*>(at(row, 2 * c)); }
};

// Transposing read: within 16 lanes, lane i gets element i % 4 of the 8-byte
// pieces addressed by lanes 4 e + i / 4, e = 0..3.
__device__ __forceinline__ i16x4_t la_tr(const uint16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(p));
}

// Rows r0 .. r0 + 7 (r0 a multiple of 8) of column c0 + (lane % 16).
template <int W>
__device__ __forceinline__ bf16x8_t la_col8(const LaRows<W>& tile, int r0, int c0, int l) {
  const int k = l & 15;
  const int row = r0 + (k >> 2), byte = 2 * c0 + 8 * (k & 3);
  const i16x4_t lo = la_tr(reinterpret_cast<const uint16_t*>(tile.at(row, byte)));
  const i16x4_t hi = la_tr(reinterpret_cast<const uint16_t*>(tile.at(row + 4, byte)));
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ f32x4_t la_mfma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Eight fp32 values as sums of N bf16 operands: their roundings, the rests'
// roundings, ...  The rest v - bf16(v) is exact in fp32; the two-term dot product
// with (-1, 0) or (0, -1) forms it in one instruction, from the packed pair (a half
// that is not finite spoils its neighbour's too: they are of one value column,
// which is lost then anyway).
template <int N>
__device__ __forceinline__ void la_split8(float* v, u32x4_t* t) {
  // (kept in registers: as an instruction's own constant, -1.0 does not mean the
  // packed pair that the compiler takes it for)
  uint32_t first = 0x0000bf80u, second = 0xbf800000u;
  asm("" : "+s"(first), "+s"(second));
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int r = 0; r < 4; ++r) t[i][r] = pack_bf16x2(v[2 * r], v[2 * r + 1]);
    if (i + 1 < N) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // (by itself: out of the operand of eight, the compiler takes the first pair
        // for every one of the four)
        uint32_t pair = t[i][r];
        asm("" : "+v"(pair));
        t[i][r] = pair;
        const bf16x2_t p = __builtin_bit_cast(bf16x2_t, pair);
        v[2 * r] = __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2_t, first), v[2 * r], false);
        v[2 * r + 1] = __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2_t, second), v[2 * r + 1], false);
      }
    }
  }
}

// Prefix sums over each half of a wavefront in 64 bits (row shifts, then the first
// row's total into the second).
template <int CTRL, int ROWS>
__device__ __forceinline__ double la_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ double la_prefix32(double v) {
  v += la_dpp<0x111, 0xf>(v);   // row_shr:1
  v += la_dpp<0x112, 0xf>(v);   // row_shr:2
  v += la_dpp<0x114, 0xf>(v);   // row_shr:4
  v += la_dpp<0x118, 0xf>(v);   // row_shr:8
  v += la_dpp<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
  return v;
}

// 2^c rounded to fp32 once: the power series of e^(f ln 2) to its seventh power, for
// the rest f of c to the nearest integer (the eighth is below 2^-27).  The hardware's
// exponential is off by up to an ulp, and with a fixed decay by the same in every
// chunk, which adds up over a state's memory and in the decay's gradient.
__device__ __forceinline__ float la_exp2(double c) {
  constexpr double kLn2 = 0.6931471805599453;
  constexpr double c1 = kLn2, c2 = c1 * kLn2 / 2, c3 = c2 * kLn2 / 3, c4 = c3 * kLn2 / 4, c5 = c4 * kLn2 / 5, c6 = c5 * kLn2 / 6,
                   c7 = c6 * kLn2 / 7;
  const double n = __builtin_rint(c), f = c - n;
  double p = __builtin_fma(c7, f, c6);
  p = __builtin_fma(p, f, c5);
  p = __builtin_fma(p, f, c4);
  p = __builtin_fma(p, f, c3);
  p = __builtin_fma(p, f, c2);
  p = __builtin_fma(p, f, c1);
  p = __builtin_fma(p, f, 1.0);
  // (held within an int; NaN stays in p)
  return __builtin_amdgcn_ldexpf((float)p, (int)__builtin_fmin(__builtin_fmax(n, -2000.0), 2000.0));
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

constexpr int kWalkOut = 0;     // the products alone
constexpr int kWalkState = 1;   // no rows and no output: the state at the end of the time chunk
constexpr int kWalkDq = 2;      // with the decay gradient's parts of dq: Z = q
constexpr int kWalkDk = 3;      // ... of dk: Z = k

constexpr int kLaTerms = 3;     // bf16 terms of an fp32 operand

// LDS of one walk (C: contracted columns, 64 or 128).  B and X, which both
// phases of a chunk read, are held twice: the next chunk's are loaded from the
// chunk's start; A and Z, which only the first phase reads, from its middle.
template <int C, int KIND>
struct LaTile {
  static constexpr bool kOut = KIND != kWalkState;
  static constexpr bool kZ = KIND == kWalkDq || KIND == kWalkDk;
  static constexpr int kBlk = kLaQ / 16;
  static constexpr int kRing = 16;            // chunks whose decays are at hand
  char B[2][kLaQ * 2 * C] __attribute__((aligned(1024)));
  char X[2][kLaQ * 128] __attribute__((aligned(1024)));
  char A[kOut ? kLaQ * 2 * C : 16] __attribute__((aligned(1024)));
  char Z[kZ ? kLaQ * 128 : 16] __attribute__((aligned(1024)));
  char W[kLaTerms][kOut ? kLaQ * 64 : 16] __attribute__((aligned(16)));   // by terms
  char Y[kOut ? kLaQ * 128 : 16] __attribute__((aligned(16)));     // bf16 output
  float cum[kRing][kLaQ] __attribute__((aligned(16)));   // log2 decay summed from the chunk's first step, inclusive
  float low[kRing][kLaQ] __attribute__((aligned(16)));   // what it lacks of the 64-bit sum
  float row[kRing][kLaQ];                                // factor of A S^T
  float src[kRing][kLaQ] __attribute__((aligned(16)));   // factor of X in the state update
  float end[kRing];                                  // exp(c_end)
  int bad[2];                                        // the chunk's X holds a value that is not finite
  float dot[kZ ? 4 : 1][kLaQ];                       // per wavefront: Z . (diag(row) A S^T)
  float rs[KIND == kWalkDq ? kBlk : 1][kLaQ];        // row sums of M by column block
  float cs[KIND == kWalkDq ? kBlk : 1][kLaQ] __attribute__((aligned(16)));   // column sums of M by row block
};

// One walk.  `h`, `b`: head and batch row; `slice`: its 64 value columns; `kt`:
// time chunk.
template <int C, int KIND, bool REV>
__device__ __forceinline__ void la_walk(const LaWalk& a, LaTile<C, KIND>& s, int b, int h, int slice, int kt) {
  using T = LaTile<C, KIND>;
  constexpr int NT = C / 16;                  // 16 x 16 state tiles per wavefront
  constexpr int NB = kLaQ / 16;               // 16-step blocks per chunk
  static_assert(NB == 2, "the products over a chunk's steps are one instruction deep");
  constexpr int NR = kLaQ * 2 * C / 4096;     // loads of A and B per wavefront and chunk (of X and Z: one)
  constexpr bool kOut = T::kOut;
  constexpr bool kZ = T::kZ;
  const int tid = threadIdx.x, l = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = l & 15, q = l >> 4;
  const int x0 = slice * 64;
  const int K = a.n_chunks;
  const int64_t t_begin = (int64_t)kt * a.chunk_len;
  const int64_t L = min(a.chunk_len, a.seqlen - t_begin);
  const int chunks = (int)((L + kLaQ - 1) / kLaQ);
  const int xdim = min(64, a.xdim - x0);      // value columns of this slice that exist
  const int p = 16 * w + lr;                  // this lane's value column in the slice
  auto start_of = [&](int ch) SSM_INLINE { return (int64_t)(REV ? chunks - 1 - ch : ch) * kLaQ; };
  auto steps_of = [&](int ch) SSM_INLINE { return (int)min((int64_t)kLaQ, L - start_of(ch)); };

  // Loads: each operand's next chunk is a running base, uniform across the
  // workgroup, plus 32-bit lane offsets that are the same for every full chunk
  // (one chunk of any tensor spans less than 2^31 bytes: checked on the host).
  // Rows past the sequence's last step re-read that step; lanes whose columns lie
  // past the tensor's width stay off, and those columns zero from the start.
  auto base = [&](const LaOperand& o, int col) SSM_INLINE {
    return reinterpret_cast<const char*>(o.p + ((int64_t)b * a.seqlen + t_begin + start_of(0)) * o.row +
                                         (int64_t)(h / o.share) * o.head + col);
  };
  auto hop = [&](const LaOperand& o) SSM_INLINE { return (REV ? -2 : 2) * kLaQ * o.row; };   // bytes
  const char* nA = kOut ? base(a.A, 0) : nullptr;
  const char* nB = base(a.B, 0);
  const char* nX = base(a.X, x0);
  const char* nZ = kZ ? base(a.Z, x0) : nullptr;
  constexpr int kPer = 1024 / (2 * C);        // rows of A and B per load
  // lane l of load r: row, and the source's byte in it
  auto wide_row = [&](int r) SSM_INLINE { return (w * NR + r) * kPer + l / (64 / kPer); };
  auto wide_byte = [&](int r) SSM_INLINE { return (uint32_t)(l % (64 / kPer)) * 16u ^ la_flip<2 * C>(wide_row(r)); };
  const int xrow = 8 * w + l / 8;
  const uint32_t xbyte = (uint32_t)(l % 8) * 16u ^ la_flip<128>(xrow);
  const bool xin = (int)xbyte < 2 * xdim;
  uint32_t offA[kOut ? NR : 1], offB[NR], offX, offZ = 0u;
  auto set_offsets = [&](int nt) SSM_INLINE {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const uint32_t row = (uint32_t)min(wide_row(r), nt - 1);
      if constexpr (kOut) offA[r] = row * ((uint32_t)a.A.row * 2u) + wide_byte(r);
      offB[r] = row * ((uint32_t)a.B.row * 2u) + wide_byte(r);
    }
    const uint32_t row = (uint32_t)min(xrow, nt - 1);
    offX = row * ((uint32_t)a.X.row * 2u) + xbyte;
    if constexpr (kZ) offZ = row * ((uint32_t)a.Z.row * 2u) + xbyte;
  };
  // (the ragged chunk is a forward walk's last and a backward walk's first)
  auto load_bx = [&](int to) SSM_INLINE {
#pragma unroll
    for (int r = 0; r < NR; ++r)
      if ((int)wide_byte(r) < 2 * a.cdim) load_lds(nB, offB[r], &s.B[to][(w * NR + r) * 1024]);
    if (xin) load_lds(nX, offX, &s.X[to][w * 1024]);
    nB += hop(a.B);
    nX += hop(a.X);
  };
  auto load_az = [&]() SSM_INLINE {
    if constexpr (kOut) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
        if ((int)wide_byte(r) < 2 * a.cdim) load_lds(nA, offA[r], &s.A[(w * NR + r) * 1024]);
      nA += hop(a.A);
    }
    if constexpr (kZ) {
      if (xin) load_lds(nZ, offZ, &s.Z[w * 1024]);
      nZ += hop(a.Z);
    }
  };

  // Decays.  Every eight chunks each wavefront sums those of two, one in each
  // half: eight chunks ahead, of eight steps loaded eight chunks before that.
  const float* gb = a.decay + (int64_t)b * a.decay_b + t_begin * a.decay_t + h;
  float g = 0.0f;      // this lane's step
  float csum = 0.0f;   // log2 decay of this half's chunks
  const int half = l >> 5, step = l & 31;
  static_assert(kLaQ == 32, "two chunks' decays fit a wavefront");
  auto get_decays = [&](int first) SSM_INLINE {
    const int ch = first + 2 * w + half;
    const int nt = ch < chunks ? steps_of(ch) : 0;
    g = step < nt ? gb[(start_of(ch) + step) * a.decay_t] : 0.0f;
  };
  auto sum_decays = [&](int first) SSM_INLINE {
    // exp2 of anything below -150 is 0 in fp32: decays are held above -160, so
    // that a decay of minus infinity (forget everything) leaves the differences
    // of sums finite.  Sums are held as two floats (from 64 bits): W needs
    // their differences, which one float would give to 2^-24 of the sums only.
    const int to = (first + 2 * w + half) % T::kRing;
    const float one = g * kLog2e;
    const double c = la_prefix32((double)(one < -160.0f ? -160.0f : one));
    const double c_end = __shfl(c, 31, 32);
    const float hi = (float)c;
    const float to_here = la_exp2(c), to_end = la_exp2(c_end - c);
    csum += (float)c_end;
    s.cum[to][step] = hi;
    s.low[to][step] = (float)(c - (double)hi);
    s.row[to][step] = (REV ? to_end : to_here) * a.row_scale;
    s.src[to][step] = (REV ? to_here : to_end) * a.src_scale;
    if (step == 31) s.end[to] = to_here;
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

  if (tid < 2) s.bad[tid] = 0;
  if (a.cdim < C || xdim < 64) {
    auto clear = [&](char* t, int bytes) SSM_INLINE {
      for (int e = 16 * tid; e < bytes; e += 16 * 256) *reinterpret_cast<u32x4_t*>(t + e) = u32x4_t{0u, 0u, 0u, 0u};
    };
    clear(s.B[0], sizeof(s.B));
    clear(s.X[0], sizeof(s.X));
    if constexpr (kOut) clear(s.A, sizeof(s.A));
    if constexpr (kZ) clear(s.Z, sizeof(s.Z));
  }
  if constexpr (kOut) {
    // W's block beyond the triangle
    for (int e = tid; e < kLaTerms * 256; e += 256) {
      const int k = e >> 8, i = (e >> 4) & 15, j = e & 15;
      *reinterpret_cast<uint16_t*>(LaRows<64>{s.W[k]}.at(i + (REV ? 16 : 0), 2 * (j + (REV ? 0 : 16)))) = 0;
    }
  }
  block_sync();

  set_offsets(steps_of(0));
  load_bx(0);
  load_az();
  get_decays(0);
  sum_decays(0);
  if (chunks > 8) get_decays(8);
  loaded<0>();
  block_sync();

  f32x4_t accY[kOut ? NB : 1];
  // Outputs of chunk ch leave a chunk late.  A lane holds four consecutive columns
  // of step 16 n + lr (xdim is a multiple of 8).  bf16 rows are gathered in LDS and
  // leave as whole lines; a wavefront's own share of a row is a quarter of one
  // (prompts of 8 x 2048, 40 heads: 225 us stored from the registers, 213 so).
  auto gather = [&]() SSM_INLINE {
    if (a.out_bf16) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
        *reinterpret_cast<uint2*>(LaRows<128>{s.Y}.at(16 * n + lr, 2 * (16 * w + 4 * q))) =
            make_uint2(pack_bf16x2(accY[n][0], accY[n][1]), pack_bf16x2(accY[n][2], accY[n][3]));
    }
  };
  auto store = [&](int ch) SSM_INLINE {
    const int64_t t0 = start_of(ch);
    const int nt = steps_of(ch);
    const int64_t o0 = (((int64_t)b * a.seqlen + t_begin + t0) * a.nheads + h) * a.xdim + x0;
    const uint32_t row = (uint32_t)a.nheads * (uint32_t)a.xdim;
    if (a.out_bf16) {
      const int r = 8 * w + l / 8, c = 8 * (l % 8);
      if (r < nt && c < xdim) {
        const u32x4_t y = *reinterpret_cast<const u32x4_t*>(LaRows<128>{s.Y}.at(r, 2 * c));
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + o0 + (uint32_t)r * row + c) = y;
      }
    } else {
      const int py = 16 * w + 4 * q;
#pragma unroll
      for (int n = 0; n < NB; ++n)
        if (py < xdim && 16 * n + lr < nt) {
          const float y[4] = {accY[n][0], accY[n][1], accY[n][2], accY[n][3]};
          store_row<float, 4>(static_cast<float*>(a.out) + o0 + (uint32_t)(16 * n + lr) * row + py, y);
        }
    }
  };
  // The state at every kLaSnap chunks from the sequence's start on, as the wavefronts
  // hold it, for the decay's gradient.  The dq walk passes a border between two chunks
  // before the later one, the dk walk before the earlier one.
  auto store_snap = [&](int ch) SSM_INLINE {
    const int border = REV ? chunks - ch : ch;
    if (a.snaps == nullptr || border % kLaSnap != 0) return;
    constexpr int kTiles = NT * 256;        // float4 of a wavefront's tiles, all four of them
    const int64_t slot = (((int64_t)b * a.nheads + h) * K + kt) * a.snap_slots + border / kLaSnap - 1;
    f32x4_t* to = reinterpret_cast<f32x4_t*>(a.snaps) + (slot * ((a.xdim + 63) / 64) + slice) * kTiles + tid;
#pragma unroll
    for (int t = 0; t < NT; ++t) to[t * 256] = accS[t];
  };
  float part = 0.0f;
  auto store_part = [&](int ch) SSM_INLINE {
    if (tid < steps_of(ch)) {
      if (s.bad[ch & 1] != 0) part = __builtin_nanf("");
      a.part[(((int64_t)slice * a.batch + b) * a.nheads + h) * a.seqlen + t_begin + start_of(ch) + tid] = part;
    }
    if (tid == 0) s.bad[ch & 1] = 0;
  };

  auto chunk = [&](int ch, auto buffer) SSM_INLINE {
    const int nt = steps_of(ch);
    constexpr int cur = decltype(buffer)::value;
    const int dec = ch % T::kRing;
    const bool more = ch + 1 < chunks;
    const LaRows<2 * C> tA{s.A}, tB{s.B[cur]};
    const LaRows<128> tX{s.X[cur]}, tZ{s.Z};
    // The previous chunk's stores, then the next one's loads: what is waited for
    // at the chunk's end has had the chunk's time.
    if constexpr (kOut) {
      if (ch > 0) {
        store(ch - 1);
        if constexpr (kZ) store_part(ch - 1);
      }
    }
    if (more) {
      if (REV ? ch == 0 : ch + 2 == chunks) set_offsets(steps_of(ch + 1));
      load_bx(cur ^ 1);
    }
    if constexpr (cur == 0) {      // (every eighth chunk is even)
      if (ch % 8 == 0 && ch + 8 < chunks) {
        sum_decays(ch + 8);
        if (ch + 16 < chunks) get_decays(ch + 16);
      }
    }

    if constexpr (kOut) {
      // Phase 1.  The triangle's three 16 x 16 tiles of G, one each for the first
      // three wavefronts, transposed: lane (q, lr)
      // holds row i = 16 ib + lr, columns j = 16 jb + 4 q + r.
      const int ib = REV ? (w == 2 ? 1 : 0) : (w == 0 ? 0 : 1);
      const int jb = REV ? (w == 0 ? 0 : 1) : (w == 2 ? 1 : 0);
      const int i = 16 * ib + lr, j0 = 16 * jb + 4 * q;
      if (w < 3) {
        f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < C / 32; ++m) acc = la_mfma(tB.op(16 * jb + lr, 4 * m + q), tA.op(i, 4 * m + q), acc);
        const float ci = s.cum[dec][i], li = s.low[dec][i];
        const f32x4_t cj = *reinterpret_cast<const f32x4_t*>(&s.cum[dec][j0]);
        const f32x4_t lj = *reinterpret_cast<const f32x4_t*>(&s.low[dec][j0]);
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float d = __builtin_amdgcn_exp2f(REV ? cj[r] - ci + (lj[r] - li) : ci - cj[r] + (li - lj[r])) * a.w_scale;
          v[r] = (REV ? j0 + r >= i : j0 + r <= i) ? acc[r] * d : 0.0f;
        }
        float rest[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int e = 0; e < kLaTerms; ++e) {
          const uint2 term = make_uint2(pack_bf16x2(rest[0], rest[1]), pack_bf16x2(rest[2], rest[3]));
          *reinterpret_cast<uint2*>(LaRows<64>{s.W[e]}.at(i, 2 * j0)) = term;
          rest[0] -= __uint_as_float(term.x << 16);
          rest[1] -= __uint_as_float(term.x & 0xffff0000u);
          rest[2] -= __uint_as_float(term.y << 16);
          rest[3] -= __uint_as_float(term.y & 0xffff0000u);
        }
        if constexpr (KIND == kWalkDq) {
          // M = W o (q k^T) below the diagonal, over this slice's columns of q
          // and k: its row and column sums, in fp32 from exact products
          f32x4_t pk = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int m = 0; m < 2; ++m) pk = la_mfma(tX.op(16 * jb + lr, 4 * m + q), tZ.op(i, 4 * m + q), pk);
          float rowsum = 0.0f;
          f32x4_t colsum;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float m = j0 + r < i && i < nt ? v[r] * pk[r] : 0.0f;
            rowsum += m;
            colsum[r] = la_row_sum(m);
          }
          rowsum = la_rows_sum(rowsum);
          if (q == 0) s.rs[jb][i] = rowsum;
          if (lr == 0) *reinterpret_cast<f32x4_t*>(&s.cs[ib][j0]) = colsum;
        }
      }
      // The entering state's readout: tiles 2 m and 2 m + 1 give the eight k slots
      // of product m (columns 32 m + 4 q + 0..3 and 32 m + 16 + 4 q + 0..3), and
      // A is read in the same order.
#pragma unroll
      for (int n = 0; n < NB; ++n) accY[n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m = 0; m < C / 32; ++m) {
        u32x4_t t[kLaTerms];
        float v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = accS[2 * m + r / 4][r % 4];
        la_split8<kLaTerms>(v, t);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          // (apart: the compiler would fetch halves of two operands with one
          // instruction, and move them into place with six)
          asm volatile("" ::: "memory");
          const bf16x8_t av = tA.op2(16 * n + lr, 32 * m + 4 * q);
#pragma unroll
          for (int e = 0; e < kLaTerms; ++e) accY[n] = la_mfma(__builtin_bit_cast(bf16x8_t, t[e]), av, accY[n]);
        }
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float f = s.row[dec][16 * n + lr];
#pragma unroll
        for (int r = 0; r < 4; ++r) accY[n][r] *= f;
      }
      if constexpr (kZ) {
        // Z . readout over this wavefront's 16 columns
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const uint2 z = tZ.four(16 * n + lr, 16 * w + 4 * q);
          float d = accY[n][0] * __uint_as_float(z.x << 16);
          d = __builtin_fmaf(accY[n][1], __uint_as_float(z.x & 0xffff0000u), d);
          d = __builtin_fmaf(accY[n][2], __uint_as_float(z.y << 16), d);
          d = __builtin_fmaf(accY[n][3], __uint_as_float(z.y & 0xffff0000u), d);
          d = la_rows_sum(d);
          if (q == 0) s.dot[w][16 * n + lr] = d;
        }
      }
      block_sync();
      if (more) load_az();
    }

    // Phase 2: Y += W X; the state moves past the chunk.
    const float e_end = s.end[dec];
    u32x4_t xw = __builtin_bit_cast(u32x4_t, la_col8(tX, 8 * q, 16 * w, l));   // X[8 q .. 8 q + 7][p]
    const f32x4_t f0 = *reinterpret_cast<const f32x4_t*>(&s.src[dec][8 * q]);
    const f32x4_t f1 = *reinterpret_cast<const f32x4_t*>(&s.src[dec][8 * q + 4]);
    if (nt < kLaQ) {   // steps past the end
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * q + e >= nt) xw[e >> 1] &= (e & 1) ? 0x0000ffffu : 0xffff0000u;
    }
    // W is zero where j comes after i, and zero times a value that is not finite
    // is not zero: such values of X are taken out here and put back into the
    // rows and the state that they reach (poison, below).
    auto mag = [&](int e) SSM_INLINE { return __builtin_bit_cast(u16x2_t, xw[e] & 0x7fff7fffu); };
    const uint32_t top = __builtin_bit_cast(
        uint32_t, __builtin_elementwise_max(__builtin_elementwise_max(mag(0), mag(1)), __builtin_elementwise_max(mag(2), mag(3))));
    const bool poison = __any(((top + 0x00800080u) & 0x80008000u) != 0u);   // an exponent of all ones
    int bad_at = REV ? -1 : kLaQ;               // column p's first (REV: last) such step
    if (poison) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t half = (e & 1) ? 0xffff0000u : 0x0000ffffu;
        if ((xw[e >> 1] & half & 0x7f807f80u) == (half & 0x7f807f80u)) {
          bad_at = REV ? max(bad_at, 8 * q + e) : min(bad_at, 8 * q + e);
          xw[e >> 1] &= ~half;
        }
      }
#pragma unroll
      for (int d = 16; d < 64; d *= 2) {
        const int o = __shfl_xor(bad_at, d);
        bad_at = REV ? max(bad_at, o) : min(bad_at, o);
      }
      if (kZ && l == 0) s.bad[cur] = 1;
    }
    if constexpr (kOut) {
      const bf16x8_t xo = __builtin_bit_cast(bf16x8_t, xw);
#pragma unroll
      for (int e = 0; e < kLaTerms; ++e)
#pragma unroll
        for (int n = 0; n < NB; ++n) accY[n] = la_mfma(xo, LaRows<64>{s.W[e]}.op(16 * n + lr, q), accY[n]);
    }
    bf16x8_t xs[kLaTerms];
    {
      u32x4_t t[kLaTerms];
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(xw[e] << 16) * (e < 2 ? f0[2 * e] : f1[2 * e - 4]);
        v[2 * e + 1] = __uint_as_float(xw[e] & 0xffff0000u) * (e < 2 ? f0[2 * e + 1] : f1[2 * e - 3]);
      }
      la_split8<kLaTerms>(v, t);
#pragma unroll
      for (int k = 0; k < kLaTerms; ++k) xs[k] = __builtin_bit_cast(bf16x8_t, t[k]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) accS[t][r] *= e_end;
      const bf16x8_t bt = la_col8(tB, 8 * q, 16 * t, l);
#pragma unroll
      for (int k = 0; k < kLaTerms; ++k) accS[t] = la_mfma(bt, xs[k], accS[t]);
    }
    if (poison) {
      if (REV ? bad_at >= 0 : bad_at < kLaQ) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) accS[t][r] = __builtin_nanf("");
      }
      if constexpr (kOut) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = __shfl(bad_at, 4 * q + r);      // of column 16 w + 4 q + r
#pragma unroll
          for (int n = 0; n < NB; ++n)
            if (REV ? 16 * n + lr <= at : 16 * n + lr >= at) accY[n][r] = __builtin_nanf("");
        }
      }
    }
    if constexpr (kOut) gather();
    if constexpr (kZ) {
      if (tid < nt) {
        part = s.dot[0][tid] + s.dot[1][tid] + s.dot[2][tid] + s.dot[3][tid];
        if constexpr (KIND == kWalkDq) {
          for (int k = 0; k <= tid >> 4; ++k) part += s.rs[k][tid];
          for (int k = tid >> 4; k < NB; ++k) part -= s.cs[k][tid];
        }
      }
    }
    loaded<0>();
    block_sync();
  };
  for (int ch = 0; ch < chunks; ch += 2) {
    if constexpr (kZ)
      if (ch > 0) store_snap(ch);
    chunk(ch, std::integral_constant<int, 0>());
    if (ch + 1 >= chunks) break;
    if constexpr (kZ && REV) store_snap(ch + 1);     // (forward, a border is even)
    chunk(ch + 1, std::integral_constant<int, 1>());
  }
  if constexpr (kOut) {
    store(chunks - 1);
    if constexpr (kZ) store_part(chunks - 1);
  }

  const int far = REV ? 0 : K - 1;
  float* dst = KIND == kWalkState ? a.chunk_out + ((int64_t)(b * K + kt) * a.nheads + h) * per
              : kt == far && a.last != nullptr ? a.last + ((int64_t)b * a.nheads + h) * per : nullptr;
  // (the lane's place is formed anew, not held through the chunks)
  int lane = threadIdx.x & 63;
  asm("" : "+v"(lane));
  const int px = 16 * w + lane % 16;
  const uint32_t at = (uint32_t)(x0 + px) * (uint32_t)a.st_x;
  if (dst != nullptr && px < xdim) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int c = 16 * t + 4 * (lane / 16);
      if (c >= a.cdim) continue;
      if (a.st_c == 1) {
        *reinterpret_cast<f32x4_t*>(dst + at + c) = accS[t];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) dst[at + (uint32_t)(c + r) * (uint32_t)a.st_c] = accS[t][r];
      }
    }
  }
  if constexpr (KIND == kWalkState) {
    // the time chunk's log2 decay: the halves of all wavefronts, in order
    float* const sums = &s.row[0][0];
    block_sync();
    if (step == 0) sums[2 * w + half] = csum;
    block_sync();
    if (slice == 0 && tid == 0) {
      float r = 0.0f;
      for (int i = 0; i < 8; ++i) r += sums[i];
      a.chunk_decay[(int64_t)(b * K + kt) * a.nheads + h] = r;
    }
  }
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
