// gfx950 kernels of libssmscan: cross entropy and distillation against a large
// vocabulary.  Everything large is one kind of product, C = A B^T of two bf16 matrices
// whose rows run along the contracted dimension, on bf16 matrix cores with fp32 sums;
// what differs is what becomes of a tile of C in the registers.
#include <algorithm>

#include "device.h"
#include "lds_load.h"
#include "model.h"
#include "vocab_plan.h"

namespace ssm {
namespace {

using namespace vocab;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));

// One side of a product, a bf16 matrix in either order:
//   along  (ACROSS false): [n][k], rows run along the contracted dimension;
//   across (ACROSS true):  [k][n], rows run across it.
struct Side {
  const uint16_t* p;
  int64_t ld;       // elements between rows
  int32_t n;        // rows or columns of C that it gives (across: a multiple of 8)
  int32_t k;        // contracted elements that it has (along: a multiple of 8); past them it counts as 0
};

// The descriptor of `rows` rows of `length` elements: reads past the last row's end give 0.
__device__ __forceinline__ i32x4_t buffer_of(const uint16_t* p, int64_t ld, int64_t rows, int64_t length) {
  const uint64_t base = (uint64_t)(uintptr_t)p;
  const uint32_t bytes = rows > 0 && length > 0 ? (uint32_t)(((rows - 1) * ld + length) * 2) : 0;
  i32x4_t d;
  d.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
  d.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xffff);
  d.z = __builtin_amdgcn_readfirstlane((int)bytes);
  d.w = 0x00020000;     // raw, 32-bit elements
  return d;
}

// A workgroup computes a tile of C, a wavefront kMi x kNi blocks of 16 x 16 of it.  A stage
// holds kK contracted elements of the tile's rows and columns; kStages of them are in LDS,
// one being multiplied while the others arrive.
//
//   Large: 256 x 256 by 2 x 4 wavefronts, 64 KB a stage, two stages.  Its products take
//     most of a stage's time, so one stage ahead is enough.
//   Small: 128 x 128 by 2 x 2 wavefronts, 32 KB a stage, four stages: where tiles are few,
//     a stage's time is the time that its data take to arrive, and three are under way.
//
// In LDS a stage's side lies as in memory, in pieces that are permuted so that an
// operand's reads meet all 64 banks once:
//   along: a row is 128 bytes; the 16-byte piece c of row r is at place
//     c ^ ((r >> 1) & 7).  An operand takes one piece of each of 16 rows.
//   across: 64 rows; the 32-byte piece c of row r is at place
//     c ^ ((r & 3) | (r >> 1 & 4)).  An operand takes one piece of each of 16 rows,
//     turned over on the way (ds_read_tr: 16 lanes read four rows of 16 elements, and
//     receive one column of four each).
struct Large {
  static constexpr int kTile = kLargeTile, kWm = 2, kWn = 4, kStages = 2;
  static constexpr int kWaves = kWm * kWn, kThreads = 64 * kWaves, kMi = kTile / kWm / 16, kNi = kTile / kWn / 16;
  static constexpr int kPerSimd = 2;
};
struct Small {
  static constexpr int kTile = kSmallTile, kWm = 2, kWn = 2, kStages = 4;
  static constexpr int kWaves = kWm * kWn, kThreads = 64 * kWaves, kMi = kTile / kWm / 16, kNi = kTile / kWn / 16;
  static constexpr int kPerSimd = 1;
};
static_assert(Large::kNi == 4 && Small::kNi == 4, "a wavefront has 64 columns of C");
static_assert(Large::kTile == 256 && Small::kTile == 128, "tiles are powers of two");

template <typename Shape>
struct Stages {
  alignas(1024) char a[Shape::kStages][Shape::kTile * kK * 2];
  alignas(1024) char b[Shape::kStages][Shape::kTile * kK * 2];
};

// acc[mi][ni][i]: C[wm * 16 kMi + mi * 16 + (lane & 15)][wn * 64 + ni * 16 + 4 * (lane >> 4) + i].
template <typename Shape>
using Acc = f4_t[Shape::kMi][4];

// A side's loads: a wavefront brings four times 1 KB of a stage.
template <typename Shape, bool ACROSS>
struct Loader {
  static constexpr int kTile = Shape::kTile;
  static_assert(kTile * kK * 2 == Shape::kWaves * 4096, "four loads");
  const uint16_t* p;
  int64_t ld;
  uint32_t off[4];
  int32_t length, k, c;
  __device__ __forceinline__ Loader(const Side& s, int64_t n0, int k0, int k1, int wave, int lane) {
    ld = s.ld;
    k = (s.k < k1 ? s.k : k1) - k0;
    length = (int32_t)(s.n - n0 < kTile ? s.n - n0 : kTile);
    if constexpr (ACROSS) {
      // kK / kWaves rows of the stage, as many at a time as make 1 KB
      constexpr int kPieces = kTile / 8, kRows = 64 / kPieces;
      p = s.p + k0 * s.ld + n0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = wave * (kK / Shape::kWaves) + j * kRows + lane / kPieces, half = lane % kPieces;
        off[j] = (uint32_t)(r * s.ld * 2) + ((half >> 1) ^ ((r & 3) | (r >> 1 & 4))) * 32 + (half & 1) * 16;
      }
      c = 0;
    } else {
      // rows wave * 32 .. + 31 of the tile, eight at a time
      p = s.p + n0 * s.ld + k0;
      c = (lane & 7) ^ ((lane >> 4) & 3);       // of rows 0..7 of 16; rows 8..15 differ in bit 2
#pragma unroll
      for (int j = 0; j < 4; ++j)
        off[j] = (uint32_t)((wave * 32 + j * 8 + (lane >> 3)) * s.ld * 2) + (uint32_t)(c ^ ((j & 1) << 2)) * 16;
    }
  }
  // The stage at contracted element `at` (from k0; past the last, zeros).
  __device__ __forceinline__ void operator()(int at, uint32_t to) const {
    if constexpr (ACROSS) {
      // (a column past the matrix is one of C that is not stored: what is read there, the
      // next row's, does not matter; past the last row there are zeros)
      const i32x4_t buffer = buffer_of(p + (int64_t)at * ld, ld, k - at < kK ? k - at : kK, length);
#pragma unroll
      for (int j = 0; j < 4; ++j) load_lds(buffer, off[j], to + j * 1024);
    } else {
      const i32x4_t buffer = buffer_of(p, ld, length, k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t past = at + (c ^ ((j & 1) << 2)) * 8 < k ? 0 : 0x80000000u;     // (descriptors end below 2^31)
        load_lds(buffer, (off[j] + at * 2) | past, to + j * 1024);
      }
    }
  }
};

// An operand's reads: 16 rows or columns of C, 32 contracted elements (half kk of a stage).
template <typename Shape, bool ACROSS>
struct Reader {
  static constexpr int kRow = Shape::kTile * 2;      // bytes of a row that runs across
  uint32_t at;
  __device__ __forceinline__ Reader(int first, int lane) {
    if constexpr (ACROSS) {
      const int r = (lane >> 4) * 8 + ((lane >> 2) & 3);
      at = r * kRow + (((first >> 4) ^ ((r & 3) | (r >> 1 & 4))) * 32) + (lane & 3) * 8;
    } else {
      at = (first + (lane & 15)) * 128 + (((lane >> 4) ^ ((lane & 15) >> 1)) & 7) * 16;
    }
  }
  // Operand i, counted in 16s from `first`.
  __device__ __forceinline__ bf16x8_t operator()(const char* side, int i, int kk) const {
    if constexpr (ACROSS) {
      // (piece first / 16 + i: first / 16 is a multiple of 4 or 8, and i below that)
      const char* q = side + (at ^ (i * 32)) + kk * 32 * kRow;
      typedef short s4_t __attribute__((ext_vector_type(4)));
      typedef short s8_t __attribute__((ext_vector_type(8)));
      const s4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4_t*)(q));
      const s4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4_t*)(q + 4 * kRow));
      return __builtin_bit_cast(bf16x8_t, (s8_t)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const bf16x8_t*>(side + i * 2048 + (at ^ (kk * 64)));
    }
  }
};

// acc = the tile at (m0, n0) of A B over the contracted elements k0 to k1 (k0 a multiple of 8).
//
// What bounds it is the matrix cores' power: in long runs of these products the clock falls
// to about 2.06 GHz.  A training step of 8192 x 2560 x 50280 (8.4 TFLOP) 7000 to 7120 us on several boxes; without any
// load from memory 5730 in place of 7156, from L2 alone 6 % less, with half the operands'
// reads 2 %, with products alone 5020.  So everything that moves fewer bits through the
// cores is worth more than anything that waits less: 16 x 16 x 32 products 7380 us, 32 x 32 x 16
// 7940; neighbours that share an operand 7295, that do not 7345; while loads issued between
// the products (7030 for 6850), quarter stages fetched four ahead (7382 for 7300) and no wait
// at all (the same) gave nothing.
//
// A stage's first half is multiplied while its second half is read, the second half
// while the next stage's first is: no product waits for LDS.  Between the halves every
// wavefront has read all of the stage, so its place is free for the stage kStages on,
// and the next stage has to be there.  (At the end nothing is on its way to the stages; a
// barrier is due before they hold anything else.)
template <typename Shape, bool A_ACROSS, bool B_ACROSS>
__device__ __forceinline__ void multiply(const Side& A, const Side& B, int64_t m0, int64_t n0, int k0, int k1, Stages<Shape>& s,
                                         Acc<Shape>& acc) {
  constexpr int kMi = Shape::kMi, kS = Shape::kStages;
  constexpr uint32_t kStage = Shape::kTile * kK * 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / Shape::kWn, wn = wave % Shape::kWn;
  const Loader<Shape, A_ACROSS> load_a(A, m0, k0, k1, wave, lane);
  const Loader<Shape, B_ACROSS> load_b(B, n0, k0, k1, wave, lane);
  const Reader<Shape, A_ACROSS> read_a(wm * kMi * 16, lane);
  const Reader<Shape, B_ACROSS> read_b(wn * 64, lane);
  const uint32_t la = lds_address(s.a[0]) + wave * 4096, lb = lds_address(s.b[0]) + wave * 4096;
#pragma unroll
  for (int mi = 0; mi < kMi; ++mi)
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) acc[mi][ni] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int stages = (k1 - k0 + kK - 1) / kK;
  auto load = [&](int t) SSM_INLINE {
    load_a(t * kK, la + (t & (kS - 1)) * kStage);
    load_b(t * kK, lb + (t & (kS - 1)) * kStage);
  };
  bf16x8_t fa[2][kMi], fb[2][4];
  auto read = [&](int t, int kk) SSM_INLINE {
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) fb[kk][ni] = read_b(s.b[t & (kS - 1)], ni, kk);
#pragma unroll
    for (int mi = 0; mi < kMi; ++mi) fa[kk][mi] = read_a(s.a[t & (kS - 1)], mi, kk);
  };
  // kMi + 4 operands read (twice as many accesses where they are turned over) among 4 kMi products
  constexpr int kOperands = kMi + 4, kReads = kMi * (A_ACROSS ? 2 : 1) + 4 * (B_ACROSS ? 2 : 1);
  constexpr int kEach = kReads / kOperands, kBeside = kMi == 8 ? 2 : 1;
  auto products = [&](int kk) SSM_INLINE {
#pragma unroll
    for (int mi = 0; mi < kMi; ++mi)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int ni = mi & 1 ? 3 - j : j;      // (neighbours share an operand)
        acc[mi][ni] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[kk][ni], fa[kk][mi], acc[mi][ni], 0, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < kOperands; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kBeside, 0);
    }
    if constexpr (kReads % kOperands != 0) __builtin_amdgcn_sched_group_barrier(0x100, kReads % kOperands, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 4 * kMi - kOperands * kBeside, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int t = 0; t < kS; ++t) load(t);
  loaded<8 * (kS - 1)>();      // (eight loads a stage)
  block_sync();
  read(0, 0);
  for (int t = 0; t < stages; ++t) {
    read(t, 1);
    products(0);
    loaded_and_read<8 * (kS - 2)>();
    block_sync();
    load(t + kS);      // (past the last stage zeros, so that the counts hold)
    read(t + 1, 0);
    products(1);
  }
  loaded_and_read<0>();
}

// Two neighbouring operands' columns of a row of C, rounded to bf16, as eight in a row:
// quarter q = lane >> 4 of the wavefront has columns 4 q .. + 3 of either; exchanged
// between neighbouring quarters, the even one of a pair has eight of the first, the odd
// one eight of the second.  first_of_eight: where they begin, of the two's 32 columns.
__device__ __forceinline__ uint4 eight_bf16(const float (&a)[4], const float (&b)[4]) {
  const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16x2(a[0], a[1]), pack_bf16x2(b[0], b[1]), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16x2(a[2], a[3]), pack_bf16x2(b[2], b[3]), false, false);
  return make_uint4(lo[0], hi[0], lo[1], hi[1]);
}
__device__ __forceinline__ int first_of_eight(int lane) { return ((lane >> 4) & 1) * 16 + (lane >> 5) * 8; }

// The tile of C that a workgroup computes.  Workgroups go round the eight XCDs, whose
// L2s are their own: each XCD gets a run of tiles, in groups of eight rows of tiles that
// go through the columns together, so that the 32 tiles under way read 8 + 4 panels.
__device__ __forceinline__ void tile_place(int id, int tiles_m, int tiles_n, int* m, int* n) {
  const int total = tiles_m * tiles_n;
  const int each = total >> 3, rest = total & 7, xcd = id & 7;
  const int t = xcd * each + (xcd < rest ? xcd : rest) + (id >> 3);
  const int group = t / (8 * tiles_n), first = group * 8;
  const int high = tiles_m - first < 8 ? tiles_m - first : 8;
  const int in = t - first * tiles_n;
  *m = first + in % high;
  *n = in / high;
}

// ----------------------------------------------------------------- the forward

// What a row's dz is formed from: dz = soft exp2(z log2 e - lse2) less hard q at its
// indices.  soft = hard = 0 for a row that takes no part.
struct RowGrad {
  float lse2, soft, hard;
  int32_t target;       // cross entropy: its column; -1 for none, -2 for a row that takes no part
};
static_assert(sizeof(RowGrad) == kRowGradBytes, "vocab_plan.h agrees");

// A row's statistics are a maximum and the sum of 2^(value - maximum).  The maximum of no
// values, or of values that are all minus infinity, is this: differences of maxima stay numbers.
constexpr float kLowest = -3.0e38f;

// What a row's indices are to the forward: the target; top indices, each looked at by every
// tile; or, of many, those in order, of which a tile takes its own.
enum StatsKind { kTarget, kTops, kSortedTops };
struct Sorted {
  const uint64_t* keys;       // [rows, top]: index << kPlaceBits | place
  const uint16_t* starts;     // [rows, tiles + 1]: how many lie before a tile's columns
};
constexpr int kPlaceBits = 10;
static_assert(1 << kPlaceBits == kMostTops, "a place fits");

// For every tile's columns a row's maximum and sum of exponentials (base 2), and the
// target's logit where it lies in them.  The logits live in the registers of a tile only:
// what leaves is 8 bytes for a row of 256 columns.  8192 x 2560 x 50280: 1690 us, 1245 TFLOP/s
// (a library's product of 8192 x 8192 x 8192 1328, of this form and size 1155 with its logits);
// 2039 x 1536 x 50280 298 us with the join, 1056 TFLOP/s.
template <typename Shape, StatsKind KIND>
__global__ void __launch_bounds__(Shape::kThreads, Shape::kPerSimd) vocab_stats_kernel(VocabArgs a, float2* __restrict__ stats,
                                                                                       float* __restrict__ picked, Sorted sorted, int tiles_m,
                                                                                       int tiles_n) {
  constexpr int kTile = Shape::kTile, kMi = Shape::kMi, kWn = Shape::kWn, kHalf = kMi * 16;
  __shared__ Stages<Shape> s;
  __shared__ float2 part[kWn * kTile];
  int tm, tn;
  tile_place(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;
  Acc<Shape> acc;
  multiply<Shape, false, false>(Side{a.x, a.x_row, a.rows, a.width}, Side{a.w, a.w_row, a.vocab, a.width}, m0, n0, 0, a.width, s, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / kWn, wn = wave % kWn;
  const int n = wn * 64 + 4 * (lane >> 4);          // + ni * 16 + i
  const int columns = (int)(a.vocab - n0 < kTile ? a.vocab - n0 : kTile);
  // The indices of half the tile's rows at a time, of which a thread holds the first kHeld
  // while the tile is dealt with; or where its row's own begin and end, and the first of those.
  constexpr int kHeld = KIND == kTops ? 16 : 1, kPer = Shape::kThreads / kHalf;
  int64_t held[kHeld];
  int own = 0, own_end = 0;
  const int own_row = threadIdx.x / kPer;
  auto entries_of = [&](int half) SSM_INLINE {
    const int64_t left = a.rows - (m0 + half * kHalf);
    return (uint32_t)(left < 0 ? 0 : left > kHalf ? kHalf : left) * (uint32_t)a.top;
  };
  auto hold = [&](int half) SSM_INLINE {
    if constexpr (KIND == kTops) {
      const uint32_t entries = entries_of(half);
      const int64_t* at = a.index + (m0 + half * kHalf) * a.top;
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const uint32_t e = threadIdx.x + j * Shape::kThreads;
        held[j] = e < entries ? at[e] : -1;
      }
    } else {
      const int64_t row = m0 + half * kHalf + own_row;
      own = own_end = 0;
      if (row < a.rows) {
        const uint16_t* at = sorted.starts + row * (tiles_n + 1) + tn;
        own = at[0] + threadIdx.x % kPer;
        own_end = at[1];
      }
      if (own < own_end) held[0] = sorted.keys[row * a.top + own];
    }
  };
  if constexpr (KIND != kTarget) hold(0);
#pragma unroll
  for (int mi = 0; mi < kMi; ++mi) {
    const int m = wm * kHalf + mi * 16 + (lane & 15);
    float top = -__builtin_inff();
#pragma unroll
    for (int ni = 0; ni < 4; ++ni)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float z = n + ni * 16 + i < columns ? acc[mi][ni][i] * a.scale : -__builtin_inff();
        acc[mi][ni][i] = z;
        top = __builtin_fmaxf(top, z);
      }
    if constexpr (KIND == kTarget) {
      if (m0 + m < a.rows) {
        const int64_t v = a.index[m0 + m], d = v - n0 - n;
        if (v >= 0 && d >= 0 && d < 64 && (d & 12) == 0 && n + d < columns) {
          float z = 0.0f;
#pragma unroll
          for (int ni = 0; ni < 4; ++ni)
#pragma unroll
            for (int i = 0; i < 4; ++i) z = d == ni * 16 + i ? acc[mi][ni][i] : z;
          picked[m0 + m] = z;
        }
      }
    }
    top = __builtin_fmaxf(top, __shfl_xor(top, 16));
    top = __builtin_fmaxf(top, __shfl_xor(top, 32));
    const float top2 = __builtin_fmaxf(top * kLog2e, kLowest);
    float sum = 0.0f;
#pragma unroll
    for (int ni = 0; ni < 4; ++ni)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[mi][ni][i], kLog2e, -top2));
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (lane < 16) part[wn * kTile + m] = make_float2(top2, sum);
  }
  block_sync();
  const int m = threadIdx.x;
  if (m < kTile && m0 + m < a.rows) {
    float2 r = part[m];
#pragma unroll
    for (int w = 1; w < kWn; ++w) {
      const float2 o = part[w * kTile + m];
      const float top = __builtin_fmaxf(r.x, o.x);
      r.y = r.y * __builtin_amdgcn_exp2f(r.x - top) + o.y * __builtin_amdgcn_exp2f(o.x - top);
      r.x = top;
    }
    stats[(int64_t)tn * a.rows + m0 + m] = r;
  }
  if constexpr (KIND != kTarget) {
    // The logits at the rows' indices, by way of LDS, half the rows at a time: 16-byte
    // piece c of row r is at place c ^ (r & 15).
    float* z = reinterpret_cast<float*>(s.a[0]);
    static_assert(sizeof(Stages<Shape>) >= kHalf * kTile * 4, "half the tile in fp32 fits");
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      block_sync();
      if (wm == half) {
#pragma unroll
        for (int mi = 0; mi < kMi; ++mi)
#pragma unroll
          for (int ni = 0; ni < 4; ++ni) {
            const int piece = (n >> 2) + ni * 4;
            *reinterpret_cast<f4_t*>(z + (mi * 16 + (lane & 15)) * kTile + (piece ^ (lane & 15)) * 4) = acc[mi][ni];
          }
      }
      block_sync();
      const int64_t first = (m0 + half * kHalf) * a.top;
      auto logit = [&](uint32_t r, uint32_t col) SSM_INLINE { return z[r * kTile + ((col >> 2) ^ (r & 15)) * 4 + (col & 3)]; };
      if constexpr (KIND == kTops) {
        auto pick = [&](uint32_t e, int64_t v) SSM_INLINE {
          const int64_t d = v - n0;
          if (v >= 0 && d >= 0 && d < columns) a.logits[first + e] = logit(e / (uint32_t)a.top, (uint32_t)d);
        };
#pragma unroll
        for (int j = 0; j < kHeld; ++j) pick(threadIdx.x + j * Shape::kThreads, held[j]);
        const uint32_t entries = entries_of(half);
#pragma unroll 4
        for (uint32_t e = threadIdx.x + kHeld * Shape::kThreads; e < entries; e += Shape::kThreads) pick(e, a.index[first + e]);
      } else {
        while (own < own_end) {
          const int64_t at = first + (int64_t)own_row * a.top;
          a.logits[at + (held[0] & (kMostTops - 1))] = logit(own_row, (uint32_t)((held[0] >> kPlaceBits) - n0));
          own += kPer;
          if (own < own_end) held[0] = sorted.keys[at + own];
        }
      }
      if (half == 0) hold(1);
    }
  }
}

// The same for up to 16 rows, where the weights' way from memory is all that counts.  x
// lies in LDS, in the order in which the matrix cores take it; every wavefront reads an
// equal share of the vocabulary's rows, 16 at a time, straight to registers, with eight
// lines of 16 x 64 elements under way and no barrier between them.  Bound by HBM: one row x
// 2560 x 50280 reads 257 MB in 50 us, 5.1 TB/s.  (A call 54.7 us; with twelve lines 54.5, with
// non-temporal loads 61.7: part of the weights is still in the last cache from the call
// before.  16 x 4096 x 50280, 412 MB: 99.8, 97.5 and 96.2.)
// What becomes of the logits: statistics and the target's logit, statistics, or dz of a
// piece of the vocabulary (a.w and a.vocab are then the piece's).
enum FewKind { kFewTarget, kFewStats, kFewDz };
struct FewOut {
  float2* stats;
  float* picked;
  const RowGrad* rows;      // dz [rows, ldz], padded with zeros
  uint16_t* dz;
  int64_t ldz, v0;
};
template <int KMAX, FewKind KIND>
__global__ void __launch_bounds__(512, 2) vocab_few_kernel(VocabArgs a, FewOut out, int share) {
  constexpr int kAhead = 8;
  __shared__ alignas(1024) char xs[KMAX / 32 * 1024];       // [32 contracted elements][lane][8 elements]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quarter = lane >> 4;          // of 32 contracted elements
  const int lines = (a.width + 63) / 64, pieces = (a.width + 7) / 8;
  for (int e = threadIdx.x; e < lines * 8 * 16; e += 512) {
    const int c = e >> 4, m = e & 15;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < pieces) v = *reinterpret_cast<const uint4*>(a.x + (int64_t)(m < a.rows ? m : a.rows - 1) * a.x_row + c * 8);
    *reinterpret_cast<uint4*>(xs + (c >> 2) * 1024 + ((c & 3) * 16 + m) * 16) = v;
  }
  const int id = blockIdx.x * 8 + wave;
  const int64_t first = (int64_t)id * share;
  const int columns = (int)(first >= a.vocab ? 0 : a.vocab - first < share ? a.vocab - first : share);
  const int steps = (columns + 15) / 16 * lines;
  const bool has_row = (lane & 15) < a.rows;
  int64_t target = -1;              // of row lane & 15, counted from the share's first column
  RowGrad g{0.0f, 0.0f, 0.0f, -2};
  if (KIND == kFewTarget && has_row) {
    const int64_t v = a.index[lane & 15];
    target = v < 0 ? -1 : v - first;
  }
  if (KIND == kFewDz && has_row) {
    g = out.rows[lane & 15];
    target = g.target < 0 ? -1 : g.target - out.v0 - first;
  }
  bf16x8_t w[kAhead][2];
  int load_group = 0, load_line = 0;      // what is loaded next
  // A group of 16 rows through a buffer descriptor, so that what lies past a row's end is 0, as in x: an
  // infinity there, of whatever row it is, would make the sum a NaN.  (16 rows stay within 2^27 bytes.)
  constexpr uint32_t kPast = 0x80000000u;
  const uint16_t* group = a.w;
  uint32_t off = 0;       // of the lane's row and its first element
  auto begin_row = [&]() SSM_INLINE {
    // (columns past the share repeat its last)
    const int at = load_group * 16, c = at + (lane & 15);
    group = a.w + (first + at) * a.w_row;
    off = (uint32_t)(((c < columns ? c : columns - 1) - at) * (int)a.w_row * 2 + quarter * 16);
  };
  auto load = [&](bf16x8_t (&f)[2]) SSM_INLINE {
    const auto buffer = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(group), 0, 0x7fffffff, 0x00020000);
    const int k = load_line * 64;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
      f[kk] = __builtin_bit_cast(bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(
                                               buffer, k + kk * 32 + quarter * 8 < a.width ? off : kPast, (k + kk * 32) * 2, 0));
    if (++load_line == lines) {
      load_line = 0;
      ++load_group;
      begin_row();
    }
  };
  if (steps > 0) begin_row();
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (u < steps) load(w[u]);
  block_sync();
  f4_t acc = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
  float top2 = kLowest, sum = 0.0f;                // of row lane & 15, over this lane's columns
  int line = 0, n = 4 * quarter;                   // columns n .. + 3 of the share
  auto step = [&](const bf16x8_t (&f)[2]) SSM_INLINE {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[kk], *reinterpret_cast<const bf16x8_t*>(xs + (line * 2 + kk) * 1024 + lane * 16),
                                                    acc, 0, 0, 0);
    if (++line < lines) return;
    line = 0;
    if constexpr (KIND == kFewDz) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = g.soft * __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i], a.scale * kLog2e, -g.lse2));
        const float d = g.target == -2 ? 0.0f : p - (n + i == target ? g.hard : 0.0f);
        if (has_row && n + i < columns) out.dz[(lane & 15) * out.ldz + first + n + i] = f32_to_bf16_rne(d);
      }
    } else {
      float top = top2;
      float z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = acc[i] * a.scale;
        z[i] = n + i < columns ? v * kLog2e : -__builtin_inff();
        top = __builtin_fmaxf(top, z[i]);
        if (KIND == kFewTarget && target == n + i && n + i < columns) out.picked[lane & 15] = v;
      }
      sum *= __builtin_amdgcn_exp2f(top2 - top);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += __builtin_amdgcn_exp2f(z[i] - top);
      top2 = top;
    }
    acc = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    n += 16;
  };
  for (int at = 0; at < steps; at += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (at + u < steps) {
        step(w[u]);
        if (at + u + kAhead < steps) load(w[u]);
      }
  }
  if constexpr (KIND == kFewDz) {
    // the padding, by the wavefront of the last column
    if (columns > 0 && first + columns == a.vocab && has_row)
      for (int64_t c = a.vocab + quarter; c < out.ldz; c += 4) out.dz[(lane & 15) * out.ldz + c] = 0;
  } else {
#pragma unroll
    for (int o = 16; o < 64; o *= 2) {
      const float t = __shfl_xor(top2, o), v = __shfl_xor(sum, o), top = __builtin_fmaxf(top2, t);
      sum = sum * __builtin_amdgcn_exp2f(top2 - top) + v * __builtin_amdgcn_exp2f(t - top);
      top2 = top;
    }
    if (lane < 16 && has_row) out.stats[(int64_t)id * a.rows + lane] = make_float2(top2, sum);
  }
}

// The logits at the indices of few rows, one wavefront for each: at most 16 top reads of a row
// of weights.
__global__ void __launch_bounds__(256) vocab_pick_kernel(VocabArgs a) {
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (e >= a.rows * a.top) return;
  const int64_t v = a.index[e];
  if (v < 0 || v >= a.vocab) return;
  const uint16_t* x = a.x + e / a.top * a.x_row;
  const uint16_t* w = a.w + v * a.w_row;
  float z = 0.0f;
  for (int k = lane * 8; k < a.width; k += 512) {
    float xv[8], wv[8];
    Vec16<uint16_t>::unpack(*reinterpret_cast<const uint4*>(x + k), xv);
    Vec16<uint16_t>::unpack(*reinterpret_cast<const uint4*>(w + k), wv);
#pragma unroll
    for (int i = 0; i < 8; ++i) z = __builtin_fmaf(xv[i], wv[i], z);
  }
#pragma unroll
  for (int o = 1; o < 64; o *= 2) z += __shfl_xor(z, o);
  if (lane == 0) a.logits[e] = z * a.scale;
}

// What one row's indices and teacher logits say, over a wavefront: whether the row
// counts (an index that is in the vocabulary and not without weight), whether an index
// lies past the vocabulary, and the softmax of the teacher's.
struct Teacher {
  bool counts, past;
  float top, sum;       // the largest of the teacher's logits, and the sum of e^((logit - top) / temperature)
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
      const float l = a.teacher[row * a.top + k];
      top = top != top ? top : (l != l ? l : __builtin_fmaxf(top, l));
    }
  }
  t.top = wave_max(top);
  t.past = __any(past);
  t.counts = !t.past && t.top != -__builtin_inff();
  float sum = 0.0f;
  for (int k = lane; k < a.top; k += 64)
    if (a.index[row * a.top + k] >= 0) sum += __builtin_amdgcn_exp2f((a.teacher[row * a.top + k] - t.top) * t2);
  t.sum = wave_sum(sum);
  return t;
}

// A row's indices in the vocabulary as keys in order, all ones for the others, by a wavefront
// in n (a power of two, at least top) words of LDS; all wavefronts of a workgroup together.
__device__ __forceinline__ void sort_row(const VocabArgs& a, int64_t row, int n, int lane, uint64_t* keys) {
  for (int i = lane; i < n; i += 64) {
    uint64_t key = ~0ull;
    if (row < a.rows && i < a.top) {
      const int64_t v = a.index[row * a.top + i];
      if (v >= 0 && v < a.vocab) key = (uint64_t)v << kPlaceBits | i;
    }
    keys[i] = key;
  }
  block_sync();
  for (int k = 2; k <= n; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      for (int i = lane; i < n / 2; i += 64) {
        const int lo = (i & ~(j - 1)) * 2 + (i & (j - 1)), hi = lo + j;
        const uint64_t x = keys[lo], y = keys[hi];
        if ((x > y) == ((lo & k) == 0)) keys[lo] = y, keys[hi] = x;
      }
      block_sync();
    }
}

// The forward's: rows' keys and where each tile of 2^shift columns begins among them.  4096
// rows of 64 indices 13 us, of 1024 105: a sort's 21 or 55 rounds through LDS.
__global__ void __launch_bounds__(256) vocab_sort_kernel(VocabArgs a, uint64_t* __restrict__ out, uint16_t* __restrict__ starts, int shift,
                                                         int tiles_n, int n) {
  __shared__ uint64_t sorted[4][kMostTops];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * 4 + wave;
  uint64_t* keys = sorted[wave];
  sort_row(a, row, n, lane, keys);
  if (row >= a.rows) return;
  for (int i = lane; i < a.top; i += 64) out[row * a.top + i] = keys[i];
  uint16_t* s = starts + row * (tiles_n + 1);
  auto tile_of = [&](int i) SSM_INLINE {
    const uint64_t t = keys[i] >> kPlaceBits >> shift;
    return t < (uint64_t)tiles_n ? (int)t : tiles_n;
  };
  for (int i = lane; i <= a.top; i += 64) {
    const int to = i < a.top ? tile_of(i) : tiles_n;
    for (int t = i ? tile_of(i - 1) + 1 : 0; t <= to; ++t) s[t] = (uint16_t)i;
  }
}

// A row's log sum of exponentials from its pieces', and its loss.  A workgroup of 1024
// threads takes `each` rows (a power of two up to 16), 1024 / each threads a row for the
// pieces and a wavefront a row for the loss.  Short and by reads: 8192 rows of 197 pieces (13 MB)
// 6.5 us; with 4096 rows' 64 teacher logits 8.3.
template <bool ONE>
__global__ void __launch_bounds__(1024) vocab_loss_kernel(VocabArgs a, const float2* __restrict__ stats,
                                                          const float* __restrict__ picked, int pieces, int each) {
  __shared__ float2 part[1024];
  __shared__ float logs[16];
  const int64_t row0 = (int64_t)blockIdx.x * each;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  {
    const int64_t row = row0 + (threadIdx.x & (each - 1));
    const int per = 1024 / each;
    float2 r = make_float2(kLowest, 0.0f);
    if (row < a.rows) {
#pragma unroll 4
      for (int n = threadIdx.x / each; n < pieces; n += per) {
        const float2 v = stats[(int64_t)n * a.rows + row];
        const float top = __builtin_fmaxf(r.x, v.x);
        r.y = r.y * __builtin_amdgcn_exp2f(r.x - top) + v.y * __builtin_amdgcn_exp2f(v.x - top);
        r.x = top;
      }
    }
    part[threadIdx.x] = r;
  }
  for (int half = 512; half >= each; half /= 2) {
    block_sync();
    if (threadIdx.x < half) {
      const float2 r = part[threadIdx.x], v = part[threadIdx.x + half];
      const float top = __builtin_fmaxf(r.x, v.x);
      part[threadIdx.x] = make_float2(top, r.y * __builtin_amdgcn_exp2f(r.x - top) + v.y * __builtin_amdgcn_exp2f(v.x - top));
    }
  }
  block_sync();
  if (threadIdx.x < each && row0 + threadIdx.x < a.rows) {
    const float2 r = part[threadIdx.x];
    // r.x is the largest logit in base 2, of which ln 2 gives back its value to an ulp
    const float lse = __builtin_fmaf(r.x, kLn2, __builtin_amdgcn_logf(r.y) * kLn2);
    a.lse[row0 + threadIdx.x] = lse;
    logs[threadIdx.x] = lse;
    if constexpr (ONE) {
      const int64_t v = a.index[row0 + threadIdx.x];
      float loss = 0.0f;
      if (v >= a.vocab) loss = __builtin_nanf("");
      else if (v >= 0) loss = (lse - picked[row0 + threadIdx.x]) + a.z_loss * lse * lse;
      a.loss[row0 + threadIdx.x] = loss;
    }
  }
  if constexpr (!ONE) {
    block_sync();
    const int64_t row = row0 + wave;
    if (wave >= each || row >= a.rows) return;
    const float lse = logs[wave];
    const Teacher t = teacher_of(a, row, lane);
    float loss = 0.0f;
    for (int k = lane; k < a.top; k += 64) {
      const int64_t v = a.index[row * a.top + k];
      if (v < 0 || v >= a.vocab) a.logits[row * a.top + k] = 0.0f;
    }
    if (t.past) loss = __builtin_nanf("");
    else if (t.counts) {
      const float t2 = kLog2e / a.temperature;
      const float logsum = __builtin_amdgcn_logf(t.sum);
      for (int k = lane; k < a.top; k += 64) {
        const float l2 = (a.teacher[row * a.top + k] - t.top) * t2 - logsum;     // log2 q
        const float q = __builtin_amdgcn_exp2f(l2);
        if (a.index[row * a.top + k] >= 0 && q != 0.0f)
          loss = __builtin_fmaf(q, __builtin_fmaf(l2, kLn2, lse - a.logits[row * a.top + k]), loss);
      }
      loss = wave_sum(loss) * a.temperature * a.temperature;
    }
    if (lane == 0) a.loss[row] = loss;
  }
}

// ---------------------------------------------------------------- the gradients

// A wavefront a row: what its dz is formed from, and (for dweight) its x, zeros where the
// row takes no part, whatever x holds there.  Distillation: also hard q for each of the
// row's indices, where the same index twice has the sum of both: in order, they lie together.
// 8192 rows of 2560 14 us, 4096 rows of 1536 with 64 indices 14, with 1024 126 (comparing every
// pair: 20 and 2840).
template <bool ONE>
__global__ void __launch_bounds__(256) vocab_rows_kernel(VocabArgs a, RowGrad* __restrict__ rows, float* __restrict__ hard,
                                                         uint16_t* __restrict__ x, int n) {
  __shared__ uint64_t sorted[ONE ? 1 : 4][ONE ? 1 : kMostTops];
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  uint64_t* keys = sorted[ONE ? 0 : threadIdx.x >> 6];
  if constexpr (!ONE) sort_row(a, row, n, lane, keys);
  if (row >= a.rows) return;
  RowGrad g{0.0f, 0.0f, 0.0f, -2};
  const float lse = a.lse_in[row];
  if constexpr (ONE) {
    const int64_t v = a.index[row];
    if (v >= 0 && v < a.vocab) {
      const float d = a.dloss[row] * a.scale;
      g = RowGrad{lse * kLog2e, d * __builtin_fmaf(2.0f * a.z_loss, lse, 1.0f), d, (int32_t)v};
    }
  } else {
    const Teacher t = teacher_of(a, row, lane);
    if (t.counts) {
      // (a.scale is over the temperature: its square leaves one of them)
      const float d = a.dloss[row] * a.temperature * a.temperature * a.scale;
      g = RowGrad{lse * kLog2e, d, d, -1};
      const float t2 = kLog2e / a.temperature, by = d / t.sum;
      const int64_t at = row * a.top;
      for (int i = lane; i < a.top; i += 64) {
        const uint64_t v = keys[i] >> kPlaceBits;
        if (v >= (uint64_t)a.vocab) break;
        int e = i;
        while (e > 0 && keys[e - 1] >> kPlaceBits == v) --e;
        float q = 0.0f;
        for (; e < a.top && keys[e] >> kPlaceBits == v; ++e)
          q += __builtin_amdgcn_exp2f((a.teacher[at + (keys[e] & (kMostTops - 1))] - t.top) * t2);
        hard[at + (keys[i] & (kMostTops - 1))] = q * by;
      }
    }
  }
  if (lane == 0) rows[row] = g;
  if (x != nullptr) {
    const uint4* from = reinterpret_cast<const uint4*>(a.x + row * a.x_row);
    uint4* to = reinterpret_cast<uint4*>(x + row * a.width);
#pragma unroll 4
    for (int e = lane; e < a.width / 8; e += 64) to[e] = g.target == -2 ? make_uint4(0, 0, 0, 0) : from[e];
  }
}

// dz of a piece of the vocabulary, [rows, ldz] and padded with zeros, from the logits,
// computed once more: storing them in the forward would cost 2 rows vocab bytes of memory
// and gain a quarter of the step.  dz is rounded to bf16 (2^-8 of each element), the matrix
// cores' type: a piece of fp32 would double its bytes and triple its products.  8192 x 2560 x
// 16384: 600 us, 1145 TFLOP/s, with 268 MB written.
template <typename Shape>
__global__ void __launch_bounds__(Shape::kThreads, Shape::kPerSimd) vocab_dz_kernel(VocabArgs a, const RowGrad* __restrict__ rows, int64_t v0, int columns,
                                                          uint16_t* __restrict__ dz, int64_t ldz, int tiles_m, int tiles_n) {
  constexpr int kTile = Shape::kTile, kMi = Shape::kMi;
  __shared__ Stages<Shape> s;
  int tm, tn;
  tile_place(blockIdx.x, tiles_m, tiles_n, &tm, &tn);
  const int64_t m0 = (int64_t)tm * kTile, n0 = (int64_t)tn * kTile;
  Acc<Shape> acc;
  multiply<Shape, false, false>(Side{a.x, a.x_row, a.rows, a.width}, Side{a.w + v0 * a.w_row, a.w_row, columns, a.width}, m0, n0, 0,
                                a.width, s, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / Shape::kWn, wn = wave % Shape::kWn;
  const float s2 = a.scale * kLog2e;
#pragma unroll
  for (int mi = 0; mi < kMi; ++mi) {
    const int64_t m = m0 + wm * kMi * 16 + mi * 16 + (lane & 15);
    RowGrad g{0.0f, 0.0f, 0.0f, -2};
    if (m < a.rows) g = rows[m];
    const int64_t target = g.target < 0 ? -1 : g.target - v0;
#pragma unroll
    for (int ni = 0; ni < 4; ni += 2) {
      float d[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t n = n0 + wn * 64 + (ni + h) * 16 + 4 * (lane >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = g.soft * __builtin_amdgcn_exp2f(__builtin_fmaf(acc[mi][ni + h][i], s2, -g.lse2));
          d[h][i] = g.target == -2 || n + i >= columns ? 0.0f : p - (n + i == target ? g.hard : 0.0f);
        }
      }
      const uint4 v = eight_bf16(d[0], d[1]);
      const int64_t n = n0 + wn * 64 + ni * 16 + first_of_eight(lane);
      if (m < a.rows && n < ldz) *reinterpret_cast<uint4*>(dz + m * ldz + n) = v;
    }
  }
}

// Distillation: dz at the teacher's indices, formed from the stored logits in place of
// the rounded softmax, so that p - q is rounded once.  4096 x 64 indices 7 us a piece.
__global__ void __launch_bounds__(256) vocab_fix_kernel(VocabArgs a, const RowGrad* __restrict__ rows, const float* __restrict__ hard,
                                                        int64_t v0, int columns, uint16_t* __restrict__ dz, int64_t ldz) {
  const int64_t entries = (int64_t)a.rows * a.top;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < entries; e += (int64_t)gridDim.x * 256) {
    const int64_t v = a.index[e], n = v - v0;
    if (v < v0 || n >= columns) continue;
    const int64_t row = e / a.top;
    const RowGrad g = rows[row];
    if (g.target == -2) continue;
    const float p = g.soft * __builtin_amdgcn_exp2f(__builtin_fmaf(a.logits_in[e], kLog2e, -g.lse2));
    dz[row * ldz + n] = f32_to_bf16_rne(p - hard[e]);
  }
}

// What becomes of a tile of C: added to fp32 sums (`add`: of those there are; no other
// workgroup has the tile), which are stored, or, with out, rounded to bf16.
template <typename Shape>
__device__ __forceinline__ void store_tile(Acc<Shape>& acc, int64_t m0, int64_t n0, int rows, int columns, float* sum, bool add,
                                           uint16_t* out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / Shape::kWn, wn = wave % Shape::kWn;
#pragma unroll
  for (int mi = 0; mi < Shape::kMi; ++mi) {
    const int64_t m = m0 + wm * Shape::kMi * 16 + mi * 16 + (lane & 15);
#pragma unroll
    for (int ni = 0; ni < 4; ni += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t n = n0 + wn * 64 + (ni + h) * 16 + 4 * (lane >> 4);
        f4_t* at = reinterpret_cast<f4_t*>(sum + m * columns + n);
        if (m < rows && n < columns) {
          if (add) acc[mi][ni + h] += *at;
          if (!out) *at = acc[mi][ni + h];
        }
      }
      if (out) {
        float v[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[h][i] = acc[mi][ni + h][i];
        const uint4 w = eight_bf16(v[0], v[1]);
        const int64_t n = n0 + wn * 64 + ni * 16 + first_of_eight(lane);
        if (m < rows && n < columns) *reinterpret_cast<uint4*>(out + m * columns + n) = w;
      }
    }
  }
}

// A piece's two products, side by side so that neither leaves CUs idle alone:
//   dweight[v0 ..] = dz^T x, the rows in slices, and its part of dx = dz weight, the piece's
//   columns in slices.
// 8192 x 2560 x 16384: 1055 us, 1300 TFLOP/s, as the library's largest products.
struct Products {
  const uint16_t* dz;       // [rows, ldz], zeros from `columns` on
  int64_t ldz;
  const uint16_t* x;        // [rows, width]
  const uint16_t* w;        // the piece's rows of weight
  int64_t w_row;
  float* x_sums;            // [slices][rows, width]
  float* w_sums;            // [slices][columns, width]
  uint16_t* dx;             // NULL: the sums
  uint16_t* dw;             // the piece's rows; NULL: the sums
  int32_t x_add;            // x_sums hold those of the pieces before
  int32_t rows, width, columns;
  int32_t x_slice, w_slice;       // contracted elements of a slice, multiples of kK
  int32_t tiles_m, tiles_n, tiles_d;
  int32_t x_items, w_items;
  int32_t x_first;
};

template <typename Shape>
__global__ void __launch_bounds__(Shape::kThreads, Shape::kPerSimd) vocab_products_kernel(Products a) {
  __shared__ Stages<Shape> s;
  const int first = a.x_first ? a.x_items : a.w_items;
  const bool dx = ((int)blockIdx.x < first) == (a.x_first != 0);
  const int id = (int)blockIdx.x < first ? blockIdx.x : blockIdx.x - first;
  const int tiles = dx ? a.tiles_m : a.tiles_n, each = tiles * a.tiles_d, slice = id / each;
  int tm, tn;
  tile_place(id % each, tiles, a.tiles_d, &tm, &tn);
  const int64_t m0 = (int64_t)tm * Shape::kTile, n0 = (int64_t)tn * Shape::kTile;
  Acc<Shape> acc;
  if (dx) {
    const int k0 = slice * a.x_slice, end = (a.columns + 7) & ~7, k1 = k0 + a.x_slice < end ? k0 + a.x_slice : end;
    multiply<Shape, false, true>(Side{a.dz, a.ldz, a.rows, end}, Side{a.w, a.w_row, a.width, a.columns}, m0, n0, k0, k1, s, acc);
    store_tile<Shape>(acc, m0, n0, a.rows, a.width, a.x_sums + (int64_t)slice * a.rows * a.width, a.x_add != 0, a.dx);
  } else {
    const int k0 = slice * a.w_slice, k1 = k0 + a.w_slice < a.rows ? k0 + a.w_slice : a.rows;
    multiply<Shape, true, true>(Side{a.dz, a.ldz, (int32_t)a.ldz, a.rows}, Side{a.x, a.width, a.width, a.rows}, m0, n0, k0, k1, s, acc);
    store_tile<Shape>(acc, m0, n0, a.columns, a.width, a.w_sums + (int64_t)slice * a.columns * a.width, false, a.dw);
  }
}

// bf16 from the sums of its parts, in order; four elements a thread.  (Two of 4096 x 1536: 11 us.)
__global__ void __launch_bounds__(256) vocab_sum_kernel(const float4* __restrict__ sums, int parts, int64_t each, uint2* __restrict__ out) {
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < each; e += (int64_t)gridDim.x * 256) {
    float4 v = sums[e];
#pragma unroll 4
    for (int p = 1; p < parts; ++p) {
      const float4 o = sums[p * each + e];
      v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
    }
    out[e] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

template <FewKind KIND>
void launch_few(const Few& few, const VocabArgs& a, const FewOut& out, hipStream_t s) {
  auto k = a.width <= kFewWidth / 2 ? vocab_few_kernel<kFewWidth / 2, KIND> : vocab_few_kernel<kFewWidth, KIND>;
  hipLaunchKernelGGL(k, dim3((unsigned)few.groups), dim3(512), 0, s, a, out, (int)few.share);
}

unsigned fours(int64_t n) { return (unsigned)((n + 3) / 4); }

void launch_sum(const float* sums, int parts, int64_t elems, uint16_t* out, hipStream_t s) {
  const int64_t each = elems / 4;
  hipLaunchKernelGGL(vocab_sum_kernel, dim3((unsigned)std::min<int64_t>((each + 255) / 256, 1 << 20)), dim3(256), 0, s,
                     reinterpret_cast<const float4*>(sums), parts, each, reinterpret_cast<uint2*>(out));
}

// The words in which a row's indices are put in order.
int sort_words(const VocabArgs& a) {
  int n = 64;
  while (n < a.top) n *= 2;
  return n;
}

template <typename Shape>
void launch_stats(const VocabArgs& a, const FwdParts& at, float2* stats, float* picked, hipStream_t s) {
  const int tm = (int)tiles(a.rows, Shape::kTile), tn = (int)tiles(a.vocab, Shape::kTile);
  Sorted sorted{};
  if (at.sorted) {
    uint64_t* keys = reinterpret_cast<uint64_t*>(a.work + at.keys);
    uint16_t* starts = reinterpret_cast<uint16_t*>(a.work + at.starts);
    hipLaunchKernelGGL(vocab_sort_kernel, dim3(fours(a.rows)), dim3(256), 0, s, a, keys, starts, Shape::kTile == 256 ? 8 : 7, tn, sort_words(a));
    sorted = Sorted{keys, starts};
  }
  auto k = !a.teacher ? vocab_stats_kernel<Shape, kTarget> : at.sorted ? vocab_stats_kernel<Shape, kSortedTops> : vocab_stats_kernel<Shape, kTops>;
  hipLaunchKernelGGL(k, dim3((unsigned)(tm * tn)), dim3(Shape::kThreads), 0, s, a, stats, picked, sorted, tm, tn);
}

template <typename Shape>
void launch_dz(const VocabArgs& a, const RowGrad* rows, int64_t v0, int columns, uint16_t* dz, int64_t ldz, hipStream_t s) {
  const int tm = (int)tiles(a.rows, Shape::kTile), tn = (int)tiles(columns, Shape::kTile);
  hipLaunchKernelGGL(vocab_dz_kernel<Shape>, dim3((unsigned)(tm * tn)), dim3(Shape::kThreads), 0, s, a, rows, v0, columns, dz, ldz, tm,
                     tn);
}

template <typename Shape>
void launch_products(Products& p, int x_slices, int w_slices, hipStream_t s) {      // (0 slices: not wanted)
  p.tiles_m = (int32_t)tiles(p.rows, Shape::kTile);
  p.tiles_n = (int32_t)tiles(p.columns, Shape::kTile);
  p.tiles_d = (int32_t)tiles(p.width, Shape::kTile);
  p.x_items = p.tiles_m * p.tiles_d * x_slices;
  p.w_items = p.tiles_n * p.tiles_d * w_slices;
  p.x_first = p.x_slice >= p.w_slice;      // the longer ones first
  hipLaunchKernelGGL(vocab_products_kernel<Shape>, dim3((unsigned)(p.x_items + p.w_items)), dim3(Shape::kThreads), 0, s, p);
}

}  // namespace

hipError_t launch_vocab_fwd(const VocabArgs& a, hipStream_t s) {
  const FwdParts at(a);
  float2* stats = reinterpret_cast<float2*>(a.work + at.stats);
  float* picked = reinterpret_cast<float*>(a.work + at.picked);
  const bool one = a.teacher == nullptr;
  if (at.few.few) {
    FewOut out{};
    out.stats = stats;
    out.picked = picked;
    if (one) launch_few<kFewTarget>(at.few, a, out, s);
    else launch_few<kFewStats>(at.few, a, out, s);
    if (!one) hipLaunchKernelGGL(vocab_pick_kernel, dim3(fours(a.rows * a.top)), dim3(256), 0, s, a);
  } else if (at.large) {
    launch_stats<Large>(a, at, stats, picked, s);
  } else {
    launch_stats<Small>(a, at, stats, picked, s);
  }
  int each = 1;
  while (each < 16 && each < a.rows) each *= 2;
  auto l = one ? vocab_loss_kernel<true> : vocab_loss_kernel<false>;
  hipLaunchKernelGGL(l, dim3((unsigned)((a.rows + each - 1) / each)), dim3(1024), 0, s, a, stats, picked, (int)at.pieces, each);
  return hipGetLastError();
}

hipError_t launch_vocab_bwd(const VocabArgs& a, hipStream_t s) {
  const BwdParts at(a);
  const Cut& cut = at.cut;
  RowGrad* rows = reinterpret_cast<RowGrad*>(a.work + at.rows);
  float* hard = reinterpret_cast<float*>(a.work + at.hard);
  uint16_t* x = reinterpret_cast<uint16_t*>(a.work + at.x);
  uint16_t* dz = reinterpret_cast<uint16_t*>(a.work + at.dz);
  float* x_sums = reinterpret_cast<float*>(a.work + at.x_sums);
  float* w_sums = reinterpret_cast<float*>(a.work + at.w_sums);
  const bool one = a.teacher == nullptr;
  auto rk = one ? vocab_rows_kernel<true> : vocab_rows_kernel<false>;
  hipLaunchKernelGGL(rk, dim3(fours(a.rows)), dim3(256), 0, s, a, rows, hard, a.dw ? x : nullptr, one ? 0 : sort_words(a));
  int x_slices = 0;
  for (int64_t v0 = 0; v0 < a.vocab; v0 += cut.piece) {
    const Piece piece(a, cut, v0);
    const int columns = piece.columns;
    const Few few(a, columns);
    if (few.few) {
      VocabArgs part_of = a;
      part_of.w = a.w + v0 * a.w_row;
      part_of.vocab = columns;
      FewOut out{};
      out.rows = rows;
      out.dz = dz;
      out.ldz = at.ldz;
      out.v0 = v0;
      launch_few<kFewDz>(few, part_of, out, s);
    } else if (large_tiles(a.rows, columns, a.width, std::max(1, a.cus))) {
      launch_dz<Large>(a, rows, v0, columns, dz, at.ldz, s);
    } else {
      launch_dz<Small>(a, rows, v0, columns, dz, at.ldz, s);
    }
    if (!one)
      hipLaunchKernelGGL(vocab_fix_kernel, dim3((unsigned)std::min<int64_t>(((int64_t)a.rows * a.top + 255) / 256, 1 << 16)), dim3(256), 0,
                         s, a, rows, hard, v0, columns, dz, at.ldz);
    Products p{};
    p.dz = dz;
    p.ldz = at.ldz;
    p.x = x;
    p.w = a.w + v0 * a.w_row;
    p.w_row = a.w_row;
    p.rows = a.rows;
    p.width = a.width;
    p.columns = columns;
    p.x_slice = piece.x_slice;
    p.w_slice = piece.w_slice;
    // dx is rounded once, behind the last piece: by its products, or over the slices
    const bool last = v0 + columns == a.vocab;
    p.x_sums = x_sums;
    p.x_add = v0 > 0;
    p.dx = last && cut.x_slices == 1 ? a.dx : nullptr;
    p.w_sums = w_sums;
    uint16_t* dw = a.dw ? a.dw + v0 * a.width : nullptr;
    p.dw = cut.w_slices == 1 ? dw : nullptr;
    if (cut.large) launch_products<Large>(p, a.dx ? piece.x_slices : 0, a.dw ? piece.w_slices : 0, s);
    else launch_products<Small>(p, a.dx ? piece.x_slices : 0, a.dw ? piece.w_slices : 0, s);
    if (dw && !p.dw) launch_sum(w_sums, piece.w_slices, (int64_t)columns * a.width, dw, s);
    x_slices = std::max(x_slices, piece.x_slices);      // (the last piece may have fewer)
  }
  if (a.dx && cut.x_slices > 1) launch_sum(x_sums, x_slices, (int64_t)a.rows * a.width, a.dx, s);
  return hipGetLastError();
}

}  // namespace ssm
