// gfx950 kernels of libssmscan: the gated linear recurrence
// h_t = a_t h_{t-1} + m_t u_t for each channel, its gradients and its single-token
// step.  Both directions read every tensor once (gscan_kernel.h: the chain of tiles).
#include <algorithm>

#include "gscan_kernel.h"

namespace ssm {
namespace {

// Steps of a wavefront, what its registers hold, and wavefronts of a tile.  More steps need
// fewer words of the chain and put more loads under way; the registers of two workgroups of
// 8 wavefronts a CU hold 16 (us, 8 x 2048 x 5120 and 1 x 65537 x 2560, steps x wavefronts: 16 x 8
// 152 and 197, 8 x 16 143 and 217, 8 x 8 165 and 335, 16 x 4 161 and 282, 16 x 16 164 and 199).
constexpr int kFwdSteps = 16, kFwdWaves = 8;
constexpr int kBwdSteps = 8, kBwdWaves = 8;       // (back, a step keeps three times as much)
constexpr int kFwdApart = kGsSegment / kFwdSteps, kBwdApart = kGsSegment / kBwdSteps;      // wavefronts between stored states

static_assert(kFwdWaves == kGsWaves && kBwdWaves == kGsWaves && kGsFwdTile == kFwdSteps * kFwdWaves && kGsBwdTile == kBwdSteps * kBwdWaves, "model.h agrees");
static_assert(kGsFwdTile % kGsSegment == 0 && kGsBwdTile % kGsSegment == 0, "tiles begin with a stored state");

// Three forms of the kernels: the plain one; one whose outputs go past the caches; and one for
// short sequences, several strips of which share a workgroup.
enum Form { kPlain, kStream, kShort };

// The tile that a workgroup takes: its place in the chain and its strip; short sequences have
// one tile, and strips are told by wavefronts.
template <Form FORM>
__device__ __forceinline__ void take_tile(const Chain& c, int* tile, int* strip) {
  int n = blockIdx.x;
  if (FORM != kShort && c.tiles > 1) {
    __shared__ uint32_t taken;
    if (threadIdx.x == 0) taken = atomicAdd(c.next, 1u);
    block_sync();
    n = (int)__builtin_amdgcn_readfirstlane(taken);
  }
  *tile = FORM == kShort ? 0 : n / c.strips;
  *strip = FORM == kShort ? n : n % c.strips;
}

// Where a wavefront's steps lie.
template <int CH, int kSteps, Form FORM>
struct Place {
  int64_t b, t0, left, tok;      // batch row; first step; steps of the sequence from there; token
  int64_t d;                     // the lane's first channel
  int n;                         // steps of this wavefront's kSteps that there are
  bool in;                       // whether the channel is
  __device__ __forceinline__ Place(const GscanArgs& a, const Chain& c, int tile, int strip, int steps, int wave, int lane) {
    const int per_row = (int)((a.width + 64 * CH - 1) / (64 * CH));
    b = strip / per_row;
    d = (int64_t)(strip % per_row) * (64 * CH) + lane * CH;
    const bool there = FORM != kShort || strip < c.strips;      // (the last workgroup's may not be)
    in = d < a.width && there;
    t0 = (int64_t)tile * steps + wave * kSteps;
    left = there ? a.seqlen - t0 : -1;
    n = left < 0 ? 0 : left > kSteps ? kSteps : (int)left;
    tok = b * a.seqlen + t0;
  }
  // Byte offset of the lane's channels in a row of values of `size` bytes, in the
  // wavefront's step j (not needed where all steps are there).
  __device__ __forceinline__ uint32_t off(int size, int j = 0) const { return in && j < n ? (uint32_t)d * size : kNowhere; }
};

// The forward.  A wavefront's steps are h -> P_j h + H_j with P and H running products and
// sums, so what enters it is all that is missing when its loads are through: the wavefronts'
// last (P, H) meet in LDS, the tile's in the chain.  Bound by HBM: x, r and i are read once,
// out written once.  8 x 2048 x 5120 bf16 with all three (671 MB) 143 us, 4.7 TB/s; 1 x 65537 x
// 2560 of two tensors (1007 MB) 195 us, 5.2 TB/s, what a large copy reaches (5.1).  An odd width reads
// the lines at the borders of strips twice: 3 x 1021 x 1537 fp32 (76 MB) 26 us and bf16 (39 MB) 21.
template <typename T, bool RATE, bool LERP, bool GATE, int CH, Form FORM>
__global__ void __launch_bounds__(64 * kFwdWaves, 4) gscan_fwd_kernel(GscanArgs a, Chain c) {
  __shared__ float2 parts[kFwdWaves][CH][64];
  __shared__ float enter[FORM == kShort ? kFwdWaves : 1][CH][64];      // at a strip's first wavefront
  int tile, strip;
  take_tile<FORM>(c, &tile, &strip);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = FORM == kShort ? wave & -c.waves : 0;      // of the strip's wavefronts
  if (FORM == kShort) strip = (strip * kFwdWaves + wave) / c.waves;
  constexpr int kSteps = kFwdSteps;
  constexpr bool kGrow = RATE && LERP;      // (a rate below 0; without LERP its m is NaN)
  const Place<CH, kSteps, FORM> at(a, c, tile, strip, kGsFwdTile, wave - first, lane);
  const uint32_t off = at.off(sizeof(T));
  float rate2[CH], P[kSteps][CH], H[kSteps][CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) rate2[k] = RATE && at.in ? a.rate[at.d + k] * kLog2e : 0.0f;
  auto steps = [&](auto whole) SSM_INLINE {
    constexpr bool kWhole = decltype(whole)::value;      // all kSteps are there
    // all loads first: a wavefront has 16 steps of three tensors under way
    const Rows rx(a.x, at.tok, a.x_row, sizeof(T)), rr(a.r, at.tok, a.r_row, sizeof(T)), ri(a.i, at.tok, a.i_row, sizeof(T));
    uint32_t x[kSteps], r[kSteps], i[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const uint32_t o = kWhole ? off : at.off(sizeof(T), j);
      r[j] = load_raw<T, CH>(rr, j, o);
      if constexpr (GATE) i[j] = load_raw<T, CH>(ri, j, o);
      x[j] = load_raw<T, CH>(rx, j, o);
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float ea, em;
        decay<RATE, LERP>(gate_exp<!RATE>(raw_value<T>(r[j], k)), rate2[k], &ea, &em);
        float u = raw_value<T>(x[j], k);
        if constexpr (GATE) u *= gate_open(gate_exp<false>(raw_value<T>(i[j], k)));
        u *= em;
        if (!kWhole && j >= at.n) ea = 1.0f, u = 0.0f;
        P[j][k] = j ? P[j - 1][k] * ea : ea;
        H[j][k] = j ? __builtin_fmaf(ea, H[j - 1][k], u) : u;
      }
  };
  if (at.n == kSteps) steps(std::true_type{});
  else steps(std::false_type{});
#pragma unroll
  for (int k = 0; k < CH; ++k) parts[wave][k][lane] = make_float2(P[kSteps - 1][k], H[kSteps - 1][k]);
  block_sync();
  if (wave == first) {
    float hin[CH];
    if (FORM != kShort && c.tiles > 1) {
      float tp[CH], th[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        tp[k] = P[kSteps - 1][k], th[k] = H[kSteps - 1][k];
#pragma unroll
        for (int w = 1; w < kFwdWaves; ++w) {
          const float2 v = parts[w][k][lane];
          tp[k] *= v.x;
          th[k] = onward<kGrow>(v.x, th[k], v.y);
        }
      }
      chain_enter<kGrow, CH>(c, strip, tile, tp, th, hin);
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) hin[k] = a.initial && at.in ? a.initial[at.b * a.width + at.d + k] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) enter[first][k][lane] = hin[k];
  }
  block_sync();
  float h[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    h[k] = enter[first][k][lane];
    for (int w = first; w < wave; ++w) {
      const float2 v = parts[w][k][lane];
      h[k] = onward<kGrow>(v.x, h[k], v.y);
    }
  }
  if (at.n == 0) return;
  if (a.states && (wave - first) % kFwdApart == 0 && at.in) {
    float* s = a.states + (at.b * ((a.seqlen + kGsSegment - 1) / kGsSegment) + at.t0 / kGsSegment) * a.width + at.d;
#pragma unroll
    for (int k = 0; k < CH; ++k) s[k] = h[k];
  }
  float v[CH];
  auto stores = [&](auto whole, auto type) SSM_INLINE {
    using Tout = decltype(type);
    const Rows ro(a.out, at.tok, a.width, sizeof(Tout));
    const uint32_t off = at.off(sizeof(Tout));
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
#pragma unroll
      for (int k = 0; k < CH; ++k) v[k] = onward<kGrow>(P[j][k], h[k], H[j][k]);      // (past the last step the last one's)
      store_raw<FORM == kStream, Tout, CH>(ro, j, decltype(whole)::value ? off : at.off(sizeof(Tout), j), v);
    }
  };
  if (at.n == kSteps) {
    if (a.out_bf16) stores(std::true_type{}, uint16_t{});
    else stores(std::true_type{}, float{});
  } else {
    if (a.out_bf16) stores(std::false_type{}, uint16_t{});
    else stores(std::false_type{}, float{});
  }
  if (a.last && at.n == at.left && at.in) {
#pragma unroll
    for (int k = 0; k < CH; ++k) a.last[at.b * a.width + at.d + k] = v[k];
  }
}

// The gradients.  g_t = dout_t + a_{t+1} g_{t+1} is the same recurrence back in time: a
// wavefront knows what leaves it for a zero gradient entering, the chain runs from the last
// tile to the first.  The states before each step, which e needs, come forward from the one
// stored every kGsSegment steps, by the same composition over at most 4 wavefronts.  x, r and
// i stay in LDS as they were loaded between the two passes, a, m and g in registers; the
// sigmoids are taken twice: registers that held those too would spill.  Bound by HBM: 4 x 2048 x 5120 bf16 reads four
// tensors and the states and writes three, 608 MB in 145 us, 4.2 TB/s; 3 x 1021 x 1537 fp32 (133 MB)
// 38 us and bf16 (67 MB) 31, one value a lane.
template <typename T, bool RATE, bool LERP, bool GATE, int CH, Form FORM>
__global__ void __launch_bounds__(64 * kBwdWaves, 4) gscan_bwd_kernel(GscanArgs a, Chain c) {
  __shared__ uint32_t kept[kBwdWaves][3][kBwdSteps][64];      // x, r and i as they lie in memory, for the second pass
  __shared__ float2 parts[kBwdWaves][CH][64];
  __shared__ float ahead[kBwdWaves][CH][64];      // forward: what leaves a wavefront for a zero state entering
  __shared__ float enter[FORM == kShort ? kBwdWaves : 1][CH][64];      // at a strip's first wavefront
  int back, strip;
  take_tile<FORM>(c, &back, &strip);
  const int tile = c.tiles - 1 - back;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = FORM == kShort ? wave & -c.waves : 0, last = FORM == kShort ? first + c.waves - 1 : kBwdWaves - 1;
  if (FORM == kShort) strip = (strip * kBwdWaves + wave) / c.waves;
  constexpr int kSteps = kBwdSteps;
  constexpr bool kGrow = RATE && LERP;
  const Place<CH, kSteps, FORM> at(a, c, tile, strip, kGsBwdTile, wave - first, lane);
  const uint32_t off = at.off(sizeof(T));
  // the state stored last before the wavefront's steps
  float rate[CH], h[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) rate[k] = RATE && at.in ? a.rate[at.d + k] : 0.0f, h[k] = 0.0f;
  if (at.n > 0 && at.in) {
    const float* s = a.states_in + (at.b * ((a.seqlen + kGsSegment - 1) / kGsSegment) + at.t0 / kGsSegment) * a.width + at.d;
#pragma unroll
    for (int k = 0; k < CH; ++k) h[k] = s[k];
  }
  // what a step keeps in registers: its decay, the input's coefficient and the gradient
  float A[kSteps][CH], M[kSteps][CH], g[kSteps][CH], p[CH], q[CH], f[CH];
  auto steps = [&](auto whole, auto type) SSM_INLINE {
    constexpr bool kWhole = decltype(whole)::value;
    using Tout = decltype(type);
    const Rows rx(a.x, at.tok, a.x_row, sizeof(T)), rr(a.r, at.tok, a.r_row, sizeof(T)), ri(a.i, at.tok, a.i_row, sizeof(T));
    const Rows rg(a.dout, at.tok, a.width, sizeof(Tout));
    const uint32_t off_g = at.off(sizeof(Tout));
    uint32_t x[kSteps], r[kSteps], i[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const uint32_t o = kWhole ? off : at.off(sizeof(T), j);
      r[j] = load_raw<T, CH>(rr, j, o);
      if constexpr (GATE) i[j] = load_raw<T, CH>(ri, j, o);
      x[j] = load_raw<T, CH>(rx, j, o);
      load_values<Tout, CH>(rg, j, kWhole ? off_g : at.off(sizeof(Tout), j), g[j]);
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) f[k] = 0.0f;
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        decay<RATE, LERP>(gate_exp<!RATE>(raw_value<T>(r[j], k)), rate[k] * kLog2e, &A[j][k], &M[j][k]);
        float u = raw_value<T>(x[j], k);
        if constexpr (GATE) u *= gate_open(gate_exp<false>(raw_value<T>(i[j], k)));
        if (!kWhole && j >= at.n) A[j][k] = 1.0f, M[j][k] = 0.0f;
        f[k] = __builtin_fmaf(A[j][k], f[k], M[j][k] * u);
      }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      kept[wave][0][j][lane] = x[j];
      kept[wave][1][j][lane] = r[j];
      if constexpr (GATE) kept[wave][2][j][lane] = i[j];
    }
    // back through the wavefront's steps: what leaves it for a zero gradient entering
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      p[k] = A[kSteps - 1][k], q[k] = A[kSteps - 1][k] * g[kSteps - 1][k];
#pragma unroll
      for (int j = kSteps - 2; j >= 0; --j) {
        p[k] *= A[j][k];
        q[k] = A[j][k] * (q[k] + g[j][k]);
      }
    }
  };
  if (at.n == kSteps) {
    if (a.out_bf16) steps(std::true_type{}, uint16_t{});
    else steps(std::true_type{}, float{});
  } else {
    if (a.out_bf16) steps(std::false_type{}, uint16_t{});
    else steps(std::false_type{}, float{});
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    parts[wave][k][lane] = make_float2(p[k], q[k]);
    ahead[wave][k][lane] = f[k];
  }
  block_sync();
  if (wave == last) {
    float gin[CH];
    if (FORM != kShort && c.tiles > 1) {
      float tp[CH], tq[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        tp[k] = p[k], tq[k] = q[k];
#pragma unroll
        for (int w = kBwdWaves - 2; w >= 0; --w) {
          const float2 v = parts[w][k][lane];
          tp[k] *= v.x;
          tq[k] = onward<kGrow>(v.x, tq[k], v.y);
        }
      }
      chain_enter<kGrow, CH>(c, strip, back, tp, tq, gin);
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) gin[k] = a.dlast && at.in ? a.dlast[at.b * a.width + at.d + k] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) enter[first][k][lane] = gin[k];
  }
  block_sync();
  // the gradient entering from behind, and the state entering from before
  float carry[CH], sum[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    carry[k] = enter[first][k][lane];
    for (int w = last; w > wave; --w) {
      const float2 v = parts[w][k][lane];
      carry[k] = onward<kGrow>(v.x, carry[k], v.y);
    }
    for (int w = first + (wave - first) / kBwdApart * kBwdApart; w < wave; ++w) h[k] = onward<kGrow>(parts[w][k][lane].x, h[k], ahead[w][k][lane]);
    sum[k] = 0.0f;
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      g[j][k] += carry[k];
      carry[k] = A[j][k] * g[j][k];
    }
  }
  if (a.dinitial && at.t0 == 0 && at.in) {
#pragma unroll
    for (int k = 0; k < CH; ++k) a.dinitial[at.b * a.width + at.d + k] = carry[k];
  }
  // forward again, with the states on the way
  auto gradients = [&](auto whole) SSM_INLINE {
    const Rows rx(a.dx, at.tok, a.width, sizeof(T)), rr(a.dr, at.tok, a.width, sizeof(T)), ri(a.di, at.tok, a.width, sizeof(T));
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const uint32_t o = decltype(whole)::value ? off : at.off(sizeof(T), j);
      float dx[CH], dr[CH], di[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float u = raw_value<T>(kept[wave][0][j][lane], k);
        const float er = gate_exp<true>(raw_value<T>(kept[wave][1][j][lane], k));
        const float rpos = gate_open(er), gm = g[j][k] * M[j][k];
        dx[k] = gm;
        if constexpr (GATE) {
          const float ei = gate_exp<true>(raw_value<T>(kept[wave][2][j][lane], k));
          const float pos = gate_open(ei);
          u *= pos;
          dx[k] *= pos;
          di[k] = gm * u * (ei * pos);
        }
        const float by = g[j][k] * __builtin_fmaf(A[j][k], h[k], u * decay_slope<LERP>(A[j][k], M[j][k]));
        const float rneg = er * rpos;
        if constexpr (RATE) {
          const float bp = by * rpos;
          sum[k] -= decltype(whole)::value || j < at.n ? bp : 0.0f;
          dr[k] = -bp * rate[k] * rneg;
        } else {
          dr[k] = by * rneg;      // (by rpos would be about rpos^2 where it is small, and lost below 1e-38)
        }
        h[k] = __builtin_fmaf(A[j][k], h[k], M[j][k] * u);
      }
      store_raw<FORM == kStream, T, CH>(rx, j, o, dx);
      store_raw<FORM == kStream, T, CH>(rr, j, o, dr);
      if constexpr (GATE) store_raw<FORM == kStream, T, CH>(ri, j, o, di);
    }
  };
  if (at.n == kSteps) gradients(std::true_type{});
  else gradients(std::false_type{});
  if (RATE && a.part) {
    block_sync();
#pragma unroll
    for (int k = 0; k < CH; ++k) ahead[wave][k][lane] = sum[k];
    block_sync();
    if (wave == first && at.in) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float s = ahead[first][k][lane];
        for (int w = first + 1; w <= last; ++w) s += ahead[w][k][lane];
        a.part[(at.b * c.tiles + tile) * a.width + at.d + k] = s;
      }
    }
  }
}

// Before a chain: everything unwritten but the first group's state, and no tile taken.
// (4 to 6 us beside kernels of 80 to 200, mostly a launch: 1 x 65537 x 2560 writes 11 MB.)
__global__ void __launch_bounds__(256) gscan_begin_kernel(Chain c, const float* __restrict__ first, int64_t width, int ch) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, stride = (int64_t)gridDim.x * 256;
  const int64_t each = 64 * ch, parts = (int64_t)c.strips * c.tiles * each, states = (int64_t)c.strips * c.groups * each;
  for (int64_t j = n; j < parts; j += stride) c.parts[j] = ~0ull;
  const int64_t per_row = (width + each - 1) / each;
  for (int64_t j = n; j < states; j += stride) {
    const int64_t strip = j / each / c.groups;
    uint32_t w = kUnwritten;
    if (j / each % c.groups == 0) {
      // (a channel's place: the wavefront's channels are stored a word of each lane at a time)
      const int64_t at = j % each, d = strip % per_row * each + at % 64 * ch + at / 64;
      w = first && d < width ? word_of(first[strip / per_row * width + d]) : 0;
    }
    c.states[j] = w;
  }
  if (n == 0) *c.next = 0;
}

// One token: an element a lane.  256 x 8192 bf16 (34 MB with the states) 8.2 us a call from call to
// call on the same tensors, which the caches hold, 8.9 over three sets of them in turn; 1 x 2560 2.8,
// a launch's least.
template <typename T, bool RATE, bool LERP, bool GATE>
__global__ void __launch_bounds__(256) gscan_step_kernel(GscanArgs a) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.batch * a.width) return;
  const int64_t b = e / a.width, d = e % a.width;
  float ea, em;
  decay<RATE, LERP>(gate_exp<!RATE>(Io<T>::cvt(Io<T>::load(a.r, b * a.r_row + d))), RATE ? a.rate[d] * kLog2e : 0.0f, &ea, &em);
  float u = Io<T>::cvt(Io<T>::load(a.x, b * a.x_row + d));
  if constexpr (GATE) u *= gate_open(gate_exp<false>(Io<T>::cvt(Io<T>::load(a.i, b * a.i_row + d))));
  const float h = __builtin_fmaf(ea, a.initial[e], em * u);
  a.last[e] = h;
  if (a.out_bf16) Io<uint16_t>::store(a.out, e, h);
  else Io<float>::store(a.out, e, h);
}

// out[y][d] = sum of part[n][d] over slice y of n rows, in a fixed order: 16 wavefronts take
// every sixteenth row of 64 columns.  (128 rows of 5120: 4 us.  In one slice, and in up to 64 and
// those then, forward and back: 8192 rows of 1024 329 and 314 us, 4096 of 512 115 and 108, 2048
// of 1024 179 and 175, 512 of 1024 158 and 159.)
__global__ void __launch_bounds__(1024) gscan_sum_kernel(const float* __restrict__ part, float* __restrict__ out, int64_t n, int64_t each,
                                                         int64_t width) {
  __shared__ float t[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t d = (int64_t)blockIdx.x * 64 + lane, from = blockIdx.y * each, to = from + each < n ? from + each : n;
  float s = 0.0f;
  if (d < width) {
#pragma unroll 8
    for (int64_t i = from + wave; i < to; i += 16) s += part[i * width + d];
  }
  t[wave][lane] = s;
  block_sync();
  if (wave == 0 && d < width) {
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) r += t[i][lane];
    out[blockIdx.y * width + d] = r;
  }
}

// The kernel for a type and the three choices, and the form (a lane's one bf16 value is never a
// whole line's).
#define SSM_GSCAN_PICK(kernel, ...)                                                                                  \
  (a.rate ? (a.lerp ? (a.i ? kernel<true, true, true, __VA_ARGS__> : kernel<true, true, false, __VA_ARGS__>)       \
                    : (a.i ? kernel<true, false, true, __VA_ARGS__> : kernel<true, false, false, __VA_ARGS__>))    \
          : (a.lerp ? (a.i ? kernel<false, true, true, __VA_ARGS__> : kernel<false, true, false, __VA_ARGS__>)     \
                    : (a.i ? kernel<false, false, true, __VA_ARGS__> : kernel<false, false, false, __VA_ARGS__>)))
#define SSM_GSCAN_FORM(kernel, ...)                                                 \
  (l.c.waves < kGsWaves ? SSM_GSCAN_PICK(kernel, __VA_ARGS__, kShort)               \
   : stream             ? SSM_GSCAN_PICK(kernel, __VA_ARGS__, kStream)              \
                        : SSM_GSCAN_PICK(kernel, __VA_ARGS__, kPlain))
template <bool RATE, bool LERP, bool GATE, typename T, int CH, Form FORM>
constexpr auto fwd_kernel = &gscan_fwd_kernel<T, RATE, LERP, GATE, CH, FORM>;
template <bool RATE, bool LERP, bool GATE, typename T, int CH, Form FORM>
constexpr auto bwd_kernel = &gscan_bwd_kernel<T, RATE, LERP, GATE, CH, FORM>;
template <bool RATE, bool LERP, bool GATE, typename T>
constexpr auto step_kernel = &gscan_step_kernel<T, RATE, LERP, GATE>;

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Neighbouring channels of a lane: two bf16 values in one access where every tensor's rows
// allow it, one where not.
int channels(const GscanArgs& a, DT in) {
  const uintptr_t out = a.out_bf16 ? 4 : 8;
  return in == DT::BF16 && a.width % 2 == 0 && a.x_row % 2 == 0 && a.r_row % 2 == 0 && (!a.i || a.i_row % 2 == 0) &&
                 aligned(a.x, 4) && aligned(a.r, 4) && aligned(a.i, 4) && aligned(a.out, out) && aligned(a.dout, out) &&
                 aligned(a.dx, 4) && aligned(a.dr, 4) && aligned(a.di, 4)
             ? 2
             : 1;
}

// Outputs go past the caches where their rows are whole lines of 128 bytes (us, with and
// without: forward of 8 x 2048 x 5120 bf16 143 / 147, 2 x 2048 x 5120 43.6 / 48.2, 1 x 65537 x
// 2560 196 / 201; forward and back 4 x 2048 x 5120 224 / 232, fp32 2 x 1024 x 5120 107 / 118).
// A line written in parts does not take it: 3 x 1021 x 1537 fp32, forward and back, 71 / 67.
// (Loads past the caches: 8 x 2048 x 5120 141, but 1 x 2048 x 5120 34.6 in place of 32.3.)
bool streams(int64_t width, int size) { return width * size % 128 == 0; }

void begin(const Layout& l, const float* first, int64_t width, hipStream_t s) {
  if (l.c.tiles <= 1) return;
  const int64_t n = (int64_t)l.c.strips * l.c.tiles * 64 * l.ch;
  const unsigned blocks = (unsigned)(n / 1024 < 1 ? 1 : n / 1024 > 2048 ? 2048 : n / 1024);
  hipLaunchKernelGGL(gscan_begin_kernel, dim3(blocks), dim3(256), 0, s, l.c, first, width, l.ch);
}

}  // namespace

hipError_t launch_gscan_fwd(const GscanArgs& a, DT in, hipStream_t s) {
  const Layout l = gscan_layout(a.batch, a.seqlen, a.width, kGsFwdTile, channels(a, in), a.work);
  begin(l, a.initial, a.width, s);
  const bool stream = streams(a.width, a.out_bf16 ? 2 : 4);
  auto k = in == DT::F32 ? SSM_GSCAN_FORM(fwd_kernel, float, 1)
           : l.ch == 2   ? SSM_GSCAN_FORM(fwd_kernel, uint16_t, 2)
           : l.c.waves < kGsWaves ? SSM_GSCAN_PICK(fwd_kernel, uint16_t, 1, kShort)
                                  : SSM_GSCAN_PICK(fwd_kernel, uint16_t, 1, kPlain);
  hipLaunchKernelGGL(k, dim3((unsigned)l.blocks), dim3(64 * kFwdWaves), 0, s, a, l.c);
  return hipGetLastError();
}

hipError_t launch_gscan_bwd(const GscanArgs& a, DT in, hipStream_t s) {
  const Layout l = gscan_layout(a.batch, a.seqlen, a.width, kGsBwdTile, channels(a, in), a.work);
  begin(l, a.dlast, a.width, s);
  const bool stream = streams(a.width, in == DT::F32 ? 4 : 2);
  auto k = in == DT::F32 ? SSM_GSCAN_FORM(bwd_kernel, float, 1)
           : l.ch == 2   ? SSM_GSCAN_FORM(bwd_kernel, uint16_t, 2)
           : l.c.waves < kGsWaves ? SSM_GSCAN_PICK(bwd_kernel, uint16_t, 1, kShort)
                                  : SSM_GSCAN_PICK(bwd_kernel, uint16_t, 1, kPlain);
  hipLaunchKernelGGL(k, dim3((unsigned)l.blocks), dim3(64 * kBwdWaves), 0, s, a, l.c);
  if (a.drate) {
    const int64_t rows = a.batch * l.c.tiles, slices = gscan_sum_slices(rows), each = (rows + slices - 1) / slices;
    const unsigned strips = (unsigned)((a.width + 63) / 64);
    float* sums = slices > 1 ? a.part + rows * a.width : a.drate;
    hipLaunchKernelGGL(gscan_sum_kernel, dim3(strips, (unsigned)slices), dim3(1024), 0, s, a.part, sums, rows, each, a.width);
    if (slices > 1) hipLaunchKernelGGL(gscan_sum_kernel, dim3(strips), dim3(1024), 0, s, sums, a.drate, slices, slices, a.width);
  }
  return hipGetLastError();
}

hipError_t launch_gscan_step(const GscanArgs& a, DT in, hipStream_t s) {
  auto k = in == DT::F32 ? SSM_GSCAN_PICK(step_kernel, float) : SSM_GSCAN_PICK(step_kernel, uint16_t);
  hipLaunchKernelGGL(k, dim3((unsigned)((a.batch * a.width + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssm
