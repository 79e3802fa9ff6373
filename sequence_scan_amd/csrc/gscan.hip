// gfx950 kernels of libssmscan: the gated linear recurrence
// h_t = a_t h_{t-1} + m_t u_t for each channel, its gradients and its single-token
// step.  Both directions read every tensor once (gscan_kernel.h: the chain of tiles).
#include <algorithm>

#include "gscan_kernel.h"

namespace ssm {
namespace {

constexpr int kSteps = 16;         // steps of a wavefront: what its registers hold
constexpr int kFwdWaves = 8;       // tiles of 128 steps forward
constexpr int kBwdWaves = 4;       // ... and 64 back, which keeps twice as much of each

static_assert(kGsFwdTile == kSteps * kFwdWaves && kGsBwdTile == kSteps * kBwdWaves, "model.h agrees");
static_assert(kGsSegment == 2 * kSteps, "stored states enter every other wavefront");

// The tile that a workgroup takes: its place in the chain and its strip.
__device__ __forceinline__ void take_tile(const Chain& c, int* tile, int* strip) {
  int n = blockIdx.x;
  if (c.tiles > 1) {
    __shared__ uint32_t taken;
    if (threadIdx.x == 0) taken = atomicAdd(c.next, 1u);
    block_sync();
    n = (int)__builtin_amdgcn_readfirstlane(taken);
  }
  *tile = n / c.strips;
  *strip = n % c.strips;
}

template <typename T, bool RATE, bool LERP, bool GATE, int CH>
__global__ void __launch_bounds__(64 * kFwdWaves, 4) gscan_fwd_kernel(GscanArgs a, Chain c) {
  __shared__ float2 parts[kFwdWaves][CH][64];
  __shared__ float enter[CH][64];
  int tile, strip;
  take_tile(c, &tile, &strip);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per_row = (int)((a.width + 64 * CH - 1) / (64 * CH));
  const int64_t b = strip / per_row;
  const int d0 = strip % per_row * (64 * CH) + lane * CH;
  const bool in = d0 < a.width;
  const uint32_t d = in ? d0 : 0;             // (lanes past the width repeat the first channels)
  const int64_t t0 = (int64_t)tile * kGsFwdTile + wave * kSteps;
  const int64_t left = a.seqlen - t0;
  const int n = left < 0 ? 0 : left > kSteps ? kSteps : (int)left;
  const int64_t tok = b * a.seqlen + t0;
  float rate[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) rate[k] = RATE ? a.rate[d + k] : 0.0f;

  // all loads first: a wavefront has 16 steps of three tensors under way
  uint32_t x[kSteps], r[kSteps], i[kSteps];
#pragma unroll
  for (int j = 0; j < kSteps; ++j)
    if (j < n) {
      x[j] = load_raw<T, CH>(a.x, tok + j, a.x_row, d);
      r[j] = load_raw<T, CH>(a.r, tok + j, a.r_row, d);
      if constexpr (GATE) i[j] = load_raw<T, CH>(a.i, tok + j, a.i_row, d);
    }
  float P[kSteps][CH], H[kSteps][CH], p[CH], h[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) p[k] = 1.0f, h[k] = 0.0f;
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    if (j < n) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const Decay e = decay<RATE, LERP>(raw_value<T>(r[j], k), rate[k]);
        float u = raw_value<T>(x[j], k);
        if constexpr (GATE) {
          float pos, neg;
          sigmoids(raw_value<T>(i[j], k), &pos, &neg);
          u *= pos;
        }
        p[k] *= e.a;
        h[k] = __builtin_fmaf(e.a, h[k], e.m * u);
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) P[j][k] = p[k], H[j][k] = h[k];
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) parts[wave][k][lane] = make_float2(p[k], h[k]);
  block_sync();
  if (wave == 0) {
    float hin[CH];
    if (c.tiles > 1) {
      float tp[CH], th[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        tp[k] = p[k], th[k] = h[k];
#pragma unroll
        for (int w = 1; w < kFwdWaves; ++w) {
          const float2 v = parts[w][k][lane];
          tp[k] *= v.x;
          th[k] = __builtin_fmaf(v.x, th[k], v.y);
        }
      }
      chain_enter<CH>(c, strip, tile, tp, th, hin);
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) hin[k] = a.initial ? a.initial[b * a.width + d + k] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) enter[k][lane] = hin[k];
  }
  block_sync();
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    h[k] = enter[k][lane];
    for (int w = 0; w < wave; ++w) {
      const float2 v = parts[w][k][lane];
      h[k] = __builtin_fmaf(v.x, h[k], v.y);
    }
  }
  if (!in || n == 0) return;
  if (a.states && wave % 2 == 0) {
    float* s = a.states + (b * ((a.seqlen + kGsSegment - 1) / kGsSegment) + t0 / kGsSegment) * a.width + d;
#pragma unroll
    for (int k = 0; k < CH; ++k) s[k] = h[k];
  }
  float v[CH];
#pragma unroll
  for (int j = 0; j < kSteps; ++j)
    if (j < n) {
#pragma unroll
      for (int k = 0; k < CH; ++k) v[k] = __builtin_fmaf(P[j][k], h[k], H[j][k]);
      if (a.out_bf16) store_raw<uint16_t, CH>(a.out, tok + j, a.width, d, v);
      else store_raw<float, CH>(a.out, tok + j, a.width, d, v);
    }
  if (a.last && n == left) {
#pragma unroll
    for (int k = 0; k < CH; ++k) a.last[b * a.width + d + k] = v[k];
  }
}

// Of a gate's two sigmoids the smaller one, with the argument's sign: the larger is one
// less it, to an ulp.
__device__ __forceinline__ float small_sigmoid(float pos, float neg) { return pos < neg ? -pos : neg; }
__device__ __forceinline__ void both_sigmoids(float s, float* pos, float* neg) {
  const float m = __builtin_fabsf(s), o = 1.0f - m;
  const bool shut = __float_as_int(s) < 0;
  *pos = shut ? m : o;
  *neg = shut ? o : m;
}

template <typename T, bool RATE, bool LERP, bool GATE, int CH>
__global__ void __launch_bounds__(64 * kBwdWaves, 2) gscan_bwd_kernel(GscanArgs a, Chain c) {
  __shared__ float2 parts[kBwdWaves][CH][64];
  __shared__ float half[kBwdWaves][CH][64];
  __shared__ float enter[CH][64];
  int back, strip;
  take_tile(c, &back, &strip);
  const int tile = c.tiles - 1 - back;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per_row = (int)((a.width + 64 * CH - 1) / (64 * CH));
  const int64_t b = strip / per_row;
  const int d0 = strip % per_row * (64 * CH) + lane * CH;
  const bool in = d0 < a.width;
  const uint32_t d = in ? d0 : 0;
  const int64_t t0 = (int64_t)tile * kGsBwdTile + wave * kSteps;
  const int64_t left = a.seqlen - t0;
  const int n = left < 0 ? 0 : left > kSteps ? kSteps : (int)left;
  const int64_t tok = b * a.seqlen + t0;
  float rate[CH], h[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) rate[k] = RATE ? a.rate[d + k] : 0.0f, h[k] = 0.0f;
  if (wave % 2 == 0 && n > 0) {
    const float* s = a.states_in + (b * ((a.seqlen + kGsSegment - 1) / kGsSegment) + t0 / kGsSegment) * a.width + d;
#pragma unroll
    for (int k = 0; k < CH; ++k) h[k] = s[k];
  }
  uint32_t x[kSteps], r[kSteps], i[kSteps];
  float g[kSteps][CH];
#pragma unroll
  for (int j = 0; j < kSteps; ++j)
    if (j < n) {
      x[j] = load_raw<T, CH>(a.x, tok + j, a.x_row, d);
      r[j] = load_raw<T, CH>(a.r, tok + j, a.r_row, d);
      if constexpr (GATE) i[j] = load_raw<T, CH>(a.i, tok + j, a.i_row, d);
      if (a.out_bf16) {
        const uint32_t w = load_raw<uint16_t, CH>(a.dout, tok + j, a.width, d);
#pragma unroll
        for (int k = 0; k < CH; ++k) g[j][k] = raw_value<uint16_t>(w, k);
      } else {
#pragma unroll
        for (int k = 0; k < CH; ++k) g[j][k] = static_cast<const float*>(a.dout)[(tok + j) * a.width + d + k];
      }
    }
  // per step and channel: the decay, the input's coefficient and the gates' sigmoids
  float A[kSteps][CH], M[kSteps][CH], sr[kSteps][CH], si[kSteps][CH];
  float enters[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) enters[k] = h[k];
#pragma unroll
  for (int j = 0; j < kSteps; ++j)
    if (j < n) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const Decay e = decay<RATE, LERP>(raw_value<T>(r[j], k), rate[k]);
        A[j][k] = e.a;
        M[j][k] = e.m;
        sr[j][k] = small_sigmoid(e.pos, e.neg);
        float u = raw_value<T>(x[j], k);
        if constexpr (GATE) {
          float pos, neg;
          sigmoids(raw_value<T>(i[j], k), &pos, &neg);
          si[j][k] = small_sigmoid(pos, neg);
          u *= pos;
        }
        h[k] = __builtin_fmaf(e.a, h[k], e.m * u);
      }
    }
  // back through the wavefront's steps: what leaves it for a zero gradient entering
  float p[CH], q[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) p[k] = 1.0f, q[k] = 0.0f;
#pragma unroll
  for (int j = kSteps - 1; j >= 0; --j)
    if (j < n) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        p[k] *= A[j][k];
        q[k] = A[j][k] * (q[k] + g[j][k]);
      }
    }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    parts[wave][k][lane] = make_float2(p[k], q[k]);
    half[wave][k][lane] = h[k];
  }
  block_sync();
  if (wave == kBwdWaves - 1) {
    float gin[CH];
    if (c.tiles > 1) {
      float tp[CH], tq[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        tp[k] = p[k], tq[k] = q[k];
#pragma unroll
        for (int w = kBwdWaves - 2; w >= 0; --w) {
          const float2 v = parts[w][k][lane];
          tp[k] *= v.x;
          tq[k] = __builtin_fmaf(v.x, tq[k], v.y);
        }
      }
      chain_enter<CH>(c, strip, back, tp, tq, gin);
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) gin[k] = a.dlast ? a.dlast[b * a.width + d + k] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) enter[k][lane] = gin[k];
  }
  block_sync();
  // the gradient entering from behind, and the state entering from before
  float carry[CH], sum[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    carry[k] = enter[k][lane];
    for (int w = kBwdWaves - 1; w > wave; --w) {
      const float2 v = parts[w][k][lane];
      carry[k] = __builtin_fmaf(v.x, carry[k], v.y);
    }
    h[k] = wave % 2 == 0 ? enters[k] : half[wave - 1][k][lane];
    sum[k] = 0.0f;
  }
#pragma unroll
  for (int j = kSteps - 1; j >= 0; --j)
    if (j < n) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        g[j][k] += carry[k];
        carry[k] = A[j][k] * g[j][k];
      }
    }
  if (a.dinitial && t0 == 0 && in) {
#pragma unroll
    for (int k = 0; k < CH; ++k) a.dinitial[b * a.width + d + k] = carry[k];
  }
  // forward again, with the states on the way
#pragma unroll
  for (int j = 0; j < kSteps; ++j)
    if (j < n) {
      float dx[CH], dr[CH], di[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const float xv = raw_value<T>(x[j], k);
        float pos = 1.0f, neg = 0.0f, rpos, rneg;
        if constexpr (GATE) both_sigmoids(si[j][k], &pos, &neg);
        both_sigmoids(sr[j][k], &rpos, &rneg);
        const float u = xv * pos, gm = g[j][k] * M[j][k];
        Decay e;
        e.a = A[j][k];
        e.m = M[j][k];
        const float by = g[j][k] * __builtin_fmaf(e.a, h[k], u * decay_slope<LERP>(e));
        dx[k] = gm * pos;
        di[k] = gm * u * neg;
        if constexpr (RATE) {
          const float bp = by * rpos;
          sum[k] -= bp;
          dr[k] = -bp * rate[k] * rneg;
        } else {
          dr[k] = by * rneg;
        }
        h[k] = __builtin_fmaf(e.a, h[k], e.m * u);
      }
      if (in) {
        store_raw<T, CH>(a.dx, tok + j, a.width, d, dx);
        store_raw<T, CH>(a.dr, tok + j, a.width, d, dr);
        if constexpr (GATE) store_raw<T, CH>(a.di, tok + j, a.width, d, di);
      }
    }
  if (RATE && a.part) {
    block_sync();
#pragma unroll
    for (int k = 0; k < CH; ++k) half[wave][k][lane] = sum[k];
    block_sync();
    if (wave == 0 && in) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float s = half[0][k][lane];
#pragma unroll
        for (int w = 1; w < kBwdWaves; ++w) s += half[w][k][lane];
        a.part[(b * c.tiles + tile) * a.width + d + k] = s;
      }
    }
  }
}

// Before a chain: everything unwritten but the first group's state, and no tile taken.
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

template <typename T, bool RATE, bool LERP, bool GATE>
__global__ void __launch_bounds__(256) gscan_step_kernel(GscanArgs a) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.batch * a.width) return;
  const int64_t b = e / a.width, d = e % a.width;
  auto get = [&](const void* p, int64_t row) SSM_INLINE { return raw_value<T>(load_raw<T, 1>(p, b, row, (uint32_t)d), 0); };
  const Decay c = decay<RATE, LERP>(get(a.r, a.r_row), RATE ? a.rate[d] : 0.0f);
  float u = get(a.x, a.x_row);
  if constexpr (GATE) {
    float pos, neg;
    sigmoids(get(a.i, a.i_row), &pos, &neg);
    u *= pos;
  }
  const float h[1] = {__builtin_fmaf(c.a, a.initial[e], c.m * u)};
  a.last[e] = h[0];
  if (a.out_bf16) store_raw<uint16_t, 1>(a.out, b, a.width, (uint32_t)d, h);
  else store_raw<float, 1>(a.out, b, a.width, (uint32_t)d, h);
}

// out[d] = sum over n rows of part[n][d], in a fixed order: 16 wavefronts take every
// sixteenth row of 64 columns.
__global__ void __launch_bounds__(1024) gscan_sum_kernel(const float* __restrict__ part, float* __restrict__ out, int64_t n,
                                                         int64_t width) {
  __shared__ float t[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t d = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (d < width) {
#pragma unroll 8
    for (int64_t i = wave; i < n; i += 16) s += part[i * width + d];
  }
  t[wave][lane] = s;
  block_sync();
  if (wave == 0 && d < width) {
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) r += t[i][lane];
    out[d] = r;
  }
}

// The kernel for a type and the three choices.
#define SSM_GSCAN_PICK(kernel, ...)                                                                                  \
  (a.rate ? (a.lerp ? (a.i ? kernel<true, true, true, __VA_ARGS__> : kernel<true, true, false, __VA_ARGS__>)       \
                    : (a.i ? kernel<true, false, true, __VA_ARGS__> : kernel<true, false, false, __VA_ARGS__>))    \
          : (a.lerp ? (a.i ? kernel<false, true, true, __VA_ARGS__> : kernel<false, true, false, __VA_ARGS__>)     \
                    : (a.i ? kernel<false, false, true, __VA_ARGS__> : kernel<false, false, false, __VA_ARGS__>)))
template <bool RATE, bool LERP, bool GATE, typename T, int CH>
constexpr auto fwd_kernel = &gscan_fwd_kernel<T, RATE, LERP, GATE, CH>;
template <bool RATE, bool LERP, bool GATE, typename T, int CH>
constexpr auto bwd_kernel = &gscan_bwd_kernel<T, RATE, LERP, GATE, CH>;
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

struct Layout {
  Chain c;
  int ch;
  int64_t bytes;     // of the chain's workspace
};
Layout layout(int64_t batch, int64_t seqlen, int64_t width, int64_t steps, int ch, char* work) {
  Layout l{};
  l.ch = ch;
  const int64_t each = 64 * ch;
  l.c.strips = (int32_t)(batch * ((width + each - 1) / each));
  l.c.tiles = (int32_t)((seqlen + steps - 1) / steps);
  l.c.groups = (l.c.tiles + kGsGroup - 1) / kGsGroup;
  if (l.c.tiles > 1) {
    const int64_t parts = (int64_t)l.c.strips * l.c.tiles * each * 8, states = (int64_t)l.c.strips * l.c.groups * each * 4;
    l.c.parts = reinterpret_cast<uint64_t*>(work);
    l.c.states = reinterpret_cast<uint32_t*>(work + parts);
    l.c.next = reinterpret_cast<uint32_t*>(work + parts + states);
    l.bytes = parts + states + 16;
  }
  return l;
}

void begin(const Layout& l, const float* first, int64_t width, hipStream_t s) {
  if (l.c.tiles <= 1) return;
  const int64_t n = (int64_t)l.c.strips * l.c.tiles * 64 * l.ch;
  const unsigned blocks = (unsigned)(n / 1024 < 1 ? 1 : n / 1024 > 2048 ? 2048 : n / 1024);
  hipLaunchKernelGGL(gscan_begin_kernel, dim3(blocks), dim3(256), 0, s, l.c, first, width, l.ch);
}

}  // namespace

int64_t gscan_chain_bytes(int64_t batch, int64_t seqlen, int64_t width, bool backward) {
  // (strips of single channels are as many or more bytes than those of two)
  const int64_t steps = backward ? kGsBwdTile : kGsFwdTile;
  return std::max(layout(batch, seqlen, width, steps, 1, nullptr).bytes, layout(batch, seqlen, width, steps, 2, nullptr).bytes);
}

hipError_t launch_gscan_fwd(const GscanArgs& a, DT in, hipStream_t s) {
  const Layout l = layout(a.batch, a.seqlen, a.width, kGsFwdTile, channels(a, in), a.work);
  begin(l, a.initial, a.width, s);
  auto k = in == DT::F32 ? SSM_GSCAN_PICK(fwd_kernel, float, 1)
           : l.ch == 2   ? SSM_GSCAN_PICK(fwd_kernel, uint16_t, 2)
                         : SSM_GSCAN_PICK(fwd_kernel, uint16_t, 1);
  hipLaunchKernelGGL(k, dim3((unsigned)(l.c.strips * l.c.tiles)), dim3(64 * kFwdWaves), 0, s, a, l.c);
  return hipGetLastError();
}

hipError_t launch_gscan_bwd(const GscanArgs& a, DT in, hipStream_t s) {
  const Layout l = layout(a.batch, a.seqlen, a.width, kGsBwdTile, channels(a, in), a.work);
  begin(l, a.dlast, a.width, s);
  auto k = in == DT::F32 ? SSM_GSCAN_PICK(bwd_kernel, float, 1)
           : l.ch == 2   ? SSM_GSCAN_PICK(bwd_kernel, uint16_t, 2)
                         : SSM_GSCAN_PICK(bwd_kernel, uint16_t, 1);
  hipLaunchKernelGGL(k, dim3((unsigned)(l.c.strips * l.c.tiles)), dim3(64 * kBwdWaves), 0, s, a, l.c);
  if (a.drate)
    hipLaunchKernelGGL(gscan_sum_kernel, dim3((unsigned)((a.width + 63) / 64)), dim3(1024), 0, s, a.part, a.drate,
                       a.batch * l.c.tiles, a.width);
  return hipGetLastError();
}

hipError_t launch_gscan_step(const GscanArgs& a, DT in, hipStream_t s) {
  auto k = in == DT::F32 ? SSM_GSCAN_PICK(step_kernel, float) : SSM_GSCAN_PICK(step_kernel, uint16_t);
  hipLaunchKernelGGL(k, dim3((unsigned)((a.batch * a.width + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssm
