// gfx950 kernels of libssmscan: the gated linear recurrence
// h_t = a_t h_{t-1} + m_t u_t for each channel, its gradients and its single-token
// step.  A thread walks one channel of one batch row.
#include "gscan_kernel.h"

namespace ssm {
namespace {

template <typename T>
__device__ __forceinline__ float at(const void* p, int64_t i) {
  return Io<T>::cvt(Io<T>::load(p, i));
}

__device__ __forceinline__ void put(void* p, int64_t i, float v, int bf16) {
  if (bf16) Io<uint16_t>::store(p, i, v);
  else Io<float>::store(p, i, v);
}
__device__ __forceinline__ float get(const void* p, int64_t i, int bf16) {
  return bf16 ? at<uint16_t>(p, i) : at<float>(p, i);
}

template <typename T, bool RATE, bool LERP, bool GATE>
__global__ void __launch_bounds__(256) gscan_fwd_kernel(GscanArgs a) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.batch * a.width) return;
  const int64_t b = e / a.width, d = e % a.width;
  const float rate = RATE ? a.rate[d] : 0.0f;
  const int64_t segments = (a.seqlen + kGsSegment - 1) / kGsSegment;
  float h = a.initial ? a.initial[e] : 0.0f;
  for (int64_t t = 0; t < a.seqlen; ++t) {
    const int64_t tok = b * a.seqlen + t;
    if (a.states && t % kGsSegment == 0) a.states[(b * segments + t / kGsSegment) * a.width + d] = h;
    const Decay c = decay<RATE, LERP>(at<T>(a.r, tok * a.r_row + d), rate);
    float u = at<T>(a.x, tok * a.x_row + d);
    if constexpr (GATE) {
      float pos, neg;
      sigmoids(at<T>(a.i, tok * a.i_row + d), &pos, &neg);
      u *= pos;
    }
    h = __builtin_fmaf(c.a, h, c.m * u);
    put(a.out, tok * a.width + d, h, a.out_bf16);
  }
  if (a.last) a.last[e] = h;
}

template <typename T, bool RATE, bool LERP, bool GATE>
__global__ void __launch_bounds__(256) gscan_bwd_kernel(GscanArgs a) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.batch * a.width) return;
  const int64_t b = e / a.width, d = e % a.width;
  const float rate = RATE ? a.rate[d] : 0.0f;
  const int64_t segments = (a.seqlen + kGsSegment - 1) / kGsSegment;
  float carry = a.dlast ? a.dlast[e] : 0.0f, sum = 0.0f;
  float before[kGsSegment];
  for (int64_t s = segments - 1; s >= 0; --s) {
    const int64_t t0 = s * kGsSegment;
    const int n = (int)(a.seqlen - t0 < kGsSegment ? a.seqlen - t0 : kGsSegment);
    float h = a.states_in[(b * segments + s) * a.width + d];
#pragma unroll
    for (int j = 0; j < kGsSegment; ++j) {
      before[j] = h;
      if (j < n) {
        const int64_t tok = b * a.seqlen + t0 + j;
        const Decay c = decay<RATE, LERP>(at<T>(a.r, tok * a.r_row + d), rate);
        float u = at<T>(a.x, tok * a.x_row + d), pos, neg;
        if constexpr (GATE) {
          sigmoids(at<T>(a.i, tok * a.i_row + d), &pos, &neg);
          u *= pos;
        }
        h = __builtin_fmaf(c.a, h, c.m * u);
      }
    }
#pragma unroll
    for (int j = kGsSegment - 1; j >= 0; --j) {
      if (j < n) {
        const int64_t tok = b * a.seqlen + t0 + j;
        const Decay c = decay<RATE, LERP>(at<T>(a.r, tok * a.r_row + d), rate);
        const float x = at<T>(a.x, tok * a.x_row + d);
        float pos = 1.0f, neg = 0.0f;
        if constexpr (GATE) sigmoids(at<T>(a.i, tok * a.i_row + d), &pos, &neg);
        const float u = x * pos;
        const float g = get(a.dout, tok * a.width + d, a.out_bf16) + carry;
        const float grad_e = g * __builtin_fmaf(c.a, before[j], u * decay_slope<LERP>(c));
        const float gm = g * c.m;
        Io<T>::store(a.dx, tok * a.width + d, gm * pos);
        if constexpr (GATE) Io<T>::store(a.di, tok * a.width + d, gm * u * neg);
        Io<T>::store(a.dr, tok * a.width + d, grad_e * c.neg * (RATE ? -rate * c.pos : 1.0f));
        sum = __builtin_fmaf(-grad_e, c.pos, sum);
        carry = c.a * g;
      }
    }
  }
  if (a.dinitial) a.dinitial[e] = carry;
  if (a.drate) a.part[e] = sum;
}

template <typename T, bool RATE, bool LERP, bool GATE>
__global__ void __launch_bounds__(256) gscan_step_kernel(GscanArgs a) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.batch * a.width) return;
  const int64_t b = e / a.width, d = e % a.width;
  const Decay c = decay<RATE, LERP>(at<T>(a.r, b * a.r_row + d), RATE ? a.rate[d] : 0.0f);
  float u = at<T>(a.x, b * a.x_row + d);
  if constexpr (GATE) {
    float pos, neg;
    sigmoids(at<T>(a.i, b * a.i_row + d), &pos, &neg);
    u *= pos;
  }
  const float h = __builtin_fmaf(c.a, a.initial[e], c.m * u);
  a.last[e] = h;
  put(a.out, e, h, a.out_bf16);
}

__global__ void __launch_bounds__(256) gscan_sum_kernel(const float* __restrict__ part, float* __restrict__ out, int64_t n,
                                                        int64_t width) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (d >= width) return;
  float s = 0.0f;
  for (int64_t i = 0; i < n; ++i) s += part[i * width + d];
  out[d] = s;
}

// The kernel for a type and the three choices.
#define SSM_GSCAN_PICK(kernel, T)                                                                          \
  (a.rate ? (a.lerp ? (a.i ? kernel<T, true, true, true> : kernel<T, true, true, false>)                  \
                    : (a.i ? kernel<T, true, false, true> : kernel<T, true, false, false>))               \
          : (a.lerp ? (a.i ? kernel<T, false, true, true> : kernel<T, false, true, false>)                \
                    : (a.i ? kernel<T, false, false, true> : kernel<T, false, false, false>)))

unsigned blocks(int64_t n) { return (unsigned)((n + 255) / 256); }

}  // namespace

hipError_t launch_gscan_fwd(const GscanArgs& a, DT in, hipStream_t s) {
  auto k = in == DT::F32 ? SSM_GSCAN_PICK(gscan_fwd_kernel, float) : SSM_GSCAN_PICK(gscan_fwd_kernel, uint16_t);
  hipLaunchKernelGGL(k, dim3(blocks(a.batch * a.width)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_gscan_bwd(const GscanArgs& a, DT in, hipStream_t s) {
  auto k = in == DT::F32 ? SSM_GSCAN_PICK(gscan_bwd_kernel, float) : SSM_GSCAN_PICK(gscan_bwd_kernel, uint16_t);
  hipLaunchKernelGGL(k, dim3(blocks(a.batch * a.width)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_gscan_step(const GscanArgs& a, DT in, hipStream_t s) {
  auto k = in == DT::F32 ? SSM_GSCAN_PICK(gscan_step_kernel, float) : SSM_GSCAN_PICK(gscan_step_kernel, uint16_t);
  hipLaunchKernelGGL(k, dim3(blocks(a.batch * a.width)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_gscan_sum(const float* part, float* out, int64_t n, int64_t width, hipStream_t s) {
  hipLaunchKernelGGL(gscan_sum_kernel, dim3(blocks(width)), dim3(256), 0, s, part, out, n, width);
  return hipGetLastError();
}

}  // namespace ssm
