// gfx950 kernels of libssmscan: linear attention with a decay for each head,
// S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t: the chunked forward
// (linattn_kernel.h), the states at time chunk borders, and the single-token
// step.
#include <algorithm>

#include "linattn_kernel.h"

namespace ssm {
namespace {

template <int C>
__global__ void __launch_bounds__(256, 3) la_fwd_kernel(LaWalk a) {
  __shared__ LaTile<C, kWalkOut> s;
  int bh, slice;
  la_place(blockIdx.x, a.batch * a.nheads, (a.xdim + 63) / 64, &bh, &slice);
  la_walk<C, kWalkOut, false>(a, s, bh / a.nheads, bh % a.nheads, slice, blockIdx.y);
}

template <int C, bool REV>
__global__ void __launch_bounds__(256, 3) la_state_kernel(LaWalk a) {
  __shared__ LaTile<C, kWalkState> s;
  int bh, slice;
  la_place(blockIdx.x, a.batch * a.nheads, (a.xdim + 63) / 64, &bh, &slice);
  la_walk<C, kWalkState, REV>(a, s, bh / a.nheads, bh % a.nheads, slice, blockIdx.y + (REV ? 1 : 0));
}

// Composes the time chunks' (decay, end state) pairs in walking order; slot k
// then holds the state that enters chunk k + 1 (back in time: that leaves chunk k
// at its start, the gradient of the state entering it).
template <bool REV>
__global__ void __launch_bounds__(256) la_carry_kernel(LaWalk a) {
  const int64_t per = (int64_t)a.xdim * a.cdim;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= per) return;
  const int h = blockIdx.y;
  const int64_t b = blockIdx.z;
  const int K = a.n_chunks;
  constexpr int kAhead = 8;      // slots loaded before the first of them is stored
  float S = 0.0f;
  for (int i0 = 0; i0 + 1 < K; i0 += kAhead) {
    float end[kAhead], decay[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i + 1 >= K) break;
      const int64_t slot = (b * K + (REV ? K - 1 - i0 - i : i0 + i)) * a.nheads + h;
      end[i] = a.chunk_out[slot * per + e];
      decay[i] = a.chunk_decay[slot];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i + 1 >= K) break;
      const int64_t slot = (b * K + (REV ? K - 1 - i0 - i : i0 + i)) * a.nheads + h;
      S = __builtin_fmaf(__builtin_amdgcn_exp2f(decay[i]), S, end[i]);
      a.chunk_out[slot * per + e] = S;
    }
  }
}

// One token: each state row (dk values of one dv channel) is read and written
// once, 16 bytes per lane, LPR lanes per row; its product with q is summed
// over those lanes.  A thread takes two rows of one head, all loads first.  Memory
// bounds it: 64 sequences of 80 heads of 128 x 64 (337 MB) take 57 us, 5.9 TB/s; one
// sequence 3.9 us.
template <typename Tin, typename Tout, int LPR>
__global__ void __launch_bounds__(256) la_step_kernel(LaStep a) {
  constexpr int RPB = 256 / LPR;
  const int p0 = (int)(blockIdx.x * (2 * RPB) + threadIdx.x / LPR);
  const int q = (int)(threadIdx.x % LPR);
  if (p0 >= a.dv) return;                  // whole rows leave together
  const int h = blockIdx.y;
  const int64_t b = blockIdx.z;
  const int64_t bh = b * a.nheads + h;
  const bool in = 4 * q < a.dk;
  const int c = in ? 4 * q : 0;
  const int64_t qk = (b * a.ngroups + h / (a.nheads / a.ngroups)) * a.dk + c;
  const bool live1 = p0 + RPB < a.dv;      // the second row, or the first again
  int64_t row[2];
  row[0] = bh * a.dv + p0;
  row[1] = live1 ? row[0] + RPB : row[0];
  float4 s4[2];
  float v[2], kv[4], qv[4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    s4[r] = load_stream4(a.state + row[r] * a.dk + c);
    v[r] = ld_in(static_cast<const Tin*>(a.v) + row[r]);
  }
  load4<Tin>(a.k, qk, kv);
  load4<Tin>(a.q, qk, qv);
  const float d = __builtin_amdgcn_exp2f(a.decay[b * a.decay_b + h] * kLog2e);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (r == 1 && !live1) break;
    float hs[4] = {s4[r].x, s4[r].y, s4[r].z, s4[r].w};
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hs[i] = __builtin_fmaf(d, hs[i], v[r] * kv[i]);
      y = __builtin_fmaf(qv[i], hs[i], y);
    }
    if (in) store_stream4(a.state_out + row[r] * a.dk + c, make_float4(hs[0], hs[1], hs[2], hs[3]));
    else y = 0.0f;
    y = la_row_sum(y);
    if constexpr (LPR == 32) {
      const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(y), __float_as_uint(y), false, false);
      y = __uint_as_float(t[0]) + __uint_as_float(t[1]);
    }
    if constexpr (LPR == 64) y = la_rows_sum(y);
    if (q == 0) Io<Tout>::store(a.out, row[r], y * a.scale);
  }
}

template <typename Tin, typename Tout>
void launch_step_t(const LaStep& a, hipStream_t s) {
  const int lpr = a.dk <= 64 ? 16 : a.dk <= 128 ? 32 : 64;
  const int rows = 2 * (256 / lpr);
  const dim3 grid((unsigned)((a.dv + rows - 1) / rows), (unsigned)a.nheads, (unsigned)a.batch);
  if (lpr == 16) hipLaunchKernelGGL((la_step_kernel<Tin, Tout, 16>), grid, dim3(256), 0, s, a);
  else if (lpr == 32) hipLaunchKernelGGL((la_step_kernel<Tin, Tout, 32>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((la_step_kernel<Tin, Tout, 64>), grid, dim3(256), 0, s, a);
}

dim3 walk_grid(const LaWalk& a, int chunks) {
  return dim3((unsigned)((int64_t)a.batch * a.nheads * ((a.xdim + 63) / 64)), (unsigned)chunks);
}

}  // namespace

hipError_t launch_la_states(const LaWalk& a, bool rev, hipStream_t s) {
  const dim3 grid = walk_grid(a, a.n_chunks - 1);
  const dim3 carry((unsigned)(((int64_t)a.xdim * a.cdim + 255) / 256), (unsigned)a.nheads, (unsigned)a.batch);
  const bool wide = a.cdim > 64;
  if (rev) {
    if (wide) hipLaunchKernelGGL((la_state_kernel<128, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((la_state_kernel<64, true>), grid, dim3(256), 0, s, a);
    hipLaunchKernelGGL(la_carry_kernel<true>, carry, dim3(256), 0, s, a);
  } else {
    if (wide) hipLaunchKernelGGL((la_state_kernel<128, false>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((la_state_kernel<64, false>), grid, dim3(256), 0, s, a);
    hipLaunchKernelGGL(la_carry_kernel<false>, carry, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_la_fwd(const LaWalk& a, hipStream_t s) {
  const dim3 grid = walk_grid(a, a.n_chunks);
  if (a.cdim > 64) hipLaunchKernelGGL(la_fwd_kernel<128>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(la_fwd_kernel<64>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_la_step(const LaStep& a, DT in, DT out, hipStream_t s) {
  if (in == DT::F32 && out == DT::F32) launch_step_t<float, float>(a, s);
  else if (in == DT::F32) launch_step_t<float, uint16_t>(a, s);
  else if (out == DT::F32) launch_step_t<uint16_t, float>(a, s);
  else launch_step_t<uint16_t, uint16_t>(a, s);
  return hipGetLastError();
}

}  // namespace ssm
