// gfx950 kernels of libssmscan: the gradients of linear attention with a decay
// for each head.
//
// dq, dk and dv are walks of the forward's form (linattn_kernel.h).  The decay's
// gradient is dg_t = <exp(g_t) S_{t-1}, dS_t>.  Inside a chunk, with S the state
// that enters it, R the gradient of the state that leaves it, and
// M_us = exp(c_u - c_s) scale (q_u . k_s)(dout_u . v_s) for s < u,
//   dg_t = sum_{s < t <= u} M_us + sum_{u >= t} a_u + sum_{s < t} b_s + X,
//   a_u = scale exp(c_u) q_u . (S^T dout_u),  b_s = exp(c_end - c_s) k_s . (R^T v_s),
//   X = exp(c_end) <S, R>.
// The first sum is a suffix sum of M's row sums less its column sums, whose terms
// are fp32 and exact products, so that no difference of rounded values enters it;
// a and b are by-products of the dq and dk walks' readouts.  X follows from chunk
// to chunk: <S, R> at a chunk's end is X + sum b, at its start X + sum a; it
// is a plain dot product of two states where the walks end or a time chunk
// does, which bounds how far rounding travels.
#include <algorithm>

#include "linattn_kernel.h"

namespace ssm {
namespace {

// Three walks in one launch: the slots of a head are the slices of dq, of dk and
// of dv, side by side on one XCD, so that its rows are fetched once.
template <int CK, int CV>
__global__ void __launch_bounds__(256, 2) la_bwd_kernel(LaBwd a) {
  union Tiles {
    LaTile<CV, kWalkDq> dq;
    LaTile<CV, kWalkDk> dk;
    LaTile<CK, kWalkOut> dv;
  };
  __shared__ __attribute__((aligned(16))) char raw[sizeof(Tiles)];
  const int nk = (a.dq.xdim + 63) / 64, nv = (a.dv.xdim + 63) / 64;
  int bh, slot;
  la_place(blockIdx.x, a.dq.batch * a.dq.nheads, 2 * nk + nv, &bh, &slot);
  const int b = bh / a.dq.nheads, h = bh % a.dq.nheads, kt = blockIdx.y;
  if (slot < nk) la_walk<CV, kWalkDq, false>(a.dq, *reinterpret_cast<LaTile<CV, kWalkDq>*>(raw), b, h, slot, kt);
  else if (slot < 2 * nk) la_walk<CV, kWalkDk, true>(a.dk, *reinterpret_cast<LaTile<CV, kWalkDk>*>(raw), b, h, slot - nk, kt);
  else la_walk<CK, kWalkOut, true>(a.dv, *reinterpret_cast<LaTile<CK, kWalkOut>*>(raw), b, h, slot - 2 * nk, kt);
}

__device__ __forceinline__ float wave_total(float v) { return la_rows_sum(la_row_sum(v)); }

constexpr int kLaDecayChunks = kLaBwdChunk / kLaQ;   // matrix chunks per time chunk, at most

// The decay's gradient of one (batch row, head) and time chunk, from the walks'
// per-step parts.
__global__ void __launch_bounds__(256) la_decay_kernel(LaBwd a) {
  __shared__ float sA[kLaDecayChunks], sB[kLaDecayChunks], sdot[4], ssum[4];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int H = a.dq.nheads, K = a.dq.n_chunks;
  const int b = blockIdx.x / H, h = blockIdx.x % H, kt = blockIdx.y;
  const int64_t t_begin = (int64_t)kt * a.dq.chunk_len;
  const int64_t L = min(a.dq.chunk_len, a.dq.seqlen - t_begin);
  const int chunks = (int)((L + kLaQ - 1) / kLaQ);
  const int64_t per = (int64_t)a.dq.xdim * a.dq.cdim;
  const float* S = kt < K - 1 ? a.fwd_states + ((int64_t)(b * K + kt) * H + h) * per
                   : a.dlast != nullptr ? a.last_state + ((int64_t)b * H + h) * per : nullptr;
  const float* R = kt < K - 1 ? a.rev_states + ((int64_t)(b * K + kt + 1) * H + h) * per
                   : a.dlast != nullptr ? a.dlast + ((int64_t)b * H + h) * per : nullptr;
  float dot = 0.0f;
  if (S != nullptr)
    for (int64_t e = tid; e < per; e += 256) dot = __builtin_fmaf(S[e], R[e], dot);
  dot = wave_total(dot);
  if (l == 0) sdot[w] = dot;
  const int nk = (a.dq.xdim + 63) / 64;
  const int64_t plane = (int64_t)a.dq.batch * H * a.dq.seqlen;
  const int64_t at0 = ((int64_t)b * H + h) * a.dq.seqlen + t_begin;
  auto parts = [&](int c, float* da, float* db) SSM_INLINE {
    const int64_t t = (int64_t)c * kLaQ + l;
    *da = *db = 0.0f;
    if (l < kLaQ && t < L)
      for (int i = 0; i < nk; ++i) {
        *da += a.dq.part[i * plane + at0 + t];
        *db += a.dk.part[i * plane + at0 + t];
      }
  };
  for (int c = w; c < chunks; c += 4) {
    float da, db;
    parts(c, &da, &db);
    da = wave_total(da);
    db = wave_total(db);
    if (l == 0) {
      sA[c] = da;
      sB[c] = db;
    }
  }
  block_sync();
  const float end = sdot[0] + sdot[1] + sdot[2] + sdot[3];
  float sum = 0.0f;
  for (int c = w; c < chunks; c += 4) {
    float X = end;
    for (int i = chunks - 1; i > c; --i) X += sA[i] - sB[i];
    X -= sB[c];
    float da, db;
    parts(c, &da, &db);
    float one = 1.0f, pre = db;
    affine_wave_scan(one, pre);
    pre -= db;                                   // sum of b before this step
    float suf = __shfl(da, 63 - l);              // steps in reverse order
    one = 1.0f;
    affine_wave_scan(one, suf);
    suf = __shfl(suf, 63 - l);
    const float g = suf + pre + X;
    const int64_t t = (int64_t)c * kLaQ + l;
    if (l < kLaQ && t < L) {
      sum += g;
      if (!a.fixed_decay) a.ddecay[((int64_t)b * a.dq.seqlen + t_begin + t) * H + h] = g;
    }
  }
  if (a.fixed_decay) {
    sum = wave_total(sum);
    if (l == 0) ssum[w] = sum;
    block_sync();
    if (tid == 0) a.ddecay[(int64_t)(b * K + kt) * H + h] = ssum[0] + ssum[1] + ssum[2] + ssum[3];
  }
}

// Sums over the heads that share q and k, in head order; four columns per thread.
template <typename Tout>
__global__ void __launch_bounds__(256) la_group_sum_kernel(const float* in, Tout* out, int64_t n4, int dim4, int share) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const int64_t rg = i / dim4;
  const int d = (int)(i % dim4);
  const float* p = in + (rg * share * dim4 + d) * 4;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < share; ++k) {
    const float4 t = *reinterpret_cast<const float4*>(p + (int64_t)k * dim4 * 4);
    v[0] += t.x;
    v[1] += t.y;
    v[2] += t.z;
    v[3] += t.w;
  }
  store_row<Tout, 4>(out + i * 4, v);
}

__global__ void __launch_bounds__(256) la_decay_sum_kernel(const float* in, float* out, int64_t n, int nheads) {
  const int h = (int)(blockIdx.x * 256 + threadIdx.x);
  if (h >= nheads) return;
  float s = 0.0f;
  for (int64_t i = 0; i < n; ++i) s += in[i * nheads + h];
  out[h] = s;
}

}  // namespace

hipError_t launch_la_bwd(const LaBwd& a, hipStream_t s) {
  const int nk = (a.dq.xdim + 63) / 64, nv = (a.dv.xdim + 63) / 64;
  const dim3 grid((unsigned)((int64_t)a.dq.batch * a.dq.nheads * (2 * nk + nv)), (unsigned)a.dq.n_chunks);
  const bool wk = a.dv.cdim > 64, wv = a.dq.cdim > 64;
  if (wk && wv) hipLaunchKernelGGL((la_bwd_kernel<128, 128>), grid, dim3(256), 0, s, a);
  else if (wk) hipLaunchKernelGGL((la_bwd_kernel<128, 64>), grid, dim3(256), 0, s, a);
  else if (wv) hipLaunchKernelGGL((la_bwd_kernel<64, 128>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((la_bwd_kernel<64, 64>), grid, dim3(256), 0, s, a);
  hipLaunchKernelGGL(la_decay_kernel, dim3((unsigned)(a.dq.batch * a.dq.nheads), (unsigned)a.dq.n_chunks), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_la_group_sum(const float* in, void* out, bool out_bf16, int64_t rows, int ngroups, int share, int dim,
                               hipStream_t s) {
  const int64_t n4 = rows * ngroups * (dim / 4);
  const dim3 grid((unsigned)((n4 + 255) / 256));
  if (out_bf16)
    hipLaunchKernelGGL(la_group_sum_kernel<uint16_t>, grid, dim3(256), 0, s, in, static_cast<uint16_t*>(out), n4, dim / 4, share);
  else
    hipLaunchKernelGGL(la_group_sum_kernel<float>, grid, dim3(256), 0, s, in, static_cast<float*>(out), n4, dim / 4, share);
  return hipGetLastError();
}

hipError_t launch_la_decay_sum(const float* in, float* out, int64_t n, int nheads, hipStream_t s) {
  hipLaunchKernelGGL(la_decay_sum_kernel, dim3((unsigned)((nheads + 255) / 256)), dim3(256), 0, s, in, out, n, nheads);
  return hipGetLastError();
}

}  // namespace ssm
