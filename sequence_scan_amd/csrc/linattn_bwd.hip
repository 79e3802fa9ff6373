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
// to chunk: <S, R> at a chunk's end is X + sum b, at its start X + sum a; it is a
// plain dot product of two states where the walks or a time chunk start and end,
// which bounds how far rounding travels.  A fixed decay's gradient is the sum over all
// steps, in which the errors of X that neighbouring steps share add up: there the dq
// and dk walks keep S and R every four chunks, and X starts anew from each pair.  Of 6
// x 5926 steps of 5 heads, the sums were off by 2.6e-6 without, by 1.6e-6 with states
// every eight chunks and by 7e-7 with every four; 4 x 2048, 40 heads took 427, 464
// and 514 us then.
//
// Measured: 4 x 2048, 40 heads of 128 x 128, 434 us (a fixed decay: 523), of which the
// decay's kernel is 14 us; the bytes that have to move would take 114 us at a copy's
// rate.  The walks' registers leave two workgroups per CU, so that the chunks' chains bound
// it as in the forward.
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
  // (the tiles' own alignment: their swizzled addresses are formed by it)
  __shared__ __attribute__((aligned(alignof(Tiles)))) char raw[sizeof(Tiles)];
  static_assert(__alignof__(raw) == alignof(Tiles) && alignof(Tiles) == 1024, "the tiles' place");
  const int nk = (a.dq.xdim + 63) / 64, nv = (a.dv.xdim + 63) / 64;
  int bh, slot;
  la_place(blockIdx.x, a.dq.batch * a.dq.nheads, 2 * nk + nv, &bh, &slot);
  const int b = bh / a.dq.nheads, h = bh % a.dq.nheads, kt = blockIdx.y;
  if (slot < nk) la_walk<CV, kWalkDq, false>(a.dq, *reinterpret_cast<LaTile<CV, kWalkDq>*>(raw), b, h, slot, kt);
  else if (slot < 2 * nk) la_walk<CV, kWalkDk, true>(a.dk, *reinterpret_cast<LaTile<CV, kWalkDk>*>(raw), b, h, slot - nk, kt);
  else la_walk<CK, kWalkOut, true>(a.dv, *reinterpret_cast<LaTile<CK, kWalkOut>*>(raw), b, h, slot - 2 * nk, kt);
}

__device__ __forceinline__ double wave_total(double v) {
  const double p = la_prefix32(v);
  return __shfl(p, 31) + __shfl(p, 63);
}

constexpr int kLaDecayChunks = kLaBwdChunk / kLaQ;   // matrix chunks per time chunk, at most
constexpr int kDecayWaves = 16, kDecayEach = kLaDecayChunks / kDecayWaves;

// The decay's gradient of one (batch row, head) and time chunk, from the walks'
// per-step parts: a wavefront per matrix chunk, a lane per step, all parts loaded
// first.  The recursion for <S, R> runs from the time chunk's end; at its start it
// has to arrive at <S, R> there, which is known too.  What it misses by is the
// rounding that it gathered, and is taken off each chunk in proportion to its
// distance from the end.
__global__ void __launch_bounds__(64 * kDecayWaves) la_decay_kernel(LaBwd a) {
  __shared__ double sA[kLaDecayChunks], sB[kLaDecayChunks], sdot[kLaSnapParts + 1][kDecayWaves], ssum[kDecayWaves];
  const int tid = threadIdx.x, l = tid & 63, w = tid >> 6;
  const int H = a.dq.nheads, K = a.dq.n_chunks;
  const int b = blockIdx.x / H, h = blockIdx.x % H, kt = blockIdx.y;
  const int64_t t_begin = (int64_t)kt * a.dq.chunk_len;
  const int64_t L = min(a.dq.chunk_len, a.dq.seqlen - t_begin);
  const int chunks = (int)((L + kLaQ - 1) / kLaQ);
  const int64_t per = (int64_t)a.dq.xdim * a.dq.cdim;
  const int nk = (a.dq.xdim + 63) / 64;
  const int64_t plane = (int64_t)a.dq.batch * H * a.dq.seqlen;
  const int64_t at0 = ((int64_t)b * H + h) * a.dq.seqlen + t_begin;
  float da[kDecayEach], db[kDecayEach];
  double back[kDecayEach], upto[kDecayEach];
#pragma unroll
  for (int i = 0; i < kDecayEach; ++i) {
    const int64_t t = (int64_t)(w + kDecayWaves * i) * kLaQ + l;
    da[i] = db[i] = 0.0f;
    if (l < kLaQ && t < L)
      for (int n = 0; n < nk; ++n) {
        da[i] += a.dq.part[n * plane + at0 + t];
        db[i] += a.dk.part[n * plane + at0 + t];
      }
  }
  // <S, R> where the time chunk starts and ends, and at the states kept in between
  const int64_t bh = ((int64_t)b * H + h) * per;
  auto slot = [&](int k) SSM_INLINE { return ((int64_t)(b * K + k) * H + h) * per; };
  const int each = a.dq.snaps != nullptr ? kLaSnap : kLaDecayChunks;     // chunks from one to the next
  const int parts = (chunks + each - 1) / each;
  for (int e = 0; e <= parts; ++e) {
    const float* S;
    const float* R;
    int64_t n = per;
    if (e == 0) {
      S = kt > 0 ? a.fwd_states + slot(kt - 1) : a.initial != nullptr ? a.initial + bh : nullptr;
      R = kt > 0 ? a.rev_states + slot(kt) : a.initial != nullptr ? a.dinitial + bh : nullptr;
    } else if (e == parts) {
      S = kt < K - 1 ? a.fwd_states + slot(kt) : a.dlast != nullptr ? a.last_state + bh : nullptr;
      R = kt < K - 1 ? a.rev_states + slot(kt + 1) : a.dlast != nullptr ? a.dlast + bh : nullptr;
    } else {
      n = (int64_t)nk * (a.dq.cdim > 64 ? 8192 : 4096);
      const int64_t at = ((((int64_t)b * H + h) * K + kt) * a.dq.snap_slots + e - 1) * n;
      S = a.dq.snaps + at;
      R = a.dk.snaps + at;
    }
    double dot = 0.0;
    if (S != nullptr)
      for (int64_t i = 4 * tid; i < n; i += 4 * 64 * kDecayWaves) {   // n is a multiple of 64
        const float4 x = *reinterpret_cast<const float4*>(S + i), y = *reinterpret_cast<const float4*>(R + i);
        dot += (double)x.x * y.x + (double)x.y * y.y + ((double)x.z * y.z + (double)x.w * y.w);
      }
    dot = wave_total(dot);
    if (l == 0) sdot[e][w] = dot;
  }
#pragma unroll
  for (int i = 0; i < kDecayEach; ++i) {
    // the sum of a from each step on (in reverse order of the steps), that of b up to it
    back[i] = la_prefix32((double)__shfl(da[i], 31 - l, 32));
    upto[i] = la_prefix32((double)db[i]);
    if (l == 31) {
      sA[w + kDecayWaves * i] = back[i];
      sB[w + kDecayWaves * i] = upto[i];
    }
  }
  block_sync();
  // Lane e: <S, R> at border e; and lane i: the sum of A - B over the chunks from i on.
  double border = 0.0;
  if (l <= parts)
    for (int i = 0; i < kDecayWaves; ++i) border += sdot[l][i];
  static_assert(kLaDecayChunks == 64, "a lane per chunk");
  const int rev = 63 - l;
  double from = la_prefix32(rev < chunks ? sA[rev] - sB[rev] : 0.0);
  const double half = __shfl(from, 31);
  from = __shfl(from + (l > 31 ? half : 0.0), rev);
  double sum = 0.0;
#pragma unroll
  for (int n = 0; n < kDecayEach; ++n) {
    const int c = w + kDecayWaves * n;
    if (c >= chunks) continue;
    // this chunk's part: from its end back, and what its start misses by
    const int first = c / each * each, last = min(first + each, chunks);
    const double after = last < 64 ? __shfl(from, last) : 0.0;
    const double end = __shfl(border, c / each + 1);
    const double miss = end - __shfl(border, c / each) + (__shfl(from, first) - after);
    const double X = end + (__shfl(from, c) - (sA[c] - sB[c]) - after) - sB[c] -
                     miss * ((double)(last - c) - 0.5) / (double)(last - first);
    const double g = __shfl(back[n], 31 - l, 32) + (upto[n] - db[n]) + X;
    const int64_t t = (int64_t)c * kLaQ + l;
    if (l < kLaQ && t < L) {
      sum += g;
      if (!a.fixed_decay) a.ddecay[((int64_t)b * a.dq.seqlen + t_begin + t) * H + h] = (float)g;
    }
  }
  if (a.fixed_decay) {
    sum = wave_total(sum);
    if (l == 0) ssum[w] = sum;
    block_sync();
    if (tid == 0) {
      double r = 0.0;
#pragma unroll
      for (int i = 0; i < kDecayWaves; ++i) r += ssum[i];
      // (as two floats: the time chunks' parts can be much larger than their sum)
      const int64_t at = ((int64_t)(b * K + kt) * H + h) * 2;
      a.ddecay[at] = (float)r;
      a.ddecay[at + 1] = (float)(r - (double)(float)r);
    }
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
  double s = 0.0;
  for (int64_t i = 0; i < n; ++i) {
    const float2 p = *reinterpret_cast<const float2*>(in + (i * nheads + h) * 2);
    s += (double)p.x + (double)p.y;
  }
  out[h] = (float)s;
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
  hipLaunchKernelGGL(la_decay_kernel, dim3((unsigned)(a.dq.batch * a.dq.nheads), (unsigned)a.dq.n_chunks),
                     dim3(64 * kDecayWaves), 0, s, a);
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
