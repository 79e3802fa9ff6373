// gfx950 kernels of libssmscan: the norm before a block with its residual add
// (norm_kernel.h), and the join of the backward's column sums.
#include <algorithm>

#include "norm_kernel.h"

namespace ssm {
namespace {

// Column sums of the row blocks: a workgroup takes 64 columns, its wavefronts
// every 16th row block each, and the 16 partial sums are added in order.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float* part, int blocks, int sums, int64_t width, float* o0,
                                                         float* o1, float* o2) {
  __shared__ float t[16][64];
  const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t d = (int64_t)blockIdx.x * 64 + l;
  const int k = blockIdx.y;
  float* out = k == 0 ? o0 : k == 1 ? o1 : o2;
  if (out == nullptr) return;
  float s = 0.0f;
  if (d < width) {
#pragma unroll 8
    for (int b = w; b < blocks; b += 16) s += part[((int64_t)b * sums + k) * width + d];
  }
  t[w][l] = s;
  block_sync();
  if (w == 0 && d < width) {
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) r += t[i][l];
    out[d] = r;
  }
}

}  // namespace

int norm_row_blocks(const NormArgs& a) { return (int)norm_shape(a, kNormBwdPerCu).grid.x; }

hipError_t launch_norm_sums(const float* part, int blocks, int sums, int64_t width, float* const out[3], hipStream_t s) {
  hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)((width + 63) / 64), (unsigned)sums), dim3(1024), 0, s, part, blocks,
                     sums, width, out[0], out[1], out[2]);
  return hipGetLastError();
}

hipError_t launch_add_norm(const NormArgs& a, DT in, DT res, hipStream_t s) {
  if (in == DT::F32 && res == DT::F32) launch_norm_fwd_t<kModeAdd, float, float>(a, s);
  else if (in == DT::F32) launch_norm_fwd_t<kModeAdd, float, uint16_t>(a, s);
  else if (res == DT::F32) launch_norm_fwd_t<kModeAdd, uint16_t, float>(a, s);
  else launch_norm_fwd_t<kModeAdd, uint16_t, uint16_t>(a, s);
  return hipGetLastError();
}

hipError_t launch_add_norm_bwd(const NormArgs& a, DT in, DT res, hipStream_t s) {
  if (in == DT::F32 && res == DT::F32) launch_norm_bwd_t<kModeAdd, float, float>(a, s);
  else if (in == DT::F32) launch_norm_bwd_t<kModeAdd, float, uint16_t>(a, s);
  else if (res == DT::F32) launch_norm_bwd_t<kModeAdd, uint16_t, float>(a, s);
  else launch_norm_bwd_t<kModeAdd, uint16_t, uint16_t>(a, s);
  return hipGetLastError();
}

}  // namespace ssm
