// C-ABI host layer of libssmscan, second part (include/ssmblock.h): the norms,
// linear attention and the 4-bit products.  As in api.cpp, every check runs
// before anything is enqueued; on any non-OK status nothing has been enqueued
// and no output has been written.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/ssmblock.h"
#include "block.h"
#include "host.h"

namespace {

using namespace ssmhost;

static_assert(ssm::kNormMaxWidth == SSM_NORM_MAX_WIDTH && ssm::kNormMaxBlocks == SSM_NORM_MAX_BLOCKS,
              "block.h and ssmblock.h agree");

struct Arg {
  const char* name;
  const void* p;
  int64_t bytes;     // extent that the kernels touch
  int64_t align;     // the element's size, or what vector accesses need
  bool required;
};

// Required pointers, alignment, and outputs that overlap an input or each
// other.  `same` lists pairs (output, input) that may be one buffer.
struct Same {
  const char* out;
  const char* in;
};
ssm_status check_args(std::initializer_list<Arg> ins, std::initializer_list<Arg> outs,
                      std::initializer_list<Same> same = {}) {
  ssm_status st;
  for (const auto* list : {&ins, &outs})
    for (const Arg& a : *list) {
      if (a.required && a.p == nullptr && a.bytes > 0)
        return fail(SSM_ERR_NULL_ARG, "required pointer %s is NULL", a.name);
      if ((st = check_align(a.name, a.p, (uintptr_t)a.align)) != SSM_OK) return st;
    }
  for (const Arg& o : outs) {
    const Range ro = range(o.name, o.p, o.bytes);
    for (const Arg& i : ins) {
      bool allowed = false;
      for (const Same& s : same)
        allowed |= o.p == i.p && o.bytes == i.bytes && std::string(s.out) == o.name && std::string(s.in) == i.name;
      if (!allowed && overlaps(ro, range(i.name, i.p, i.bytes)))
        return fail(SSM_ERR_UNSUPPORTED, "%s overlaps input %s", o.name, i.name);
    }
    for (const Arg& q : outs)
      if (&q != &o && overlaps(ro, range(q.name, q.p, q.bytes)))
        return fail(SSM_ERR_UNSUPPORTED, "%s overlaps %s", o.name, q.name);
  }
  return SSM_OK;
}

// ----------------------------------------------------------------------- norms

struct NormSizes {
  int64_t elems;   // rows * width
};

ssm_status norm_check(int64_t rows, int64_t width, int64_t ngroups, float eps, int flags, int allowed,
                      std::initializer_list<ssm_dtype> types, NormSizes* sz) {
  if (rows < 0 || width < 0)
    return fail(SSM_ERR_BAD_SHAPE, "negative size (rows=%lld width=%lld)", (long long)rows, (long long)width);
  if (ngroups < 1 || width % ngroups != 0)
    return fail(SSM_ERR_UNSUPPORTED, "width=%lld must be a multiple of ngroups=%lld >= 1", (long long)width,
                (long long)ngroups);
  if (width / ngroups > SSM_NORM_MAX_WIDTH)
    return fail(SSM_ERR_UNSUPPORTED, "a norm over %lld channels is not supported (at most %d)",
                (long long)(width / ngroups), SSM_NORM_MAX_WIDTH);
  if (ngroups > 65535) return fail(SSM_ERR_UNSUPPORTED, "ngroups=%lld exceeds 65535", (long long)ngroups);
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(SSM_ERR_UNSUPPORTED, "eps must be finite and not negative");
  if ((flags & ~allowed) != 0) return fail(SSM_ERR_UNSUPPORTED, "norm flags %d: unknown bits for this call", flags);
  for (ssm_dtype t : types)
    if (!valid_dtype(t)) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype (%d)", (int)t);
  int64_t t;
  if (!mul_ok(rows, width, &sz->elems) || !mul_ok(sz->elems, 8, &t))
    return fail(SSM_ERR_BAD_SHAPE, "element count overflows int64");
  return SSM_OK;
}

// Bytes from a strided tensor's first element to its last.
ssm_status norm_extent(const char* name, int64_t rows, int64_t width, int64_t stride, int64_t esz, int64_t* bytes) {
  int64_t n;
  *bytes = 0;
  if (rows == 0 || width == 0) return SSM_OK;
  if (stride < width)
    return fail(SSM_ERR_UNSUPPORTED, "%s rows are %lld elements apart, less than width=%lld", name, (long long)stride,
                (long long)width);
  if (!mul_ok(rows, stride, &n) || !mul_ok(n, 8, &n)) return fail(SSM_ERR_BAD_SHAPE, "%s extent overflows int64", name);
  *bytes = ((rows - 1) * stride + width) * esz;
  return SSM_OK;
}

// The backward's launches: the kernel, then the join of its column sums.
template <typename Launch>
ssm_status norm_bwd_run(ssm::NormArgs& a, float* const sums[3], Launch launch, hipStream_t s) {
  const int64_t width = (int64_t)a.groups * a.width;
  const bool want = sums[0] || sums[1] || sums[2];
  a.sums = sums[2] ? 3 : 2;
  int blocks = 0;
  void* ws = nullptr;
  hipError_t e = hipSuccess;
  if (want) {
    blocks = ssm::norm_row_blocks(a);
    int64_t bytes;
    if (!mul_ok((int64_t)blocks * a.sums, width * 4, &bytes)) return fail(SSM_ERR_BAD_SHAPE, "workspace size overflows int64");
    e = ws_alloc(&ws, bytes, s);
    if (e != hipSuccess || ws == nullptr) return fail_hip("workspace allocation", (long long)bytes, e);
    a.part = static_cast<float*>(ws);
  }
  e = launch(a);
  if (e == hipSuccess && want) e = ssm::launch_norm_sums(a.part, blocks, a.sums, width, sums, s);
  if (ws) {
    const hipError_t e2 = hipFreeAsync(ws, s);
    if (e == hipSuccess) e = e2;
  }
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return ok();
}

// With no rows the column sums are zero.
ssm_status zero_sums(float* const sums[3], int64_t width, hipStream_t s) {
  for (int k = 0; k < 3; ++k)
    if (sums[k] != nullptr && width > 0) {
      const hipError_t e = ssm::launch_fill_zero(sums[k], width, s);
      if (e != hipSuccess) return fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    }
  return ok();
}

}  // namespace

extern "C" {

ssm_status ssm_add_norm_fwd(const void* x, int64_t x_stride, const void* residual, const float* weight,
                            const float* bias, const float* scale, float alpha, float eps, int flags, void* out,
                            void* residual_out, int64_t rows, int64_t width, ssm_dtype x_dtype,
                            ssm_dtype res_dtype, ssm_dtype out_dtype, void* stream) {
  NormSizes sz;
  ssm_status st = norm_check(rows, width, 1, eps, flags, SSM_NORM_CENTER, {x_dtype, res_dtype, out_dtype}, &sz);
  if (st != SSM_OK) return st;
  const int64_t sx = esize(x_dtype), sr = esize(res_dtype), so = esize(out_dtype);
  int64_t xb;
  if ((st = norm_extent("x", rows, width, x_stride, sx, &xb)) != SSM_OK) return st;
  st = check_args({{"x", x, xb, sx, true},
                   {"residual", residual, sz.elems * sr, sr, false},
                   {"weight", weight, width * 4, 4, false},
                   {"bias", bias, width * 4, 4, false},
                   {"scale", scale, width * 4, 4, false}},
                  {{"out", out, sz.elems * so, so, true}, {"residual_out", residual_out, sz.elems * sr, sr, false}},
                  {{"residual_out", "residual"}});
  if (st != SSM_OK) return st;
  if (sz.elems == 0) return ok();
  ssm::NormArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.res = residual;
  a.w = weight;
  a.bias = bias;
  a.scale = scale;
  a.alpha = alpha;
  a.eps = eps;
  a.out = out;
  a.res_out = residual_out;
  a.rows = rows;
  a.width = (int32_t)width;
  a.groups = 1;
  a.center = (flags & SSM_NORM_CENTER) != 0;
  a.out_bf16 = out_dtype == SSM_BF16;
  a.cus = device_simds() / 4;
  const hipError_t e = ssm::launch_add_norm(a, to_dt(x_dtype), to_dt(res_dtype), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_add_norm_bwd(const void* dout, const void* r, const float* weight, const void* dresidual_out,
                            const void* x, int64_t x_stride, const float* scale, float alpha, float eps, int flags,
                            void* dx, void* dresidual, float* dweight, float* dbias, float* dscale, int64_t rows,
                            int64_t width, ssm_dtype x_dtype, ssm_dtype res_dtype, ssm_dtype out_dtype,
                            void* stream) {
  NormSizes sz;
  ssm_status st = norm_check(rows, width, 1, eps, flags, SSM_NORM_CENTER, {x_dtype, res_dtype, out_dtype}, &sz);
  if (st != SSM_OK) return st;
  const int64_t sx = esize(x_dtype), sr = esize(res_dtype), so = esize(out_dtype);
  int64_t xb = 0;
  if (dscale != nullptr && (st = norm_extent("x", rows, width, x_stride, sx, &xb)) != SSM_OK) return st;
  st = check_args({{"dout", dout, sz.elems * so, so, true},
                   {"r", r, sz.elems * sr, sr, true},
                   {"weight", weight, width * 4, 4, false},
                   {"dresidual_out", dresidual_out, sz.elems * sr, sr, false},
                   {"x", x, xb, sx, dscale != nullptr},
                   {"scale", scale, width * 4, 4, false}},
                  {{"dx", dx, sz.elems * sx, sx, false},
                   {"dresidual", dresidual, sz.elems * sr, sr, false},
                   {"dweight", dweight, width * 4, 4, false},
                   {"dbias", dbias, width * 4, 4, false},
                   {"dscale", dscale, width * 4, 4, false}},
                  {{"dresidual", "dresidual_out"}});
  if (st != SSM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* const sums[3] = {dweight, dbias, dscale};
  if (sz.elems == 0) return zero_sums(sums, width, s);
  ssm::NormArgs a{};
  a.dout = dout;
  a.res = r;
  a.w = weight;
  a.dres = dresidual_out;
  a.x = x;
  a.x_stride = x_stride;
  a.scale = scale;
  a.alpha = alpha;
  a.eps = eps;
  a.out = dx;
  a.res_out = dresidual;
  a.rows = rows;
  a.width = (int32_t)width;
  a.groups = 1;
  a.center = (flags & SSM_NORM_CENTER) != 0;
  a.x_bf16 = x_dtype == SSM_BF16;
  a.cus = device_simds() / 4;
  return norm_bwd_run(a, sums, [&](const ssm::NormArgs& n) { return ssm::launch_add_norm_bwd(n, to_dt(out_dtype), to_dt(res_dtype), s); }, s);
}

ssm_status ssm_gated_norm_fwd(const void* x, int64_t x_stride, const void* z, int64_t z_stride, const float* weight,
                              const float* bias, float eps, int flags, void* out, int64_t rows, int64_t width,
                              int64_t ngroups, ssm_dtype in_dtype, ssm_dtype out_dtype, void* stream) {
  NormSizes sz;
  ssm_status st = norm_check(rows, width, ngroups, eps, flags, SSM_NORM_CENTER | SSM_NORM_GATE_LAST,
                             {in_dtype, out_dtype}, &sz);
  if (st != SSM_OK) return st;
  const int64_t si = esize(in_dtype), so = esize(out_dtype);
  int64_t xb, zb = 0;
  if ((st = norm_extent("x", rows, width, x_stride, si, &xb)) != SSM_OK) return st;
  if (z != nullptr && (st = norm_extent("z", rows, width, z_stride, si, &zb)) != SSM_OK) return st;
  st = check_args({{"x", x, xb, si, true},
                   {"z", z, zb, si, false},
                   {"weight", weight, width * 4, 4, false},
                   {"bias", bias, width * 4, 4, false}},
                  {{"out", out, sz.elems * so, so, true}});
  if (st != SSM_OK) return st;
  if (sz.elems == 0) return ok();
  ssm::NormArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.z = z;
  a.z_stride = z_stride;
  a.w = weight;
  a.bias = bias;
  a.eps = eps;
  a.out = out;
  a.rows = rows;
  a.width = (int32_t)(width / ngroups);
  a.groups = (int32_t)ngroups;
  a.center = (flags & SSM_NORM_CENTER) != 0;
  a.gate_last = (flags & SSM_NORM_GATE_LAST) != 0;
  a.out_bf16 = out_dtype == SSM_BF16;
  a.cus = device_simds() / 4;
  const hipError_t e = ssm::launch_gated_norm(a, to_dt(in_dtype), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_gated_norm_bwd(const void* dout, const void* x, int64_t x_stride, const void* z, int64_t z_stride,
                              const float* weight, const float* bias, float eps, int flags, void* dx, void* dz,
                              float* dweight, float* dbias, int64_t rows, int64_t width, int64_t ngroups,
                              ssm_dtype in_dtype, ssm_dtype out_dtype, void* stream) {
  NormSizes sz;
  ssm_status st = norm_check(rows, width, ngroups, eps, flags, SSM_NORM_CENTER | SSM_NORM_GATE_LAST,
                             {in_dtype, out_dtype}, &sz);
  if (st != SSM_OK) return st;
  const int64_t si = esize(in_dtype), so = esize(out_dtype);
  int64_t xb, zb = 0;
  if ((st = norm_extent("x", rows, width, x_stride, si, &xb)) != SSM_OK) return st;
  if (z != nullptr && (st = norm_extent("z", rows, width, z_stride, si, &zb)) != SSM_OK) return st;
  if (z == nullptr && dz != nullptr) return fail(SSM_ERR_UNSUPPORTED, "dz is given without z");
  st = check_args({{"dout", dout, sz.elems * so, so, true},
                   {"x", x, xb, si, true},
                   {"z", z, zb, si, false},
                   {"weight", weight, width * 4, 4, false},
                   {"bias", bias, width * 4, 4, false}},
                  {{"dx", dx, sz.elems * si, si, true},
                   {"dz", dz, sz.elems * si, si, z != nullptr},
                   {"dweight", dweight, width * 4, 4, false},
                   {"dbias", dbias, width * 4, 4, false}});
  if (st != SSM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* const sums[3] = {dweight, dbias, nullptr};
  if (sz.elems == 0) return zero_sums(sums, width, s);
  ssm::NormArgs a{};
  a.dout = dout;
  a.x = x;
  a.x_stride = x_stride;
  a.z = z;
  a.z_stride = z_stride;
  a.w = weight;
  a.bias = bias;
  a.eps = eps;
  a.out = dx;
  a.dz = dz;
  a.rows = rows;
  a.width = (int32_t)(width / ngroups);
  a.groups = (int32_t)ngroups;
  a.center = (flags & SSM_NORM_CENTER) != 0;
  a.gate_last = (flags & SSM_NORM_GATE_LAST) != 0;
  a.cus = device_simds() / 4;
  return norm_bwd_run(a, sums, [&](const ssm::NormArgs& n) { return ssm::launch_gated_norm_bwd(n, to_dt(in_dtype), to_dt(out_dtype), s); }, s);
}

}  // extern "C"
