// C-ABI host layer of libssmscan, second part (include/ssmblock.h): the norms,
// linear attention and the 4-bit products.  As in api.cpp, every check runs
// before anything is enqueued; on any non-OK status nothing has been enqueued
// and no output has been written.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "../../include/ssmblock.h"
#include "block.h"
#include "host_block.h"

namespace {

using namespace ssmhost;

static_assert(ssm::kNormMaxWidth == SSM_NORM_MAX_WIDTH && ssm::kNormMaxBlocks == SSM_NORM_MAX_BLOCKS,
              "block.h and ssmblock.h agree");

// ----------------------------------------------------------------------- norms

constexpr int64_t kMaxNormChannels = int64_t{1} << 24;

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
  if (width > kMaxNormChannels)
    return fail(SSM_ERR_UNSUPPORTED, "width=%lld exceeds %lld", (long long)width, (long long)kMaxNormChannels);
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
ssm_status norm_bwd_run(Workspace& work, ssm::NormArgs& a, float* const sums[3], Launch launch, hipStream_t s) {
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
    e = work.get(&ws, bytes, s);
    if (e != hipSuccess || ws == nullptr) return fail_hip("workspace allocation", (long long)bytes, e);
    a.part = static_cast<float*>(ws);
  }
  e = launch(a);
  if (e == hipSuccess && want) e = ssm::launch_norm_sums(a.part, blocks, a.sums, width, sums, s);
  e = work.done(e, s);
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

// ------------------------------------------------------------ linear attention

static_assert(ssm::kLaMaxDim == SSM_LINATTN_MAX_DIM && ssm::kLaMaxStepDk == SSM_LINATTN_MAX_STEP_DK,
              "block.h and ssmblock.h agree");

struct LaSizes {
  int64_t rows;      // batch * seqlen
  int64_t v;         // elements of v and out
  int64_t qk;        // elements of q and k, packed
  int64_t state;     // elements of a state
  int64_t decay;     // elements of the decay
};

ssm_status la_check(int64_t batch, int64_t seqlen, int64_t nheads, int64_t ngroups, int64_t dk, int64_t dv, int flags,
                    float scale, std::initializer_list<ssm_dtype> types, LaSizes* sz) {
  if (batch < 0 || seqlen < 0 || nheads < 0 || ngroups < 0 || dk < 0 || dv < 0)
    return fail(SSM_ERR_BAD_SHAPE, "negative size (batch=%lld seqlen=%lld nheads=%lld ngroups=%lld dk=%lld dv=%lld)",
                (long long)batch, (long long)seqlen, (long long)nheads, (long long)ngroups, (long long)dk, (long long)dv);
  if (ngroups < 1 || nheads < 1 || nheads % ngroups != 0)
    return fail(SSM_ERR_UNSUPPORTED, "nheads=%lld must be a positive multiple of ngroups=%lld", (long long)nheads,
                (long long)ngroups);
  if (nheads > 65535) return fail(SSM_ERR_UNSUPPORTED, "nheads=%lld exceeds 65535", (long long)nheads);
  if (batch > 65535) return fail(SSM_ERR_UNSUPPORTED, "batch=%lld exceeds 65535", (long long)batch);
  if (dk < 1 || dv < 1 || dv > (1 << 24))
    return fail(SSM_ERR_UNSUPPORTED, "dk=%lld and dv=%lld must be positive, dv at most 2^24", (long long)dk, (long long)dv);
  if ((flags & ~SSM_LINATTN_FIXED_DECAY) != 0) return fail(SSM_ERR_UNSUPPORTED, "linear attention flags %d: unknown bits", flags);
  if (!std::isfinite(scale)) return fail(SSM_ERR_UNSUPPORTED, "scale must be finite");
  for (ssm_dtype t : types)
    if (!valid_dtype(t)) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype (%d)", (int)t);
  int64_t t;
  if (!mul_ok(batch, seqlen, &sz->rows) || !mul_ok(sz->rows, nheads, &sz->decay) || !mul_ok(sz->decay, dv, &sz->v) ||
      !mul_ok(sz->v, 8, &t) || !mul_ok(sz->rows, ngroups, &t) || !mul_ok(t, dk, &sz->qk) || !mul_ok(sz->qk, 8, &t) ||
      !mul_ok(sz->decay, dk, &t) || !mul_ok(t, 8, &t) || !mul_ok(batch * nheads, dk, &t) || !mul_ok(t, dv, &sz->state) ||
      !mul_ok(sz->state, 8, &t))
    return fail(SSM_ERR_BAD_SHAPE, "element count overflows int64");
  if (flags & SSM_LINATTN_FIXED_DECAY) sz->decay = nheads;
  return SSM_OK;
}

// What the chunked form needs besides.
ssm_status la_check_chunked(int64_t batch, int64_t nheads, int64_t dk, int64_t dv, ssm_dtype in_dtype, int slots) {
  if (in_dtype != SSM_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "chunked linear attention takes bf16 inputs (its products run on bf16 matrix cores)");
  if (dk % 8 != 0 || dv % 8 != 0 || dk > SSM_LINATTN_MAX_DIM || dv > SSM_LINATTN_MAX_DIM)
    return fail(SSM_ERR_UNSUPPORTED, "dk=%lld and dv=%lld must be multiples of 8, at most %d", (long long)dk, (long long)dv,
                SSM_LINATTN_MAX_DIM);
  if (batch * nheads * slots * 256 > kMaxThreads)
    return fail(SSM_ERR_UNSUPPORTED, "batch * nheads = %lld exceeds the grid", (long long)(batch * nheads));
  return SSM_OK;
}

ssm_status la_rows(const char* name, int64_t rows, int64_t width, int64_t row, int64_t* bytes) {
  *bytes = 0;
  if (rows == 0) return SSM_OK;
  if (row < width || row % 8 != 0 || row > (int64_t{1} << 24))
    return fail(SSM_ERR_UNSUPPORTED, "%s rows are %lld elements apart: a multiple of 8 from %lld to 2^24 is supported", name,
                (long long)row, (long long)width);
  int64_t t;
  if (!mul_ok(rows, row * 2, &t)) return fail(SSM_ERR_BAD_SHAPE, "%s extent overflows int64", name);
  *bytes = ((rows - 1) * row + width) * 2;
  return SSM_OK;
}

// Time chunks of a forward.  A workgroup walks 64 value columns of one (batch
// row, head), and three fit a CU: one round of them, up to 24 time chunks of at
// least 256 steps; past that two per CU, of at least 128 steps, since a time chunk
// costs a fixed part and the carry runs over all of them (microseconds, dk = dv =
// 128 where not said):
//   1 x 65537, 16 heads of 64 x 128: 16 chunks 362, 24 322, 32 339, 48 330
//   1 x 16384, 32 heads: 8 chunks 263, 12 253, 16 270    4 x 2048, 32 heads: 1 chunk 142, 2 145, 3 136, 4 146
//   1 x 8192, 8 heads: 16 chunks 61, 32 49, 48 53         1 x 2048, 8 heads: 4 chunks 58, 16 30, 32 31
//   1 x 131072, 2 heads of 128 x 64: 256 chunks 99, 384 107
// More workgroups than CUs are not cut: 4 x 2048, 40 heads: 1 chunk 173, 2 175.
void choose_la_plan(int64_t batch, int64_t seqlen, int64_t nheads, int64_t dv, int simds, ssm_plan* p) {
  const int64_t wgs = std::max<int64_t>(1, batch * nheads * ((dv + 63) / 64));
  const int64_t cus = std::max(1, simds / 4);
  int64_t chunks = 1;
  if (wgs <= cus) {
    chunks = 3 * cus / wgs;
    if (chunks > 24 || seqlen / chunks < 256) chunks = std::min(2 * cus / wgs, std::max<int64_t>(1, seqlen / 128));
  }
  int64_t len = seqlen > 0 ? ceil_div(seqlen, chunks) : 1;
  if (chunks > 1) len = (len + ssm::kLaQ - 1) / ssm::kLaQ * ssm::kLaQ;
  *p = ssm_plan{};
  p->chunk_len = std::max<int64_t>(1, len);
  p->n_chunks = ceil_div(seqlen, p->chunk_len);
}

// Time chunks of a backward: at most kLaBwdChunk steps each, and more where its
// three walks leave CUs idle.  The walks differ in length, so six workgroups per CU
// (two fit) even them out better than two, down to 256 steps (microseconds, dk = dv
// = 128, 2 and 6 per CU): 1 x 4096, 40 heads 356, 301; 1 x 8192, 8 heads 162, 152;
// with at least 512 steps in place of 256: 166, and 1 x 2048, 8 heads 100 in place of 75.
void choose_la_bwd_plan(int64_t batch, int64_t seqlen, int64_t nheads, int64_t slots, int simds, ssm_plan* p) {
  const int64_t wgs = std::max<int64_t>(1, batch * nheads * slots);
  const int64_t cus = std::max(1, simds / 4);
  int64_t chunks = ceil_div(seqlen, ssm::kLaBwdChunk);
  if (wgs <= cus) chunks = std::max(chunks, std::min(6 * cus / wgs, seqlen / 256));
  chunks = std::max<int64_t>(1, chunks);
  const int64_t len = (ceil_div(seqlen, chunks) + ssm::kLaQ - 1) / ssm::kLaQ * ssm::kLaQ;
  *p = ssm_plan{};
  p->chunk_len = std::max<int64_t>(ssm::kLaQ, len);
  p->n_chunks = ceil_div(seqlen, p->chunk_len);
}

ssm::LaOperand la_operand(const void* p, int64_t row, int64_t dim, int64_t share) {
  ssm::LaOperand o{};
  o.p = static_cast<const uint16_t*>(p);
  o.row = row;
  o.head = (int32_t)dim;
  o.share = (int32_t)share;
  return o;
}

// ------------------------------------------------------------ 4-bit products

ssm_status q4_check(int64_t m, int64_t n, int64_t k, int64_t group, std::initializer_list<ssm_dtype> types) {
  if (m < 0 || n < 0 || k < 0 || group < 0)
    return fail(SSM_ERR_BAD_SHAPE, "negative size (m=%lld n=%lld k=%lld group=%lld)", (long long)m, (long long)n, (long long)k,
                (long long)group);
  if (group != 32 && group != 64 && group != 128)
    return fail(SSM_ERR_UNSUPPORTED, "group=%lld is not supported (32, 64 or 128)", (long long)group);
  if (k % group != 0) return fail(SSM_ERR_UNSUPPORTED, "k=%lld must be a multiple of group=%lld", (long long)k, (long long)group);
  for (ssm_dtype t : types)
    if (!valid_dtype(t)) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype (%d)", (int)t);
  int64_t t;
  if (!mul_ok(n, k, &t) || !mul_ok(t, 8, &t) || !mul_ok(m, n, &t) || !mul_ok(t, 8, &t))
    return fail(SSM_ERR_BAD_SHAPE, "element count overflows int64");
  // (16 threads per column in a grid; 1024 of padding in 32-bit indexes; 65535
  // blocks of 5 rows)
  if (n > (1 << 28) - 1024 || k > INT32_MAX - 1024 || m > 65535ll * 5)
    return fail(SSM_ERR_UNSUPPORTED, "m=%lld, n=%lld or k=%lld exceeds what the kernel indexes", (long long)m, (long long)n,
                (long long)k);
  return SSM_OK;
}

}  // namespace

extern "C" {

ssm_status ssm_workspace(void* memory, int64_t bytes) {
  g_offer = Offer{nullptr, 0};
  if (bytes < 0) return fail(SSM_ERR_BAD_SHAPE, "negative size (bytes=%lld)", (long long)bytes);
  const ssm_status st = check_align("memory", memory, 16);
  if (st != SSM_OK) return st;
  if (memory != nullptr) g_offer = Offer{memory, bytes};
  return ok();
}

int64_t ssm_workspace_bytes(void) { return g_wanted; }

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
  Workspace work;
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
  return norm_bwd_run(work, a, sums, [&](const ssm::NormArgs& n) { return ssm::launch_add_norm_bwd(n, to_dt(out_dtype), to_dt(res_dtype), s); }, s);
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
  Workspace work;
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
  return norm_bwd_run(work, a, sums, [&](const ssm::NormArgs& n) { return ssm::launch_gated_norm_bwd(n, to_dt(in_dtype), to_dt(out_dtype), s); }, s);
}

ssm_status ssm_linattn_plan_query(int64_t batch, int64_t seqlen, int64_t nheads, int64_t dk, int64_t dv,
                                  ssm_plan* plan) {
  if (plan == nullptr) return fail(SSM_ERR_NULL_ARG, "required pointer plan is NULL");
  LaSizes sz;
  ssm_status st = la_check(batch, seqlen, nheads, 1, dk, dv, 0, 1.0f, {}, &sz);
  if (st == SSM_OK) st = la_check_chunked(batch, nheads, dk, dv, SSM_BF16, 2);
  if (st != SSM_OK) return st;
  choose_la_plan(batch, seqlen, nheads, dv, device_simds(), plan);
  return ok();
}

ssm_status ssm_linattn_fwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v, int64_t v_row,
                           const float* log_decay, int flags, float scale, const float* initial_state, void* out,
                           float* last_state, int64_t batch, int64_t seqlen, int64_t nheads, int64_t ngroups,
                           int64_t dk, int64_t dv, ssm_dtype in_dtype, ssm_dtype out_dtype, void* stream,
                           const ssm_plan* plan_in) {
  Workspace work;
  LaSizes sz;
  ssm_status st = la_check(batch, seqlen, nheads, ngroups, dk, dv, flags, scale, {in_dtype, out_dtype}, &sz);
  if (st == SSM_OK) st = la_check_chunked(batch, nheads, dk, dv, in_dtype, 2);
  int64_t qb, kb, vb;
  if (st == SSM_OK) st = la_rows("q", sz.rows, ngroups * dk, q_row, &qb);
  if (st == SSM_OK) st = la_rows("k", sz.rows, ngroups * dk, k_row, &kb);
  if (st == SSM_OK) st = la_rows("v", sz.rows, nheads * dv, v_row, &vb);
  if (st != SSM_OK) return st;
  const bool some = sz.rows > 0;
  st = check_args({{"q", q, qb, 16, true},
                   {"k", k, kb, 16, true},
                   {"v", v, vb, 16, true},
                   {"log_decay", log_decay, some ? sz.decay * 4 : 0, 4, true},
                   {"initial_state", initial_state, sz.state * 4, 16, false}},
                  {{"out", out, sz.v * esize(out_dtype), 16, true}, {"last_state", last_state, sz.state * 4, 16, false}},
                  {{"last_state", "initial_state"}});
  if (st != SSM_OK) return st;
  ssm_plan plan;
  if (plan_in != nullptr) {
    plan = *plan_in;
    if (plan.chunk_len < 1) return fail(SSM_ERR_UNSUPPORTED, "plan.chunk_len must be >= 1");
    plan.n_chunks = ceil_div(seqlen, plan.chunk_len);
    if (plan.n_chunks > 1 && plan.chunk_len % ssm::kLaQ != 0)
      return fail(SSM_ERR_UNSUPPORTED, "plan.chunk_len=%lld must be a multiple of %d when it cuts the sequence",
                  (long long)plan.chunk_len, ssm::kLaQ);
    if (plan.n_chunks > 65535) return fail(SSM_ERR_UNSUPPORTED, "plan gives more than 65535 chunks");
  } else {
    choose_la_plan(batch, seqlen, nheads, dv, device_simds(), &plan);
  }
  const int64_t K = std::max<int64_t>(1, plan.n_chunks);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool in_place = initial_state != nullptr && initial_state == last_state;
  if (batch == 0) return ok();
  hipError_t e = hipSuccess;
  if (seqlen == 0) {
    if (last_state != nullptr && !in_place)
      e = initial_state ? ssm::launch_copy_f32(last_state, initial_state, sz.state, s)
                        : ssm::launch_fill_zero(last_state, sz.state, s);
    return e == hipSuccess ? ok() : fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  }
  const bool fixed = (flags & SSM_LINATTN_FIXED_DECAY) != 0;
  const int64_t share = nheads / ngroups;
  ssm::LaWalk a{};
  a.A = la_operand(q, q_row, dk, share);
  a.B = la_operand(k, k_row, dk, share);
  a.X = la_operand(v, v_row, dv, 1);
  a.decay = log_decay;
  a.decay_t = fixed ? 0 : nheads;
  a.decay_b = fixed ? 0 : seqlen * nheads;
  a.out = out;
  a.first = initial_state;
  a.last = last_state;
  a.seqlen = seqlen;
  a.chunk_len = K > 1 ? plan.chunk_len : seqlen;
  a.st_x = dk;
  a.st_c = 1;
  a.n_chunks = (int32_t)K;
  a.batch = (int32_t)batch;
  a.nheads = (int32_t)nheads;
  a.xdim = (int32_t)dv;
  a.cdim = (int32_t)dk;
  a.out_bf16 = out_dtype == SSM_BF16;
  a.w_scale = scale;
  a.row_scale = scale;
  a.src_scale = 1.0f;
  void* ws = nullptr;
  if (K > 1) {
    // the workgroups that read the initial state are then not those that write
    // the last one: an in-place state is read from a copy
    int64_t n_state, n_decay;
    if (!mul_ok(sz.state, K, &n_state) || !mul_ok(batch * nheads, K, &n_decay))
      return fail(SSM_ERR_BAD_SHAPE, "workspace size overflows int64");
    Pieces w;
    const int64_t at_state = w.add(n_state), at_decay = w.add(n_decay), at_copy = w.add(in_place ? sz.state : 0);
    if (!w.fits) return fail(SSM_ERR_BAD_SHAPE, "workspace size overflows int64");
    e = work.get(&ws, w.floats * 4, s);
    if (e != hipSuccess || ws == nullptr) return fail_hip("workspace allocation", (long long)(w.floats * 4), e);
    float* f = static_cast<float*>(ws);
    a.chunk_out = f + at_state;
    a.chunk_states = a.chunk_out;
    a.chunk_decay = f + at_decay;
    if (in_place) {
      e = ssm::launch_copy_f32(f + at_copy, initial_state, sz.state, s);
      a.first = f + at_copy;
    }
    if (e == hipSuccess) e = ssm::launch_la_states(a, false, s);
  }
  if (e == hipSuccess) e = ssm::launch_la_fwd(a, s);
  e = work.done(e, s);
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_linattn_bwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v, int64_t v_row,
                           const float* log_decay, int flags, float scale, const float* initial_state,
                           const void* dout, const float* dlast_state, void* dq, void* dk_, void* dv_,
                           float* dlog_decay, float* dinitial_state, int64_t batch, int64_t seqlen, int64_t nheads,
                           int64_t ngroups, int64_t dk, int64_t dv, ssm_dtype in_dtype, ssm_dtype grad_dtype,
                           void* stream) {
  Workspace work;
  LaSizes sz;
  ssm_status st = la_check(batch, seqlen, nheads, ngroups, dk, dv, flags, scale, {in_dtype, grad_dtype}, &sz);
  if (st == SSM_OK) st = la_check_chunked(batch, nheads, dk, dv, in_dtype, 6);
  int64_t qb, kb, vb;
  if (st == SSM_OK) st = la_rows("q", sz.rows, ngroups * dk, q_row, &qb);
  if (st == SSM_OK) st = la_rows("k", sz.rows, ngroups * dk, k_row, &kb);
  if (st == SSM_OK) st = la_rows("v", sz.rows, nheads * dv, v_row, &vb);
  if (st != SSM_OK) return st;
  const int64_t sg = esize(grad_dtype);
  const bool some = sz.rows > 0;
  const bool fixed = (flags & SSM_LINATTN_FIXED_DECAY) != 0;
  st = check_args({{"q", q, qb, 16, true},
                   {"k", k, kb, 16, true},
                   {"v", v, vb, 16, true},
                   {"log_decay", log_decay, some ? sz.decay * 4 : 0, 4, true},
                   {"initial_state", initial_state, sz.state * 4, 16, false},
                   {"dout", dout, sz.v * 2, 16, true},
                   {"dlast_state", dlast_state, sz.state * 4, 16, false}},
                  {{"dq", dq, sz.qk * sg, 16, true},
                   {"dk", dk_, sz.qk * sg, 16, true},
                   {"dv", dv_, sz.v * sg, 16, true},
                   {"dlog_decay", dlog_decay, sz.decay * 4, 4, true},
                   {"dinitial_state", dinitial_state, sz.state * 4, 16, false}});
  if (st != SSM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (!some) {
    if (fixed) e = ssm::launch_fill_zero(dlog_decay, sz.decay, s);
    if (e == hipSuccess && dinitial_state != nullptr && sz.state > 0)
      e = dlast_state ? ssm::launch_copy_f32(dinitial_state, dlast_state, sz.state, s)
                      : ssm::launch_fill_zero(dinitial_state, sz.state, s);
    return e == hipSuccess ? ok() : fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  }
  const int64_t nk = (dk + 63) / 64, nv = (dv + 63) / 64, share = nheads / ngroups;
  ssm_plan plan;
  choose_la_bwd_plan(batch, seqlen, nheads, 2 * nk + nv, device_simds(), &plan);
  const int64_t K = plan.n_chunks;
  if (K > 65535) return fail(SSM_ERR_UNSUPPORTED, "seqlen=%lld gives more than 65535 time chunks", (long long)seqlen);
  if (share > 1 && sz.qk / 4 > kMaxThreads)
    return fail(SSM_ERR_UNSUPPORTED, "q and k of %lld elements exceed the grid that sums their heads' gradients", (long long)sz.qk);
  const int64_t q_chunks = (std::min(seqlen, plan.chunk_len) + ssm::kLaQ - 1) / ssm::kLaQ;
  const int64_t snap_slots = fixed ? (q_chunks - 1) / ssm::kLaSnap : 0;
  int64_t n_state, n_heads, n_part, n_grad, n_snap;
  if (!mul_ok(sz.state, K, &n_state) || !mul_ok(batch * nheads, K, &n_heads) || !mul_ok(sz.rows * nheads, nk, &n_part) ||
      !mul_ok(sz.rows * nheads, dk, &n_grad) ||
      !mul_ok(n_heads, snap_slots * nk * (dv > 64 ? 8192 : 4096), &n_snap))
    return fail(SSM_ERR_BAD_SHAPE, "workspace size overflows int64");
  Pieces w;
  const bool cut = K > 1;
  const int64_t at_pq = w.add(n_part), at_pk = w.add(n_part), at_fwd = w.add(cut ? n_state : 0),
                at_rev = w.add(cut ? n_state : 0), at_fd = w.add(cut ? n_heads : 0), at_rd = w.add(cut ? n_heads : 0),
                at_last = w.add(dlast_state ? sz.state : 0),
                at_init = w.add(initial_state ? sz.state : 0), at_dq = w.add(share > 1 ? n_grad : 0),
                at_dk = w.add(share > 1 ? n_grad : 0), at_dec = w.add(fixed ? 2 * n_heads : 0), at_sq = w.add(n_snap), at_sk = w.add(n_snap);
  if (!w.fits) return fail(SSM_ERR_BAD_SHAPE, "workspace size overflows int64");
  void* ws = nullptr;
  e = work.get(&ws, w.floats * 4, s);
  if (e != hipSuccess || ws == nullptr) return fail_hip("workspace allocation", (long long)(w.floats * 4), e);
  float* f = static_cast<float*>(ws);

  const ssm::LaOperand oq = la_operand(q, q_row, dk, share), ok_ = la_operand(k, k_row, dk, share),
                       ov = la_operand(v, v_row, dv, 1), od = la_operand(dout, nheads * dv, dv, 1);
  ssm::LaWalk base{};
  base.decay = log_decay;
  base.decay_t = fixed ? 0 : nheads;
  base.decay_b = fixed ? 0 : seqlen * nheads;
  base.seqlen = seqlen;
  base.chunk_len = plan.chunk_len;
  base.n_chunks = (int32_t)K;
  base.batch = (int32_t)batch;
  base.nheads = (int32_t)nheads;
  base.out_bf16 = grad_dtype == SSM_BF16;
  base.w_scale = scale;
  base.snap_slots = (int32_t)snap_slots;
  // the states at time chunk borders, values v (forward) and dout (back)
  ssm::LaWalk fs = base, rs = base;
  fs.B = ok_;
  fs.X = ov;
  fs.first = initial_state;
  fs.chunk_out = f + at_fwd;
  fs.chunk_decay = f + at_fd;
  fs.src_scale = 1.0f;
  rs.B = oq;
  rs.X = od;
  rs.first = dlast_state;
  rs.chunk_out = f + at_rev;
  rs.chunk_decay = f + at_rd;
  rs.src_scale = scale;
  for (ssm::LaWalk* p : {&fs, &rs}) {
    p->xdim = (int32_t)dv;
    p->cdim = (int32_t)dk;
    p->st_x = dk;
    p->st_c = 1;
  }
  ssm::LaBwd a{};
  a.dq = base;
  a.dq.A = od;
  a.dq.B = ov;
  a.dq.X = ok_;
  a.dq.Z = oq;
  a.dq.out = share > 1 ? static_cast<void*>(f + at_dq) : dq;
  a.dq.first = initial_state;
  a.dq.last = dlast_state ? f + at_last : nullptr;
  a.dq.chunk_states = f + at_fwd;
  a.dq.part = f + at_pq;
  a.dq.snaps = snap_slots > 0 ? f + at_sq : nullptr;
  a.dq.row_scale = scale;
  a.dq.src_scale = 1.0f;
  a.dk = base;
  a.dk.A = ov;
  a.dk.B = od;
  a.dk.X = oq;
  a.dk.Z = ok_;
  a.dk.out = share > 1 ? static_cast<void*>(f + at_dk) : dk_;
  a.dk.first = dlast_state;
  a.dk.chunk_states = f + at_rev;
  a.dk.part = f + at_pk;
  a.dk.snaps = snap_slots > 0 ? f + at_sk : nullptr;
  a.dk.row_scale = 1.0f;
  a.dk.src_scale = scale;
  for (ssm::LaWalk* p : {&a.dq, &a.dk}) {   // values k and q: states read transposed
    p->xdim = (int32_t)dk;
    p->cdim = (int32_t)dv;
    p->st_x = 1;
    p->st_c = dk;
    if (share > 1) p->out_bf16 = 0;
  }
  a.dv = base;
  a.dv.A = ok_;
  a.dv.B = oq;
  a.dv.X = od;
  a.dv.out = dv_;
  a.dv.first = dlast_state;
  a.dv.last = dinitial_state;
  a.dv.chunk_states = f + at_rev;
  a.dv.row_scale = 1.0f;
  a.dv.src_scale = scale;
  a.dv.xdim = (int32_t)dv;
  a.dv.cdim = (int32_t)dk;
  a.dv.st_x = dk;
  a.dv.st_c = 1;
  a.fwd_states = f + at_fwd;
  a.rev_states = f + at_rev;
  a.last_state = f + at_last;
  a.dlast = dlast_state;
  a.initial = initial_state;
  a.dinitial = f + at_init;
  a.dk.last = initial_state ? f + at_init : nullptr;
  a.ddecay = fixed ? f + at_dec : dlog_decay;
  a.fixed_decay = fixed ? 1 : 0;
  if (cut) e = ssm::launch_la_states(fs, false, s);
  if (cut && e == hipSuccess) e = ssm::launch_la_states(rs, true, s);
  if (e == hipSuccess) e = ssm::launch_la_bwd(a, s);
  if (share > 1) {
    const bool b16 = grad_dtype == SSM_BF16;
    if (e == hipSuccess) e = ssm::launch_la_group_sum(f + at_dq, dq, b16, sz.rows, (int)ngroups, (int)share, (int)dk, s);
    if (e == hipSuccess) e = ssm::launch_la_group_sum(f + at_dk, dk_, b16, sz.rows, (int)ngroups, (int)share, (int)dk, s);
  }
  if (fixed && e == hipSuccess) e = ssm::launch_la_decay_sum(f + at_dec, dlog_decay, batch * K, (int)nheads, s);
  e = work.done(e, s);
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_linattn_state_update(const float* state, float* state_out, const void* q, const void* k, const void* v,
                                    const float* log_decay, int flags, float scale, void* out, int64_t batch,
                                    int64_t nheads, int64_t ngroups, int64_t dk, int64_t dv, ssm_dtype in_dtype,
                                    ssm_dtype out_dtype, void* stream) {
  LaSizes sz;
  ssm_status st = la_check(batch, 1, nheads, ngroups, dk, dv, flags, scale, {in_dtype, out_dtype}, &sz);
  if (st != SSM_OK) return st;
  if (dk % 4 != 0 || dk > SSM_LINATTN_MAX_STEP_DK)
    return fail(SSM_ERR_UNSUPPORTED, "dk=%lld must be a multiple of 4, at most %d", (long long)dk, SSM_LINATTN_MAX_STEP_DK);
  const int64_t si = esize(in_dtype);
  st = check_args({{"state", state, sz.state * 4, 16, true},
                   {"q", q, sz.qk * si, 4 * si, true},
                   {"k", k, sz.qk * si, 4 * si, true},
                   {"v", v, sz.v * si, si, true},
                   {"log_decay", log_decay, batch > 0 ? sz.decay * 4 : 0, 4, true}},
                  {{"state_out", state_out, sz.state * 4, 16, true}, {"out", out, sz.v * esize(out_dtype), esize(out_dtype), true}},
                  {{"state_out", "state"}});
  if (st != SSM_OK) return st;
  if (batch == 0) return ok();
  ssm::LaStep a{};
  a.state = state;
  a.state_out = state_out;
  a.q = q;
  a.k = k;
  a.v = v;
  a.decay = log_decay;
  a.decay_b = (flags & SSM_LINATTN_FIXED_DECAY) ? 0 : nheads;
  a.out = out;
  a.scale = scale;
  a.batch = (int32_t)batch;
  a.nheads = (int32_t)nheads;
  a.ngroups = (int32_t)ngroups;
  a.dk = (int32_t)dk;
  a.dv = (int32_t)dv;
  const hipError_t e = ssm::launch_la_step(a, to_dt(in_dtype), to_dt(out_dtype), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_q4_matvec(const void* x, int64_t x_row, const uint8_t* codes, const void* scales, const uint8_t* zeros,
                         const float* bias, void* out, int64_t m, int64_t n, int64_t k, int64_t group,
                         ssm_dtype in_dtype, ssm_dtype scale_dtype, ssm_dtype out_dtype, void* stream) {
  Workspace work;
  ssm_status st = q4_check(m, n, k, group, {in_dtype, scale_dtype, out_dtype});
  if (st != SSM_OK) return st;
  const int64_t si = esize(in_dtype), ss = esize(scale_dtype), so = esize(out_dtype);
  int64_t xb = 0;
  if (m > 0 && k > 0) {
    int64_t t;
    if (x_row < k || x_row * si % 16 != 0)
      return fail(SSM_ERR_UNSUPPORTED, "x rows are %lld elements apart: at least k=%lld and a multiple of 16 bytes is supported",
                  (long long)x_row, (long long)k);
    if (!mul_ok(m, x_row, &t) || !mul_ok(t, 8, &t)) return fail(SSM_ERR_BAD_SHAPE, "x extent overflows int64");
    xb = ((m - 1) * x_row + k) * si;
  }
  const bool some = m > 0 && n > 0;
  st = check_args({{"x", x, xb, 16, some},
                   {"codes", codes, n * k / 2, 16, some},
                   {"scales", scales, n * (k / group) * ss, ss, some},
                   {"zeros", zeros, n * (k / group), 1, false},
                   {"bias", bias, n * 4, 4, false}},
                  {{"out", out, m * n * so, so, true}});
  if (st != SSM_OK) return st;
  if (!some) return ok();
  ssm::Q4Args a{};
  a.x = x;
  a.x_row = x_row;
  a.codes = codes;
  a.scales = scales;
  a.zeros = zeros;
  a.bias = bias;
  a.out = out;
  a.m = (int32_t)m;
  a.n = (int32_t)n;
  a.k = (int32_t)k;
  a.group = (int32_t)group;
  a.x_bf16 = in_dtype == SSM_BF16;
  a.scale_bf16 = scale_dtype == SSM_BF16;
  a.out_bf16 = out_dtype == SSM_BF16;
  a.cus = device_simds() / 4;
  hipStream_t s = static_cast<hipStream_t>(stream);
  void* ws = nullptr;
  hipError_t e = hipSuccess;
  if (const int64_t bytes = ssm::q4_image_bytes(a)) {
    e = work.get(&ws, bytes, s);
    if (e != hipSuccess || ws == nullptr) return fail_hip("workspace allocation", (long long)bytes, e);
    a.image = static_cast<char*>(ws);
  }
  e = ssm::launch_q4(a, s);
  e = work.done(e, s);
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return ok();
}

ssm_status ssm_q4_quantize(const void* w, uint8_t* codes, void* scales, uint8_t* zeros, int64_t n, int64_t k,
                           int64_t group, ssm_dtype w_dtype, ssm_dtype scale_dtype, void* stream) {
  ssm_status st = q4_check(0, n, k, group, {w_dtype, scale_dtype});
  if (st != SSM_OK) return st;
  const int64_t sw = esize(w_dtype), ss = esize(scale_dtype), groups = n * (k / group);
  if (groups > kMaxThreads) return fail(SSM_ERR_UNSUPPORTED, "n * k / group exceeds the grid");
  st = check_args({{"w", w, n * k * sw, sw, true}},
                  {{"codes", codes, n * k / 2, 1, true}, {"scales", scales, groups * ss, ss, true}, {"zeros", zeros, groups, 1, true}});
  if (st != SSM_OK) return st;
  if (groups == 0) return ok();
  const hipError_t e = ssm::launch_q4_quantize(w, w_dtype == SSM_BF16, codes, scales, scale_dtype == SSM_BF16, zeros, groups,
                                               (int)group, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // extern "C"
