// C-ABI host layer of libssmscan, third part (include/ssmmodel.h): the gated linear
// recurrence and the losses over a vocabulary.  As in api.cpp, every check runs before
// anything is enqueued; on any non-OK status nothing has been enqueued and no output
// has been written.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/ssmmodel.h"
#include "gscan_plan.h"
#include "host_block.h"
#include "model.h"
#include "vocab_plan.h"

namespace {

using namespace ssmhost;

static_assert(ssm::kGsSegment == SSM_GSCAN_SEGMENT && ssm::kVocabPieceBytes == SSM_VOCAB_PIECE_BYTES &&
                  ssm::vocab::kMostTops == SSM_DISTILL_MAX_TOP,
              "model.h, vocab_plan.h and ssmmodel.h agree");

// ------------------------------------------------------ gated linear recurrence

constexpr int64_t kGsMostRow = int64_t{1} << 24;      // elements between rows, and channels

struct GsSizes {
  int64_t tokens;    // batch * seqlen
  int64_t elems;     // ... * width
  int64_t state;     // batch * width
  int64_t states;    // elements of the stored states
};

// tiles: the call runs over tiles of steps (a single token's does not).
ssm_status gs_check(int64_t batch, int64_t seqlen, int64_t width, int flags, std::initializer_list<ssm_dtype> types,
                    bool tiles, GsSizes* sz) {
  if (batch < 0 || seqlen < 0 || width < 0)
    return fail(SSM_ERR_BAD_SHAPE, "negative size (batch=%lld seqlen=%lld width=%lld)", (long long)batch, (long long)seqlen,
                (long long)width);
  if ((flags & ~SSM_GSCAN_LERP) != 0) return fail(SSM_ERR_UNSUPPORTED, "recurrence flags %d: unknown bits", flags);
  for (ssm_dtype t : types)
    if (!valid_dtype(t)) return fail(SSM_ERR_UNSUPPORTED, "unknown dtype (%d)", (int)t);
  int64_t t;
  if (!mul_ok(batch, seqlen, &sz->tokens) || !mul_ok(sz->tokens, width, &sz->elems) || !mul_ok(sz->elems, 16, &t) ||
      !mul_ok(batch, width, &sz->state) || !mul_ok(sz->state, 16, &t))
    return fail(SSM_ERR_BAD_SHAPE, "element count overflows int64");
  if (sz->state > INT32_MAX - 1023 || width > kGsMostRow)
    return fail(SSM_ERR_UNSUPPORTED, "batch * width = %lld exceeds 2^31 - 1024 or width = %lld 2^24", (long long)sz->state, (long long)width);
  sz->states = sz->state * ceil_div(seqlen, SSM_GSCAN_SEGMENT);
  // a workgroup of 512 threads for every 64 channels of a row and 128 steps, back 64 (one
  // limit for both: what runs forward can have its gradients)
  if (tiles && ceil_div(seqlen, ssm::kGsBwdTile) * batch * ceil_div(width, 64) > kMaxThreads / 512)
    return fail(SSM_ERR_UNSUPPORTED, "batch=%lld by seqlen=%lld by width=%lld exceeds the grid", (long long)batch, (long long)seqlen,
                (long long)width);
  return SSM_OK;
}

// Bytes from the first token's first channel to the last token's last.
ssm_status gs_rows(const char* name, const void* p, int64_t tokens, int64_t width, int64_t row, int64_t esz, int64_t* bytes) {
  *bytes = 0;
  if (p == nullptr || tokens == 0 || width == 0) return SSM_OK;
  if (row < width)
    return fail(SSM_ERR_UNSUPPORTED, "%s rows are %lld elements apart, less than width=%lld", name, (long long)row,
                (long long)width);
  if (row > kGsMostRow)
    return fail(SSM_ERR_UNSUPPORTED, "%s rows are %lld elements apart: more than 2^24", name, (long long)row);
  int64_t n;
  if (!mul_ok(tokens, row, &n) || !mul_ok(n, 8, &n)) return fail(SSM_ERR_BAD_SHAPE, "%s extent overflows int64", name);
  *bytes = ((tokens - 1) * row + width) * esz;
  return SSM_OK;
}

ssm_status launched(hipError_t e) {
  return e == hipSuccess ? ok() : fail(SSM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}

// -------------------------------------------------- losses over a vocabulary

constexpr int64_t kVocabMost = int64_t{1} << 30, kVocabRows = int64_t{1} << 22, kVocabTiles = int64_t{1} << 22,
                  kVocabElems = int64_t{1} << 37;

struct VocabSizes {
  int64_t xb, wb;     // bytes that x and weight span
  int64_t tops;       // rows * top
};

ssm_status vocab_check(const void* x, int64_t x_row, const void* w, int64_t w_row, int64_t rows, int64_t width, int64_t vocab,
                       int64_t top, float scale, ssm_dtype in_dtype, VocabSizes* sz) {
  if (rows < 0 || width < 0 || vocab < 0 || top < 0)
    return fail(SSM_ERR_BAD_SHAPE, "negative size (rows=%lld width=%lld vocab=%lld top=%lld)", (long long)rows, (long long)width,
                (long long)vocab, (long long)top);
  if (in_dtype != SSM_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "the losses take bf16 rows and weights (their products run on bf16 matrix cores)");
  if (width % 8 != 0 || width < 8 || width > SSM_VOCAB_MAX_WIDTH)
    return fail(SSM_ERR_UNSUPPORTED, "width=%lld must be a positive multiple of 8, at most %d", (long long)width, SSM_VOCAB_MAX_WIDTH);
  if (vocab < 1 || vocab > kVocabMost || rows > kVocabRows)
    return fail(SSM_ERR_UNSUPPORTED, "vocab=%lld must be from 1 to 2^30 and rows=%lld at most 2^22", (long long)vocab, (long long)rows);
  if (rows * width > kVocabElems || vocab * width > kVocabElems)
    return fail(SSM_ERR_UNSUPPORTED, "rows=%lld or vocab=%lld by width=%lld exceeds 2^37 elements", (long long)rows, (long long)vocab,
                (long long)width);
  if (ceil_div(rows, ssm::kVocabTile) * ceil_div(vocab, ssm::kVocabTile) > kVocabTiles)
    return fail(SSM_ERR_UNSUPPORTED, "rows=%lld by vocab=%lld exceeds 2^22 tiles of 256 by 256", (long long)rows, (long long)vocab);
  if (top < 1 || top > SSM_DISTILL_MAX_TOP)
    return fail(SSM_ERR_UNSUPPORTED, "top=%lld must be from 1 to %d", (long long)top, SSM_DISTILL_MAX_TOP);
  if (!std::isfinite(scale)) return fail(SSM_ERR_UNSUPPORTED, "scale must be finite");
  const struct {
    const char* name;
    const void* p;
    int64_t n, row;
    int64_t* bytes;
  } sides[2] = {{"x", x, rows, x_row, &sz->xb}, {"weight", w, vocab, w_row, &sz->wb}};
  for (const auto& m : sides) {
    *m.bytes = 0;
    if (m.n == 0) continue;
    if (m.row < width || m.row % 8 != 0 || m.row > ssm::kVocabMaxLd)
      return fail(SSM_ERR_UNSUPPORTED, "%s rows are %lld elements apart: a multiple of 8 from %lld to 2^22 is supported", m.name,
                  (long long)m.row, (long long)width);
    *m.bytes = ((m.n - 1) * m.row + width) * 2;
  }
  sz->tops = rows * top;
  return SSM_OK;
}

ssm::VocabArgs vocab_args(const void* x, int64_t x_row, const void* w, int64_t w_row, const int64_t* index, float scale,
                          int64_t rows, int64_t width, int64_t vocab, int64_t top) {
  ssm::VocabArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.x_row = x_row;
  a.w = static_cast<const uint16_t*>(w);
  a.w_row = w_row;
  a.index = index;
  a.scale = scale;
  a.temperature = 1.0f;
  a.rows = (int32_t)rows;
  a.width = (int32_t)width;
  a.vocab = (int32_t)vocab;
  a.top = (int32_t)top;
  a.cus = device_simds() / 4;
  return a;
}

ssm_status check_temperature(float scale, float temperature) {
  if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(scale / temperature) ||
      !std::isnormal(temperature * temperature))
    return fail(SSM_ERR_UNSUPPORTED, "temperature must be positive and finite, its square a normal number and scale / temperature finite");
  return SSM_OK;
}

ssm_status vocab_run(Workspace& work, ssm::VocabArgs& a, bool backward, hipStream_t s) {
  const int64_t bytes = backward ? ssm::vocab_bwd_bytes(a) : ssm::vocab_fwd_bytes(a);
  void* ws = nullptr;
  hipError_t e = work.get(&ws, bytes, s);
  if (e != hipSuccess || ws == nullptr) return fail_hip("workspace allocation", (long long)bytes, e);
  a.work = static_cast<char*>(ws);
  e = backward ? ssm::launch_vocab_bwd(a, s) : ssm::launch_vocab_fwd(a, s);
  return launched(work.done(e, s));
}

// With no rows the weights' gradient is zero.
ssm_status no_rows(void* dweight, int64_t vocab, int64_t width, hipStream_t s) {
  if (dweight == nullptr) return ok();
  return launched(ssm::launch_fill_zero(static_cast<float*>(dweight), vocab * width / 2, s));
}

}  // namespace

extern "C" {

ssm_status ssm_gscan_fwd(const void* x, int64_t x_row, const void* r, int64_t r_row, const void* i, int64_t i_row,
                         const float* rate, int flags, const float* initial_state, void* out, float* last_state,
                         float* states, int64_t batch, int64_t seqlen, int64_t width, ssm_dtype in_dtype,
                         ssm_dtype out_dtype, void* stream) {
  Workspace work;
  GsSizes sz;
  ssm_status st = gs_check(batch, seqlen, width, flags, {in_dtype, out_dtype}, true, &sz);
  const int64_t si = esize(in_dtype), so = esize(out_dtype);
  int64_t xb, rb, ib;
  if (st == SSM_OK) st = gs_rows("x", x, sz.tokens, width, x_row, si, &xb);
  if (st == SSM_OK) st = gs_rows("r", r, sz.tokens, width, r_row, si, &rb);
  if (st == SSM_OK) st = gs_rows("i", i, sz.tokens, width, i_row, si, &ib);
  if (st != SSM_OK) return st;
  const bool some = sz.elems > 0;
  st = check_args({{"x", x, x ? xb : some, si, true},
                   {"r", r, r ? rb : some, si, true},
                   {"i", i, ib, si, false},
                   {"rate", rate, width * 4, 4, false},
                   {"initial_state", initial_state, sz.state * 4, 4, false}},
                  {{"out", out, sz.elems * so, so, true},
                   {"last_state", last_state, sz.state * 4, 4, false},
                   {"states", states, sz.states * 4, 4, false}},
                  {{"last_state", "initial_state"}});
  if (st != SSM_OK) return st;
  if (sz.state == 0) return ok();
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (seqlen == 0) {
    if (last_state == nullptr || last_state == initial_state) return ok();
    return launched(initial_state ? ssm::launch_copy_f32(last_state, initial_state, sz.state, s)
                                  : ssm::launch_fill_zero(last_state, sz.state, s));
  }
  ssm::GscanArgs a{};
  a.x = x;
  a.r = r;
  a.i = i;
  a.x_row = x_row;
  a.r_row = r_row;
  a.i_row = i_row;
  a.rate = rate;
  a.lerp = (flags & SSM_GSCAN_LERP) != 0;
  a.initial = initial_state;
  a.out = out;
  a.last = last_state;
  a.states = states;
  a.batch = batch;
  a.seqlen = seqlen;
  a.width = width;
  a.out_bf16 = out_dtype == SSM_BF16;
  void* ws = nullptr;
  hipError_t e = hipSuccess;
  const int64_t bytes = ssm::gscan_chain_bytes(batch, seqlen, width, false);
  if (bytes > 0) {
    e = work.get(&ws, bytes, s);
    if (e != hipSuccess || ws == nullptr) return fail_hip("workspace allocation", (long long)bytes, e);
    a.work = static_cast<char*>(ws);
  }
  e = ssm::launch_gscan_fwd(a, to_dt(in_dtype), s);
  return launched(work.done(e, s));
}

ssm_status ssm_gscan_bwd(const void* x, int64_t x_row, const void* r, int64_t r_row, const void* i, int64_t i_row,
                         const float* rate, int flags, const float* states, const void* dout,
                         const float* dlast_state, void* dx, void* dr, void* di, float* drate, float* dinitial_state,
                         int64_t batch, int64_t seqlen, int64_t width, ssm_dtype in_dtype, ssm_dtype out_dtype,
                         void* stream) {
  Workspace work;
  GsSizes sz;
  ssm_status st = gs_check(batch, seqlen, width, flags, {in_dtype, out_dtype}, true, &sz);
  const int64_t si = esize(in_dtype), so = esize(out_dtype);
  int64_t xb, rb, ib;
  if (st == SSM_OK) st = gs_rows("x", x, sz.tokens, width, x_row, si, &xb);
  if (st == SSM_OK) st = gs_rows("r", r, sz.tokens, width, r_row, si, &rb);
  if (st == SSM_OK) st = gs_rows("i", i, sz.tokens, width, i_row, si, &ib);
  if (st != SSM_OK) return st;
  if (rate == nullptr && drate != nullptr) return fail(SSM_ERR_UNSUPPORTED, "drate is given without rate");
  if (i == nullptr && di != nullptr) return fail(SSM_ERR_UNSUPPORTED, "di is given without i");
  const bool some = sz.elems > 0;
  st = check_args({{"x", x, x ? xb : some, si, true},
                   {"r", r, r ? rb : some, si, true},
                   {"i", i, ib, si, false},
                   {"rate", rate, width * 4, 4, false},
                   {"states", states, sz.states * 4, 4, true},
                   {"dout", dout, sz.elems * so, so, true},
                   {"dlast_state", dlast_state, sz.state * 4, 4, false}},
                  {{"dx", dx, sz.elems * si, si, true},
                   {"dr", dr, sz.elems * si, si, true},
                   {"di", di, sz.elems * si, si, i != nullptr},
                   {"drate", drate, width * 4, 4, false},
                   {"dinitial_state", dinitial_state, sz.state * 4, 4, false}});
  if (st != SSM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (!some) {
    if (drate != nullptr) e = ssm::launch_fill_zero(drate, width, s);
    if (e == hipSuccess && dinitial_state != nullptr)
      e = dlast_state ? ssm::launch_copy_f32(dinitial_state, dlast_state, sz.state, s)
                      : ssm::launch_fill_zero(dinitial_state, sz.state, s);
    return launched(e);
  }
  ssm::GscanArgs a{};
  a.x = x;
  a.r = r;
  a.i = i;
  a.x_row = x_row;
  a.r_row = r_row;
  a.i_row = i_row;
  a.rate = rate;
  a.lerp = (flags & SSM_GSCAN_LERP) != 0;
  a.states_in = states;
  a.dout = dout;
  a.dlast = dlast_state;
  a.dx = dx;
  a.dr = dr;
  a.di = di;
  a.drate = drate;
  a.dinitial = dinitial_state;
  a.batch = batch;
  a.seqlen = seqlen;
  a.width = width;
  a.out_bf16 = out_dtype == SSM_BF16;
  const int64_t chain = ssm::gscan_chain_bytes(batch, seqlen, width, true);
  const int64_t rows = batch * ceil_div(seqlen, ssm::kGsBwdTile);
  const int64_t bytes = chain + (drate != nullptr ? (rows + ssm::gscan_sum_slices(rows)) * width * 4 : 0);
  if (bytes > 0) {
    void* ws = nullptr;
    e = work.get(&ws, bytes, s);
    if (e != hipSuccess || ws == nullptr) return fail_hip("workspace allocation", (long long)bytes, e);
    a.work = static_cast<char*>(ws);
    if (drate != nullptr) a.part = reinterpret_cast<float*>(a.work + chain);
  }
  e = ssm::launch_gscan_bwd(a, to_dt(in_dtype), s);
  return launched(work.done(e, s));
}

ssm_status ssm_gscan_update(const float* state, float* state_out, const void* x, int64_t x_row, const void* r,
                            int64_t r_row, const void* i, int64_t i_row, const float* rate, int flags, void* out,
                            int64_t batch, int64_t width, ssm_dtype in_dtype, ssm_dtype out_dtype, void* stream) {
  GsSizes sz;
  ssm_status st = gs_check(batch, 1, width, flags, {in_dtype, out_dtype}, false, &sz);
  const int64_t si = esize(in_dtype), so = esize(out_dtype);
  int64_t xb, rb, ib;
  if (st == SSM_OK) st = gs_rows("x", x, batch, width, x_row, si, &xb);
  if (st == SSM_OK) st = gs_rows("r", r, batch, width, r_row, si, &rb);
  if (st == SSM_OK) st = gs_rows("i", i, batch, width, i_row, si, &ib);
  if (st != SSM_OK) return st;
  const bool some = sz.elems > 0;
  st = check_args({{"x", x, x ? xb : some, si, true},
                   {"r", r, r ? rb : some, si, true},
                   {"i", i, ib, si, false},
                   {"rate", rate, width * 4, 4, false},
                   {"state", state, sz.state * 4, 4, true}},
                  {{"out", out, sz.elems * so, so, true}, {"state_out", state_out, sz.state * 4, 4, true}},
                  {{"state_out", "state"}});
  if (st != SSM_OK) return st;
  if (!some) return ok();
  ssm::GscanArgs a{};
  a.x = x;
  a.r = r;
  a.i = i;
  a.x_row = x_row;
  a.r_row = r_row;
  a.i_row = i_row;
  a.rate = rate;
  a.lerp = (flags & SSM_GSCAN_LERP) != 0;
  a.initial = state;
  a.last = state_out;
  a.out = out;
  a.batch = batch;
  a.seqlen = 1;
  a.width = width;
  a.out_bf16 = out_dtype == SSM_BF16;
  return launched(ssm::launch_gscan_step(a, to_dt(in_dtype), static_cast<hipStream_t>(stream)));
}

ssm_status ssm_xent_fwd(const void* x, int64_t x_row, const void* weight, int64_t w_row, const int64_t* target,
                        float scale, float z_loss, float* loss, float* lse, int64_t rows, int64_t width,
                        int64_t vocab, ssm_dtype in_dtype, void* stream) {
  Workspace work;
  VocabSizes sz;
  ssm_status st = vocab_check(x, x_row, weight, w_row, rows, width, vocab, 1, scale, in_dtype, &sz);
  if (st != SSM_OK) return st;
  if (!std::isfinite(z_loss)) return fail(SSM_ERR_UNSUPPORTED, "z_loss must be finite");
  st = check_args({{"x", x, sz.xb, 16, true}, {"weight", weight, rows ? sz.wb : 0, 16, true}, {"target", target, rows * 8, 8, true}},
                  {{"loss", loss, rows * 4, 4, true}, {"lse", lse, rows * 4, 4, true}});
  if (st != SSM_OK || rows == 0) return st == SSM_OK ? ok() : st;
  ssm::VocabArgs a = vocab_args(x, x_row, weight, w_row, target, scale, rows, width, vocab, 1);
  a.z_loss = z_loss;
  a.loss = loss;
  a.lse = lse;
  return vocab_run(work, a, false, static_cast<hipStream_t>(stream));
}

ssm_status ssm_xent_bwd(const float* dloss, const void* x, int64_t x_row, const void* weight, int64_t w_row,
                        const int64_t* target, float scale, float z_loss, const float* lse, void* dx, void* dweight,
                        int64_t rows, int64_t width, int64_t vocab, ssm_dtype in_dtype, void* stream) {
  Workspace work;
  VocabSizes sz;
  ssm_status st = vocab_check(x, x_row, weight, w_row, rows, width, vocab, 1, scale, in_dtype, &sz);
  if (st != SSM_OK) return st;
  if (!std::isfinite(z_loss)) return fail(SSM_ERR_UNSUPPORTED, "z_loss must be finite");
  st = check_args({{"dloss", dloss, rows * 4, 4, true},
                   {"x", x, sz.xb, 16, true},
                   {"weight", weight, rows ? sz.wb : 0, 16, true},
                   {"target", target, rows * 8, 8, true},
                   {"lse", lse, rows * 4, 4, true}},
                  {{"dx", dx, rows * width * 2, 16, false}, {"dweight", dweight, vocab * width * 2, 16, false}});
  if (st != SSM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows == 0) return no_rows(dweight, vocab, width, s);
  if (dx == nullptr && dweight == nullptr) return ok();
  ssm::VocabArgs a = vocab_args(x, x_row, weight, w_row, target, scale, rows, width, vocab, 1);
  a.z_loss = z_loss;
  a.dloss = dloss;
  a.lse_in = lse;
  a.dx = static_cast<uint16_t*>(dx);
  a.dw = static_cast<uint16_t*>(dweight);
  return vocab_run(work, a, true, s);
}

ssm_status ssm_distill_fwd(const void* x, int64_t x_row, const void* weight, int64_t w_row, const int64_t* index,
                           const float* teacher, float scale, float temperature, float* loss, float* lse,
                           float* logits, int64_t rows, int64_t width, int64_t vocab, int64_t top, ssm_dtype in_dtype,
                           void* stream) {
  Workspace work;
  VocabSizes sz;
  ssm_status st = vocab_check(x, x_row, weight, w_row, rows, width, vocab, top, scale, in_dtype, &sz);
  if (st == SSM_OK) st = check_temperature(scale, temperature);
  if (st != SSM_OK) return st;
  st = check_args({{"x", x, sz.xb, 16, true},
                   {"weight", weight, rows ? sz.wb : 0, 16, true},
                   {"index", index, sz.tops * 8, 8, true},
                   {"teacher", teacher, sz.tops * 4, 4, true}},
                  {{"loss", loss, rows * 4, 4, true}, {"lse", lse, rows * 4, 4, true}, {"logits", logits, sz.tops * 4, 4, true}});
  if (st != SSM_OK || rows == 0) return st == SSM_OK ? ok() : st;
  ssm::VocabArgs a = vocab_args(x, x_row, weight, w_row, index, scale / temperature, rows, width, vocab, top);
  a.teacher = teacher;
  a.temperature = temperature;
  a.loss = loss;
  a.lse = lse;
  a.logits = logits;
  return vocab_run(work, a, false, static_cast<hipStream_t>(stream));
}

ssm_status ssm_distill_bwd(const float* dloss, const void* x, int64_t x_row, const void* weight, int64_t w_row,
                           const int64_t* index, const float* teacher, float scale, float temperature,
                           const float* lse, const float* logits, void* dx, void* dweight, int64_t rows,
                           int64_t width, int64_t vocab, int64_t top, ssm_dtype in_dtype, void* stream) {
  Workspace work;
  VocabSizes sz;
  ssm_status st = vocab_check(x, x_row, weight, w_row, rows, width, vocab, top, scale, in_dtype, &sz);
  if (st == SSM_OK) st = check_temperature(scale, temperature);
  if (st != SSM_OK) return st;
  st = check_args({{"dloss", dloss, rows * 4, 4, true},
                   {"x", x, sz.xb, 16, true},
                   {"weight", weight, rows ? sz.wb : 0, 16, true},
                   {"index", index, sz.tops * 8, 8, true},
                   {"teacher", teacher, sz.tops * 4, 4, true},
                   {"lse", lse, rows * 4, 4, true},
                   {"logits", logits, sz.tops * 4, 4, true}},
                  {{"dx", dx, rows * width * 2, 16, false}, {"dweight", dweight, vocab * width * 2, 16, false}});
  if (st != SSM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows == 0) return no_rows(dweight, vocab, width, s);
  if (dx == nullptr && dweight == nullptr) return ok();
  ssm::VocabArgs a = vocab_args(x, x_row, weight, w_row, index, scale / temperature, rows, width, vocab, top);
  a.teacher = teacher;
  a.temperature = temperature;
  a.dloss = dloss;
  a.lse_in = lse;
  a.logits_in = logits;
  a.dx = static_cast<uint16_t*>(dx);
  a.dw = static_cast<uint16_t*>(dweight);
  return vocab_run(work, a, true, s);
}

}  // extern "C"
