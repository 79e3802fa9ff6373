// Host-only stand-ins for the model operators' kernel launchers (model.h), linked with
// fake_runtime.cpp: each reads the first and the last byte of every buffer, and of every
// part of the workspace that its plan (gscan_plan.h, vocab_plan.h) lays out, at the extent
// that the kernels index.  Nothing is computed.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>

#include "../../sequence_scan_amd/csrc/gscan_plan.h"
#include "../../sequence_scan_amd/csrc/vocab_plan.h"

namespace {
long g_model_launches = 0;

void touch(const char* what, const void* p, int64_t n, int64_t esize) {
  if (n <= 0) return;
  if (!p) {
    std::fprintf(stderr, "launcher got NULL %s for %lld elements\n", what, (long long)n);
    std::abort();
  }
  const volatile unsigned char* c = static_cast<const volatile unsigned char*>(p);
  (void)c[0];
  (void)c[n * esize - 1];
}
void maybe(const char* what, const void* p, int64_t n, int64_t esize) {
  if (p) touch(what, p, n, esize);
}
void fail(const char* what) {
  std::fprintf(stderr, "inconsistent plan: %s\n", what);
  std::abort();
}
int64_t es(ssm::DT t) { return t == ssm::DT::F32 ? 4 : 2; }

void gates(const ssm::GscanArgs& a, ssm::DT in, int64_t tokens) {
  touch("x", a.x, (tokens - 1) * a.x_row + a.width, es(in));
  touch("r", a.r, (tokens - 1) * a.r_row + a.width, es(in));
  if (a.i) touch("i", a.i, (tokens - 1) * a.i_row + a.width, es(in));
  maybe("rate", a.rate, a.width, 4);
  ++g_model_launches;
}

void chain(const ssm::GscanArgs& a, int64_t steps, bool backward) {
  const int64_t bytes = ssm::gscan_chain_bytes(a.batch, a.seqlen, a.width, backward);
  if (bytes % 16) fail("chain bytes");
  for (int ch = 1; ch <= 2; ++ch) {
    const ssm::Layout l = ssm::gscan_layout(a.batch, a.seqlen, a.width, steps, ch, a.work);
    const ssm::Chain& c = l.c;
    if ((int64_t)c.tiles * steps < a.seqlen || (int64_t)(c.tiles - 1) * steps >= a.seqlen) fail("tiles");
    if ((int64_t)c.groups * c.group < c.tiles || (int64_t)(c.groups - 1) * c.group >= c.tiles) fail("groups");
    if (l.bytes > bytes) fail("chain bytes");
    if (c.tiles == 1) continue;
    const int64_t each = 64 * ch;
    touch("parts", c.parts, (int64_t)c.strips * c.tiles * each, 8);
    touch("states", c.states, (int64_t)c.strips * c.groups * each, 4);
    touch("next", c.next, 1, 4);
    if ((char*)c.states < (char*)(c.parts + (int64_t)c.strips * c.tiles * each) ||
        (char*)c.next < (char*)(c.states + (int64_t)c.strips * c.groups * each) || (char*)(c.next + 1) > a.work + bytes)
      fail("chain parts overlap");
  }
}

struct Region {
  int64_t at, bytes;
};
// The parts of a workspace: apart, inside it and readable.
void regions(const char* work, int64_t bytes, std::initializer_list<Region> all) {
  for (const Region& r : all) {
    if (r.bytes == 0) continue;
    if (r.at % 16 || r.at + r.bytes > bytes) fail("workspace part");
    touch("workspace", work + r.at, r.bytes, 1);
    for (const Region& o : all)
      if (&o != &r && o.bytes && r.at < o.at + o.bytes && o.at < r.at + r.bytes) fail("workspace parts overlap");
  }
}

void head(const ssm::VocabArgs& a) {
  touch("x", a.x, (int64_t)(a.rows - 1) * a.x_row + a.width, 2);
  touch("weight", a.w, (int64_t)(a.vocab - 1) * a.w_row + a.width, 2);
  touch("index", a.index, (int64_t)a.rows * a.top, 8);
  maybe("teacher", a.teacher, (int64_t)a.rows * a.top, 4);
  if (a.cus < 1 || (!a.teacher && a.top != 1) || !(a.temperature > 0)) fail("arguments");
  ++g_model_launches;
}
}  // namespace

extern "C" long fake_model_launches(void) { return g_model_launches; }

namespace ssm {

hipError_t launch_gscan_fwd(const GscanArgs& a, DT in, hipStream_t) {
  const int64_t tokens = a.batch * a.seqlen, state = a.batch * a.width, segments = (a.seqlen + kGsSegment - 1) / kGsSegment;
  gates(a, in, tokens);
  maybe("initial", a.initial, state, 4);
  maybe("last", a.last, state, 4);
  maybe("states", a.states, state * segments, 4);
  touch("out", a.out, tokens * a.width, a.out_bf16 ? 2 : 4);
  chain(a, kGsFwdTile, false);
  return hipSuccess;
}

hipError_t launch_gscan_bwd(const GscanArgs& a, DT in, hipStream_t) {
  const int64_t tokens = a.batch * a.seqlen, state = a.batch * a.width, segments = (a.seqlen + kGsSegment - 1) / kGsSegment;
  gates(a, in, tokens);
  touch("states", a.states_in, state * segments, 4);
  touch("dout", a.dout, tokens * a.width, a.out_bf16 ? 2 : 4);
  maybe("dlast", a.dlast, state, 4);
  touch("dx", a.dx, tokens * a.width, es(in));
  touch("dr", a.dr, tokens * a.width, es(in));
  if (a.i) touch("di", a.di, tokens * a.width, es(in));
  maybe("dinitial", a.dinitial, state, 4);
  if (a.drate) {
    touch("drate", a.drate, a.width, 4);
    const int64_t rows = a.batch * ((a.seqlen + kGsBwdTile - 1) / kGsBwdTile);
    touch("part", a.part, (rows + gscan_sum_slices(rows)) * a.width, 4);
  }
  chain(a, kGsBwdTile, true);
  return hipSuccess;
}

hipError_t launch_gscan_step(const GscanArgs& a, DT in, hipStream_t) {
  gates(a, in, a.batch);
  touch("state", a.initial, a.batch * a.width, 4);
  touch("state_out", a.last, a.batch * a.width, 4);
  touch("out", a.out, a.batch * a.width, a.out_bf16 ? 2 : 4);
  return hipSuccess;
}

hipError_t launch_vocab_fwd(const VocabArgs& a, hipStream_t) {
  using namespace vocab;
  head(a);
  touch("loss", a.loss, a.rows, 4);
  touch("lse", a.lse, a.rows, 4);
  if (a.teacher) touch("logits", a.logits, (int64_t)a.rows * a.top, 4);
  const FwdParts at(a);
  const int64_t tile = at.large ? kLargeTile : kSmallTile;
  if (at.few.few ? at.pieces * at.few.share < a.vocab || at.pieces != at.few.groups * 8 : at.pieces * tile < a.vocab) fail("pieces");
  if (at.few.few && (a.rows > kFewRows || a.width > kFewWidth)) fail("few");
  regions(a.work, vocab_fwd_bytes(a), {{at.stats, at.pieces * a.rows * 8},
                                       {at.picked, a.teacher ? 0 : (int64_t)a.rows * 4},
                                       {at.keys, at.sorted ? (int64_t)a.rows * a.top * 8 : 0},
                                       {at.starts, at.sorted ? a.rows * (at.pieces + 1) * 2 : 0}});
  return hipSuccess;
}

hipError_t launch_vocab_bwd(const VocabArgs& a, hipStream_t) {
  using namespace vocab;
  head(a);
  touch("dloss", a.dloss, a.rows, 4);
  touch("lse", a.lse_in, a.rows, 4);
  if (a.teacher) touch("logits", a.logits_in, (int64_t)a.rows * a.top, 4);
  maybe("dx", a.dx, (int64_t)a.rows * a.width, 2);
  maybe("dweight", a.dw, (int64_t)a.vocab * a.width, 2);
  const BwdParts at(a);
  const int64_t rw = (int64_t)a.rows * a.width;
  if (at.ldz % kK || at.ldz < at.cut.piece || at.ldz > kVocabMaxLd || at.cut.piece < 1 ||
      (at.cut.piece < a.vocab && at.cut.piece % kVocabTile))
    fail("piece");
  if (a.rows * at.ldz * 2 > kVocabPieceBytes && at.cut.piece > kVocabPieceLeast) fail("piece bytes");
  int first = 0, slices = 0, pieces = 0;
  for (int64_t v0 = 0; v0 < a.vocab; v0 += at.cut.piece, ++pieces) {
    const Piece p(a, at.cut, v0);
    if (p.x_slice % kK || p.w_slice % kK || (int64_t)p.x_slices * p.x_slice < p.columns || (int64_t)(p.x_slices - 1) * p.x_slice >= p.columns ||
        (int64_t)p.w_slices * p.w_slice < a.rows || (int64_t)(p.w_slices - 1) * p.w_slice >= a.rows || p.w_slices > at.cut.w_slices)
      fail("slices");
    if (p.w_slices > 1 && at.cut.pieces > 1) fail("slices of rows in pieces");
    if (v0 == 0) first = p.x_slices;
    slices = std::max(slices, p.x_slices);
  }
  if (pieces != at.cut.pieces || slices > at.cut.x_slices || first < slices) fail("slices");
  regions(a.work, vocab_bwd_bytes(a),
          {{at.rows, a.rows * (int64_t)kRowGradBytes},
           {at.hard, a.teacher ? (int64_t)a.rows * a.top * 4 : 0},
           {at.x, a.dw ? rw * 2 : 0},
           {at.dz, a.rows * at.ldz * 2},
           {at.x_sums, a.dx && (pieces > 1 || at.cut.x_slices > 1) ? slices * rw * 4 : 0},
           {at.w_sums, a.dw && at.cut.w_slices > 1 ? at.cut.w_slices * at.cut.piece * a.width * 4 : 0}});
  return hipSuccess;
}

}  // namespace ssm
