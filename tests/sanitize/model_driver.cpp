// Drives every entry point of ssmmodel.h through its host layer over the fake runtime and
// launchers (fake_runtime.cpp, fake_model.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer: buffers of exactly their documented sizes, empty sizes,
// absent and in-place tensors, rejected calls (which launch nothing), offered workspaces
// and an allocation that fails; then the plans of many sizes.  Prints "model driver ok".
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../../include/ssmmodel.h"
#include "../../sequence_scan_amd/csrc/gscan_plan.h"
#include "../../sequence_scan_amd/csrc/vocab_plan.h"

extern "C" void fake_fail_next_alloc(void);
extern "C" long fake_launches(void);
extern "C" long fake_model_launches(void);
extern "C" long fake_live_allocs(void);

namespace {
int g_failures = 0;
std::vector<void*> g_bufs;

void* buf(int64_t elems, int64_t esize) {
  if (elems <= 0) return nullptr;
  void* p = nullptr;
  if (posix_memalign(&p, 16, (size_t)(elems * esize)) != 0) std::abort();
  std::memset(p, 0, (size_t)(elems * esize));
  g_bufs.push_back(p);
  return p;
}
float* fbuf(int64_t n) { return static_cast<float*>(buf(n, 4)); }
int64_t* ibuf(int64_t n) { return static_cast<int64_t*>(buf(n, 8)); }
void release() {
  for (void* p : g_bufs) std::free(p);
  g_bufs.clear();
}
int64_t es(ssm_dtype t) { return t == SSM_F32 ? 4 : 2; }

void expect(const char* what, ssm_status got, ssm_status want) {
  if (got != want) {
    std::fprintf(stderr, "%s: status %d, expected %d; last error: %s\n", what, (int)got, (int)want, ssm_last_error());
    ++g_failures;
  }
}
long launches() { return fake_launches() + fake_model_launches(); }

// The call with its workspace from the pool, offered (exactly what it wants, and too
// little), and with an allocation that fails.
template <typename F>
void each_way(const char* what, F call) {
  expect(what, call(), SSM_OK);
  const int64_t n = ssm_workspace_bytes();
  if (n == 0) return;
  for (int64_t room : {n, n - 1}) {
    expect(what, ssm_workspace(buf(room, 1), room), SSM_OK);
    expect(what, call(), SSM_OK);
    if (ssm_workspace_bytes() != n) {
      std::fprintf(stderr, "%s: wants %lld bytes, then %lld\n", what, (long long)n, (long long)ssm_workspace_bytes());
      ++g_failures;
    }
  }
  const long before = launches();
  fake_fail_next_alloc();
  expect(what, call(), SSM_ERR_HIP);
  if (launches() != before) {
    std::fprintf(stderr, "%s: launched without its workspace\n", what);
    ++g_failures;
  }
}

void gscan(int64_t batch, int64_t seqlen, int64_t width, ssm_dtype in, ssm_dtype out, bool some) {
  const int64_t tokens = batch * seqlen, e = tokens * width, state = batch * width, row = some ? 3 * width + 1 : width;
  const int64_t span = e ? (tokens - 1) * row + width : 0, states = state * ((seqlen + SSM_GSCAN_SEGMENT - 1) / SSM_GSCAN_SEGMENT);
  void *x = buf(span, es(in)), *r = buf(span, es(in)), *i = some ? buf(span, es(in)) : nullptr;
  float *rate = some ? fbuf(width) : nullptr, *S = fbuf(state), *last = fbuf(state), *kept = fbuf(states);
  void* o = buf(e, es(out));
  each_way("gscan_fwd", [&] { return ssm_gscan_fwd(x, row, r, row, i, row, rate, 0, some ? S : nullptr, o, last, kept, batch, seqlen, width, in, out, nullptr); });
  each_way("gscan_fwd in place", [&] { return ssm_gscan_fwd(x, row, r, row, i, row, rate, SSM_GSCAN_LERP, S, o, S, nullptr, batch, seqlen, width, in, out, nullptr); });
  void *dx = buf(e, es(in)), *dr = buf(e, es(in)), *di = some ? buf(e, es(in)) : nullptr;
  float *drate = some ? fbuf(width) : nullptr, *dS = fbuf(state);
  each_way("gscan_bwd", [&] { return ssm_gscan_bwd(x, row, r, row, i, row, rate, 0, kept, o, some ? S : nullptr, dx, dr, di, drate, some ? dS : nullptr,
                                                   batch, seqlen, width, in, out, nullptr); });
  if (seqlen == 1)
    for (float* to : {S, last})
      expect("gscan_update", ssm_gscan_update(S, to, x, row, r, row, i, row, rate, 0, o, batch, width, in, out, nullptr), SSM_OK);
  release();
}

void losses(int64_t rows, int64_t width, int64_t vocab, int64_t top, bool apart) {
  const int64_t xr = width + (apart ? 24 : 0), wr = width + (apart ? 8 : 0);
  void *x = buf(rows ? (rows - 1) * xr + width : 0, 2), *w = buf((vocab - 1) * wr + width, 2);
  int64_t *t = ibuf(rows), *idx = ibuf(rows * top);
  float *loss = fbuf(rows), *lse = fbuf(rows), *teacher = fbuf(rows * top), *logits = fbuf(rows * top), *dloss = fbuf(rows);
  void *dx = buf(rows * width, 2), *dw = buf(vocab * width, 2);
  each_way("xent_fwd", [&] { return ssm_xent_fwd(x, xr, w, wr, t, 1.0f, 0.0f, loss, lse, rows, width, vocab, SSM_BF16, nullptr); });
  each_way("distill_fwd", [&] { return ssm_distill_fwd(x, xr, w, wr, idx, teacher, 1.0f, 2.0f, loss, lse, logits, rows, width, vocab, top, SSM_BF16, nullptr); });
  for (int wants = 0; wants < 4; ++wants) {
    void *gx = wants & 1 ? dx : nullptr, *gw = wants & 2 ? dw : nullptr;
    each_way("xent_bwd", [&] { return ssm_xent_bwd(dloss, x, xr, w, wr, t, 1.0f, 0.1f, lse, gx, gw, rows, width, vocab, SSM_BF16, nullptr); });
    each_way("distill_bwd", [&] { return ssm_distill_bwd(dloss, x, xr, w, wr, idx, teacher, 1.0f, 2.0f, lse, logits, gx, gw, rows, width, vocab, top,
                                                         SSM_BF16, nullptr); });
  }
  release();
}

// Plans alone, of sizes whose tensors need not be there: what fake_model.cpp checks of them, by arithmetic.
void plans() {
  using namespace ssm;
  for (int64_t rows : {1, 16, 17, 100, 1000, 8192, 100003, 1 << 22})
    for (int64_t width : {8, 64, 1000, 2560, 4096, 4104, 65536})
      for (int64_t vocab : {1, 255, 257, 5000, 50280, 262144, 1 << 22, 1 << 26, 1 << 30}) {
        const int64_t t = (rows + 255) / 256 * ((vocab + 255) / 256);
        if (t > 1 << 22 || rows * width > int64_t{1} << 37 || vocab * width > int64_t{1} << 37) continue;      // (refused)
        for (int both = 1; both < 4; ++both) {
          VocabArgs a{};
          uint16_t some = 0;
          a.rows = (int32_t)rows;
          a.width = (int32_t)width;
          a.vocab = (int32_t)vocab;
          a.top = 1;
          a.cus = 256;
          a.temperature = 1;
          a.dx = both & 1 ? &some : nullptr;
          a.dw = both & 2 ? &some : nullptr;
          const vocab::BwdParts at(a);
          int64_t pieces = 0, first = 0;
          bool good = at.cut.piece >= 1 && at.ldz <= kVocabMaxLd && vocab_bwd_bytes(a) > 0 && vocab_fwd_bytes(a) > 0;
          if (!good) {
            std::fprintf(stderr, "plan of %lld x %lld x %lld\n", (long long)rows, (long long)width, (long long)vocab);
            ++g_failures;
            continue;
          }
          for (int64_t v0 = 0; v0 < vocab; v0 += at.cut.piece, ++pieces) {
            const vocab::Piece p(a, at.cut, v0);
            good = good && p.columns >= 1 && (int64_t)p.x_slices * p.x_slice >= p.columns && (int64_t)p.w_slices * p.w_slice >= rows;
            // items of a launch stay within a grid of 2^32 threads and an int
            const int64_t tile = at.cut.large ? vocab::kLargeTile : vocab::kSmallTile;
            const int64_t items = vocab::tiles(rows, tile) * vocab::tiles(width, tile) * p.x_slices +
                                  vocab::tiles(p.columns, tile) * vocab::tiles(width, tile) * p.w_slices;
            good = good && items < (int64_t{1} << 23);
            if (v0 == 0) first = p.x_slices;
            good = good && p.x_slices <= first && first <= at.cut.x_slices;
          }
          if (!good || pieces != at.cut.pieces) {
            std::fprintf(stderr, "plan of %lld x %lld x %lld: %lld pieces of %lld, %lld slices of %d\n", (long long)rows, (long long)width,
                         (long long)vocab, (long long)pieces, (long long)at.cut.piece, (long long)first, at.cut.x_slices);
            ++g_failures;
          }
        }
      }
}
}  // namespace

int main() {
  for (ssm_dtype in : {SSM_F32, SSM_BF16})
    for (ssm_dtype out : {SSM_F32, SSM_BF16})
      for (bool some : {false, true})
        for (int64_t L : {0, 1, 31, 64, 65, 128, 129, 700, 9000}) gscan(3, L, L == 9000 ? 5 : 130, in, out, some);
  gscan(0, 5, 8, SSM_F32, SSM_F32, true);
  gscan(2, 5, 0, SSM_F32, SSM_F32, true);
  for (bool apart : {false, true}) {
    losses(0, 64, 100, 3, apart);
    losses(1, 8, 1, 1, apart);
    losses(5, 72, 300, 7, apart);
    losses(300, 64, 513, 20, apart);
    losses(1000, 16, 700, 2, apart);
    losses(16, 4096, 300, 1024, apart);
    losses(16, 4104, 300, 3, apart);
  }
  losses(70000, 8, 2600, 1, false);
  plans();
  if (fake_live_allocs() != 0) {
    std::fprintf(stderr, "%ld workspace allocations not freed\n", fake_live_allocs());
    ++g_failures;
  }
  if (g_failures) return 1;
  std::printf("model driver ok\n");
  return 0;
}
