// Drives every entry point of ssmblock.h through its host layer over the fake
// runtime and launchers (fake_runtime.cpp, fake_block.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer: buffers of exactly their
// documented sizes, empty sizes, in-place and absent tensors, rejected calls (which
// launch nothing), and a workspace allocation that fails.  Prints "block driver ok".
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../../include/ssmblock.h"

extern "C" void fake_fail_next_alloc(void);
extern "C" long fake_launches(void);
extern "C" long fake_block_launches(void);
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
uint8_t* cbuf(int64_t n) { return static_cast<uint8_t*>(buf(n, 1)); }
int64_t es(ssm_dtype t) { return t == SSM_F32 ? 4 : 2; }

void expect(const char* what, ssm_status got, ssm_status want) {
  if (got != want) {
    std::fprintf(stderr, "%s: status %d, expected %d; last error: %s\n", what, (int)got, (int)want, ssm_last_error());
    ++g_failures;
  }
}
long launches() { return fake_launches() + fake_block_launches(); }
template <typename F>
void rejected(const char* what, ssm_status want, F call) {
  const long before = launches();
  expect(what, call(), want);
  if (launches() != before) {
    std::fprintf(stderr, "%s: a rejected call launched a kernel\n", what);
    ++g_failures;
  }
}

// The call with its workspace offered: exactly what it wants, and too little.
template <typename F>
void offered(const char* what, F call) {
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
}

const ssm_dtype kTypes[] = {SSM_F32, SSM_BF16};

void add_norm(int64_t rows, int64_t width) {
  for (ssm_dtype xt : kTypes)
    for (ssm_dtype rt : kTypes)
      for (ssm_dtype ot : kTypes) {
        const int64_t n = rows * width, stride = width + 3;
        void* x = buf(rows > 0 ? (rows - 1) * stride + width : 0, es(xt));
        void *r = buf(n, es(rt)), *ro = buf(n, es(rt)), *out = buf(n, es(ot)), *dx = buf(n, es(xt)), *dr = buf(n, es(rt));
        float *w = fbuf(width), *b = fbuf(width), *sc = fbuf(width), *dw = fbuf(width), *db = fbuf(width), *ds = fbuf(width);
        auto fwd = [&](const void* res, void* res_out, float* wt) {
          return ssm_add_norm_fwd(x, stride, res, wt, wt ? b : nullptr, wt ? sc : nullptr, 0.5f, 1e-5f, SSM_NORM_CENTER, out, res_out,
                                  rows, width, xt, rt, ot, nullptr);
        };
        expect("add_norm", fwd(r, ro, w), SSM_OK);
        expect("add_norm in place", fwd(r, r, w), SSM_OK);
        expect("add_norm bare", fwd(nullptr, nullptr, nullptr), SSM_OK);
        auto bwd = [&](void* dro, void* dres, float* w1, float* b1, float* s1, void* px) {
          return ssm_add_norm_bwd(out, r, w, dro, x, stride, sc, 0.5f, 1e-5f, 0, px, dres, w1, b1, s1, rows, width, xt, rt, ot, nullptr);
        };
        offered("add_norm_bwd", [&] { return bwd(ro, dr, dw, db, ds, dx); });
        expect("add_norm_bwd in place", bwd(ro, ro, dw, nullptr, nullptr, dx), SSM_OK);
        expect("add_norm_bwd bare", bwd(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr), SSM_OK);
        if (n > 0) {
          fake_fail_next_alloc();
          rejected("add_norm_bwd without workspace", SSM_ERR_HIP, [&] { return bwd(ro, dr, dw, db, ds, dx); });
          rejected("add_norm out on x", SSM_ERR_UNSUPPORTED, [&] {
            return ssm_add_norm_fwd(x, stride, r, w, b, sc, 1, 1e-5f, 0, x, ro, rows, width, xt, rt, ot, nullptr);
          });
          rejected("add_norm short rows", SSM_ERR_UNSUPPORTED, [&] {
            return ssm_add_norm_fwd(x, width - 1, r, w, b, sc, 1, 1e-5f, 0, out, ro, rows, width, xt, rt, ot, nullptr);
          });
        }
      }
}

void gated_norm(int64_t rows, int64_t width, int64_t groups) {
  for (ssm_dtype it : kTypes)
    for (ssm_dtype ot : kTypes)
      for (int flags : {0, SSM_NORM_CENTER, SSM_NORM_GATE_LAST}) {
        const int64_t n = rows * width, sx = width + 5, sz = 2 * width;
        void *x = buf(rows > 0 ? (rows - 1) * sx + width : 0, es(it)), *z = buf(rows > 0 ? (rows - 1) * sz + width : 0, es(it));
        void *out = buf(n, es(ot)), *dx = buf(n, es(it)), *dz = buf(n, es(it));
        float *w = fbuf(width), *b = fbuf(width), *dw = fbuf(width), *db = fbuf(width);
        for (void* g : {z, static_cast<void*>(nullptr)}) {
          expect("gated_norm", ssm_gated_norm_fwd(x, sx, g, sz, w, b, 1e-5f, flags, out, rows, width, groups, it, ot, nullptr), SSM_OK);
          auto bwd = [&](float* w1, float* b1) {
            return ssm_gated_norm_bwd(out, x, sx, g, sz, w, b, 1e-5f, flags, dx, g ? dz : nullptr, w1, b1, rows, width, groups, it, ot, nullptr);
          };
          offered("gated_norm_bwd", [&] { return bwd(dw, db); });
          expect("gated_norm_bwd without sums", bwd(nullptr, nullptr), SSM_OK);
        }
        if (n > 0) {
          fake_fail_next_alloc();
          rejected("gated_norm_bwd without workspace", SSM_ERR_HIP, [&] {
            return ssm_gated_norm_bwd(out, x, sx, z, sz, w, b, 1e-5f, flags, dx, dz, dw, db, rows, width, groups, it, ot, nullptr);
          });
          rejected("gated_norm_bwd dz without z", SSM_ERR_UNSUPPORTED, [&] {
            return ssm_gated_norm_bwd(out, x, sx, nullptr, 0, w, b, 1e-5f, flags, dx, dz, dw, db, rows, width, groups, it, ot, nullptr);
          });
          rejected("gated_norm_bwd missing dz", SSM_ERR_NULL_ARG, [&] {
            return ssm_gated_norm_bwd(out, x, sx, z, sz, w, b, 1e-5f, flags, dx, nullptr, dw, db, rows, width, groups, it, ot, nullptr);
          });
        }
      }
}

void linattn(int64_t B, int64_t L, int64_t H, int64_t G, int64_t K, int64_t V) {
  for (ssm_dtype ot : kTypes)
    for (int flags : {0, SSM_LINATTN_FIXED_DECAY}) {
      const int64_t T = B * L, row = 2 * G * K + H * V + 8;
      // q, k and v packed in one tensor of rows
      uint16_t* qkv = static_cast<uint16_t*>(buf(T > 0 ? (T - 1) * row + 2 * G * K + H * V : 0, 2));
      const void *q = qkv, *k = qkv ? qkv + G * K : nullptr, *v = qkv ? qkv + 2 * G * K : nullptr;
      float* g = fbuf(flags ? H : T * H);
      float *st = fbuf(B * H * K * V), *st2 = fbuf(B * H * K * V), *st3 = fbuf(B * H * K * V);
      void* out = buf(T * H * V, es(ot));
      auto fwd = [&](const float* first, float* last, const ssm_plan* p) {
        return ssm_linattn_fwd(q, row, k, row, v, row, g, flags, 0.5f, first, out, last, B, L, H, G, K, V, SSM_BF16, ot, nullptr, p);
      };
      expect("linattn", fwd(st, st2, nullptr), SSM_OK);
      expect("linattn in place", fwd(st, st, nullptr), SSM_OK);
      expect("linattn stateless", fwd(nullptr, nullptr, nullptr), SSM_OK);
      ssm_plan p{};
      for (int64_t c : {32, 64, 96}) {
        p.chunk_len = c;
        offered("linattn plan", [&] { return fwd(st, st, &p); });
        expect("linattn plan", fwd(nullptr, st2, &p), SSM_OK);
      }
      if (L > 32 && B > 0) {
        p.chunk_len = 32;
        fake_fail_next_alloc();
        rejected("linattn without workspace", SSM_ERR_HIP, [&] { return fwd(st, st2, &p); });
        p.chunk_len = 33;
        rejected("linattn plan 33", SSM_ERR_UNSUPPORTED, [&] { return fwd(st, st2, &p); });
        p.chunk_len = 0;
        rejected("linattn plan 0", SSM_ERR_UNSUPPORTED, [&] { return fwd(st, st2, &p); });
      }
      void *dout = buf(T * H * V, 2), *dq = buf(T * G * K, es(ot)), *dk = buf(T * G * K, es(ot)), *dv = buf(T * H * V, es(ot));
      float* dg = fbuf(flags ? H : T * H);
      auto bwd = [&](const float* first, const float* dlast, float* dfirst) {
        return ssm_linattn_bwd(q, row, k, row, v, row, g, flags, 0.5f, first, dout, dlast, dq, dk, dv, dg, dfirst, B, L, H, G, K, V,
                               SSM_BF16, ot, nullptr);
      };
      offered("linattn_bwd", [&] { return bwd(st, st2, st3); });
      expect("linattn_bwd bare", bwd(nullptr, nullptr, nullptr), SSM_OK);
      expect("linattn_bwd dlast", bwd(nullptr, st2, nullptr), SSM_OK);
      expect("linattn_bwd initial", bwd(st, nullptr, st3), SSM_OK);
      if (T > 0) {
        fake_fail_next_alloc();
        rejected("linattn_bwd without workspace", SSM_ERR_HIP, [&] { return bwd(st, st2, st3); });
        rejected("linattn_bwd dinitial on dlast", SSM_ERR_UNSUPPORTED, [&] { return bwd(st, st2, st2); });
      }
    }
}

void linattn_step(int64_t B, int64_t H, int64_t G, int64_t K, int64_t V) {
  for (ssm_dtype it : kTypes)
    for (ssm_dtype ot : kTypes)
      for (int flags : {0, SSM_LINATTN_FIXED_DECAY}) {
        float *st = fbuf(B * H * K * V), *st2 = fbuf(B * H * K * V), *g = fbuf(flags ? H : B * H);
        void *q = buf(B * G * K, es(it)), *k = buf(B * G * K, es(it)), *v = buf(B * H * V, es(it)), *out = buf(B * H * V, es(ot));
        for (float* to : {st, st2})
          expect("linattn step", ssm_linattn_state_update(st, to, q, k, v, g, flags, 1, out, B, H, G, K, V, it, ot, nullptr), SSM_OK);
      }
}

void q4(int64_t m, int64_t n, int64_t k, int64_t group) {
  for (ssm_dtype it : kTypes)
    for (ssm_dtype st : kTypes)
      for (ssm_dtype ot : kTypes) {
        const int64_t row = k + 8, g = n * (k / group);
        void *x = buf(m > 0 && k > 0 ? (m - 1) * row + k : 0, es(it)), *out = buf(m * n, es(ot)), *sc = buf(g, es(st)), *w = buf(n * k, es(it));
        uint8_t *codes = cbuf(n * k / 2), *zeros = cbuf(g);
        float* bias = fbuf(n);
        auto call = [&](const uint8_t* z, const float* b) {
          return ssm_q4_matvec(x, row, codes, sc, z, b, out, m, n, k, group, it, st, ot, nullptr);
        };
        offered("q4", [&] { return call(zeros, bias); });
        expect("q4 bare", call(nullptr, nullptr), SSM_OK);
        expect("q4 quantize", ssm_q4_quantize(w, codes, sc, zeros, n, k, group, it, st, nullptr), SSM_OK);
        if (m > 16 && n > 0 && k > 0) {
          fake_fail_next_alloc();
          rejected("q4 without workspace", SSM_ERR_HIP, [&] { return call(zeros, bias); });
          rejected("q4 short rows", SSM_ERR_UNSUPPORTED, [&] {
            return ssm_q4_matvec(x, k - 8, codes, sc, zeros, bias, out, m, n, k, group, it, st, ot, nullptr);
          });
        }
      }
}
}  // namespace

int main() {
  for (int64_t rows : {0, 1, 5, 40})
    for (int64_t width : {0, 1, 7, 64, 513}) add_norm(rows, width);
  for (int64_t rows : {0, 1, 9}) {
    gated_norm(rows, 0, 1);
    for (int64_t g : {1, 2, 6}) gated_norm(rows, 12 * g, g);
  }
  for (int64_t L : {0, 1, 31, 64, 129, 4500}) {
    linattn(1, L, 1, 1, 8, 8);
    linattn(2, L, 4, 2, 72, 16);
    linattn(1, L, 3, 3, 16, 128);
  }
  linattn(0, 5, 2, 1, 64, 64);
  for (int64_t B : {0, 1, 3}) {
    linattn_step(B, 1, 1, 4, 1);
    linattn_step(B, 6, 2, 256, 5);
  }
  for (int64_t m : {0, 1, 5, 17, 70})
    for (int64_t n : {0, 1, 33})
      for (int64_t k : {0, 128, 640})
        for (int64_t group : {32, 64, 128}) q4(m, n, k, group);
  for (void* p : g_bufs) std::free(p);
  if (fake_live_allocs() != 0) {
    std::fprintf(stderr, "%ld workspaces were not freed\n", fake_live_allocs());
    ++g_failures;
  }
  if (g_failures) return 1;
  std::printf("block driver ok: %ld launches\n", launches());
  return 0;
}
