// Plans at the ends of their range, through the host layer over the fake runtime and
// launchers, built with AddressSanitizer and UndefinedBehaviorSanitizer: time chunks as long as an int64_t
// goes (one chunk), and planners asked for sequences that long.  The launchers abort on
// a plan that does not cover the sequence.  Prints "plan driver ok".
#include <cstdint>
#include <cstdio>
#include <vector>

#include "../../include/ssmblock.h"

extern "C" long fake_launches(void);
extern "C" long fake_block_launches(void);

namespace {
int g_failures = 0;
void expect(const char* what, bool good) {
  if (good) return;
  std::fprintf(stderr, "%s; last error: %s\n", what, ssm_last_error());
  ++g_failures;
}
}  // namespace

int main() {
  constexpr int64_t kMost = INT64_MAX, L = 40, D = 64;
  std::vector<float> b[12];
  for (auto& v : b) v.assign((size_t)(L * D * 16), 0.0f);
  ssm_plan p{};

  for (int64_t c : {kMost, kMost - 5, kMost / 2}) {
    p = ssm_plan{};
    p.chunk_len = c;
    long before = fake_block_launches();
    expect("linattn", ssm_linattn_fwd(b[0].data(), D, b[1].data(), D, b[2].data(), D, b[3].data(), 0, 1.0f, nullptr, b[4].data(),
                                      b[5].data(), 1, L, 1, 1, D, D, SSM_BF16, SSM_F32, nullptr, &p) == SSM_OK);
    expect("linattn: one walk", fake_block_launches() == before + 1);

    p.states_per_wave = 4;
    before = fake_launches();
    expect("scan", ssm_scan_fwd_plan(b[0].data(), b[1].data(), b[2].data(), b[3].data(), b[4].data(), nullptr, nullptr, nullptr, 0,
                                b[5].data(), b[6].data(), 1, L, D, 16, SSM_F32, SSM_F32, nullptr, &p) == SSM_OK);
    expect("scan: launched", fake_launches() > before);
  }
  // no rows of a sequence as long as can be: planned, and nothing to run
  expect("linattn plan", ssm_linattn_plan_query(0, kMost, 1, D, D, &p) == SSM_OK && p.chunk_len >= 1 && p.n_chunks >= 1 &&
                             p.n_chunks - 1 <= (kMost - 1) / p.chunk_len);
  expect("linattn without rows", ssm_linattn_fwd(b[0].data(), D, b[1].data(), D, b[2].data(), D, b[3].data(), 0, 1.0f, nullptr,
                                                 b[4].data(), nullptr, 0, kMost, 1, 1, D, D, SSM_BF16, SSM_F32, nullptr,
                                                 nullptr) == SSM_OK);
  if (g_failures) return 1;
  std::printf("plan driver ok\n");
  return 0;
}
