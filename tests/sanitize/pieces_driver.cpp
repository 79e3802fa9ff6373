// The pieces of the vocabulary that the losses' gradients take: for each "rows width vocab
// dx dw" of the arguments, one line "pieces columns slices last_columns last_slices w_slices"
// for 256 CUs.
#include <cstdio>
#include <cstdlib>

#include "../../sequence_scan_amd/csrc/vocab_plan.h"

int main(int argc, char** argv) {
  using namespace ssm;
  for (int i = 1; i + 4 < argc; i += 5) {
    uint16_t some = 0;
    VocabArgs a{};
    a.rows = std::atoi(argv[i]);
    a.width = std::atoi(argv[i + 1]);
    a.vocab = std::atoi(argv[i + 2]);
    a.dx = std::atoi(argv[i + 3]) ? &some : nullptr;
    a.dw = std::atoi(argv[i + 4]) ? &some : nullptr;
    a.top = 1;
    a.cus = 256;
    const vocab::Cut cut = vocab::choose_cut(a);
    const vocab::Piece last(a, cut, (cut.pieces - 1) * cut.piece);
    std::printf("%d %lld %d %d %d %d\n", cut.pieces, (long long)cut.piece, cut.x_slices, last.columns, last.x_slices, cut.w_slices);
  }
  return 0;
}
