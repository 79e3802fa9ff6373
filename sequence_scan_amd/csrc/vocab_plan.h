// How the losses over a vocabulary are cut: tiles, pieces of the vocabulary, slices of
// the contracted dimensions, and the parts of the workspace.  Host code only.
#ifndef SSMSCAN_VOCAB_PLAN_H
#define SSMSCAN_VOCAB_PLAN_H

#include <algorithm>
#include <cstdint>

#include "model.h"

namespace ssm {
namespace vocab {

constexpr int kK = 64;              // contracted elements in a stage
constexpr int kLargeTile = 256, kSmallTile = 128;      // rows and columns of a workgroup's tile
constexpr int kFewRows = 16;        // rows that are one matrix operand
constexpr int kFewWidth = 4096;     // ... whose x fits LDS
constexpr int kRowGradBytes = 16;
constexpr int kMostTops = 1024;     // teacher's logits of a row

inline int64_t tiles(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }
inline int64_t padded(int64_t n) { return (n + kK - 1) / kK * kK; }

// What a product's tiles take, in units of about 10 ns: rounds of `cus` workgroups, of
// `start` and `stage` for each kK contracted elements.  With these the shapes are chosen
// (us, forward, Large / Small tiles): 249 x 2384 x 550 55.5 / 28.3, 600 x 1168 x 5059 35.7 /
// 21.1, 64 x 2560 x 50280 69.8 / 59.6, 333 x 768 x 32003 32.6 / 41.6, 1747 x 2824 x 20240 239 /
// 304, 2039 x 1536 x 50280 309 / 468.
struct Times {
  int64_t stage, start;
};
constexpr Times kLargeTimes{140, 500}, kSmallTimes{65, 250};
inline int64_t item(const Times& t, int64_t k) { return t.start + t.stage * (padded(k) / kK); }

inline bool large_tiles(int64_t rows, int64_t columns, int64_t k, int64_t cus) {
  const int64_t l = tiles(tiles(rows, kLargeTile) * tiles(columns, kLargeTile), cus) * item(kLargeTimes, k);
  const int64_t s = tiles(tiles(rows, kSmallTile) * tiles(columns, kSmallTile), cus) * item(kSmallTimes, k);
  return l <= s;
}

// Time that n1 items of k1 and then n2 of k2 take, on `cus` CUs that take the next when free.
inline int64_t makespan(int64_t n1, int64_t k1, int64_t n2, int64_t k2, int64_t cus) {
  const int64_t full = n1 / cus, rest = n1 % cus;
  const int64_t early = full * k1, late = early + (rest ? k1 : 0);       // when CUs turn to the second kind
  if (n2 == 0) return late;
  int64_t end = early + std::max<int64_t>(1, n2 / cus) * k2;      // (no earlier: ends of items of the CUs that turned early)
  for (;; end += k2) {
    const int64_t done = (cus - rest) * ((end - early) / k2) + (end > late ? rest * ((end - late) / k2) : 0);
    if (done >= n2) return end > late ? end : late;
  }
}

// (The least piece: each piece reads and writes dx's fp32 sums once, and few columns are few
// tiles.  Loss and gradients, ms, of pieces of 1024 / 4096 / 8192 / 16384 columns: 32768 x 1024 x
// 50280 - / 15.9 / 13.0 / 12.9, 65536 x 2560 x 20000 - / 22.8 / 22.5 / 22.6; gradients of 65536 x
// 1024 x 30000 25.4 / 16.1.  Below 32768 rows kVocabPieceBytes decides: half of it 2.26 in
// place of 2.28 at 4096 x 1536 x 50280, but 7.21 for 7.00 at 8192 x 2560, 7.80 for 6.41 at 16384 x
// 1024; four times 7.04, 6.40.)
// The backward's cut: columns of a piece of the vocabulary, slices of the contracted
// dimensions of dx (the piece's columns) and dweight (the rows), and the tiles.
struct Cut {
  int64_t piece;
  int pieces, x_slices, w_slices;
  bool large;
};

// Of the pieces whose dz fits kVocabPieceBytes, and the slices, those for which the tiles
// of dz and of the products take least.  A piece or a slice more costs its fp32 sums once
// written and read, about 8 bytes an element at 5 TB/s.  (8192 x 2560 x 50280: pieces of 64 tiles
// and a rest of 5, whose tiles go round the CUs without a gap, 7300 us in place of 7360 in
// four equal ones.  Rows in slices: the gradients of 6135 x 304 x 1341 157 -> 67 us; columns
// in up to 64: 20 x 1272 x 55589 196 -> 112.)
inline Cut choose_cut(const VocabArgs& a) {
  const int64_t cus = std::max(1, a.cus), tv = tiles(a.vocab, kVocabTile);
  const int64_t most = std::min(
      tv, std::max(kVocabPieceLeast, std::min(kVocabMaxLd, kVocabPieceBytes / 2 / std::max(1, a.rows))) / kVocabTile);
  const bool one = most == tv;
  Cut best{};
  int64_t least = INT64_MAX;
  const int64_t step = std::max<int64_t>(1, most / 16);
  for (int64_t tn = most; tn == most || (!one && tn > most / 2); tn -= step) {
    const int64_t columns = std::min<int64_t>(tn * kVocabTile, a.vocab), whole = a.vocab / columns, rest = a.vocab % columns;
    for (int large = 1; large >= (one ? 0 : 1); --large) {
      const int64_t tile = large ? kLargeTile : kSmallTile;
      const Times& t = large ? kLargeTimes : kSmallTimes;
      const int64_t tm = tiles(a.rows, tile), td = tiles(a.width, tile);
      for (int64_t xs = 1; xs <= (one ? 64 : 8); xs *= 2) {
        if (xs > 1 && (!a.dx || columns / xs < 512)) break;
        for (int64_t ws = 1; ws <= (one ? 16 : 1); ws *= 2) {
          if (ws > 1 && (!a.dw || a.rows / ws < 256)) break;
          auto cost_of = [&](int64_t c) {
            const int64_t nx = a.dx ? tm * td * xs : 0, nw = a.dw ? tiles(c, tile) * td * ws : 0;
            const int64_t kx = item(t, (c + xs - 1) / xs), kw = item(t, (a.rows + ws - 1) / ws);
            const int64_t z = tiles(tiles(a.rows, kLargeTile) * tiles(c, kLargeTile), cus) * item(kLargeTimes, a.width);
            return (kx >= kw ? makespan(nx, kx, nw, kw, cus) : makespan(nw, kw, nx, kx, cus)) + (one ? 0 : z);
          };
          const int64_t parts = (whole + (rest != 0)) * xs;
          const int64_t cost = whole * cost_of(columns) + (rest ? cost_of(rest) : 0) +
                               (parts > 1 ? 400 + parts * a.rows * a.width / 6250 : 0) +
                               (ws > 1 ? 400 + ws * (int64_t)a.vocab * a.width / 6250 : 0);
          if (cost < least) {
            least = cost;
            best = Cut{columns, (int)(whole + (rest != 0)), (int)xs, (int)ws, large != 0};
          }
        }
      }
    }
  }
  return best;
}

// Consecutive parts of the workspace.
struct Parts {
  int64_t bytes = 0;
  int64_t add(int64_t n) {
    const int64_t at = bytes;
    bytes += (n + 255) / 256 * 256;
    return at;
  }
};

// Few rows' weights are streamed, each wavefront of the device an equal share of them (as
// many as x in LDS leaves room for).
struct Few {
  bool few;
  int64_t share, groups;
  Few(const VocabArgs& a, int64_t columns) {
    few = a.rows <= kFewRows && a.width <= kFewWidth;
    const int64_t waves = (int64_t)std::max(1, a.cus) * 8 * (a.width <= kFewWidth / 2 ? 2 : 1);
    share = (columns + waves - 1) / waves;
    groups = (columns + share * 8 - 1) / (share * 8);
  }
};

struct FwdParts : Parts {
  Few few;
  bool large, sorted;
  int64_t pieces, stats, picked, keys, starts;
  explicit FwdParts(const VocabArgs& a) : few(a, a.vocab) {
    large = large_tiles(a.rows, a.vocab, a.width, std::max(1, a.cus));
    pieces = few.few ? few.groups * 8 : tiles(a.vocab, large ? kLargeTile : kSmallTile);
    stats = add(pieces * a.rows * 8);
    picked = add(a.teacher ? 0 : (int64_t)a.rows * 4);
    // Every tile reads its rows' indices, or they are put in order once and a tile finds its
    // own (us, forward, read by all / in order): 100 x 512 x 5000 with 1024 logits a row (34 MB of
    // reads) 96 / 109, 500 x 768 x 32000 with 100 (50 MB) 42 / 49, 4096 x 1536 x 50280 with 65
    // (420 MB) 586 / 567, with 128 713 / 572, with 1024 2489 / 771.
    sorted = a.teacher && !few.few && pieces * a.rows * a.top * 8 > (int64_t{1} << 27);
    keys = add(sorted ? (int64_t)a.rows * a.top * 8 : 0);
    starts = add(sorted ? a.rows * (pieces + 1) * 2 : 0);
  }
};

struct BwdParts : Parts {
  Cut cut;
  int64_t rows, hard, x, dz, x_sums, w_sums;
  int64_t ldz;
  explicit BwdParts(const VocabArgs& a) : cut(choose_cut(a)) {
    ldz = padded(cut.piece);
    rows = add((int64_t)a.rows * kRowGradBytes);
    hard = add(a.teacher ? (int64_t)a.rows * a.top * 4 : 0);
    x = add(a.dw ? (int64_t)a.rows * a.width * 2 : 0);
    dz = add(a.rows * ldz * 2);
    x_sums = add(a.dx && (cut.pieces > 1 || cut.x_slices > 1) ? cut.x_slices * (int64_t)a.rows * a.width * 4 : 0);
    w_sums = add(a.dw && cut.w_slices > 1 ? cut.w_slices * cut.piece * a.width * 4 : 0);
  }
};

// One piece of the vocabulary: its columns, and its products' slices.
struct Piece {
  int64_t v0;
  int columns, x_slice, x_slices, w_slice, w_slices;
  Piece(const VocabArgs& a, const Cut& cut, int64_t from) : v0(from) {
    columns = (int)std::min<int64_t>(cut.piece, a.vocab - v0);
    x_slice = (int)padded((columns + cut.x_slices - 1) / cut.x_slices);
    w_slice = (int)padded((a.rows + cut.w_slices - 1) / cut.w_slices);
    x_slices = (columns + x_slice - 1) / x_slice;
    w_slices = (a.rows + w_slice - 1) / w_slice;
  }
};

}  // namespace vocab

inline int64_t vocab_fwd_bytes(const VocabArgs& a) { return vocab::FwdParts(a).bytes; }
inline int64_t vocab_bwd_bytes(const VocabArgs& a) { return vocab::BwdParts(a).bytes; }

}  // namespace ssm

#endif  // SSMSCAN_VOCAB_PLAN_H
