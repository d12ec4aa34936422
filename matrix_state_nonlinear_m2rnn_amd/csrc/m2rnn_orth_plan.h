// How the products of the orthogonalised update are cut into tiles: the cost model and its measured figures.  Plain C++.
#pragma once

#include <algorithm>

namespace m2rnn {

constexpr long kOrthPad = 64;  // sides are rounded up to it
constexpr int kOrthK = 32;     // contraction of a stage

inline long ceil_div(long a, long b) { return (a + b - 1) / b; }

// Tiles that a product is cut into: their sides, workgroups that a CU holds, a stage's time (us) where it holds one, two, ...
// of them, and the operations a us that all CUs together reach (the card's power, then); measured over products of 192 to 8192 a
// side.
struct OrthShape {
  int TM, TN, held;
  double stage[4], rate;
};
constexpr OrthShape kShapes[] = {{256, 256, 1, {2.15}, 9.6e8},
                                 {192, 192, 1, {1.35}, 9.6e8},
                                 {128, 128, 2, {0.95, 1.25}, 9.5e8},
                                 {128, 64, 3, {0.5, 0.63, 1.0}, 8.8e8},
                                 {96, 96, 3, {0.6, 0.87, 1.28}, 9.2e8},
                                 {64, 64, 4, {0.4, 0.45, 0.55, 0.85}, 8.4e8},
                                 {64, 64, 2, {0.3, 0.5}, 8.4e8}};  // five stages in LDS
constexpr int kShapeCount = sizeof(kShapes) / sizeof(kShapes[0]);

// How a product runs: its tiles, the parts of its contraction, and the time that this should take (us).
struct Cut {
  int shape = 0, splits = 1, tiles = 1, gi = 1, gj = 1;
  double us = 0.0;
};

// The time of `groups` workgroups of `stages` stages: whole rounds of what the CUs hold, then the fullest CU of the rest.
inline double rounds_us(const OrthShape& h, long groups, long stages) {
  const long load = ceil_div(groups, 256), full = load / h.held, rest = load % h.held;
  return (full * h.stage[h.held - 1] + (rest ? h.stage[rest - 1] : 0.0)) * stages;
}

// How a product of K terms runs; `cut`: its contraction may be cut (X X^T: the longer side.  For the others it is the shorter
// one, and over matrices of 64 to 16384 rows a cut never paid).
inline Cut cut_product(long batch, long rows, long cols, long K, bool sym, bool cut) {
  Cut best;
  const long stages = K / kOrthK;
  for (int i = 0; i < kShapeCount; ++i) {
    const OrthShape& h = kShapes[i];
    const long gi = ceil_div(rows, h.TM), gj = ceil_div(cols, h.TN);
    const long tiles = sym ? gi * (gi + 1) / 2 * (h.TM / h.TN) : gi * gj;
    for (int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (s > stages || (s > 1 && !cut)) break;
      const long groups = tiles * batch * s;
      if (s > 1 && groups > 256L * h.held) break;
      const double work = (double)tiles * batch * h.TM * h.TN * K * 6.0;
      double us = std::max(rounds_us(h, groups, ceil_div(stages, s)), work / h.rate) + 6.0;
      if (s > 1) us += 4.0 + (double)groups * h.TM * h.TN * 8.0 / 4e6;  // the parts written and read, one more launch
      if (best.us == 0.0 || us < best.us) {
        best.shape = i;
        best.splits = s;
        best.tiles = (int)tiles;
        best.gi = (int)gi;
        best.gj = (int)gj;
        best.us = us;
      }
    }
  }
  return best;
}

// The products of a step over matrices of rows x cols: their sides with m the shorter, also rounded up (what a contraction takes), and how
// X X^T, b A + c A A and a X + B X run.
struct OrthCuts {
  long m, n, mp, np;
  Cut gram, poly, next;
  OrthCuts(long batch, long rows, long cols)
      : m(std::min(rows, cols)), n(std::max(rows, cols)), mp(ceil_div(m, kOrthPad) * kOrthPad), np(ceil_div(n, kOrthPad) * kOrthPad),
        gram(cut_product(batch, mp, mp, np, true, true)), poly(cut_product(batch, mp, mp, mp, true, false)),
        next(cut_product(batch, mp, np, mp, false, false)) {}
};

}  // namespace m2rnn
