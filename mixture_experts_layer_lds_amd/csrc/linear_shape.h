// Which kernel a linear layer's call takes: a rule on its sizes alone, in plain
// C++, so that a test compiles and asks it by itself.
#pragma once

#include <algorithm>
#include <cmath>

namespace moe {

// What a call's rule knows: T * k rows of E experts, or plain rows with one matrix.
struct LinearSizes {
  int rows, E;
  bool grouped;
  int N, K;
  bool gated;   // forward: SwiGLU
};

constexpr long blocks(long n, long size) { return (n + size - 1) / size; }

// Experts that have rows at most, and the rows of one were they spread evenly.
inline int used_groups(const LinearSizes& a) { return !a.grouped ? 1 : a.rows < a.E ? a.rows : a.E; }
inline int mean_rows(const LinearSizes& a) { return a.grouped ? (int)blocks(a.rows, a.E) : a.rows; }

// The tiles' shapes (LinearShape), and how long one takes for `groups` products of
// m x c over q: the rounds of its items over the chip, times an item's stages and
// what it has besides.  Measured, us a stage with every CU at work and us an item besides:
//                               stage of          stage   besides
//   Tile256  256 x 256          64 q              1.75    3.5
//   Tile128  128 x 128, two a CU  64 q              1.08    2.5
//   Pair64   64 x 64, two a CU    2 x 64 q          1.4     3
//   Quad64   64 x 64            4 x 64 q          2.0     2.3
//   Tile288  288 x 256          64 q              1.97    3.5
// A tile of few rows takes 0.4 of a full one and more by its rows.  Rows of experts
// spread: m is their mean, its root the deviation, and the tiles are the expected
// number.  Tile288 is for them (products with rows on m): of experts with 256 rows,
// or a multiple, on average half would need a tile more of 256.  us by the rule without
// it and with it: 32 experts of 256 rows on average, 4096 -> 7168 gradient of the rows 701
// and 556, 2048 -> 7168 forward 300-315 and 292; 8 of 1024, 4096 x 14336 forward 850 and 742,
// 28672 x 4096 gradient of the rows 2180 and 1660, but its forward 1480 and 1490.
// The large tiles do most work a round, the small ones fill the chip where the
// product is small.  us by shape in that order, the rule's choice by *:
//   forward     8192 x 4096 x 2048 (rows, N, K)     105*  125   -     -
//               2048 x 2048 x 1024                  29    15.6* 22.7  35.9
//               4096 x 512 x 1024                   26.9  13.7  13.6* 19.0
//               256 x 4096 x 7168                   131   81    44    37*
//   gradient of the matrices, 8192 x 1024 x 512     207   116   56    47*
struct ShapeCost {
  int BM, BC, q, occupancy;
  double stage, besides;
  double of(long groups, long m, bool spread, long c, long q_len, int cus) const {
    double tiles = (double)blocks(m, BM);
    if (spread) {
      const double deviation = std::sqrt((double)m);
      tiles = 1.0;
      for (long at = BM; at < m + 4 * deviation; at += BM) tiles += 0.5 * std::erfc((at - m) / (deviation * 1.41421356));
    }
    const double fill = std::min(1.0, m / (tiles * BM));
    const double rounds = std::ceil(std::round(groups * tiles) * blocks(c, BC) / ((double)cus * occupancy));
    return rounds * (blocks(q_len, q) * stage * (0.4 + 0.6 * fill) + besides);
  }
};
constexpr ShapeCost kShapeCosts[] = {
    {256, 256, 64, 1, 1.75, 3.5}, {128, 128, 64, 2, 1.08, 2.5}, {64, 64, 128, 2, 1.4, 3.0}, {64, 64, 256, 1, 2.0, 2.3},
    {288, 256, 64, 1, 1.97, 3.5}};
enum LinearTile { kTile256, kTile128, kPair64, kQuad64, kTile288 };

// The shape that takes least; `rows_on_m`: m are rows.
inline LinearTile least_tile(bool rows_on_m, long groups, long m, bool spread, long c, long q, int cus) {
  int best = 0;
  double least = kShapeCosts[0].of(groups, m, spread, c, q, cus);
  for (int i = 1; i < (rows_on_m ? 5 : 4); i++) {
    const double cost = kShapeCosts[i].of(groups, m, spread, c, q, cus);
    if (cost < least) least = cost, best = i;
  }
  return (LinearTile)best;
}

inline LinearTile forward_tile(const LinearSizes& a, int cus) {
  return least_tile(true, used_groups(a), mean_rows(a), a.grouped, a.N, a.K, cus);
}
inline LinearTile grad_x_tile(const LinearSizes& a, int cus) {
  return least_tile(true, used_groups(a), mean_rows(a), a.grouped, a.K, a.N, cus);
}
inline LinearTile grad_w_tile(const LinearSizes& a, int cus) {
  return least_tile(false, a.E, a.N, false, a.K, mean_rows(a), cus);
}

// Few rows an expert: the weights' stream, on tiles of 16 or 32 rows.  Experts'
// rows spread, and one with a row more than the tile reads its weights again, so
// theirs go to half the rows that plain ones do (us, gate-up and down of the layer,
// on 16, on 32 and on the large tiles: 8 of 32 experts of 7168 x 2048, 64 tokens, 16
// rows an expert 337 + 176, 312 + 175, 309 + 220; 128 tokens - , 470 + 214, 313 + 223;
// 64 skewed experts of 3584 x 640, 128 tokens 110 + 63, 108 + 69, 138 + 58).
// The rule knows the mean alone: an expert with most of the rows reads its weights once
// for every 32 of them here.  us on the stream and on the large tiles, with no, half,
// three quarters and 0.95 of the rows on one expert: 96 experts of 4096 x 7168, 16 rows on
// average 938 and 915, 1066 and 987, 1150 and 980, 886 and 664; 64 of 1280 x 3584, 8 rows
// 101 and 136, 112 and 134, 110 and 132, 47 and 59.
// Of items of 4, 2 or 1 blocks of weight rows those that take least: the rounds over
// the CUs, times the blocks and a third of one for the rows' copies and the waves'
// meeting (2 experts of 28672 x 4096, one row each: 94 us on 4 blocks, 3.5 rounds, 81
// on 2, 7 rounds)
struct StreamItem {
  int nb, mb;   // blocks of 16 weight rows and of 16 rows; nb 0: the large tiles
};
inline StreamItem stream_item(const LinearSizes& a, int cus) {
  const int mean = mean_rows(a), of_one = a.grouped ? 8 : 16;
  if (mean > 2 * of_one) return {0, 0};
  const int mb = mean <= of_one ? 1 : 2, least = mb == 2 || a.gated ? 2 : 1;
  int nb = 2;
  long best = -1;
  for (int n = mb == 2 ? 2 : 4; n >= least; n /= 2) {
    const long cost = blocks(used_groups(a) * blocks(a.N, 16 * n), cus) * (3 * n + 1);
    if (best < 0 || cost < best) best = cost, nb = n;
  }
  return {nb, mb};
}

}  // namespace moe
