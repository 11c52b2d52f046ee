// Which tiles a product of the linear layer's kernels takes.  Host code only.
#pragma once

#include <stdint.h>

namespace arcs {

inline int64_t linear_tiles(int64_t n, int64_t t) { return (n + t - 1) / t; }

// One product of the tile kernels: C[m, n] = sum_k A[m, k] B[n, k], and its tiles.
//   FORWARD  m: V, n: N, k: D    rows of both operands run along k
//   DHIDDEN  m: D, n: N, k: V    rows of A (the weight) run along m
//   DWEIGHT  m: D, n: V, k: N    rows of both run along m and n
enum LinearMode { kLinForward, kLinDhidden, kLinDweight };
struct LinearShape {
  int rows;     // of the tile along n; 0: no tiles (the few-rows kernel)
  int columns;  // of the tile along m
  int workers;  // workgroups that share all tiles evenly, each a part of k of some; 0: whole tiles
};

// What a product costs in tiles of a kind, in microseconds: `start` for the launch and the first
// loads, then for each round of tiles `step` (`alone` where no compute unit has two) for
// each 128 bytes of k and `end` for the results; shared tiles cost their parts' way
// through memory (bytes per microsecond) and `join` for the second launch.  Fitted to the times
// of 47 sizes of the forward product and 42 of each gradient in bfloat16, 13 of each in float32 (17 .. 4,096
// rows, 200 .. 130,000 columns, k of 100 .. 11,008), measured in every kind and sharing: what the
// costs name takes 0.4 % longer in the geometric mean than the best, 24 % at most (of 13 us).  On
// both sides of the choice, for instance, forward: 4,096 x 4,096 x 4,096 125 us in 256 x 256
// and 148 in 128 x 128; 512 x 11,008 x 4,096 63 in 128 x 128, 92 in 256 x 256 shared; 256 x
// 4,096 x 4,096 23 in 64 x 64, 26 in 128 x 128 shared.  (256 x 128, 256 x 64 and 128 x 64 in
// bfloat16, other depths of k and four waves of 128 x 128 each gained less than 1 % somewhere.)
struct TileCost {
  int columns, rows, slots;  // slots: workgroups that the card holds at once
  double alone, step, end, start, join, rate;
};
constexpr TileCost kCostsBf16[] = {
    {256, 256, 256, 1.50, 1.50, 6.6, 2.0, 2.6, 5.6e6},
    {128, 128, 512, 0.69, 1.08, 3.1, 2.0, 6.2, 6.1e6},
    {64, 64, 512, 0.29, 0.52, 1.8, 2.0, 4.2, 3.2e6},
    {128, 32, 512, 0.34, 0.61, 1.8, 2.0, 5.0, 3.5e6},  // not in DWEIGHT
};
constexpr TileCost kCostsF32[] = {
    {128, 64, 512, 1.12, 2.03, 1.3, 2.6, 5.3, 4.6e6},
    {64, 64, 512, 0.63, 1.25, 0.8, 3.0, 4.8, 3.9e6},
    {128, 32, 512, 0.77, 1.37, 1.2, 2.5, 5.8, 4.3e6},  // not in DWEIGHT
};

// The tiles of a product: of those built for the mode and type, and of the ways to share them,
// the ones that cost least.
inline LinearShape linear_shape(int mode, int64_t M, int64_t N, int64_t K, bool bf16) {
  const TileCost* costs = bf16 ? kCostsBf16 : kCostsF32;
  const int kinds = (bf16 ? 4 : 3) - (mode == kLinDweight ? 1 : 0);
  const double steps = (double)linear_tiles(K, bf16 ? 64 : 32);
  LinearShape best = {0, 0, 0};
  double least = 0.0;
  for (int i = 0; i < kinds; ++i) {
    const TileCost& c = costs[i];
    if (c.rows > 32 && c.rows > 2 * N && mode != kLinDweight) continue;  // mostly empty
    const double all = (double)linear_tiles(M, c.columns) * (double)linear_tiles(N, c.rows);
    for (int workers = 0; workers <= 512; workers = workers == 0 ? 128 : workers * 2) {
      double cost = c.start;
      if (workers > 0) {
        if (all > 400 || all * steps < workers) continue;
        cost += c.join + c.end + all * steps / workers * (workers <= 256 ? c.alone : c.step) +
                (all + workers) * c.columns * c.rows * 8.0 / c.rate;
      } else if (all <= 256) {
        cost += steps * c.alone + c.end;
      } else {
        const double rounds = all / c.slots;
        cost += (rounds < 4.0 ? __builtin_ceil(rounds) : rounds + 0.5) * (steps * c.step + c.end);
      }
      if (best.rows == 0 || cost < least) {
        least = cost;
        best = {c.rows, c.columns, workers};
      }
    }
  }
  return best;
}

}  // namespace arcs
