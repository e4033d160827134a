// Choice between the kernels of one product by an estimate of their times.
#pragma once

#include <stdint.h>

namespace fp8q {

// A tile's rows of activations and of weights, in one number.
constexpr int tile_id(int bm, int bn) { return 1000 * bm + bn; }

// A tiled kernel's times in ns, its launch and the ring's first fill included
// in `start`: for each 128 k with up to half of the CUs at work, with one
// workgroup on each CU and with two (they overlap where two fit, else they
// follow each other), and for a tile's end.  `split` is the factor on the k
// part where K is no multiple of 128: a row's 128 bytes then lie in two lines.
struct TileVariant {
  int tile;    // what the launch is told
  int bm, bn;  // rows of activations and of weights
  double start, idle, one, two, end, split;
};

// The kernel for few rows: a workgroup of it holds 16 weight rows and 32, 64 or
// 128 activation rows and its 8 waves take a chunk each.  In ns, for each of those
// activation rows: a chunk with up to half of the CUs at work and with all, and
// each round of workgroups.
struct FewRowsCost {
  double start, idle, one, round, split;
};

// The variant that takes least for M x weight_rows x K, or 0 where the kernel
// for few rows does; the tiles take K in steps of `step`.  The constants are
// fitted to measured times of every kernel at random shapes (M 33 to 5800,
// weight rows 64 to 8192, K 128 to 9000).  Against the best kernel of each
// shape the choice costs 0.6% on average and 16% at most over 200 int8 shapes,
// 0.2% and 15% over 138 E4M3 ones; over 40 of both that were not fitted, 1.6%
// and 18%.  (With 17 to 32 rows it matters where weight rows make several rounds
// of few-row workgroups: 32 x 32768 x 512 takes 10.4 us in those, 6.8 in tiles.)
template <int N>
inline int pick_variant(const TileVariant (&variants)[N], const FewRowsCost& few, int64_t M,
                        int64_t weight_rows, int64_t K, int step, int cus) {
  auto blocks = [](int64_t x, int64_t b) { return (x + b - 1) / b; };
  if (M <= 16) return 0;
  const bool whole = K % 128 == 0;
  const int64_t rows = M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const int64_t n_few = blocks(M, rows) * blocks(weight_rows, 16);
  const int64_t rounds = blocks(n_few, cus);
  const bool idle = 2 * (n_few - (rounds - 1) * cus) <= cus;
  const double few_k = (double)(blocks(K, 1024) * 8) * (whole ? 1.0 : few.split);
  double least = few.start + (double)rows * (few_k * ((double)(rounds - 1) * few.one +
                                                      (idle ? few.idle : few.one)) +
                                             (double)rounds * few.round);
  const double chunks = (double)(blocks(K, step) * step) / 128.0;
  int best = 0;
  for (const TileVariant& v : variants) {
    const int64_t n = blocks(M, v.bm) * blocks(weight_rows, v.bn);
    const int64_t pairs = n / (2 * cus), rest = n % (2 * cus);
    const double last = rest == 0 ? 0 : rest > cus ? v.two : 2 * rest > cus ? v.one : v.idle;
    const double t = v.start + chunks * (whole ? 1.0 : v.split) * ((double)pairs * v.two + last) +
                     (double)(2 * pairs + (rest > cus ? 2 : rest > 0 ? 1 : 0)) * v.end;
    if (t < least) {
      least = t;
      best = v.tile;
    }
  }
  return best;
}

}  // namespace fp8q
