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
// and 18%.  From 17 to 32 rows, outside the fit (60 shapes of each, weight rows
// to 65536): 0.3% and 11%, 0.1% and 2%; the kernel for few rows alone would cost
// 5% and 94%, 6% and 88% (32 x 32768 x 512: 10.4 us, 6.8 in tiles).
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

// int8 products (i8_tiles.hip): kernel times with 4096 weight rows, K = 7168, in
// us, by number of rows:
//   rows          64    128   256   384   512   768   1024  2048  4096
//   few rows      10.2  15.7  29
//   32 x 64       14.2  14.3  18.3  31
//   64 x 64       17.0  17.1  17.5  21.6  21.5  39    43
//   128 x 128     23.6  24.7  24.7  24.9  25.2  26.1  28.6  52    108
//   256 x 128                             38          41    50    102
//   256 x 256           68    68    68    69    69    69    70    86-90
// (64 x 128 tiles take 18.6 to 20.5 us up to 512 rows: with them beside the four
// kept, 0.3% less time over 160 random shapes.)  The two smallest have rings of
// three chunks of A and four of W and share a CU.
constexpr TileVariant kI8Variants[] = {
    {tile_id(32, 64), 32, 64, 2750, 179, 185, 255, 620, 1.15},
    {tile_id(64, 64), 64, 64, 2510, 228, 251, 306, 1250, 1.19},
    {tile_id(128, 128), 128, 128, 3000, 321, 398, 844, 2130, 1.18},
    {tile_id(256, 128), 256, 128, 1850, 551, 739, 1435, 6200, 1.19},
    {tile_id(256, 256), 256, 256, 5210, 972, 1147, 2418, 8110, 1.07}};
constexpr FewRowsCost kI8Few = {2350, 1.12, 1.65, 10.4, 1.07};

// Rows, weight rows and K of an int8 product to its kernel.
inline int pick_i8(int64_t M, int64_t weight_rows, int64_t K, int cus) {
  return pick_variant(kI8Variants, kI8Few, M, weight_rows, K, 256, cus);
}

// The gated block on E4M3 operands (gated_gemm.hip): kernel times with F = 2048
// (4096 weight rows), K = 7168, in us, by number of rows:
//   rows          1     32    64    128   256   512   1024  2048  4096
//   few rows      7.2   7.8   10.8  16.7  32
//   64 x 128                  24.2  24.2  24.5  26    40    79    157
//   128 x 128                       31    31    31    35    68
//   256 x 128                             48    48    49    56    112
//   256 x 256                       58    79    79    79    80    100
constexpr TileVariant kGatedVariants[] = {
    {tile_id(64, 128), 64, 128, 3340, 350, 390, 601, 1260, 1.0},
    {tile_id(128, 128), 128, 128, 950, 441, 530, 982, 3900, 1.0},
    {tile_id(256, 128), 256, 128, 0, 713, 814, 1587, 6000, 1.0},
    {tile_id(256, 256), 256, 256, 0, 1277, 1454, 2903, 7800, 1.0}};
constexpr FewRowsCost kGatedFew = {1970, 1.26, 1.59, 14.3, 1.0};

// Rows, 2F weight rows and K of a gated block on E4M3 operands to its kernel.
inline int pick_gated(int64_t M, int64_t weight_rows, int64_t K, int cus) {
  return pick_variant(kGatedVariants, kGatedFew, M, weight_rows, K, 128, cus);
}

}  // namespace fp8q
