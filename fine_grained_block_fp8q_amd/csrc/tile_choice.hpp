// Choice between the kernels of one product by an estimate of their times.
#pragma once

#include <stdint.h>

namespace fp8q {

// A tiled kernel's costs in ns: for each 128 k with under half of the CUs at
// work, with one workgroup on each CU and with two on each (they overlap where
// two fit, else they follow each other), and for a tile's end.
struct TileVariant {
  int tile;    // what the launch is told
  int bm, bn;  // rows of activations and of weights
  double idle, one, two, end;
};

// The variant that takes least for M x weight_rows x 128 chunks, or 0 where the
// kernel for few rows does: that one reads (16 + rows) * 128 bytes a chunk for
// 16 weight rows, at 80 bytes a ns and CU, and a workgroup of it holds up to
// 128 rows.  Besides, what one workgroup waits for before its first product and
// after its last: 0.5 us where few rows are served, 1.8 for a tile's ring to
// fill, and about 4 us (2 at 64 rows, where two share a CU) for each further
// round of few-row workgroups.
// Estimate and measurement of int8 products, us (3.5 of it the launch):
//   120 x 897 x 592     few rows 5.2 / 5.4    64-row tiles 8.1 / 7.2
//   911 x 1333 x 176    few rows 13.4 / 12.7  64-row tiles 7.4 / 6.6
//   74 x 1393 x 4736    few rows 12.5 / 10.7  64-row tiles 16.8 / 16.5
//   1679 x 5586 x 656   64-row tiles 21.7 / 25.5  128-row tiles 20.2 / 25.3
template <int N>
inline int pick_variant(const TileVariant (&variants)[N], int64_t M, int64_t weight_rows,
                        int64_t chunks, int cus) {
  auto blocks = [](int64_t x, int64_t b) { return (x + b - 1) / b; };
  if (M <= 32) return 0;
  const int64_t few = M <= 64 ? 64 : 128;
  const int64_t rounds = blocks(blocks(M, few) * blocks(weight_rows, 16), cus);
  double least = (double)(rounds * chunks) * (16 + few) * 1.6 + 500.0 +
                 (double)(rounds - 1) * (few == 64 ? 2000.0 : 4000.0);
  int best = 0;
  for (const TileVariant& v : variants) {
    const int64_t n = blocks(M, v.bm) * blocks(weight_rows, v.bn);
    const int64_t pairs = n / (2 * cus), rest = n % (2 * cus);
    const double last = rest == 0 ? 0 : rest > cus ? v.two : 2 * rest > cus ? v.one : v.idle;
    const double t = 1800.0 + (double)chunks * ((double)pairs * v.two + last) +
                     (double)(2 * pairs + (rest > cus ? 2 : rest > 0 ? 1 : 0)) * v.end;
    if (t < least) {
      least = t;
      best = v.tile;
    }
  }
  return best;
}

}  // namespace fp8q
