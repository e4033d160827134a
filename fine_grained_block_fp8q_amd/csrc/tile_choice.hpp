// Choice between the kernels of one product by an estimate of their times.
#pragma once

#include <stdint.h>

namespace fp8q {

// A tiled kernel's costs in ns, measured at K = 7168: for each 128 k with under
// half of the CUs at work, with one workgroup on each CU and with two on each
// (they overlap where two fit, else they follow each other), and once a tile.
struct TileVariant {
  int tile;    // what the launch is told
  int bm, bn;  // rows of activations and of weights
  double idle, one, two, end;
};

// The variant that takes least for M x weight_rows x 128 chunks, or 0 where the
// kernel for few rows does: that one reads (16 + rows) * 128 bytes a chunk for
// 16 weight rows, at 80 bytes a ns and CU, and each of its workgroups holds up
// to 128 rows.
template <int N>
inline int pick_variant(const TileVariant (&variants)[N], int64_t M, int64_t weight_rows,
                        int64_t chunks, int cus) {
  auto blocks = [](int64_t x, int64_t b) { return (x + b - 1) / b; };
  if (M <= 32) return 0;
  const int64_t few = M <= 64 ? 64 : 128;
  double least = (double)blocks(blocks(M, few) * blocks(weight_rows, 16), cus) * (double)chunks *
                 (16 + few) * 1.6;
  int best = 0;
  for (const TileVariant& v : variants) {
    const int64_t n = blocks(M, v.bm) * blocks(weight_rows, v.bn);
    const int64_t pairs = n / (2 * cus), rest = n % (2 * cus);
    const double last = rest == 0 ? 0 : rest > cus ? v.two : 2 * rest > cus ? v.one : v.idle;
    const double t = (double)chunks * ((double)pairs * v.two + last) +
                     (double)(2 * pairs + (rest > cus ? 2 : rest > 0 ? 1 : 0)) * v.end;
    if (t < least) {
      least = t;
      best = v.tile;
    }
  }
  return best;
}

}  // namespace fp8q
