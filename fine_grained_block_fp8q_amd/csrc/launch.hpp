// Size of one launch.
#pragma once

#include <stdint.h>

namespace fp8q {

// Workgroups that one launch takes along x.  The runtime keeps a dimension's
// lanes in 32 bits: of a launch with more it runs their number modulo 2^32 and
// reports success.  Calls of more work than this go out in several launches, or
// are refused.
constexpr int64_t max_blocks(int threads) { return 0xFFFFFFFFll / threads; }

}  // namespace fp8q
