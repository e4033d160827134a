// Tokens grouped by expert, in groups of 128 that never straddle experts.
//
// Expert e's n_e = off[e+1] - off[e] rows take ceil(n_e / 128) groups, the
// experts' groups follow each other: the columns of a transposed operand, of
// which only an expert's last group has some past its last row.
#pragma once

#include "fp8q_device.hpp"

namespace fp8q {

// Most groups of M rows in G experts (off is on the device, so the host can only
// bound them): min(G, M) experts with rows, each 127 short of a group at most.
__host__ __device__ inline int64_t expert_groups_most(int64_t M, int64_t G) {
  return (M + 127 * (G < M ? G : M)) / 128;
}

struct ExpertSpan {
  int status;   // -1: off is invalid; 0: not there (past the last group); 1: found
  int first;    // found: the group's (or the expert's) first row
  int rows;     // found: rows of the group (1 .. 128), or of the expert
  int group0;   // found by expert: its first group
};

__device__ __forceinline__ int groups_of(int rows) { return (rows + 127) >> 7; }

// Every wave that calls (all its lanes do) comes to the same answer by itself:
// lane l covers PL consecutive experts, a wave scan does the rest.
//   BY_GROUP: the rows of group `want`;  else: expert `want`'s groups.
// off is valid if 0 = off[0] <= ... <= off[G] <= M and the groups are at most
// `most`.
template <bool BY_GROUP>
__device__ __forceinline__ ExpertSpan expert_span(const int32_t* off, int G, int64_t M,
                                                  int64_t most, int want) {
  const int lane = threadIdx.x & 63;
  const int PL = (G + 63) >> 6;  // uniform
  const int e0 = lane * PL;
  constexpr int UP = 4;  // experts whose offsets are loaded together
  int o0[UP + 1];
  auto load = [&](int i, int (&o)[UP + 1]) {
#pragma unroll
    for (int u = 0; u <= UP; ++u) {
      const int at = e0 + i + u;
      o[u] = off[at < G ? at : G];
    }
  };
  load(0, o0);
  // f(expert, its first row, its rows) of the lane's experts, until it says so
  auto each = [&](auto f) {
    for (int i = 0; i < PL; i += UP) {
      int o[UP + 1];
      if (i == 0) {
#pragma unroll
        for (int u = 0; u <= UP; ++u) o[u] = o0[u];
      } else {
        load(i, o);
      }
#pragma unroll
      for (int u = 0; u < UP; ++u)
        if (i + u < PL && e0 + i + u < G && f(e0 + i + u, o[u], o[u + 1] - o[u])) return;
    }
  };
  int sum = 0;
  bool bad = lane == 0 && (off[0] != 0 || (int64_t)off[G] > M);
  each([&](int, int lo, int n) {
    bad = bad || n < 0 || lo < 0;
    sum += groups_of(n);
    return false;
  });
  ExpertSpan r = {-1, 0, 0, 0};
  if (__ballot(bad) != 0) return r;
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(inc, d);
    if (lane >= d) inc += v;
  }
  if ((int64_t)__builtin_amdgcn_readlane(inc, 63) > most) return r;
  int at = inc - sum, first = 0, rows = 0, group0 = 0;
  const bool mine = BY_GROUP ? want >= at && want < inc : want >= e0 && want < e0 + PL;
  if (mine)
    each([&](int e, int lo, int n) {
      const int g = groups_of(n);
      if (BY_GROUP ? want < at + g : want == e) {
        const int skip = BY_GROUP ? (want - at) * 128 : 0;
        first = lo + skip;
        rows = BY_GROUP && n - skip > 128 ? 128 : n - skip;
        group0 = at;
        return true;
      }
      at += g;
      return false;
    });
  const uint64_t who = __ballot(mine);
  r.status = 0;
  if (who == 0) return r;
  const int l = __builtin_ctzll(who);
  r.status = 1;
  r.first = __builtin_amdgcn_readlane(first, l);
  r.rows = __builtin_amdgcn_readlane(rows, l);
  r.group0 = __builtin_amdgcn_readlane(group0, l);
  return r;
}

#ifdef FP8Q_DEBUG_CHECKS
// Set by a launch that found invalid offsets (debug builds): read and cleared by
// the host entry points after their synchronization.  (One in each file.)
static __device__ int g_experts_error = 0;

static inline hipError_t take_experts_error(hipStream_t stream, int* flag) {
  const int zero = 0;
  hipError_t e = hipMemcpyFromSymbolAsync(flag, HIP_SYMBOL(g_experts_error), sizeof(int), 0,
                                          hipMemcpyDeviceToHost, stream);
  if (e == hipSuccess) e = hipStreamSynchronize(stream);
  if (e == hipSuccess && *flag)
    e = hipMemcpyToSymbol(HIP_SYMBOL(g_experts_error), &zero, sizeof(int), 0,
                          hipMemcpyHostToDevice);
  return e;
}
#endif

// Whether off is invalid; debug builds note it for the host.
__device__ __forceinline__ bool invalid(const ExpertSpan& s) {
#ifdef FP8Q_DEBUG_CHECKS
  if (s.status < 0 && blockIdx.x == 0 && threadIdx.x == 0) g_experts_error = 1;
#endif
  return s.status < 0;
}

}  // namespace fp8q
