// Grouped (per-expert) block-scaled FP8 GEMM on the tile of gemm_tile.hpp:
// row-count buckets, persistent schedule from the device offsets.
#pragma once

#include "gemm_tile.hpp"

namespace fp8q {

// Grouped configurations: 256-row tiles cover an expert's tokens (decode
// batches hold at most 256) so each expert's weights stream once, and 256
// weight rows per tile (8 waves of 64 x 128, as in the dense tile) so each
// expert's activation rows are re-read from L2 by N/256 tiles rather than
// N/128 (at 128 weight rows the activation reads outweighed the weight
// stream in large tiles and held the weight stream below the copy rate).
// Only the tile's live rows are staged (64, 128, 160, 192 or 256), and the
// LDS this frees deepens the ring: 3 stages up to 160 rows, 2 above.  A
// 2-stage ring streams the weights markedly slower than a 3-stage one once
// the activation rows share the loads, so 160 rows (most experts of a
// 256-expert top-8 routing of 4096 tokens hold 103..157) get a bucket of
// their own: the largest that still fits 3 stages in 160 KiB.
constexpr int kGroupedBN = 256;
// 160- and 192-row tiles hold experts of 129..192 rows: their waves take 48
// rows each, so for up to 144 rows the fourth row of waves has none and
// skips its MFMAs (64-row waves would run three full waves for 129 rows).
// CAST: 0, or 1 + the scale mode of activations quantized inside the GEMM
// (the same LDS ring: the cast writes the codes where the loads would).
// OP: kOpFp8, or kOpWide16 for the precise mode (no cast).
// GATED: the gated block (kGroupedBN/2 output columns a tile).
template <int ROWS, int S, int CAST = 0, int OP = kOpFp8, int GATED = 0>
using GroupedCfg = GemmCfg<(ROWS == 160 || ROWS == 192 ? 192 : 256), kGroupedBN, 4, 2, S, ROWS, 0,
                           OP, 0, CAST, GATED>;
constexpr int kS64 = 3, kS128 = 3, kS160 = 3, kS192 = 2, kS256 = 2;

// Grouped variant, persistent: one workgroup per CU (the grid grows only if a
// workgroup would otherwise walk more than 64 tiles).  Each workgroup derives
// the whole schedule from the device offsets, in LDS, once: it ranks the
// experts by row count and orders them for a balanced, largest-first
// schedule (snake_position) when the tiles fill few rounds, takes a prefix
// sum of ceil(M_e / 256) in that order, and maps each of its own tiles to
// (expert, m-tile, n-tile), one tile per lane.  It then runs the tiles one
// after the other, each with the instantiation for its live row count.
// Paying the set-up once per CU rather than once per tile (a kernel of one
// workgroup per tile spent about 4 us per workgroup on launch and set-up
// that the single resident workgroup of a CU cannot overlap).

// Position of the expert of rank r (0 = most rows) among G experts dealt to
// the 8 XCD runs in snake order: ranks 0..7 go to runs 0..7, ranks 8..15 to
// runs 7..0, and so on; run b holds its experts in rank order, and the runs
// follow each other.  A bijection on [0, G).
__device__ __forceinline__ int snake_position(int r, int G) {
  const int round = r / kXcds, i = r % kXcds;
  const int bin = (round & 1) ? kXcds - 1 - i : i;
  const int full = G / kXcds, m = G % kXcds;
  const bool last_odd = (full & 1) != 0;  // direction of the partial last round
  int start = bin * full;
  for (int b = 0; b < bin; ++b) start += (m > 0 && (last_odd ? b >= kXcds - m : b < m)) ? 1 : 0;
  return start + round;
}

__host__ __device__ constexpr int cmax(int a, int b) { return a > b ? a : b; }

#ifdef FP8Q_DEBUG_CHECKS
// Set by a grouped launch that found invalid offsets (debug builds): read and
// cleared by the host entry points after their synchronization.
// (One flag in each file that launches the kernel.)
static __device__ int g_offsets_error = 0;

static inline hipError_t take_offsets_error(hipStream_t stream, int* flag) {
  const int zero = 0;
  hipError_t e = hipMemcpyFromSymbolAsync(flag, HIP_SYMBOL(g_offsets_error), sizeof(int), 0,
                                          hipMemcpyDeviceToHost, stream);
  if (e == hipSuccess) e = hipStreamSynchronize(stream);
  if (e == hipSuccess && *flag)
    e = hipMemcpyToSymbol(HIP_SYMBOL(g_offsets_error), &zero, sizeof(int), 0,
                          hipMemcpyHostToDevice);
  return e;
}
#endif
constexpr int kMaxExpertsLds = 1024;
constexpr int kGroupedThreads = 512;
constexpr int kGroupedLds =
    cmax(cmax(GroupedCfg<64, kS64>::LDS_BYTES, GroupedCfg<128, kS128>::LDS_BYTES),
         cmax(cmax(GroupedCfg<160, kS160>::LDS_BYTES, GroupedCfg<192, kS192>::LDS_BYTES),
              GroupedCfg<256, kS256>::LDS_BYTES));
static_assert(GroupedCfg<64, kS64>::THREADS == kGroupedThreads &&
                  GroupedCfg<256, kS256>::THREADS == kGroupedThreads,
              "all grouped configurations use the same workgroup");

// CAST: 0 = FP8 activation codes and scales in A / SA; 1 + scale mode = BF16
// activations in A (SA unused), quantized inside the tiles.  OP: kOpFp8, or
// kOpWide16 (the precise mode, with CAST = 0).
// GATED: W is [G][2F][K] with N = F output columns; gu as in TileArgs.
template <int CAST, int OP = kOpFp8, int GATED = 0>
__global__ __launch_bounds__(kGroupedThreads) void grouped_gemm_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ SA, int64_t M_total,
    const int32_t* __restrict__ off, int G, const uint8_t* __restrict__ W,
    const float* __restrict__ SW, int64_t N, int64_t K, void* __restrict__ C, int out_bf16,
    int tiles_n, int lpt_max_tiles, uint16_t* __restrict__ gu, int act) {
  constexpr int T = kGroupedThreads;
  constexpr int BM = 256;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kGroupedLds];
  static_assert((3 * kMaxExpertsLds + 1) * 4 <= kGroupedLds, "prefix scratch fits in LDS");
  static_assert(kMaxExpertsLds % 64 == 0, "one wave scans the experts");
  int* mt_prefix = reinterpret_cast<int*>(smem);  // [G + 1], reused by the tiles' rings
  int* rows_of = mt_prefix + kMaxExpertsLds + 1;  // [G] rows of expert e
  int* expert_at = rows_of + kMaxExpertsLds;      // [G] expert at tile-order position p
  auto mtiles = [](int rows) { return rows > 0 ? (rows + BM - 1) / BM : 0; };

  // Number of real tiles, computed by every wave on its own from the offsets
  // (a lane sum and a wave reduction, no barrier), so that workgroups without
  // a tile leave before any LDS work.
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  // The same pass validates the offsets (0 = off[0] <= ... <= off[G] <=
  // M_total): every wave of every workgroup reads the same values and comes
  // to the same verdict, and with invalid offsets the whole launch returns
  // here, before any load or store.
  int sum_mt = 0;
  bool bad = lane == 0 && (off[0] != 0 || (int64_t)off[G] > M_total);
  for (int e = lane; e < G; e += 64) {
    const int lo = off[e], hi = off[e + 1];
    bad = bad || hi < lo;
    sum_mt += mtiles(hi - lo);
  }
  if (__ballot(bad) != 0) {
#ifdef FP8Q_DEBUG_CHECKS
    if (blockIdx.x == 0 && tid == 0) g_offsets_error = 1;
#endif
    return;
  }
  for (int d = 32; d >= 1; d >>= 1) sum_mt += __shfl_xor(sum_mt, d);
  // (equal in every lane; readfirstlane keeps everything derived from it scalar)
  const int total = __builtin_amdgcn_readfirstlane(sum_mt) * tiles_n;  // real tiles
  // Persistent schedule.  XCD x (= workgroup id mod 8) takes a contiguous run
  // of the real tiles, [x*q8 + min(x, r8), ...), so the n-tiles of one expert
  // share that expert's rows of A in one L2.  The K8 workgroups of an XCD walk
  // its run in rounds of K8 tiles in snake order (workgroup k takes run
  // position k in even rounds and K8-1-k in odd ones), which pairs the
  // largest tiles of a largest-first order with the smallest.  The host sizes
  // the grid so that no workgroup has more than 64 rounds.
  const int bid = blockIdx.x;
  const int K8 = gridDim.x / kXcds;
  const int x = bid % kXcds, k = bid / kXcds;
  const int q8 = total / kXcds, r8 = total % kXcds;
  const int run0 = x * q8 + (x < r8 ? x : r8);
  const int len = q8 + (x < r8 ? 1 : 0);
  if (k >= len) return;  // no tile for this workgroup

  for (int e = tid; e < G; e += T) rows_of[e] = off[e + 1] - off[e];
  __syncthreads();
  // Tile order.  When the tiles fill only a few rounds of the chip
  // (lpt_max_tiles = 4 per CU), the tail of the last round decides the time:
  // experts ranked by row count (largest first, ties by index) are dealt to
  // the 8 XCD runs in snake order, and each run lists its experts largest
  // first, so every XCD gets a similar share of the rows and its CUs take the
  // largest tiles first.  With many rounds, the expert order is kept: it mixes
  // tiles of different row counts (different MFMA-to-HBM ratios) in time.
  // Either way, each expert's tiles stay in one XCD run and share its L2
  // (exactly so when the runs hold equal tile counts, as with one m-tile per
  // expert).
  const bool lpt = total <= lpt_max_tiles;
  for (int e = tid; e < G; e += T) {
    int p = e;
    if (lpt) {
      const int ce = rows_of[e];
      int r = 0;
      for (int j = 0; j < G; ++j) {
        const int cj = rows_of[j];
        r += (cj > ce || (cj == ce && j < e)) ? 1 : 0;
      }
      p = snake_position(r, G);
    }
    expert_at[p] = e;
  }
  __syncthreads();

  // Prefix over tile-order positions of the number of BM-row tiles, by one
  // wave: lane l covers positions 16l .. 16l+15 (a lane sum, a shuffle scan
  // over the lanes, then the lane's 16 prefix values).
  if (tid < 64) {
    constexpr int PL = kMaxExpertsLds / 64;
    const int p0 = lane * PL;
    int sum = 0;
    for (int i = 0; i < PL; ++i)
      if (p0 + i < G) sum += mtiles(rows_of[expert_at[p0 + i]]);
    int inc = sum;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(inc, d);
      if (lane >= d) inc += v;
    }
    int run = inc - sum;
    if (lane == 0) mt_prefix[0] = 0;
    for (int i = 0; i < PL; ++i)
      if (p0 + i < G) {
        run += mtiles(rows_of[expert_at[p0 + i]]);
        mt_prefix[p0 + i + 1] = run;
      }
  }
  __syncthreads();
  // Lane r of every wave maps this workgroup's round-r tile to (expert,
  // m-tile, n-tile): tile-order position p with prefix[p] <= m-tile index <
  // prefix[p+1].  Real tiles are numbered in tile order, m-tile, then n-tile
  // fastest.
  int my_e = 0, my_mt = 0, my_tn = 0;
  const int j = lane * K8 + ((lane & 1) ? K8 - 1 - k : k);
  const bool has = j < len;
  if (has) {
    const int id = run0 + j;
    const int mt_global = id / tiles_n;
    my_tn = id % tiles_n;
    int lo = 0, hi = G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (mt_prefix[mid] <= mt_global) lo = mid; else hi = mid;
    }
    my_e = expert_at[lo];
    my_mt = mt_global - mt_prefix[lo];
  }
  // Rounds with a tile are a prefix of the lanes (j grows with the lane).
  const int n_mine = __builtin_popcountll(__ballot(has));
  __syncthreads();  // the prefix scratch is overwritten by the tiles' rings

  for (int r = 0; r < n_mine; ++r) {
    const int e = __builtin_amdgcn_readlane(my_e, r);
    const int mt = __builtin_amdgcn_readlane(my_mt, r);
    const int tn = __builtin_amdgcn_readlane(my_tn, r);
    const int64_t r0 = off[e];
    const int64_t r1 = off[e + 1];
    TileArgs t;
    t.A = A;
    t.SA = SA;
    t.W = W + (int64_t)e * (GATED ? 2 : 1) * N * K;
    t.SW = SW + (int64_t)e * (GATED ? 2 : 1) * (N / 128) * (K / 128);
    t.a_row0 = r0 + (int64_t)mt * BM;
    t.a_rows = r1;
    t.w_row0 = (int64_t)tn * (GATED ? kGroupedBN / 2 : kGroupedBN);
    t.w_rows = N;
    t.K = K;
    t.sa_ld = M_total;
    t.sw_ld = N;
    t.C = C;
    t.ldc = N;
    t.out_bf16 = out_bf16;
    t.gu = gu;
    t.act = act;
    const int64_t live = r1 - t.a_row0;  // 1 .. (>= 256 when more m-tiles follow)
    if (live <= 64)
      gemm_tile<GroupedCfg<64, kS64, CAST, OP, GATED>>(t, smem);
    else if (live <= 128)
      gemm_tile<GroupedCfg<128, kS128, CAST, OP, GATED>>(t, smem);
    else if (live <= 160)
      gemm_tile<GroupedCfg<160, kS160, CAST, OP, GATED>>(t, smem);
    else if (live <= 192)
      gemm_tile<GroupedCfg<192, kS192, CAST, OP, GATED>>(t, smem);
    else
      gemm_tile<GroupedCfg<256, kS256, CAST, OP, GATED>>(t, smem);
    __syncthreads();  // the next tile's loads reuse the ring
  }
}

}  // namespace fp8q
