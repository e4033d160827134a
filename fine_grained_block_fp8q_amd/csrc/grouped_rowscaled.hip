// Weight gradients by expert: products whose inner extent is an expert's tokens.
//
//   C[e][n][k] = sum over the expert's groups g of (a_s[g][n] b_s[g][k]) P_g[n][k],
//   P_g[n][k]  = sum over the group's 128 tokens of a_q[n][t] b_q[k][t],
//
// A = dY^T (codes [N][T]) and B = X^T (codes [K][T]) with the tokens grouped by
// expert as in experts.hpp, T = 128 times the groups there is room for.  Each P_g
// is formed by the FP8 matrix core from zero and folded into FP32 sums with the
// product of its two scales, as in the dense row-scaled GEMM.
//
// An expert has few tokens (128 .. 1024) for a large C: a tile of C has few groups
// to sum, and what costs time beside the products is the latency at a tile's start
// and the writing of C.  A persistent workgroup therefore walks tiles as one stream
// of groups: while a group is multiplied the next one's loads are on their way, a
// tile's last group's and the next tile's first one among them, and the next
// group's fragments come into registers before the current one's last products.
// Two stages of one group each in LDS (direct loads; rows of 128 bytes with
// exchanged 16-byte columns, so that fragment reads are free of conflicts).  The
// product is formed transposed (matrix-core rows are B's rows, in an order that
// gives a lane 8 consecutive k of two blocks), and the lanes of two rows exchange
// pieces, so that 8 lanes store a row's 128 bytes at once (4 lanes and 64 bytes:
// 622 us where whole lines take 522).
//
// Tiles of 256 x 256 (8 waves of 64 x 128, one workgroup a CU) where they fill the
// chip 5 times over, else 128 x 128 (4 waves of 64 x 64, two workgroups a CU), us:
//   tiles of 256 x 256         512    576    1024   1280   2048   14336
//   256 x 256                  21.4   42.7   37.0   58.9   54.1   470
//   128 x 128                  17.9   28.7   35.0   60.7   55.1   744
//
// Each XCD takes a run of the tiles (all of an expert's follow each other: its
// operands stay in that XCD's L2), cut so that the runs' groups, plus kTileCost for
// every tile, are equal; its workgroups take the run's tiles in turn.
//
// 32 experts, 8192 tokens, 4096 x 7168 in BF16 (1.88 GB of C, 2.5 groups a tile): 470
// .. 500 us, 4.2 TB/s; loads alone take 222, loads and products with nothing stored
// 395, stores of this pattern alone 350.  16 experts of 1000 tokens, 7168 x 2048: 311
// us, 1.51 PFLOP/s.

#include "experts.hpp"
#include "fp8q.h"
#include "gemm_tile.hpp"
#include "launch.hpp"

namespace fp8q {

// A tile of TN rows of A by TK rows of B, WN x WK waves of 64 x TK/WK each.
template <int TN_, int TK_, int WN_, int WK_, int PER_CU_>
struct WgCfg {
  static constexpr int TN = TN_, TK = TK_, WN = WN_, WK = WK_, PER_CU = PER_CU_;
  static constexpr int WAVES = WN * WK, THREADS = 64 * WAVES;
  static constexpr int NJ = TK / WK / 16;                     // blocks of 16 rows of B a wave
  static constexpr int A_BYTES = TN * 128, B_BYTES = TK * 128;
  static constexpr int SCALES = A_BYTES + B_BYTES;            // their place in a stage
  static constexpr int STAGE = SCALES + (TN + TK) * 4;
  static constexpr int A_LOADS = TN / 8 / WAVES, B_LOADS = TK / 8 / WAVES;  // of 1 KiB, a wave
  static constexpr int LOADS = A_LOADS + B_LOADS + 1;         // and 64 scales
  static constexpr int STORES = 4 * NJ / 2;                   // of 1 KiB in BF16, a wave and tile
  static_assert(TN == 64 * WN && (TN + TK) == 64 * WAVES, "64 rows and 64 scales a wave");
  static_assert(LOADS + 2 * STORES < 64, "vmcnt range");
};
using WgLarge = WgCfg<256, 256, 4, 2, 1>;
using WgSmall = WgCfg<128, 128, 2, 2, 2>;

constexpr int kWgExperts = 1024;
constexpr int kNonTemporal = 2;         // cache policy bit of a buffer store
constexpr int kLag = 2;                 // blocks between a product and its folding
constexpr int64_t kLargeTiles = 5;      // of 256 x 256 a CU, from which they are taken
constexpr int kTileCost = 1;            // of a tile beside its groups, in groups

template <class Cfg>
struct WgShared {
  uint8_t stage[2][Cfg::STAGE];
  int group0[kWgExperts + 1];  // groups before each expert, and all
};
static_assert(WgLarge::PER_CU * sizeof(WgShared<WgLarge>) <= 160 * 1024 &&
                  WgSmall::PER_CU * sizeof(WgShared<WgSmall>) <= 160 * 1024,
              "the workgroups of a CU fit its LDS");

// Rows r16 = 2h and 2h + 1 exchange 16-byte pieces: of the even lane's x, y and the odd
// one's, x becomes the even row's x and y, y the odd row's.
__device__ __forceinline__ void pair_rows(v4u& x, v4u& y, bool odd) {
  auto other = [](uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kDppQuadXor1, 0xF, 0xF, false);
  };
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t xo = other(x[w]), yo = other(y[w]);
    x[w] = odd ? yo : x[w];
    y[w] = odd ? y[w] : xo;
  }
}

// The rows of B that block j's matrix-core rows are: row rho = 4 q + r of blocks 2h and
// 2h + 1 is row 32 h + 8 q + r, and 4 more for the second, so that a lane's results of
// the two are 8 consecutive k.  Where row r of B keeps its 16-byte column c in LDS: by
// its place among the 16 rows of a fragment read, as swz does for A.
__device__ __forceinline__ int b_row(int rho) { return 8 * (rho >> 2) + (rho & 3); }
__device__ __forceinline__ int b_swz(int r, int c) { return swz(4 * ((r >> 3) & 3) + (r & 3), c); }

// Waits until at most STORES vector memory operations are outstanding (`stored`), or
// none.  (The choice is within the instructions here: a branch of the compiler's
// would cut a step in two.)
template <int STORES>
__device__ __forceinline__ void wait_loads(int stored) {
  asm volatile(
      "s_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 .Lnone%=\n\ts_waitcnt vmcnt(%1)\n\ts_branch .Ldone%=\n"
      ".Lnone%=:\n\ts_waitcnt vmcnt(0)\n.Ldone%=:"
      :
      : "s"(stored), "n"(STORES)
      : "memory", "scc");
}

// The experts' first groups into `group0`; false where off is invalid.  Every wave
// finds the same; the first writes.
__device__ __forceinline__ bool expert_prefix(const int32_t* off, int G, int64_t most, int* group0) {
  const int lane = threadIdx.x & 63, PL = (G + 63) >> 6, e0 = lane * PL;
  int sum = 0;
  bool bad = lane == 0 && off[0] != 0;
  for (int i = 0; i < PL; ++i)
    if (e0 + i < G) {
      const int lo = off[e0 + i], hi = off[e0 + i + 1];
      bad = bad || hi < lo;
      sum += groups_of(hi - lo);
    }
  if (__ballot(bad) != 0) return false;
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(inc, d);
    if (lane >= d) inc += v;
  }
  if ((int64_t)__builtin_amdgcn_readlane(inc, 63) > most) return false;
  if (threadIdx.x < 64) {
    int at = inc - sum;
    if (lane == 0) group0[0] = 0;
    for (int i = 0; i < PL; ++i)
      if (e0 + i < G) {
        at += groups_of(off[e0 + i + 1] - off[e0 + i]);
        group0[e0 + i + 1] = at;
      }
  }
  return true;
}

// First tile of run x of the kXcds equal ones, by cost: tiles * (groups + kTileCost) an
// expert.
__device__ __forceinline__ int run_start(const int* group0, int G, int tiles, int x) {
  auto cost = [&](int e) { return (uint64_t)tiles * (uint64_t)(group0[e] + kTileCost * e); };
  const uint64_t want = cost(G) * (uint64_t)x / kXcds;
  int lo = 0, hi = G;  // cost(lo) <= want < cost(hi), or want is the end
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cost(mid) <= want) lo = mid; else hi = mid;
  }
  const uint32_t each = (uint32_t)(group0[lo + 1] - group0[lo] + kTileCost);
  const uint64_t rest = want - cost(lo);
  // (a division of 64 bits takes long: only where one is needed)
  const uint64_t in = rest >> 32 ? rest / each : (uint32_t)rest / each;
  return lo * tiles + (int)(in < (uint64_t)tiles ? in : (uint64_t)tiles);
}

// A fragment's two 16-byte pieces.
__device__ __forceinline__ v8i frag_at(const uint8_t* lo, const uint8_t* hi, int at) {
  const v4i l = *reinterpret_cast<const v4i*>(lo + at), h = *reinterpret_cast<const v4i*>(hi + at);
  return v8i{l[0], l[1], l[2], l[3], h[0], h[1], h[2], h[3]};
}

// PRECISE: each P_g by FP16 matrix-core instructions on the codes widened to FP16.
template <class Cfg, bool PRECISE, bool OUT_BF16>
__device__ __forceinline__ void grouped_rowscaled(
    const uint8_t* A, const float* SA, const uint8_t* B, const float* SB, const int32_t* off, int G,
    int64_t T, int N, int K, void* C, int tiles_k, int tiles, WgShared<Cfg>& sh) {
  constexpr int NJ = Cfg::NJ, W = Cfg::WAVES;
  if (!expert_prefix(off, G, T / 128, sh.group0)) {
#ifdef FP8Q_DEBUG_CHECKS
    if (blockIdx.x == 0 && threadIdx.x == 0) g_experts_error = 1;
#endif
    return;
  }
  __syncthreads();
  // The workgroup's tiles: first, first + step, ... below end.  (A workgroup for every
  // tile: there are no runs to cut.)
  const bool all = (int64_t)gridDim.x >= (int64_t)tiles * G;
  int step = gridDim.x, first = blockIdx.x, end = tiles * G;
  if (!all) {
    const int x = blockIdx.x % kXcds;
    step = gridDim.x / kXcds;
    first = __builtin_amdgcn_readfirstlane(run_start(sh.group0, G, tiles, x)) +
            (int)(blockIdx.x / kXcds);
    end = __builtin_amdgcn_readfirstlane(run_start(sh.group0, G, tiles, x + 1));
  }

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / Cfg::WK, wk = wave % Cfg::WK;
  const int r16 = lane & 15, q = lane >> 4;

  // Operand loads: instruction m of an operand carries rows 8m .. 8m+7, lane l to LDS
  // byte 16 l: row l/8, physical column l%8.  (Rows past the operand's last are out
  // of its range: zeros.)
  static_assert(Cfg::A_LOADS == Cfg::B_LOADS, "as many rows of both");
  uint32_t voff_a[Cfg::A_LOADS], voff_b[Cfg::B_LOADS];
#pragma unroll
  for (int d = 0; d < Cfg::A_LOADS; ++d) {
    const int r = (d * W + wave) * 8 + (lane >> 3);
    voff_a[d] = (uint32_t)(r * T) + (uint32_t)(swz(r, lane & 7) * 16);
    voff_b[d] = (uint32_t)(r * T) + (uint32_t)(b_swz(r, lane & 7) * 16);
  }

  // The stream's next group: tile `lt`, group `lg` of its expert's `ln`.  Past the
  // last one its loads are of nothing (resources of no bytes), so that every step
  // has as many.
  int lt = first, lg = 0, ln = 0;
  __amdgpu_buffer_rsrc_t ra = make_rsrc(A, 0), rb = ra, rs = ra;
  const float* sbase = nullptr;
  int s_ld = 0, s_bytes = 0;
  auto enter = [&] {  // the first tile from lt on that has groups
    for (; lt < end; lt += step) {
      const int e = lt / tiles, in = lt - e * tiles;
      const int g0 = __builtin_amdgcn_readfirstlane(sh.group0[e]);
      ln = __builtin_amdgcn_readfirstlane(sh.group0[e + 1]) - g0;
      if (ln == 0) continue;
      const int tn = in / tiles_k, n0 = tn * Cfg::TN, k0 = (in - tn * tiles_k) * Cfg::TK;
      const int64_t t0 = (int64_t)g0 * 128;
      const int na = N - n0 < Cfg::TN ? N - n0 : Cfg::TN, nb = K - k0 < Cfg::TK ? K - k0 : Cfg::TK;
      ra = make_rsrc(A + n0 * T + t0, na * T - t0);
      rb = make_rsrc(B + k0 * T + t0, nb * T - t0);
      // Scales: the first TN/64 waves those of A, the others those of B, 64 each.
      const bool s_a = wave < Cfg::TN / 64;
      const int at = (s_a ? wave : wave - Cfg::TN / 64) * 64, live = (s_a ? na : nb) - at;
      s_ld = s_a ? N : K;
      s_bytes = live < 64 ? (live > 0 ? live * 4 : 0) : 256;
      sbase = (s_a ? SA + n0 : SB + k0) + (int64_t)g0 * s_ld + at;
      lg = -1;
      return;
    }
    ra = rb = rs = make_rsrc(A, 0);
  };
  // To the next group; before the first, to that.
  auto advance = [&] {
    if (lt < end && lg + 1 == ln) {
      lt += step;
      enter();
    }
    if (lt < end) {
      ++lg;
      rs = make_rsrc(sbase + (int64_t)lg * s_ld, s_bytes);
    }
  };
  auto issue = [&](int at) {
    uint8_t* const st = sh.stage[at];
#pragma unroll
    for (int d = 0; d < Cfg::A_LOADS; ++d)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to_lds(st + (d * W + wave) * 1024), 16, voff_a[d],
                                               lg * 128, 0, 0);
#pragma unroll
    for (int d = 0; d < Cfg::B_LOADS; ++d)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, to_lds(st + Cfg::A_BYTES + (d * W + wave) * 1024),
                                               16, voff_b[d], lg * 128, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to_lds(st + Cfg::SCALES + wave * 256), 4,
                                             (uint32_t)(lane * 4), 0, 0, 0);
  };

  // This lane's places in a stage: its row of a block of 16 and the pieces q and q+4
  // of the row (the exchange of columns goes by the row in its block).
  const int c_lo = swz(r16, q) * 16, c_hi = swz(r16, q + 4) * 16;
  const int a_lo = r16 * 128 + c_lo, a_hi = r16 * 128 + c_hi;
  const int b_lo = b_row(r16) * 128 + c_lo, b_hi = b_row(r16) * 128 + c_hi;
  const int fa = wn * 64 * 128, fb = Cfg::A_BYTES + wk * NJ * 16 * 128;
  const int fsa = Cfg::SCALES + (wn * 64 + r16) * 4;
  const int fsb = Cfg::SCALES + (Cfg::TN + wk * NJ * 16 + 8 * q) * 4;

  constexpr int OB = OUT_BF16 ? 2 : 4;
  constexpr int kStores = Cfg::STORES * OB / 2;
  constexpr int kWide = OUT_BF16 ? 4 : 2;  // blocks of 128 bytes
  const bool odd = r16 & 1;
  const uint32_t out_to =
      (uint32_t)((r16 - odd) * K * OB + (OUT_BF16 ? odd * 64 + 16 * q : odd * 16 + 32 * q));

  // What a step has in registers when it begins: its group's fragments of A, the
  // first of B, and their scales.
  v8i a[4], b[2];
  float sa[4], sa_next[4];
  v4f sb[3], sb_next;
  auto row_block = [&](const uint8_t* st, int j, v8i& f, v4f& s) {
    const int row = j / 2 * 32 + j % 2 * 4;
    f = frag_at(st + fb + b_lo, st + fb + b_hi, row * 128);
    s = *reinterpret_cast<const v4f*>(st + fsb + row * 4);
  };
  auto row_a = [&](const uint8_t* st, int i) {
    a[i] = frag_at(st + fa + a_lo, st + fa + a_hi, i * 2048);
    sa_next[i] = *reinterpret_cast<const float*>(st + fsa + i * 64);
  };

  enter();
  advance();
  issue(0);
  advance();
  if (lt < end) {
    issue(1);
    wait_vmcnt<Cfg::LOADS>();
  } else {
    wait_vmcnt<0>();
  }
  lds_barrier();
  row_block(sh.stage[0], 0, b[0], sb[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    row_a(sh.stage[0], i);
    sa[i] = sa_next[i];
  }
  int cur = 0;
  int stored = 0;  // the stores of the tile before are behind the loads in flight
  for (int t = first; t < end; t += step) {
    const int e = t / tiles, in = t - e * tiles, tn = in / tiles_k;
    const int n0 = tn * Cfg::TN + wn * 64, k0 = (in - tn * tiles_k) * Cfg::TK + wk * NJ * 16;
    const bool live = n0 < N && k0 < K;
    const int groups = __builtin_amdgcn_readfirstlane(sh.group0[e + 1] - sh.group0[e]);
    v4f acc[4][NJ];  // [16 rows of A][16 rows of B]
    auto group = [&](auto first_c) {
      constexpr bool FIRST = decltype(first_c)::value;
      // One group.  Block k = 4 j + i is folded kLag blocks later, when the matrix core
      // has written it (held in this order: the compiler would fold it at once, and
      // wait).  Before the last row of blocks every fragment of the stage is in
      // registers: the barrier there frees it for the group after the next, whose
      // loads go out at once (ahead of a tile's stores, so that they are waited for
      // without them), and makes the next group's fragments readable, which take the
      // places of those that have served.
      constexpr int kBar = 4 * (NJ - 1) - 2, kLast = 4 * (NJ - 1);
      const uint8_t *const st = sh.stage[cur], *const st_next = sh.stage[cur ^ 1];
      v4f p[kLag + 1];
      advance();
#pragma unroll
      for (int k = 0; k < 4 * NJ + kLag; ++k) {
        const int i = k % 4, j = k / 4;
        if (k < 4 * NJ) {
          if (i == 0 && j < NJ - 1) row_block(st, j + 1, b[(j + 1) % 2], sb[(j + 1) % 3]);
          v4f& o = p[k % (kLag + 1)];
          o = v4f{0.f, 0.f, 0.f, 0.f};
          if constexpr (PRECISE) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
              o = mfma_wide16(widen_quarter(b[j % 2], h), widen_quarter(a[i], h), o);
          } else {
            o = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j % 2], a[i], o, 0, 0, 0, 0, 0, 0);
          }
        }
        if (k == kBar) {
          wait_loads<kStores>(__builtin_amdgcn_readfirstlane(stored));
          stored = 0;
          lds_barrier();
          issue(cur);
        }
        if (k == kLast) row_block(st_next, 0, b[0], sb_next);
        if (k >= kLast && k < 4 * NJ) row_a(st_next, i);
        __builtin_amdgcn_sched_barrier(0);
        if (k >= kLag) {
          const int d = k - kLag;
          v4f& to = acc[d % 4][d / 4];
          if constexpr (FIRST) to = v4f{0.f, 0.f, 0.f, 0.f};
          promote_rows(to, p[d % (kLag + 1)], sa[d % 4], sb[d / 4 % 3]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      sb[0] = sb_next;
#pragma unroll
      for (int i = 0; i < 4; ++i) sa[i] = sa_next[i];
      cur ^= 1;
    };
    if (groups > 0) {
      group(std::true_type{});
      for (int g = 1; g < groups; ++g) group(std::false_type{});
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }

    // Block (i, j): the lane holds n = 16 i + r16 and k = 32 (j/2) + 8 q + 4 (j%2) .. +3.
    stored = live ? 1 : 0;
    if (!live) continue;
    uint8_t* const c0 = static_cast<uint8_t*>(C) + (((int64_t)e * N + n0) * K + k0) * OB;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NJ; j += kWide) {
        v4u x, y;
        if constexpr (OUT_BF16) {
          auto eight = [&](const v4f& l, const v4f& h) {
            return v4u{pack_bf16x2(l[0], l[1]), pack_bf16x2(l[2], l[3]), pack_bf16x2(h[0], h[1]),
                       pack_bf16x2(h[2], h[3])};
          };
          x = eight(acc[i][j], acc[i][j + 1]);
          y = eight(acc[i][j + 2], acc[i][j + 3]);
        } else {
          x = __builtin_bit_cast(v4u, acc[i][j]);
          y = __builtin_bit_cast(v4u, acc[i][j + 1]);
        }
        pair_rows(x, y, odd);
        // (The place is in the resource, not a scalar offset: for a store with one the
        // compiler puts no wait before the next instruction, which may then write the
        // data's first register before the last lanes have sent it.)
        uint8_t* const to = c0 + ((int64_t)16 * i * K + 16 * j) * OB;
        const int64_t rows = ((int64_t)14 * K + 16 * kWide) * OB;
        __builtin_amdgcn_raw_buffer_store_b128(x, make_rsrc(to, rows), out_to, 0, kNonTemporal);
        __builtin_amdgcn_raw_buffer_store_b128(y, make_rsrc(to + (int64_t)K * OB, rows), out_to, 0,
                                               kNonTemporal);
      }
  }
  // No load into LDS is under way when the wave ends (the last tile's stores may be).
  wait_loads<kStores>(__builtin_amdgcn_readfirstlane(stored));
}

template <class Cfg, bool PRECISE, bool OUT_BF16>
__global__ __launch_bounds__(Cfg::THREADS, 2) void grouped_rowscaled_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ SA, const uint8_t* __restrict__ B,
    const float* __restrict__ SB, const int32_t* __restrict__ off, int G, int64_t T, int N, int K,
    void* __restrict__ C, int tiles_k, int tiles) {
  __shared__ __attribute__((aligned(16))) WgShared<Cfg> sh;
  grouped_rowscaled<Cfg, PRECISE, OUT_BF16>(A, SA, B, SB, off, G, T, N, K, C, tiles_k, tiles, sh);
}

#ifdef FP8Q_DEBUG_CHECKS
hipError_t wgrad_offsets_error_take(hipStream_t stream, int* flag) {
  return take_experts_error(stream, flag);
}
#endif

template <class Cfg, bool PRECISE>
static hipError_t launch(const uint8_t* a_q, const float* a_s, const uint8_t* b_q, const float* b_s,
                         int64_t T, const int32_t* off, int G, int64_t N, int64_t K, void* c,
                         int out_bf16, int cus, hipStream_t stream) {
  const int64_t tiles_k = (K + Cfg::TK - 1) / Cfg::TK, tiles = (N + Cfg::TN - 1) / Cfg::TN * tiles_k;
  if (tiles > 0x7FFFFFFF / (G + 1) - 1024) return hipErrorInvalidValue;  // (tile numbers are ints)
  int64_t grid = (int64_t)cus * Cfg::PER_CU;
  if (grid > tiles * G) grid = tiles * G;
  grid = (grid + kXcds - 1) / kXcds * kXcds;
  auto kern = out_bf16 ? grouped_rowscaled_kernel<Cfg, PRECISE, true>
                       : grouped_rowscaled_kernel<Cfg, PRECISE, false>;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(Cfg::THREADS), 0, stream, a_q, a_s, b_q, b_s,
                     off, G, T, (int)N, (int)K, c, (int)tiles_k, (int)tiles);
  return hipGetLastError();
}

hipError_t launch_grouped_gemm_rowscaled(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                         const float* b_s, int64_t T, const int32_t* off, int G,
                                         int64_t N, int64_t K, void* c, int out_bf16, int precise,
                                         hipStream_t stream) {
  if (N == 0 || K == 0) return hipSuccess;
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return hipGetLastError();
  const int64_t large = (N + 255) / 256 * ((K + 255) / 256) * G;
  // (Widened to FP16, its fragments would spill.  A resource describes at most 2^32 - 1
  // bytes: 256 rows of 2^24 are one more.)
  if (large >= kLargeTiles * cus && !precise && WgLarge::TN * T <= 0xFFFFFFFFll)
    return launch<WgLarge, false>(a_q, a_s, b_q, b_s, T, off, G, N, K, c, out_bf16, cus, stream);
  return (precise ? launch<WgSmall, true> : launch<WgSmall, false>)(
      a_q, a_s, b_q, b_s, T, off, G, N, K, c, out_bf16, cus, stream);
}

}  // namespace fp8q
