// int8 products and the int8 gated block in output tiles (many rows).
//
//   Y[m][n] = (sum_k a[m][k] w[n][k]) a_s[m] w_s[n];  C = Y (+ bias), or
//   h[m][f] = act(Y[m][f]) Y[m][F + f].
//
// The scales stand outside the sum, so nothing leaves the matrix core before
// the end: a wave keeps its sums in the accumulation registers for the whole
// of K, and the loop is operand traffic and matrix instructions alone.  A wave
// of WM x WN reads WM + WN operand bytes from LDS for WM * WN products of each
// k, so the waves are as large as the registers allow: one wave a SIMD with
// 128 x 128 sums takes the 256 accumulation registers and reads 2/3 of what
// two waves of 64 x 128 would.
//
// Operands go from memory to LDS without registers, in units of 128 bytes of K
// (a cache line a row; 64-byte rows halve what the L2 delivers) of all rows of
// one operand.  A chunk is two instruction steps of 64 k.  While step 0 of
// chunk g is multiplied, the second half of its W fragments is read; while
// step 1 is, all of A's fragments of chunk g + 1 and the first half of W's.  So
// A's unit is free one step before W's, and with two units of A and three of W
// (160 KB in the largest tile) their refills go out in alternate steps, 8 loads
// a wave beside 64 products, two steps (A) and three (W) before they are needed.
// One barrier a step, a few products before its end.
//
// 4096 x 4096 x 7168: 86 to 90 us, 2650 to 2790 TOP/s.  Without the LDS reads it
// takes 83, without the loads 77, without both 72; the chip is held back by its
// power (1.95 to 2.1 GHz): 512 rows, an eighth of the CUs, take 67 where these
// do and 59 without.
//
// The product is formed transposed (weight rows are the instruction's rows), so
// a lane holds 4 consecutive outputs of one activation row; the epilogue
// scales them, passes them through the wave's share of the ring and stores
// whole rows of the tile.
//
// K is a multiple of 16.  Pieces past it, and rows past M or N, are out of
// range at the load, which then delivers zeros.

#include "activation.hpp"
#include "gemm_common.hpp"
#include "launch.hpp"
#include "tile_choice.hpp"

namespace fp8q {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int NA_, bool GATED_, bool BF16_>
struct I8Cfg {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr bool GATED = GATED_, BF16 = BF16_;
  static constexpr int BK = 128;                      // bytes of K a unit
  static constexpr int NA = NA_, NW = NA + 1;         // units of A and of W
  static constexpr int NWAVES = WAVES_M * WAVES_N, THREADS = NWAVES * 64;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int MB = WM / 16, NB = WN / 16;
  static constexpr int LA = BM / 8 / NWAVES, LW = BN / 8 / NWAVES;  // 1 KiB loads of a wave
  static constexpr int A_UNIT = BM * BK, W_UNIT = BN * BK, LDS = NA * A_UNIT + NW * W_UNIT;
  static constexpr int OBN = GATED ? BN / 2 : BN;  // output columns of the tile
  static constexpr int WNO = GATED ? WN / 2 : WN;  // and of a wave
  static_assert(BM % (8 * NWAVES) == 0 && BN % (8 * NWAVES) == 0, "whole loads for every wave");
  static_assert(WM % 16 == 0 && WN % (GATED ? 32 : 16) == 0, "whole blocks");
  static_assert(NA * LA + NW * LW < 64, "loads in flight");
  static_assert(LDS <= 160 * 1024, "LDS budget");
  // row blocks of outputs that a wave's share of the ring holds, with the
  // columns' scales: all of them or half
  static constexpr int share(int blocks) { return blocks * 16 * (WNO * (BF16 ? 2 : 4) + 16) + WN * 8; }
  static constexpr int ROW_BLOCKS = share(MB) <= LDS / NWAVES ? MB : MB / 2;
  static_assert(share(ROW_BLOCKS) <= LDS / NWAVES, "they fit it");
};

struct I8Args {
  const uint8_t* a;
  const float* a_s;
  const uint8_t* w;
  const float* w_s;
  const float* bias;
  void* c;
  int64_t M, N, K;  // N: output columns (F when gated)
  int tiles_n;
  int act;
};

// A lane offset past any operand, also with a scalar offset added.
constexpr uint32_t kOutOfRange = 0x80000000u;

// c += a . b, kept in the accumulation registers.  (As a builtin the compiler
// gives sum and addend different registers and copies most of them.)
__device__ __forceinline__ void mfma_i8(v4i& c, const v4i& a, const v4i& b) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// Orders a wave's own LDS writes and reads (the wave is its only user).
__device__ __forceinline__ void lds_wave_fence() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// Tile of workgroup `bid`: every XCD (bid mod 8) takes a contiguous run of
// tiles, which go down 4 tile rows before the next tile column, so that a run
// shares its operand rows in the XCD's L2.
__device__ __forceinline__ void xcd_run_tile(int bid, int tiles, int tiles_n, int& tm, int& tn) {
  const int x = bid % kXcds, q = tiles / kXcds, r = tiles % kXcds;
  const int id = x * q + (x < r ? x : r) + bid / kXcds;
  const int tiles_m = tiles / tiles_n;
  const int per = kGroupM * tiles_n, grp = id / per, first = grp * kGroupM;
  const int gm = tiles_m - first < kGroupM ? tiles_m - first : kGroupM;
  const int in = id - grp * per;
  // (the vector ALU divides; everything derived from the tile is to be scalar)
  tm = __builtin_amdgcn_readfirstlane(first + in % gm);
  tn = __builtin_amdgcn_readfirstlane(in / gm);
}

template <class Cfg>
__device__ __forceinline__ void i8_tile(const I8Args& p, uint8_t* smem) {
  constexpr int MB = Cfg::MB, NB = Cfg::NB, LA = Cfg::LA, LW = Cfg::LW;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave_m = wave / Cfg::WAVES_N, wave_n = wave % Cfg::WAVES_N;
  int tm, tn;
  xcd_run_tile(blockIdx.x, gridDim.x, p.tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * Cfg::BM, n0 = (int64_t)tn * Cfg::OBN;
  const int64_t K = p.K;

  const int fr = lane & 15, fq = lane >> 4;

  // ---- loads.  Load d of a wave is rows 8(d NWAVES + wave) .. +7 of the unit:
  // lane l fetches row l/8, physical piece l%8 of it.  The row block and the
  // chunk are in the scalar offset, so a load costs no vector instruction; rows
  // past M or N, and pieces past K, are out of the resource's range and come
  // as zeros.
  const int pr = lane >> 3;
  const int kc = swz(8 * (wave & 1) + pr, lane & 7) * 16;  // its byte within the 128
  // (readfirstlane: the vector ALU takes a 64-bit minimum, and a resource in
  // vector registers would be looped over at every load)
  const int a_live = __builtin_amdgcn_readfirstlane(p.M - m0 < Cfg::BM ? (int)(p.M - m0) : Cfg::BM);
  const int w_live = __builtin_amdgcn_readfirstlane(p.N - n0 < Cfg::OBN ? (int)(p.N - n0) : Cfg::OBN);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + m0 * K, (int64_t)a_live * K);
  // weight rows of the tile: with a gated block the first half of each wave's
  // rows are gate rows and the second the matching up rows, F further on
  const __amdgpu_buffer_rsrc_t rg = make_rsrc(p.w + n0 * K, (int64_t)w_live * K);
  const __amdgpu_buffer_rsrc_t ru =
      make_rsrc(p.w + ((Cfg::GATED ? p.N : 0) + n0) * K, (int64_t)w_live * K);
  constexpr int RL = 8 * Cfg::NWAVES;  // rows of the workgroup's load d
  static_assert(Cfg::WNO % RL == 0, "a load of the workgroup is all gate or all up rows");
  const uint32_t voff = (uint32_t)((wave * 8 + pr) * (int)K + kc);
  const int k_lim = (int)K - kc, ks = (int)K;
  auto load_a = [&](int g, int unit, int d) {
    const uint32_t v = g * Cfg::BK < k_lim ? voff : kOutOfRange;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        ra, to_lds(smem + unit * Cfg::A_UNIT + (d * Cfg::NWAVES + wave) * 1024), 16, v,
        g * Cfg::BK + d * RL * ks, 0, 0);
  };
  auto load_w = [&](int g, int unit, int d) {
    const uint32_t v = g * Cfg::BK < k_lim ? voff : kOutOfRange;
    const int r = d * RL, w = r / Cfg::WN, i = r % Cfg::WN;
    const bool up = Cfg::GATED && i >= Cfg::WNO;
    const int row = Cfg::GATED ? w * Cfg::WNO + i % Cfg::WNO : r;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        up ? ru : rg,
        to_lds(smem + Cfg::NA * Cfg::A_UNIT + unit * Cfg::W_UNIT + (d * Cfg::NWAVES + wave) * 1024),
        16, v, g * Cfg::BK + row * ks, 0, 0);
  };

  // ---- fragments: lane l holds row l%16, k bytes 16*(l/16) .. +15 of a step
  const int a_at = (wave_m * Cfg::WM + fr) * 128, w_at = (wave_n * Cfg::WN + fr) * 128;
  const int c0 = swz(fr, fq) * 16, c1 = swz(fr, fq + 4) * 16;
  auto read_a = [&](v4i& f, int unit, int h, int i) {
    f = *reinterpret_cast<const v4i*>(smem + unit * Cfg::A_UNIT + a_at + (h ? c1 : c0) + i * 2048);
  };
  auto read_w = [&](v4i& f, int unit, int h, int j) {
    f = *reinterpret_cast<const v4i*>(smem + Cfg::NA * Cfg::A_UNIT + unit * Cfg::W_UNIT + w_at +
                                      (h ? c1 : c0) + j * 2048);
  };

  v4i acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  // Chunks go in pairs (A has two units); past K they are zeros.
  const int chunks = (int)((K + 2 * Cfg::BK - 1) / (2 * Cfg::BK)) * 2;

  // In the order of the steady state: W of chunk 0, A of 0, W of 1, A of 1, ...
#pragma unroll
  for (int d = 0; d < LW; ++d) load_w(0, 0, d);
#pragma unroll
  for (int x = 0; x < Cfg::NA; ++x) {
#pragma unroll
    for (int d = 0; d < LA; ++d) load_a(x, x, d);
#pragma unroll
    for (int d = 0; d < LW; ++d) load_w(x + 1, x + 1, d);
  }

  // The scheduling barriers fix the order product by product: the compiler
  // left to itself reads fragments right before their products, and loads sent
  // off together block the wave's issue.  The workgroup's barrier sits kLead
  // products before a step's end, so that the matrix core has work while the
  // waves meet.
  constexpr int T = MB * NB, kLead = T >= 16 ? 4 : 0, kSpan = T - 2 * kLead;
  v4i a0[MB], a1[2][MB], w0[NB], w1[NB];
  // Step 0 of chunk g (units t of A and u of W): beside its products, the reads
  // of w1 and the loads of A of chunk g + NA into unit t, which all waves have
  // read.
  auto step0 = [&](int g, int t, int u) {
#pragma unroll
    for (int k = 0; k < T; ++k) {
      mfma_i8(acc[k / NB][k % NB], w0[k % NB], a0[k / NB]);
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (j * kSpan / NB == k) read_w(w1[j], u, 1, j);
#pragma unroll
      for (int d = 0; d < LA; ++d)
        if ((2 * d + 1) * kSpan / (2 * LA) == k) load_a(g + Cfg::NA, t, d);
      if (k == T - 1 - kLead) {
        // W's unit u is read; A and W of chunk g + 1 have landed (what was
        // issued after them: W and A of chunks g + 2 to g + NA)
        wait_vmcnt<(Cfg::NA - 1) * (LA + LW)>();
        lds_barrier();
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Step 1: the reads of A (both halves) and the first half of W of chunk
  // g + 1 (units t1 and u1), and the loads of W of chunk g + NW into unit u.
  auto step1 = [&](int g, const v4i (&x)[MB], v4i (&y)[MB], int t1, int u, int u1) {
    constexpr int R = 2 * MB + NB;
#pragma unroll
    for (int k = 0; k < T; ++k) {
      mfma_i8(acc[k / NB][k % NB], w1[k % NB], x[k / NB]);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r * kSpan / R == k) {
          if (r == 0)
            read_a(a0[0], t1, 0, 0);
          else if (r <= NB)
            read_w(w0[r - 1], u1, 0, r - 1);
          else if (r < NB + MB)
            read_a(a0[r - NB], t1, 0, r - NB);
          else
            read_a(y[r - NB - MB], t1, 1, r - NB - MB);
        }
#pragma unroll
      for (int d = 0; d < LW; ++d)
        if ((2 * d + 1) * kSpan / (2 * LW) == k) load_w(g + Cfg::NW, u, d);
      if (k == T - 1 - kLead) lds_barrier();  // A's unit of chunk g + 1 is read
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  wait_vmcnt<(Cfg::NA - 1) * LA + Cfg::NA * LW>();
  lds_barrier();
#pragma unroll
  for (int i = 0; i < MB; ++i) read_a(a0[i], 0, 0, i);
#pragma unroll
  for (int i = 0; i < MB; ++i) read_a(a1[0][i], 0, 1, i);
#pragma unroll
  for (int j = 0; j < NB; ++j) read_w(w0[j], 0, 0, j);
  lds_barrier();  // A's unit of chunk 0 is read
  int t = 0, u = 0, g = 0;
  do {  // (K >= 1: at least one pair.  With a way past the loop the sums would be
        // copied to common registers behind it, ahead of the wait below.)
    const int t1 = t + 1 == Cfg::NA ? 0 : t + 1, t2 = t1 + 1 == Cfg::NA ? 0 : t1 + 1;
    const int u1 = u + 1 == Cfg::NW ? 0 : u + 1, u2 = u1 + 1 == Cfg::NW ? 0 : u1 + 1;
    step0(g, t, u);
    step1(g, a1[0], a1[1], t1, u, u1);
    step0(g + 1, t1, u1);
    step1(g + 1, a1[1], a1[0], t2, u1, u2);
    t = t2;
    u = u2;
    g += 2;
  } while (g < chunks);
  // The last products' results, before anything else uses them: the products
  // are inline asm, of which the compiler knows no latency.  The sums are made
  // outputs of statements behind the wait, so that no use can move ahead of it.
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) asm volatile("" : "+a"(acc[i][j]));
  // The rows' and columns' scales and the bias, for the epilogue.  (Asked for
  // before the loop they would be spilled there, each with a wait of its own.)
  constexpr int CS = (Cfg::WN + 63) / 64;
  float scale[CS], bias[CS], row_scale[MB];
#pragma unroll
  for (int x = 0; x < CS; ++x) {
    const int o = (lane + 64 * x) % Cfg::WN;
    const int64_t n = n0 + wave_n * Cfg::WNO + o % Cfg::WNO;
    const int64_t nn = n < p.N ? n : p.N - 1;
    scale[x] = p.w_s[nn + (o >= Cfg::WNO ? p.N : 0)];
    bias[x] = !Cfg::GATED && p.bias ? p.bias[nn] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int64_t m = m0 + wave_m * Cfg::WM + 16 * i + fr;
    row_scale[i] = p.a_s[m < p.M ? m : p.M - 1];
  }
  wait_vmcnt<0>();
  lds_barrier();  // the ring is free: each wave takes its share for its output rows

  // ---- epilogue: block (i, j): activation row 16i + l%16, outputs
  // 16j + 4(l/16) .. +3 of the wave
  uint8_t* const mine = smem + wave * (Cfg::LDS / Cfg::NWAVES);
  float* const ws = reinterpret_cast<float*>(mine);
#pragma unroll
  for (int x = 0; x < CS; ++x) {
    const int o = (lane + 64 * x) % Cfg::WN;
    ws[o] = scale[x];
    if (!Cfg::GATED) ws[Cfg::WN + o] = bias[x];
  }
  lds_wave_fence();
  constexpr int OB = Cfg::BF16 ? 2 : 4, ROW = Cfg::WNO * OB, PITCH = ROW + 16, PER = ROW / 16;
  uint8_t* const rows = mine + Cfg::WN * 8;
  const int64_t nw = n0 + wave_n * Cfg::WNO;  // the wave's first output column
  const int live_n = (int)(p.N - nw < Cfg::WNO ? (p.N - nw > 0 ? p.N - nw : 0) : Cfg::WNO);
  // As many row blocks at a time as the wave's share holds, then one loop that
  // stores them: the code runs once a tile, and what it costs is to fetch it.
  constexpr int NO = Cfg::WNO / 16, IB = Cfg::ROW_BLOCKS;
  v4f s_w[NO], more[NO];  // more: the up rows' scales when gated, else the bias
#pragma unroll
  for (int j = 0; j < NO; ++j) {
    s_w[j] = *reinterpret_cast<const v4f*>(ws + 16 * j + 4 * fq);
    more[j] =
        *reinterpret_cast<const v4f*>(ws + (Cfg::GATED ? Cfg::WNO : Cfg::WN) + 16 * j + 4 * fq);
  }
#pragma unroll
  for (int i0 = 0; i0 < MB; i0 += IB) {
    const int64_t mb = m0 + wave_m * Cfg::WM + 16 * i0;
#pragma unroll
    for (int i = i0; i < i0 + IB; ++i)
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = (float)acc[i][j][e] * row_scale[i];
          if constexpr (Cfg::GATED) {
            const float g = v[e] * s_w[j][e];
            v[e] = (Cfg::BF16 ? act_fast(p.act, g) : act_f32(p.act, g)) *
                   ((float)acc[i][j + NB / 2][e] * row_scale[i] * more[j][e]);
          } else {
            v[e] = __builtin_fmaf(v[e], s_w[j][e], more[j][e]);
          }
        }
        uint8_t* at = rows + (16 * (i - i0) + fr) * PITCH + (16 * j + 4 * fq) * OB;
        if constexpr (Cfg::BF16)
          *reinterpret_cast<v2u*>(at) = v2u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
          *reinterpret_cast<v4f*>(at) = v4f{v[0], v[1], v[2], v[3]};
      }
    lds_wave_fence();
    const int live_m = (int)(p.M - mb < 16 * IB ? (p.M - mb > 0 ? p.M - mb : 0) : 16 * IB);
    // (rows of an odd N start anywhere: the stores are then unaligned ones)
#pragma unroll 4
    for (int x = lane; x < 16 * IB * PER; x += 64) {
      const int r = x / PER, c = x % PER, left = live_n * OB - c * 16;
      if (r >= live_m || left <= 0) continue;
      const uint8_t* from = rows + r * PITCH + c * 16;
      uint8_t* to = static_cast<uint8_t*>(p.c) + ((mb + r) * p.N + nw) * OB + c * 16;
      if (left >= 16) {
        const v4u v = *reinterpret_cast<const v4u*>(from);
        __builtin_memcpy(to, &v, 16);
      } else {
        for (int e = 0; e < left; e += OB) __builtin_memcpy(to + e, from + e, OB);
      }
    }
    lds_wave_fence();
  }
}

template <class Cfg>
__global__ __launch_bounds__(Cfg::THREADS) void i8_tile_kernel(const I8Args p) {
  // (One array for all: with a second one the compiler drains every load in
  // flight before a read of the ring.)
  __shared__ __attribute__((aligned(16))) uint8_t smem[Cfg::LDS];
  i8_tile<Cfg>(p, smem);
}

template <class Cfg>
static hipError_t launch_tiles(I8Args p, hipStream_t stream) {
  const int64_t tiles_m = (p.M + Cfg::BM - 1) / Cfg::BM, tiles_n = (p.N + Cfg::OBN - 1) / Cfg::OBN;
  if (tiles_m * tiles_n > max_blocks(Cfg::THREADS)) return hipErrorInvalidValue;
  p.tiles_n = (int)tiles_n;
  hipLaunchKernelGGL(i8_tile_kernel<Cfg>, dim3((unsigned)(tiles_m * tiles_n)), dim3(Cfg::THREADS), 0,
                     stream, p);
  return hipGetLastError();
}

template <bool GATED, bool BF16>
static hipError_t launch_tile(const I8Args& p, int tile, hipStream_t stream) {
  switch (tile) {
    case tile_id(256, 256): return launch_tiles<I8Cfg<256, 256, 2, 2, 2, GATED, BF16>>(p, stream);
    case tile_id(256, 128): return launch_tiles<I8Cfg<256, 128, 2, 2, 2, GATED, BF16>>(p, stream);
    case tile_id(128, 128): return launch_tiles<I8Cfg<128, 128, 2, 2, 2, GATED, BF16>>(p, stream);
    case tile_id(64, 64): return launch_tiles<I8Cfg<64, 64, 2, 1, 3, GATED, BF16>>(p, stream);
    default: return launch_tiles<I8Cfg<32, 64, 1, 2, 3, GATED, BF16>>(p, stream);
  }
}

hipError_t launch_i8_tiles(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s,
                           const float* bias, int64_t M, int64_t N, int64_t K, bool gated, int act,
                           void* c, int out_bf16, int tile, hipStream_t stream) {
  I8Args p{};
  p.a = reinterpret_cast<const uint8_t*>(a_q);
  p.a_s = a_s;
  p.w = reinterpret_cast<const uint8_t*>(w_q);
  p.w_s = w_s;
  p.bias = bias;
  p.c = c;
  p.M = M;
  p.N = N;
  p.K = K;
  p.act = act;
  if (gated)
    return out_bf16 ? launch_tile<true, true>(p, tile, stream)
                    : launch_tile<true, false>(p, tile, stream);
  return out_bf16 ? launch_tile<false, true>(p, tile, stream)
                  : launch_tile<false, false>(p, tile, stream);
}

hipError_t launch_i8_few(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s,
                         const float* bias, int64_t M, int64_t N, int64_t K, bool gated, int act,
                         void* c, int out_bf16, hipStream_t stream);

static hipError_t launch_i8(const int8_t* a_q, const float* a_s, const int8_t* w_q,
                            const float* w_s, const float* bias, int64_t M, int64_t N, int64_t K,
                            bool gated, int act, void* c, int out_bf16, hipStream_t stream) {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return hipGetLastError();
  const int tile = pick_i8(M, gated ? 2 * N : N, K, cus);
  if (tile == 0)
    return launch_i8_few(a_q, a_s, w_q, w_s, bias, M, N, K, gated, act, c, out_bf16, stream);
  return launch_i8_tiles(a_q, a_s, w_q, w_s, bias, M, N, K, gated, act, c, out_bf16, tile, stream);
}

hipError_t launch_gemm_i8(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s,
                          const float* bias, int64_t M, int64_t N, int64_t K, void* c,
                          int out_bf16, hipStream_t stream) {
  return launch_i8(a_q, a_s, w_q, w_s, bias, M, N, K, false, 0, c, out_bf16, stream);
}

hipError_t launch_gemm_i8_gated(const int8_t* a_q, const float* a_s, const int8_t* w_q,
                                const float* w_s, int64_t M, int64_t F, int64_t K, int act,
                                void* h, int out_bf16, hipStream_t stream) {
  return launch_i8(a_q, a_s, w_q, w_s, nullptr, M, F, K, true, act, h, out_bf16, stream);
}

}  // namespace fp8q
