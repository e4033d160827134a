// int8 products and the int8 gated block in output tiles (many rows).
//
//   Y[m][n] = (sum_k a[m][k] w[n][k]) a_s[m] w_s[n];  C = Y (+ bias), or
//   h[m][f] = act(Y[m][f]) Y[m][F + f].
//
// The scales stand outside the sum, so nothing leaves the matrix core before
// the end: a wave keeps its sums in the accumulation registers for the whole
// of K and the loop is operand traffic and matrix instructions alone.  What
// bounds it is the LDS: a wave of WM x WN reads (WM + WN) bytes of operands for
// WM * WN products of each k, so the waves are as large as the registers
// allow.  One wave a SIMD with 128 x 128 sums takes 256 accumulation registers
// and reads 2/3 of what two waves of 64 x 128 would.
//
// Operands go from memory to LDS without registers, 64 bytes of K a row and
// stage, in a ring of NS stages (NS - 1 stages in flight while one is read).
// LDS rows are 64 bytes; their 16-byte pieces are exchanged by row so that
// both the 8- and the 16-lane groups that the LDS serves together read every
// bank once.  A stage is two instruction steps of 32 k; the fragments of a step
// are read during the step before, and the one barrier of a stage lies between
// its steps, when the whole stage is already in registers: from there on its
// slot is refilled.
//
// The product is formed transposed (weight rows are the instruction's rows), so
// a lane holds 4 consecutive outputs of one activation row; the epilogue
// scales them, passes them through the wave's share of the ring and stores
// whole rows of the tile.
//
// K is a multiple of 16: pieces past it are masked at the load (out-of-range
// lanes of a buffer load deliver zeros).  Rows past M or N repeat the last one
// and are not stored.

#include "activation.hpp"
#include "gemm_common.hpp"

namespace fp8q {

typedef int v16i __attribute__((ext_vector_type(16)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int NS_, bool GATED_>
struct I8Cfg {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, NS = NS_;
  static constexpr bool GATED = GATED_;
  static constexpr int BK = 64;
  static constexpr int NWAVES = WAVES_M * WAVES_N, THREADS = NWAVES * 64;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int MB = WM / 32, NB = WN / 32;
  static constexpr int A_PIECES = BM / 16, PIECES = (BM + BN) / 16;  // 1 KiB loads
  static constexpr int LOADS = PIECES / NWAVES;
  static constexpr int STAGE = (BM + BN) * BK, LDS = STAGE * NS;
  static constexpr int OBN = GATED ? BN / 2 : BN;  // output columns of the tile
  static constexpr int WNO = GATED ? WN / 2 : WN;  // and of a wave
  static_assert(PIECES % NWAVES == 0 && A_PIECES % NWAVES == 0, "whole loads for every wave");
  static_assert(WM % 32 == 0 && WN % (GATED ? 64 : 32) == 0, "whole blocks");
  static_assert(LOADS * NS < 64 && NS >= 3, "loads in flight");
  static_assert(LDS / NWAVES >= 32 * (WNO * 4 + 16), "an output block fits the wave's share");
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
  int out_bf16, act;
};

// 16-byte piece of logical column c in LDS row r (4 pieces a row).
__device__ __forceinline__ int swz64(int r, int c) {
  return c ^ (((r >> 1) & 2) | (((r >> 1) ^ (r >> 3)) & 1));
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
  tm = first + in % gm;
  tn = in / gm;
}

template <class Cfg>
__device__ __forceinline__ void i8_tile(const I8Args& p, uint8_t* smem) {
  constexpr int MB = Cfg::MB, NB = Cfg::NB, NS = Cfg::NS, L = Cfg::LOADS;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave_m = wave / Cfg::WAVES_N, wave_n = wave % Cfg::WAVES_N;
  int tm, tn;
  xcd_run_tile(blockIdx.x, gridDim.x, p.tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * Cfg::BM, n0 = (int64_t)tn * Cfg::OBN;
  const int64_t K = p.K;

  // ---- loads.  Lane l of a 1 KiB load fetches LDS row l/4, physical piece l%4.
  const int pr = lane >> 2;
  const int kc = swz64(pr, lane & 3) * 16;  // its byte within the stage's 64
  const int64_t a_live = p.M - m0 < Cfg::BM ? p.M - m0 : Cfg::BM;
  const int64_t w_live = p.N - n0 < Cfg::OBN ? p.N - n0 : Cfg::OBN;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + m0 * K, a_live * K);
  // weight rows of the tile: with a gated block the first half of each wave's
  // rows are gate rows and the second the matching up rows, F further on
  const __amdgpu_buffer_rsrc_t rg = make_rsrc(p.w + n0 * K, w_live * K);
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(p.w + ((Cfg::GATED ? p.N : 0) + n0) * K, w_live * K);
  uint32_t voff[L];
  bool up[L];
#pragma unroll
  for (int d = 0; d < L; ++d) {
    const int m = d * Cfg::NWAVES + wave;
    int r = (d < Cfg::A_PIECES / Cfg::NWAVES ? m : m - Cfg::A_PIECES) * 16 + pr;
    int64_t live = a_live;
    up[d] = false;
    if (d >= Cfg::A_PIECES / Cfg::NWAVES) {
      live = w_live;
      if (Cfg::GATED) {
        const int w = r / Cfg::WN, i = r % Cfg::WN;
        up[d] = i >= Cfg::WNO;
        r = w * Cfg::WNO + i % Cfg::WNO;
      }
    }
    voff[d] = (uint32_t)((r < live ? r : live - 1) * K) + kc;
  }
  const int k_lim = (int)K - kc;
  auto issue = [&](int slot, int s, int d) {
    const bool is_a = d < Cfg::A_PIECES / Cfg::NWAVES;
    const uint32_t v = s * Cfg::BK < k_lim ? voff[d] : 0x80000000u;
    const int m = d * Cfg::NWAVES + wave;
    // a load's 16 rows are all gate or all up rows, the same for its wave
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        is_a ? ra : (Cfg::GATED && __builtin_amdgcn_readfirstlane(up[d])) ? ru : rg,
        to_lds(smem + slot * Cfg::STAGE + m * 1024), 16, v, s * Cfg::BK, 0, 0);
  };

  // ---- fragments: lane l holds row l%32, k bytes 16*(l/32) .. +15 of a step
  const int fr = lane & 31, fq = lane >> 5;
  const int a_at = (wave_m * Cfg::WM + fr) * 64, b_at = Cfg::BM * 64 + (wave_n * Cfg::WN + fr) * 64;
  const int c0 = swz64(fr, fq) * 16, c1 = swz64(fr, fq + 2) * 16;
  auto frag = [&](const uint8_t* at) { return *reinterpret_cast<const v4i*>(at); };

  v16i acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  // The columns' scales and bias, for the epilogue (the wave's own copy).  They
  // are asked for before the ring's loads, so that waiting for them does not
  // wait for those.
  constexpr int CS = (Cfg::WN + 63) / 64;
  float scale[CS], bias[CS];
#pragma unroll
  for (int x = 0; x < CS; ++x) {
    const int o = (lane + 64 * x) % Cfg::WN;
    const int64_t n = n0 + wave_n * Cfg::WNO + o % Cfg::WNO;
    const int64_t nn = n < p.N ? n : p.N - 1;
    scale[x] = p.w_s[nn + (o >= Cfg::WNO ? p.N : 0)];
    bias[x] = !Cfg::GATED && p.bias ? p.bias[nn] : 0.0f;
  }

  const int stages = (int)((K + Cfg::BK - 1) / Cfg::BK);
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int d = 0; d < L; ++d) issue(s, s, d);

  float* const ws = reinterpret_cast<float*>(smem + Cfg::LDS) + wave * 2 * Cfg::WN;
#pragma unroll
  for (int x = 0; x < CS; ++x) {
    const int o = (lane + 64 * x) % Cfg::WN;
    ws[o] = scale[x];
    if (!Cfg::GATED) ws[Cfg::WN + o] = bias[x];
  }

  wait_vmcnt<L*(NS - 1)>();
  lds_barrier();
  v4i a0[MB], b0[NB], a1[MB], b1[NB];
  // fragment x of a step, in the order its products want them
  constexpr int T = MB * NB, R = MB + NB;
  auto read = [&](v4i* a, v4i* b, const uint8_t* stage, int c, int x) {
    if (x == 0)
      a[0] = frag(stage + a_at + c);
    else if (x <= NB)
      b[x - 1] = frag(stage + b_at + (x - 1) * 2048 + c);
    else
      a[x - NB] = frag(stage + a_at + (x - NB) * 2048 + c);
  };
#pragma unroll
  for (int x = 0; x < R; ++x) read(a0, b0, smem, c0, x);

  // Step order is fixed by the scheduling barriers: product k, then the share
  // of the next step's reads (and of the refill's loads) that goes with it.
  // Left to itself the compiler reads fragments right before their products.
  // The barrier sits kLead products before the end of the first step, so that
  // the matrix core has work while the waves meet.
  constexpr int kLead = T >= 8 ? 2 : 0;
  constexpr int kRead = T - kLead;  // products beside which the first step's reads go
  int slot = 0;
  for (int s = 0; s < stages; ++s) {
    const uint8_t* cur = smem + slot * Cfg::STAGE;
    const int next = slot + 1 == NS ? 0 : slot + 1;
    const uint8_t* nxt = smem + next * Cfg::STAGE;
#pragma unroll
    for (int k = 0; k < T; ++k) {
      const int i = k / NB, j = k % NB;
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b0[j], a0[i], acc[i][j], 0, 0, 0);
      constexpr int per = (R + kRead - 1) / kRead;
#pragma unroll
      for (int x = k * per; x < (k + 1) * per && x < R; ++x) read(a1, b1, cur, c1, x);
      if (k == T - 1 - kLead) {
        // this wave has read the whole stage, and its loads of the next have landed
        wait_vmcnt<L*(NS - 2)>();
        lds_barrier();
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int k = 0; k < T; ++k) {
      const int i = k / NB, j = k % NB;
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b1[j], a1[i], acc[i][j], 0, 0, 0);
      constexpr int per = (R + L + T - 1) / T;
#pragma unroll
      for (int x = k * per; x < (k + 1) * per && x < R + L; ++x) {
        if (x < R)
          read(a0, b0, nxt, c0, x);
        else
          issue(slot, s + NS, x - R);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    slot = next;
  }
  wait_vmcnt<0>();
  lds_barrier();  // the ring is free: each wave takes its share for its output rows

  // ---- epilogue: block (i, j): activation row 32i + l%32, outputs
  // 32j + 8t + 4(l/32) .. +3 of the wave, t = 0..3
  uint8_t* const mine = smem + wave * (Cfg::LDS / Cfg::NWAVES);
  const int ob = p.out_bf16 ? 2 : 4;
  const int row_bytes = Cfg::WNO * ob, pitch = row_bytes + 16;
  const int64_t nw = n0 + wave_n * Cfg::WNO;  // the wave's first output column
  const int live_n = (int)(p.N - nw < Cfg::WNO ? (p.N - nw > 0 ? p.N - nw : 0) : Cfg::WNO);
  const bool vec = (p.N * ob) % 16 == 0;  // every row of C starts at a 16-byte boundary
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int64_t mb = m0 + wave_m * Cfg::WM + 32 * i;
    const int64_t m = mb + fr;
    const float s_a = p.a_s[m < p.M ? m : p.M - 1];
#pragma unroll
    for (int j = 0; j < Cfg::WNO / 32; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int o = 32 * j + 8 * t + 4 * fq;
        const v4f s_w = *reinterpret_cast<const v4f*>(ws + o);
        // gated: the up rows' scales; else the bias
        const v4f more = *reinterpret_cast<const v4f*>(ws + (Cfg::GATED ? Cfg::WNO : Cfg::WN) + o);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = (float)acc[i][j][4 * t + e] * s_a * s_w[e];
          if constexpr (Cfg::GATED)
            v[e] = act_fast(p.act, v[e]) * ((float)acc[i][j + NB / 2][4 * t + e] * s_a * more[e]);
          else
            v[e] += more[e];
        }
        if (p.out_bf16)
          *reinterpret_cast<v2u*>(mine + fr * pitch + o * 2) =
              v2u{f32_to_bf16_bits(v[0]) | f32_to_bf16_bits(v[1]) << 16,
                  f32_to_bf16_bits(v[2]) | f32_to_bf16_bits(v[3]) << 16};
        else
          *reinterpret_cast<v4f*>(mine + fr * pitch + o * 4) = v4f{v[0], v[1], v[2], v[3]};
      }
    lds_wave_fence();
    if (vec) {
      const int per_row = row_bytes / 16;
      for (int x = lane; x < 32 * per_row; x += 64) {
        const int r = x / per_row, c = x % per_row;
        if (mb + r < p.M && c * 16 < live_n * ob)
          *reinterpret_cast<v4u*>(static_cast<uint8_t*>(p.c) + ((mb + r) * p.N + nw) * ob + c * 16) =
              *reinterpret_cast<const v4u*>(mine + r * pitch + c * 16);
      }
    } else {
      for (int x = lane; x < 32 * Cfg::WNO; x += 64) {
        const int r = x / Cfg::WNO, c = x % Cfg::WNO;
        if (mb + r < p.M && c < live_n) {
          const int64_t at = (mb + r) * p.N + nw + c;
          if (p.out_bf16)
            static_cast<uint16_t*>(p.c)[at] = *reinterpret_cast<const uint16_t*>(mine + r * pitch + c * 2);
          else
            static_cast<float*>(p.c)[at] = *reinterpret_cast<const float*>(mine + r * pitch + c * 4);
        }
      }
    }
    lds_wave_fence();
  }
}

template <class Cfg>
__global__ __launch_bounds__(Cfg::THREADS) void i8_tile_kernel(const I8Args p) {
  // One array for the ring and the columns' scales behind it: with two, the
  // compiler drains every load in flight before the ring's first read.
  __shared__ __attribute__((aligned(16))) uint8_t smem[Cfg::LDS + Cfg::NWAVES * Cfg::WN * 8];
  i8_tile<Cfg>(p, smem);
}

template <class Cfg>
static hipError_t launch_tiles(I8Args p, hipStream_t stream) {
  const int64_t tiles_m = (p.M + Cfg::BM - 1) / Cfg::BM, tiles_n = (p.N + Cfg::OBN - 1) / Cfg::OBN;
  if (tiles_m * tiles_n > 0x7FFFFFFF) return hipErrorInvalidValue;
  p.tiles_n = (int)tiles_n;
  hipLaunchKernelGGL(i8_tile_kernel<Cfg>, dim3((unsigned)(tiles_m * tiles_n)), dim3(Cfg::THREADS), 0,
                     stream, p);
  return hipGetLastError();
}

template <bool GATED>
static hipError_t launch_tile(const I8Args& p, int tile, hipStream_t stream) {
  return tile == 256   ? launch_tiles<I8Cfg<256, 256, 2, 2, 4, GATED>>(p, stream)
         : tile == 128 ? launch_tiles<I8Cfg<128, 128, 2, 2, 4, GATED>>(p, stream)
                       : launch_tiles<I8Cfg<64, 128, 2, 2, 4, GATED>>(p, stream);
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
  p.out_bf16 = out_bf16;
  return gated ? launch_tile<true>(p, tile, stream) : launch_tile<false>(p, tile, stream);
}

hipError_t launch_i8_few(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s,
                         const float* bias, int64_t M, int64_t N, int64_t K, bool gated, int act,
                         void* c, int out_bf16, hipStream_t stream);

static hipError_t launch_i8(const int8_t* a_q, const float* a_s, const int8_t* w_q,
                            const float* w_s, const float* bias, int64_t M, int64_t N, int64_t K,
                            bool gated, int act, void* c, int out_bf16, hipStream_t stream) {
  if (M <= 64)
    return launch_i8_few(a_q, a_s, w_q, w_s, bias, M, N, K, gated, act, c, out_bf16, stream);
  return launch_i8_tiles(a_q, a_s, w_q, w_s, bias, M, N, K, gated, act, c, out_bf16, 256, stream);
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
