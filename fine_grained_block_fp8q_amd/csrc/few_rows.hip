// Products for few activation rows (decoding): 8-bit weights streamed once
// from memory into registers, and the whole feed-forward epilogue behind them.
//
//   int8:  Y[m][n] = (sum_k a[m][k] w[n][k]) a_s[m] w_s[n] (+ bias[n])
//   E4M3:  Y[m][n] = sum_g a_s[g][m] w_s[n/128][g] sum_{k in chunk g} a[m][k] w[n][k]
//   gated: h[m][f] = act(Y[m][f]) Y[m][F + f]
//
// At few rows the time is that of reading the weights, so nothing is shared
// through LDS on the way in: a workgroup owns 16 weight rows (8 gate and the
// 8 matching up rows when gated), its 8 waves split K in turns of 128, and a
// lane loads its operand of the matrix instruction straight from memory, 16
// bytes at a time.  4096 weight rows are then 256 workgroups, one for each CU,
// with all of a 7168-long row block in flight at once.  The 8 partial sums meet
// in LDS, in a fixed order; the int8 ones are exact in any order.
//
// The activation rows are read again by every workgroup, from the L2: at 16
// weight rows that is as many bytes as the weights for 16 activation rows,
// which the L2 delivers beside the memory stream.

#include <type_traits>

#include "activation.hpp"

namespace fp8q {

constexpr int kFewI8 = 0, kFewE4M3 = 1;
constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * 64;
constexpr int kFewChunk = 128;  // K of one wave's turn

struct FewArgs {
  const uint8_t* a;
  const float* a_s;    // int8: [M]; E4M3: [K/128][M]
  const uint8_t* w;    // [N][K] or [G][2F][K]
  const float* w_s;    // int8: [N]; E4M3: [N/128][K/128]
  const float* bias;   // int8, not gated: [N] or NULL
  const int32_t* off;  // by expert: [G + 1], else NULL
  void* c;             // [M][N], or h [M][F]
  uint16_t* gu;        // gated: Y as BF16 [M][2F], or NULL
  int64_t M, N, K;     // N: output columns (F when gated)
  int G;
  int n_blocks;        // column blocks
  int out_bf16, act;
};

#ifdef FP8Q_DEBUG_CHECKS
// Set by a launch by expert that found invalid offsets (debug builds): read
// and cleared by the host entry point after its synchronization.
__device__ int g_gated_offsets_error = 0;

hipError_t gated_offsets_error_take(hipStream_t stream, int* flag) {
  const int zero = 0;
  hipError_t e = hipMemcpyFromSymbolAsync(flag, HIP_SYMBOL(g_gated_offsets_error), sizeof(int), 0,
                                          hipMemcpyDeviceToHost, stream);
  if (e == hipSuccess) e = hipStreamSynchronize(stream);
  if (e == hipSuccess && *flag)
    e = hipMemcpyToSymbol(HIP_SYMBOL(g_gated_offsets_error), &zero, sizeof(int), 0,
                          hipMemcpyHostToDevice);
  return e;
}
#endif

// Rows of block `y` of BM rows when rows are grouped by expert: the expert's
// blocks follow those of the experts before it.  Every lane gets the same
// answer.  False where there is no such block, or the offsets are not
// 0 = off[0] <= ... <= off[G] <= M (then no block has any: nothing is written).
__device__ __forceinline__ bool find_rows(const int32_t* off, int G, int64_t M, int BM, int y,
                                          int& e, int64_t& r0, int64_t& r1) {
  const int lane = threadIdx.x & 63;
  bool bad = lane == 0 && (off[0] != 0 || (int64_t)off[G] > M);
  int before = 0, at = -1, lo_at = 0, hi_at = 0, blk = 0;
  for (int base = 0; base < G; base += 64) {
    const int i = base + lane;
    const int lo = i < G ? off[i] : 0, hi = i < G ? off[i + 1] : 0;
    bad = bad || hi < lo;
    const int n = hi > lo ? (hi - lo + BM - 1) / BM : 0;
    int inc = n;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(inc, d);
      if (lane >= d) inc += v;
    }
    const int first = before + inc - n;
    const uint64_t hit = __ballot(y >= first && y < first + n);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);
      at = base + l;
      lo_at = __shfl(lo, l);
      hi_at = __shfl(hi, l);
      blk = y - __shfl(first, l);
    }
    before += __shfl(inc, 63);
  }
  if (__ballot(bad) != 0) {
#ifdef FP8Q_DEBUG_CHECKS
    if (blockIdx.x == 0 && threadIdx.x == 0) g_gated_offsets_error = 1;
#endif
    return false;
  }
  if (at < 0) return false;
  e = __builtin_amdgcn_readfirstlane(at);
  r0 = lo_at + (int64_t)blk * BM;
  r1 = hi_at;
  return true;
}

// One chunk's operands of a lane: bytes [16q, 16q+16) and [64+16q, 64+16q+16)
// of the 128, for its weight row and its row of each activation block.
template <int MB>
struct FewOperands {
  v4i w[2];
  v4i a[MB][2];
};

template <int OP, int MB, bool GATED, bool GROUPED>
__global__ __launch_bounds__(kFewThreads) void few_rows_kernel(const FewArgs p) {
  constexpr int BM = 16 * MB;
  constexpr int U = MB == 1 ? 4 : 2;  // chunks in a batch; two batches are in flight
  constexpr bool I8 = OP == kFewI8;
  using Acc = typename std::conditional<I8, v4i, v4f>::type;
  __shared__ __attribute__((aligned(16))) float red[kFewWaves * MB * 256];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int nb = blockIdx.x % p.n_blocks, mb = blockIdx.x / p.n_blocks;

  int64_t r0 = (int64_t)mb * BM, r1 = p.M;
  const uint8_t* W = p.w;
  const float* WS = p.w_s;
  const int64_t K = p.K, N = p.N;
  const int64_t WR = GATED ? 2 * N : N;  // weight rows
  const int64_t KB = K / kFewChunk;      // E4M3: whole chunks
  if constexpr (GROUPED) {
    int e;
    if (!find_rows(p.off, p.G, p.M, BM, mb, e, r0, r1)) return;
    W += (int64_t)e * WR * K;
    WS += I8 ? (int64_t)e * WR : (int64_t)e * (WR / 128) * KB;
  }

  // this lane's weight row: row r16 of the block
  constexpr int NCOL = GATED ? 8 : 16;  // output columns of the block
  const int64_t n0 = (int64_t)nb * NCOL;
  int64_t col = n0 + (GATED ? (r16 & 7) : r16);
  col = col < N ? col : N - 1;
  const uint8_t* wp = W + (col + (GATED && r16 >= 8 ? N : 0)) * K + 16 * q;
  const uint8_t* ap[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int64_t m = r0 + 16 * i + r16;
    ap[i] = p.a + (m < r1 ? m : r1 - 1) * K + 16 * q;
  }

  const int chunks = (int)((K + kFewChunk - 1) / kFewChunk);
  const int mine = (chunks - wave + kFewWaves - 1) / kFewWaves;
  // Chunk i of this wave.  Past the wave's last chunk, and for 16-byte pieces
  // past K, the weights are read from the row's start and the activations
  // taken as zero.
  auto load = [&](FewOperands<MB>& o, int i) {
    const int64_t k = ((int64_t)i * kFewWaves + wave) * kFewChunk;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t kh = k + 64 * h;
      const bool in = i < mine && kh + 16 * q < K;
      const int64_t ks = in ? kh : 0;
      o.w[h] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(in ? wp + kh : wp - 16 * q));
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        o.a[b][h] = *reinterpret_cast<const v4i*>(in ? ap[b] + ks : ap[b] - 16 * q);
        if (!in) o.a[b][h] = v4i{0, 0, 0, 0};
      }
    }
  };

  Acc acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = Acc{0, 0, 0, 0};
  // E4M3: the scales of this lane's 4 results, which share one activation row
  // and (F is a multiple of 128) one weight block row
  const float* sw = nullptr;
  const float* sa = nullptr;
  if constexpr (!I8) {
    const int64_t blk_row = GATED ? n0 + (q >= 2 ? N : 0) : n0;
    sw = WS + blk_row / 128 * KB;
    sa = p.a_s;
  }
  auto multiply = [&](const FewOperands<MB>& o, int i) {
    if constexpr (I8) {
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(o.w[h], o.a[b][h], acc[b], 0, 0, 0);
    } else {
      const int g = i * kFewWaves + wave;
      const int gs = i < mine ? g : 0;  // past the end the partial is zero
      const float s_w = sw[gs];
      const v8i w = {o.w[0][0], o.w[0][1], o.w[0][2], o.w[0][3],
                     o.w[1][0], o.w[1][1], o.w[1][2], o.w[1][3]};
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const v8i a = {o.a[b][0][0], o.a[b][0][1], o.a[b][0][2], o.a[b][0][3],
                       o.a[b][1][0], o.a[b][1][1], o.a[b][1][2], o.a[b][1][3]};
        const v4f P = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            w, a, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
        const int64_t m = r0 + 16 * b + r16;
        const float s = sa[(int64_t)gs * p.M + (m < r1 ? m : r1 - 1)] * s_w;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[b][j] = __builtin_fmaf(P[j], s, acc[b][j]);
      }
    }
  };

  FewOperands<MB> x[U], y[U];
#pragma unroll
  for (int u = 0; u < U; ++u) load(x[u], u);
  for (int i = 0; i < mine; i += 2 * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(y[u], i + U + u);
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(x[u], i + u);
    if (i + U >= mine) break;
#pragma unroll
    for (int u = 0; u < U; ++u) load(x[u], i + 2 * U + u);
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(y[u], i + U + u);
  }

  // partial sums: red[wave][block][lane][4]
#pragma unroll
  for (int b = 0; b < MB; ++b)
    *reinterpret_cast<Acc*>(red + ((wave * MB + b) * 64 + lane) * 4) = acc[b];
  __syncthreads();
  // sum over the waves of weight row r, activation row m of the block
  auto total = [&](int m, int r) {
    const int at = ((m >> 4) * 64 + (r >> 2) * 16 + (m & 15)) * 4 + (r & 3);
    if constexpr (I8) {
      int s = 0;
#pragma unroll
      for (int v = 0; v < kFewWaves; ++v) s += reinterpret_cast<const int*>(red)[v * MB * 256 + at];
      return s;
    } else {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kFewWaves; ++v) s += red[v * MB * 256 + at];
      return s;
    }
  };
  auto store = [&](void* dst, int64_t at, float v, int bf16) {
    if (bf16)
      static_cast<uint16_t*>(dst)[at] = (uint16_t)f32_to_bf16_bits(v);
    else
      static_cast<float*>(dst)[at] = v;
  };
  for (int i = tid; i < BM * NCOL; i += kFewThreads) {
    const int m = i / NCOL, c = i % NCOL;
    const int64_t row = r0 + m, n = n0 + c;
    if (row >= r1 || n >= N) continue;
    if constexpr (GATED) {
      float g, u;
      if constexpr (I8) {
        const float s = p.a_s[row];
        g = (float)total(m, c) * s * WS[n];
        u = (float)total(m, c + 8) * s * WS[N + n];
      } else {
        g = total(m, c);
        u = total(m, c + 8);
      }
      store(p.c, row * N + n, act_fast(p.act, g) * u, p.out_bf16);
      if (p.gu) {
        store(p.gu, row * 2 * N + n, g, 1);
        store(p.gu, row * 2 * N + N + n, u, 1);
      }
    } else {
      float v = (float)total(m, c) * p.a_s[row] * WS[n];
      if (p.bias) v += p.bias[n];
      store(p.c, row * N + n, v, p.out_bf16);
    }
  }
}

template <int OP, bool GATED, bool GROUPED>
static hipError_t launch_few(FewArgs p, int64_t row_blocks_extra, hipStream_t stream) {
  constexpr int NCOL = GATED ? 8 : 16;
  const int64_t n_blocks = (p.N + NCOL - 1) / NCOL;
  const int MB = p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4;
  // by expert: sum_e ceil(M_e / BM) <= floor(M / BM) + G
  const int64_t m_blocks = (p.M + 16 * MB - 1) / (16 * MB) + row_blocks_extra;
  if (n_blocks * m_blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  p.n_blocks = (int)n_blocks;
  auto kern = MB == 1   ? few_rows_kernel<OP, 1, GATED, GROUPED>
              : MB == 2 ? few_rows_kernel<OP, 2, GATED, GROUPED>
                        : few_rows_kernel<OP, 4, GATED, GROUPED>;
  hipLaunchKernelGGL(kern, dim3((unsigned)(n_blocks * m_blocks)), dim3(kFewThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_i8_few(const int8_t* a_q, const float* a_s, const int8_t* w_q, const float* w_s,
                         const float* bias, int64_t M, int64_t N, int64_t K, bool gated, int act,
                         void* c, int out_bf16, hipStream_t stream) {
  FewArgs p{};
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
  return gated ? launch_few<kFewI8, true, false>(p, 0, stream)
               : launch_few<kFewI8, false, false>(p, 0, stream);
}

// off NULL: one dense block of weights; else G experts.
hipError_t launch_gemm_gated(const uint8_t* a_q, const float* a_s, int64_t M, const int32_t* off,
                             int G, const uint8_t* w_q, const float* w_s, int64_t F, int64_t K,
                             int act, void* h, int out_bf16, void* gu, hipStream_t stream) {
  FewArgs p{};
  p.a = a_q;
  p.a_s = a_s;
  p.w = w_q;
  p.w_s = w_s;
  p.off = off;
  p.G = G;
  p.c = h;
  p.gu = static_cast<uint16_t*>(gu);
  p.M = M;
  p.N = F;
  p.K = K;
  p.act = act;
  p.out_bf16 = out_bf16;
  if (off) return launch_few<kFewE4M3, true, true>(p, G, stream);
  return launch_few<kFewE4M3, true, false>(p, 0, stream);
}

}  // namespace fp8q
