// Products for few activation rows (decoding): 8-bit weights streamed once
// from memory into registers, and the whole feed-forward epilogue behind them.
//
//   int8:  Y[m][n] = (sum_k a[m][k] w[n][k]) a_s[m] w_s[n] (+ bias[n])
//   E4M3:  Y[m][n] = sum_g a_s[g][m] w_s[n/128][g] sum_{k in chunk g} a[m][k] w[n][k]
//   gated: h[m][f] = act(Y[m][f]) Y[m][F + f]
//
// At few rows the time is that of reading the weights.  A workgroup owns 16
// weight rows (8 gate and the 8 matching up rows when gated), so that 4096
// weight rows are 256 workgroups, one for each CU; its 8 waves split K in turns
// of 128.  A wave brings its chunks, of the weight and of the activation rows,
// into a place of its own in LDS, 8 rows of 128 bytes a load, and waits for
// nothing but its own loads; it asks for the next chunk as soon as the last one
// is in registers, and the other waves cover the wait (rings of 2 to 4 chunks
// a wave measured the same or slower: they leave room for fewer workgroups).
// The 8 partial sums meet in LDS, in a fixed order; the int8 ones are exact in
// any order.
//
// Loaded straight into registers, the operand layout of the matrix instruction
// puts consecutive lanes on different rows, and the address unit takes a load's
// 64 lanes one at a time: 16 bytes a clock and CU.  int8, 4096 x 7168 weights,
// us for 1 / 16 / 32 / 64 rows: that way 6.9 / 8.7 / 11.6 / 18, through LDS 6.5
// / 6.9 / 7.3 / 10.2, of which 3.6 is a launch that reads next to nothing; the
// weights alone take 5.9 at the rate of a large copy.  Those are of 29 MB that
// stay in the last-level cache; the kernel alone takes 5.3 for one row of them
// and 8.2 (3.6 TB/s) when they come from HBM.
//
// The activation rows are read again by every workgroup, from the L2: from 64
// rows on that is most of what a CU loads, 80 bytes a ns.

#include <type_traits>

#include "activation.hpp"
#include "gemm_common.hpp"
#include "launch.hpp"

namespace fp8q {

constexpr int kFewI8 = 0, kFewE4M3 = 1;
constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * 64;
constexpr int kFewChunk = 128;  // K of one wave's turn

struct FewArgs {
  const uint8_t* a;
  const float* a_s;    // int8: [M]; E4M3: [K/128][M]
  const uint8_t* w;    // [N][K], or [2F][K] when gated
  const float* w_s;    // int8: [N]; E4M3: [N/128][K/128]
  const float* bias;   // int8, not gated: [N] or NULL
  void* c;             // [M][N], or h [M][F]
  uint16_t* gu;        // gated: Y as BF16 [M][2F], or NULL
  int64_t M, N, K;     // N: output columns (F when gated)
  int n_blocks;        // column blocks of this launch,
  int n_first;         // and the first of them
  int out_bf16, act;
};

// A lane offset past any block of rows, also with a scalar offset added.
constexpr uint32_t kOutOfRange = 0x80000000u;

// A wave's chunk in LDS: its 16 weight rows and its 16 MB activation rows.
template <int MB>
struct FewCfg {
  static constexpr int SLOT = 2048 * (1 + MB);
  static constexpr int LDS = kFewWaves * SLOT;  // also holds the partial sums
};

template <int OP, int MB, bool GATED>
__device__ __forceinline__ void few_rows(const FewArgs& p, uint8_t* smem) {
  constexpr int BM = 16 * MB;
  constexpr bool I8 = OP == kFewI8;
  using Acc = typename std::conditional<I8, v4i, v4f>::type;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int nb = p.n_first + blockIdx.x % p.n_blocks, mb = blockIdx.x / p.n_blocks;

  const int64_t r0 = (int64_t)mb * BM;
  const int64_t K = p.K, N = p.N;
  const int64_t KB = K / kFewChunk;  // E4M3: whole chunks

  // ---- loads: lane l of a load fetches row l/8 of its 8, physical piece l%8.
  // Rows past the block's, and pieces past K, are out of the resource's range
  // and come as zeros.
  constexpr int NCOL = GATED ? 8 : 16;  // output columns of the block
  const int64_t n0 = (int64_t)nb * NCOL;
  const int live = __builtin_amdgcn_readfirstlane(p.M - r0 < BM ? (int)(p.M - r0) : BM);
  const int cols = __builtin_amdgcn_readfirstlane(N - n0 < NCOL ? (int)(N - n0) : NCOL);
  const int ks = (int)K;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + r0 * K, (int64_t)live * K);
  // the first 8 weight rows and the second: gate and up rows when gated
  const int second = GATED ? cols : cols > 8 ? cols - 8 : 0;
  const __amdgpu_buffer_rsrc_t rw0 = make_rsrc(p.w + n0 * K, (int64_t)cols * K);
  const __amdgpu_buffer_rsrc_t rw1 = make_rsrc(p.w + (n0 + (GATED ? N : 8)) * K, (int64_t)second * K);
  const int pr = lane >> 3;
  int kc[2];
  uint32_t voff[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    kc[h] = swz(8 * h + pr, lane & 7) * 16;  // its byte within the chunk
    voff[h] = (uint32_t)(pr * ks + kc[h]);
  }
  uint8_t* const mine = smem + wave * FewCfg<MB>::SLOT;
  auto load = [&](int k) {
    uint32_t v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) v[h] = k + kc[h] < ks ? voff[h] : kOutOfRange;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw0, to_lds(mine), 16, v[0], k, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw1, to_lds(mine + 1024), 16, v[1], k, 0, 0);
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to_lds(mine + 2048 * (1 + b) + 1024 * h), 16,
                                                 v[h], k + (16 * b + 8 * h) * ks, 0, 0);
  };
  // E4M3: the scales of chunk g for this lane's results: its activation rows',
  // and of its 4 weight rows, which lie in one block row (F is a multiple of 128)
  float s_a[MB], s_w = 0.f;
  const float *sa_at = nullptr, *sw_at = nullptr;
  if constexpr (!I8) {
    sa_at = p.a_s + r0;
    sw_at = p.w_s + (n0 + (GATED && q >= 2 ? N : 0)) / 128 * KB;
  }
  auto load_scales = [&](int g) {
    const int64_t gs = g < KB ? g : 0;  // past the end the products are zeros
    s_w = sw_at[gs];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int m = 16 * b + r16;
      s_a[b] = sa_at[gs * p.M + (m < live ? m : live - 1)];
    }
  };

  Acc acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = Acc{0, 0, 0, 0};
  const int chunks = (int)((K + kFewChunk - 1) / kFewChunk);
  load(wave * kFewChunk);
  if constexpr (!I8) load_scales(wave);
  for (int g = wave; g < chunks; g += kFewWaves) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    v4i w[2], a[MB][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = *reinterpret_cast<const v4i*>(mine + r16 * 128 + swz(r16, q + 4 * h) * 16);
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        a[b][h] = *reinterpret_cast<const v4i*>(mine + 2048 * (1 + b) + r16 * 128 +
                                                swz(r16, q + 4 * h) * 16);
    float s[MB];
    if constexpr (!I8) {
#pragma unroll
      for (int b = 0; b < MB; ++b) s[b] = s_a[b] * s_w;
    }
    // the chunk is in registers: ask for the next one
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    load((g + kFewWaves) * kFewChunk);
    if constexpr (!I8) load_scales(g + kFewWaves);
    if constexpr (I8) {
#pragma unroll
      for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h], a[b][h], acc[b], 0, 0, 0);
    } else {
      const v8i wf = {w[0][0], w[0][1], w[0][2], w[0][3], w[1][0], w[1][1], w[1][2], w[1][3]};
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const v8i af = {a[b][0][0], a[b][0][1], a[b][0][2], a[b][0][3],
                        a[b][1][0], a[b][1][1], a[b][1][2], a[b][1][3]};
        const v4f P = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            wf, af, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[b][j] = __builtin_fmaf(P[j], s[b], acc[b][j]);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();  // every wave is done with its chunks
  float* const red = reinterpret_cast<float*>(smem);

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
    if (row >= p.M || n >= N) continue;
    if constexpr (GATED) {
      float g, u;
      if constexpr (I8) {
        const float s = p.a_s[row];
        g = (float)total(m, c) * s * p.w_s[n];
        u = (float)total(m, c + 8) * s * p.w_s[N + n];
      } else {
        g = total(m, c);
        u = total(m, c + 8);
      }
      const float h = (I8 && !p.out_bf16 ? act_f32(p.act, g) : act_fast(p.act, g)) * u;
      store(p.c, row * N + n, h, p.out_bf16);
      if (p.gu) {
        store(p.gu, row * 2 * N + n, g, 1);
        store(p.gu, row * 2 * N + N + n, u, 1);
      }
    } else {
      float v = (float)total(m, c) * p.a_s[row] * p.w_s[n];
      if (p.bias) v += p.bias[n];
      store(p.c, row * N + n, v, p.out_bf16);
    }
  }
}

template <int OP, int MB, bool GATED>
__global__ __launch_bounds__(kFewThreads) void few_rows_kernel(const FewArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[FewCfg<MB>::LDS];
  few_rows<OP, MB, GATED>(p, smem);
}

template <int OP, bool GATED>
static hipError_t launch_few(FewArgs p, hipStream_t stream) {
  constexpr int NCOL = GATED ? 8 : 16;
  const int64_t n_blocks = (p.N + NCOL - 1) / NCOL;
  const int MB = p.M <= 16 ? 1 : p.M <= 32 ? 2 : p.M <= 64 ? 4 : 8;
  const int64_t m_blocks = (p.M + 16 * MB - 1) / (16 * MB);
  const int64_t slice = max_blocks(kFewThreads) / m_blocks;  // column blocks a launch
  if (slice == 0 || n_blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = MB == 1   ? few_rows_kernel<OP, 1, GATED>
              : MB == 2 ? few_rows_kernel<OP, 2, GATED>
              : MB == 4 ? few_rows_kernel<OP, 4, GATED>
                        : few_rows_kernel<OP, 8, GATED>;
  for (int64_t b = 0; b < n_blocks; b += slice) {
    p.n_first = (int)b;
    p.n_blocks = (int)(n_blocks - b < slice ? n_blocks - b : slice);
    hipLaunchKernelGGL(kern, dim3((unsigned)(p.n_blocks * m_blocks)), dim3(kFewThreads), 0, stream,
                       p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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
  return gated ? launch_few<kFewI8, true>(p, stream)
               : launch_few<kFewI8, false>(p, stream);
}

hipError_t launch_gated_few(const uint8_t* a_q, const float* a_s, int64_t M, const uint8_t* w_q,
                            const float* w_s, int64_t F, int64_t K, int act, void* h, int out_bf16,
                            void* gu, hipStream_t stream) {
  FewArgs p{};
  p.a = a_q;
  p.a_s = a_s;
  p.w = w_q;
  p.w_s = w_s;
  p.c = h;
  p.gu = static_cast<uint16_t*>(gu);
  p.M = M;
  p.N = F;
  p.K = K;
  p.act = act;
  p.out_bf16 = out_bf16;
  return launch_few<kFewE4M3, true>(p, stream);
}

}  // namespace fp8q
