// Activations grouped by expert, quantized along the tokens: x[M][K] -> codes of
// x^T [K][T] and scales [T/128][K], in groups of 128 tokens that never straddle
// experts (experts.hpp); T is 128 times the most groups that M rows in G experts
// can take.  Columns past an expert's last row, and past the last expert, get
// zero codes, groups past the last expert zero scales too.
//
// A workgroup takes 128 tokens and, one after the other, up to kBlocks pieces of 64
// columns, the next one's values on their way while one is worked on (finding the
// group's rows from off takes as long as a piece).  As in quantize_act_t, a column's
// maximum goes over the lane's 4 rows, the wave and the 4 waves, and the codes
// through a transposed copy in LDS.  Bound by memory (2 bytes read, 1 written).
// 32768 tokens of 256 experts, K = 7168: 217 us (953 MB with the zeros, 4.4 TB/s; one
// piece a workgroup 298); 512 tokens of 8, K = 2048: 5.6 us, a launch.

#include "experts.hpp"
#include "fp8q.h"
#include "gemm_common.hpp"
#include "launch.hpp"
#include "quant_rules.hpp"

namespace fp8q {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kEtThreads = 256, kEtRow = 144;  // bytes of a row of the tile in LDS
constexpr int kBlocks = 16, kPerCu = 16, kCus = 256;

__device__ __forceinline__ float bf16_elem(const v4u& v, int j) {
  return (j & 1) ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
}

struct TokensTile {
  float red[4][64];
  uint8_t codes[64 * kEtRow];
};

template <int MODE>
__global__ __launch_bounds__(kEtThreads) void expert_tokens_kernel(
    const uint16_t* __restrict__ x, int64_t M, int64_t K, const int32_t* __restrict__ off, int G,
    uint8_t* __restrict__ qt, float* __restrict__ st, int64_t T, int n_chunk, int blocks) {
  __shared__ __attribute__((aligned(16))) TokensTile tile;
  const int k_first = (int)(blockIdx.x % n_chunk) * blocks * 64, gb = (int)(blockIdx.x / n_chunk);
  const ExpertSpan span = expert_span<true>(off, G, M, T / 128, gb);
  if (invalid(span)) return;
  const int k_end = k_first + blocks * 64 < (int)K ? k_first + blocks * 64 : (int)K;
  const int t = threadIdx.x, rq = t >> 3, cp = t & 7, wave = t >> 6;
  uint8_t* const out = qt + (int64_t)gb * 128 + 16 * cp;
  float* const out_s = st + (int64_t)gb * K;
  if (span.rows == 0) {  // past the last group: zeros
    for (int k0 = k_first; k0 < k_end; k0 += 64) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        __builtin_nontemporal_store(v4u{0, 0, 0, 0}, reinterpret_cast<v4u*>(
                                                         out + (int64_t)(k0 + 32 * u + rq) * T));
      if (t < 64) out_s[k0 + t] = 0.f;
    }
    return;
  }
  // (rows past the group's are out of the resource's range: zeros)
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(x + (int64_t)span.first * K, (int64_t)span.rows * K * 2);
  v4u next[4];
  auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      next[i] = __builtin_amdgcn_raw_buffer_load_b128(
          rx, (uint32_t)((4 * rq + i) * K + k0 + 8 * cp) * 2u, 0, 0);
  };
  load(k_first);
  for (int k0 = k_first; k0 < k_end; k0 += 64) {
    if (k0 > k_first) __syncthreads();  // the tile is free
    v4u v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = next[i];
    if (k0 + 64 < k_end) load(k0 + 64);
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = fmaxf(fmaxf(fabsf(bf16_elem(v[0], j)), fabsf(bf16_elem(v[1], j))),
                   fmaxf(fabsf(bf16_elem(v[2], j)), fabsf(bf16_elem(v[3], j))));
#pragma unroll
      for (int d = 8; d < 64; d <<= 1) a[j] = fmaxf(a[j], __shfl_xor(a[j], d));
    }
    if ((t & 63) < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) tile.red[wave][8 * cp + j] = a[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = 8 * cp + j;
      const GroupRule r = group_rule<MODE>(
          fmaxf(fmaxf(tile.red[0][c], tile.red[1][c]), fmaxf(tile.red[2][c], tile.red[3][c])));
      if (rq == 0) out_s[k0 + c] = r.s;
      *reinterpret_cast<uint32_t*>(tile.codes + c * kEtRow + 4 * rq) =
          pack_e4m3x4(apply<MODE>(bf16_elem(v[0], j), r), apply<MODE>(bf16_elem(v[1], j), r),
                      apply<MODE>(bf16_elem(v[2], j), r), apply<MODE>(bf16_elem(v[3], j), r));
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = 32 * u + rq;  // (piece cp of it)
      __builtin_nontemporal_store(*reinterpret_cast<const v4u*>(tile.codes + row * kEtRow + 16 * cp),
                                  reinterpret_cast<v4u*>(out + (int64_t)(k0 + row) * T));
    }
  }
}

#ifdef FP8Q_DEBUG_CHECKS
hipError_t tokens_offsets_error_take(hipStream_t stream, int* flag) {
  return take_experts_error(stream, flag);
}
#endif

int64_t expert_columns(int64_t M, int64_t G) { return 128 * expert_groups_most(M, G); }

hipError_t launch_grouped_quantize_act_t(const void* x, int64_t M, int64_t K, const int32_t* off,
                                         int G, uint8_t* qt, float* st, int mode,
                                         hipStream_t stream) {
  const int64_t groups = expert_groups_most(M, G);
  if (groups == 0 || K == 0) return hipSuccess;
  // As many pieces a workgroup as leave kPerCu workgroups for each CU.
  int64_t blocks = K / 64 * groups / (kCus * kPerCu);
  blocks = blocks < 1 ? 1 : blocks > kBlocks ? kBlocks : blocks;
  const int64_t n_chunk = (K / 64 + blocks - 1) / blocks;
  if (groups > max_blocks(kEtThreads) / n_chunk) return hipErrorInvalidValue;
  auto kern = mode == 0 ? expert_tokens_kernel<0> : expert_tokens_kernel<1>;
  hipLaunchKernelGGL(kern, dim3((unsigned)(groups * n_chunk)), dim3(kEtThreads), 0, stream,
                     static_cast<const uint16_t*>(x), M, K, off, G, qt, st, 128 * groups,
                     (int)n_chunk, (int)blocks);
  return hipGetLastError();
}

}  // namespace fp8q
