// Activations grouped by expert, quantized along the tokens: x[M][K] -> codes of
// x^T [K][T] and scales [T/128][K], in groups of 128 tokens that never straddle
// experts (experts.hpp); T is 128 times the most groups that M rows in G experts
// can take.  Columns past an expert's last row, and past the last expert, get
// zero codes, groups past the last expert zero scales too.
//
// The tile of quantize_act_t: 128 tokens x 64 columns a workgroup, the column's
// maximum over the lane's 4 rows, the wave and the 4 waves, the codes through a
// transposed copy in LDS.  Bound by memory (2 bytes read, 1 written).

#include "experts.hpp"
#include "fp8q.h"
#include "gemm_common.hpp"
#include "launch.hpp"
#include "quant_rules.hpp"

namespace fp8q {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kEtThreads = 256, kEtRow = 144;  // bytes of a row of the tile in LDS

__device__ __forceinline__ float bf16_elem(const v4u& v, int j) {
  return (j & 1) ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
}

template <int MODE>
__global__ __launch_bounds__(kEtThreads) void expert_tokens_kernel(
    const uint16_t* __restrict__ x, int64_t M, int64_t K, const int32_t* __restrict__ off, int G,
    uint8_t* __restrict__ qt, float* __restrict__ st, int64_t T, int n_kblk) {
  __shared__ float red[4][64];
  __shared__ __attribute__((aligned(16))) uint8_t tile[64 * kEtRow];
  const int kb = (int)(blockIdx.x % n_kblk), gb = (int)(blockIdx.x / n_kblk);
  const ExpertSpan span = expert_span<true>(off, G, M, T / 128, gb);
  if (invalid(span)) return;
  const int t = threadIdx.x, rq = t >> 3, cp = t & 7, wave = t >> 6;
  const int k0 = kb * 64;
  // (rows past the group's are out of the resource's range: zeros)
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(x + (int64_t)span.first * K, (int64_t)span.rows * K * 2);
  v4u v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __builtin_amdgcn_raw_buffer_load_b128(
        rx, (uint32_t)((4 * rq + i) * K + k0 + 8 * cp) * 2u, 0, 0);
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
    for (int j = 0; j < 8; ++j) red[wave][8 * cp + j] = a[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = 8 * cp + j;
    const GroupRule r =
        group_rule<MODE>(fmaxf(fmaxf(red[0][c], red[1][c]), fmaxf(red[2][c], red[3][c])));
    if (rq == 0) st[(int64_t)gb * K + k0 + c] = r.s;
    *reinterpret_cast<uint32_t*>(tile + c * kEtRow + 4 * rq) =
        pack_e4m3x4(apply<MODE>(bf16_elem(v[0], j), r), apply<MODE>(bf16_elem(v[1], j), r),
                    apply<MODE>(bf16_elem(v[2], j), r), apply<MODE>(bf16_elem(v[3], j), r));
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int p = t + kEtThreads * u, row = p >> 3, piece = p & 7;
    __builtin_nontemporal_store(
        *reinterpret_cast<const v4u*>(tile + row * kEtRow + 16 * piece),
        reinterpret_cast<v4u*>(qt + (int64_t)(k0 + row) * T + (int64_t)gb * 128 + 16 * piece));
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
  const int64_t groups = expert_groups_most(M, G), n_kblk = K / 64;
  if (groups == 0 || n_kblk == 0) return hipSuccess;
  if (groups > max_blocks(kEtThreads) / n_kblk) return hipErrorInvalidValue;
  auto kern = mode == 0 ? expert_tokens_kernel<0> : expert_tokens_kernel<1>;
  hipLaunchKernelGGL(kern, dim3((unsigned)(groups * n_kblk)), dim3(kEtThreads), 0, stream,
                     static_cast<const uint16_t*>(x), M, K, off, G, qt, st, 128 * groups,
                     (int)n_kblk);
  return hipGetLastError();
}

}  // namespace fp8q
