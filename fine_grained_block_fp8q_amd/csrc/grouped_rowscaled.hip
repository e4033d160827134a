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
// An expert has few tokens (128 .. 1024) for a large C, so that the call is bound
// by writing C: 128 x 128 outputs of 1 .. 8 groups each, read once from L2 and
// written once.  A workgroup of 4 waves takes such a tile (64 x 64 a wave), two
// workgroups a CU, so that one's stores go out under the other's products.  The
// groups come into LDS by direct loads, two stages; rows of 128 bytes with
// exchanged 16-byte columns (swz), so that fragment reads are free of conflicts.
// The product is formed transposed (matrix-core rows are B's rows), so that a
// lane's four results are consecutive in k.

#include "experts.hpp"
#include "fp8q.h"
#include "gemm_tile.hpp"
#include "launch.hpp"

namespace fp8q {

constexpr int kWgTile = 128, kWgThreads = 256;
constexpr int kWgOperand = kWgTile * 128;                   // bytes of one operand's group
constexpr int kWgStage = 2 * kWgOperand + 2 * kWgTile * 4;  // and both scales'
constexpr int kWgLoads = 9;  // of one wave and group: 4 + 4 KiB of operands, scales

// PRECISE: each P_g by FP16 matrix-core instructions on the codes widened to FP16.
template <bool PRECISE>
__global__ __launch_bounds__(kWgThreads, 2) void grouped_rowscaled_kernel(
    const uint8_t* __restrict__ A, const float* __restrict__ SA, const uint8_t* __restrict__ B,
    const float* __restrict__ SB, const int32_t* __restrict__ off, int G, int64_t T, int64_t N,
    int64_t K, void* __restrict__ C, int out_bf16, int tiles_k, int tiles) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * kWgStage];
  const int e = (int)(blockIdx.x / tiles), tile = (int)(blockIdx.x % tiles);
  const ExpertSpan span = expert_span<false>(off, G, 0x7FFFFFFF, T / 128, e);
  if (invalid(span)) return;
  const int groups = groups_of(span.rows);
  const int64_t n0 = (int64_t)(tile / tiles_k) * kWgTile, k0 = (int64_t)(tile % tiles_k) * kWgTile;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave >> 1, wk = wave & 1;
  const int r16 = lane & 15, q = lane >> 4;

  v4f acc[4][4];  // [16 rows of A][16 rows of B]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // Operand loads: instruction m (0 .. 15) of an operand carries rows 8m .. 8m+7,
  // lane l to LDS byte 16 l: row l/8, physical column l%8.
  const int64_t t0 = (int64_t)span.group0 * 128;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(A + n0 * T + t0, kWgTile * T - t0);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(B + k0 * T + t0, kWgTile * T - t0);
  uint32_t voff[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int r = (d * 4 + wave) * 8 + (lane >> 3);
    voff[d] = (uint32_t)(r * T) + (uint32_t)(swz(r, lane & 7) * 16);
  }
  // Scales: waves 0, 1 the 128 of A, waves 2, 3 those of B.
  const bool s_a = wave < 2;
  const float* sbase = (s_a ? SA + span.group0 * N + n0 : SB + span.group0 * K + k0) + (wave & 1) * 64;
  const int64_t s_ld = s_a ? N : K;

  auto issue = [&](int g) {
    uint8_t* const st = smem + (g & 1) * kWgStage;
#pragma unroll
    for (int d = 0; d < 4; ++d)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to_lds(st + (d * 4 + wave) * 1024), 16, voff[d],
                                               g * 128, 0, 0);
#pragma unroll
    for (int d = 0; d < 4; ++d)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, to_lds(st + kWgOperand + (d * 4 + wave) * 1024),
                                               16, voff[d], g * 128, 0, 0);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(sbase + g * s_ld, 256);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to_lds(st + 2 * kWgOperand + wave * 256), 4,
                                             (uint32_t)(lane * 4), 0, 0, 0);
  };

  if (groups > 0) issue(0);
  for (int g = 0; g < groups; ++g) {
    if (g + 1 < groups) {
      issue(g + 1);
      wait_vmcnt<kWgLoads>();
    } else {
      wait_vmcnt<0>();
    }
    lds_barrier();
    const uint8_t* const st = smem + (g & 1) * kWgStage;
    const float* const sa_s = reinterpret_cast<const float*>(st + 2 * kWgOperand);
    v8i a[4];
    float sa[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = load_frag(st, wn * 64 + i * 16 + r16, q);
      sa[i] = sa_s[wn * 64 + i * 16 + r16];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const v8i b = load_frag(st + kWgOperand, wk * 64 + j * 16 + r16, q);
      const v4f sb = *reinterpret_cast<const v4f*>(sa_s + 128 + wk * 64 + j * 16 + 4 * q);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v4f p = {0.f, 0.f, 0.f, 0.f};
        if constexpr (PRECISE) {
#pragma unroll
          for (int h = 0; h < 4; ++h)
            p = mfma_wide16(widen_quarter(b, h), widen_quarter(a[i], h), p);
        } else {
          p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a[i], p, 0, 0, 0, 0, 0, 0);
        }
        promote_rows(acc[i][j], p, sa[i], sb);
      }
    }
    lds_barrier();  // the stage is free
  }

  // Block (i, j): the lane holds n = 16 i + r16, k = 16 j + 4 q .. +3.
  const int64_t c0 = ((int64_t)e * N + n0 + wn * 64) * K + k0 + wk * 64;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = c0 + (int64_t)(i * 16 + r16) * K + j * 16 + 4 * q;
      if (out_bf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(C) + at) =
            make_uint2(f32_to_bf16_bits(acc[i][j][0]) | (f32_to_bf16_bits(acc[i][j][1]) << 16),
                       f32_to_bf16_bits(acc[i][j][2]) | (f32_to_bf16_bits(acc[i][j][3]) << 16));
      else
        *reinterpret_cast<v4f*>(static_cast<float*>(C) + at) = acc[i][j];
    }
}

#ifdef FP8Q_DEBUG_CHECKS
hipError_t wgrad_offsets_error_take(hipStream_t stream, int* flag) {
  return take_experts_error(stream, flag);
}
#endif

hipError_t launch_grouped_gemm_rowscaled(const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                                         const float* b_s, int64_t T, const int32_t* off, int G,
                                         int64_t N, int64_t K, void* c, int out_bf16, int precise,
                                         hipStream_t stream) {
  if (N == 0 || K == 0) return hipSuccess;
  const int64_t tiles_k = K / kWgTile, tiles = N / kWgTile * tiles_k;
  if (tiles > max_blocks(kWgThreads) / G) return hipErrorInvalidValue;
  auto kern = precise ? grouped_rowscaled_kernel<true> : grouped_rowscaled_kernel<false>;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * G)), dim3(kWgThreads), 0, stream, a_q, a_s, b_q,
                     b_s, off, G, T, N, K, c, out_bf16, (int)tiles_k, (int)tiles);
  return hipGetLastError();
}

}  // namespace fp8q
