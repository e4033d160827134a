// Backward pass of the gated activation, quantized for the two gradient GEMMs.
//
// For h = act(gate) * up with Y = [gate | up] = X W^T:
//   dgate = dh * up * act'(gate),   dup = dh * act(gate),   dY = [dgate | dup];
//   dX = dY W     takes dY in 1x128 groups along the 2F features (q, s),
//   dW = dY^T X   takes dY^T in groups of 128 tokens             (qt, st).
// Both forms come from one pass: dh, gate and up are read once (6 bytes a
// feature), dY stays in FP32 registers and is never rounded to BF16, and each
// form of its codes is written once (2 + 2 bytes): bound by memory.
//
// A workgroup of 512 lanes takes 128 tokens x 128 features, so that it holds
// whole groups in both directions.  Lane (rq = t/16, l16 = t%16) owns tokens
// 4rq .. 4rq+3 at features 8 l16 .. 8 l16 + 7.  A row group's maximum is one
// DPP row's; a column group's goes over the lane's 4 tokens, the wave's 4 rq
// (shuffles) and the 8 waves (LDS).  The lane's 4 tokens of one feature are one
// word of the transposed codes, which are gathered in LDS and stored 128 bytes
// (a feature's group of tokens) to 8 lanes.
//
// Tokens past M count as zeros: the last group of tokens is a full one, and its
// codes past M are zero.

#include "activation.hpp"
#include "quant_rules.hpp"

namespace fp8q {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kBwThreads = 512;

__device__ __forceinline__ float bf16_elem(const uint4& v, int j) {
  const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
  return (j & 1) ? bf16_hi(w) : bf16_lo(w);
}

// LDS byte of token word rq (tokens 4rq..4rq+3) of feature c in a transposed
// tile: rows of 128 bytes whose 16-byte pieces are exchanged by the feature's
// octet, so that the 16 l16 of a wave write 8 different pieces.
__device__ __forceinline__ int tile_at(int c, int rq) {
  return c * 128 + (((rq >> 2) ^ (c >> 3)) & 7) * 16 + (rq & 3) * 4;
}

template <int MODE>
__global__ __launch_bounds__(kBwThreads) void gated_backward_kernel(
    const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gu, int64_t M, int64_t F, int act,
    uint8_t* __restrict__ q, float* __restrict__ s, uint8_t* __restrict__ qt,
    float* __restrict__ st, int64_t Mp, int n_fblk) {
  __shared__ float colmax[8][2][128];
  __shared__ GroupRule colrule[2][128];
  __shared__ __attribute__((aligned(16))) uint8_t tile[2][128 * 128];
  const int fb = blockIdx.x % n_fblk;
  const int64_t tb = blockIdx.x / n_fblk;
  const int t = threadIdx.x, l16 = t & 15, rq = t >> 4, wave = t >> 6;
  const int64_t m0 = tb * kGroup + 4 * rq;
  const int64_t f0 = (int64_t)fb * kGroup + 8 * l16;

  uint4 vd[4], vg[4], vu[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + i;
    if (m < M) {
      vd[i] = *reinterpret_cast<const uint4*>(dh + m * F + f0);
      vg[i] = *reinterpret_cast<const uint4*>(gu + m * 2 * F + f0);
      vu[i] = *reinterpret_cast<const uint4*>(gu + m * 2 * F + F + f0);
    } else {
      vd[i] = vg[i] = vu[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  float d[2][4][8];  // dgate, dup
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = bf16_elem(vd[i], j);
      float a, da;
      act_and_grad(act, bf16_elem(vg[i], j), a, da);
      d[0][i][j] = x * bf16_elem(vu[i], j) * da;
      d[1][i][j] = x * a;
    }

  if (q) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(d[h][i][j]));
        const GroupRule r = group_rule<MODE>(row16_max(a));
        const int64_t m = m0 + i;
        if (m < M) {
          const float* v = d[h][i];
          const v2u o = {pack_e4m3x4(apply<MODE>(v[0], r), apply<MODE>(v[1], r),
                                     apply<MODE>(v[2], r), apply<MODE>(v[3], r)),
                         pack_e4m3x4(apply<MODE>(v[4], r), apply<MODE>(v[5], r),
                                     apply<MODE>(v[6], r), apply<MODE>(v[7], r))};
          __builtin_nontemporal_store(o, reinterpret_cast<v2u*>(q + m * 2 * F + h * F + f0));
          if (l16 == 0) s[(h * (F / kGroup) + fb) * M + m] = r.s;
        }
      }
  }
  if (!qt) return;

#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a = fmaxf(fmaxf(fabsf(d[h][0][j]), fabsf(d[h][1][j])),
                      fmaxf(fabsf(d[h][2][j]), fabsf(d[h][3][j])));
      a = fmaxf(a, __shfl_xor(a, 16));
      a = fmaxf(a, __shfl_xor(a, 32));
      if ((t & 63) < 16) colmax[wave][h][8 * l16 + j] = a;
    }
  __syncthreads();
  if (t < 256) {
    const int h = t >> 7, c = t & 127;
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) a = fmaxf(a, colmax[w][h][c]);
    const GroupRule r = group_rule<MODE>(a);
    colrule[h][c] = r;
    st[tb * 2 * F + h * F + (int64_t)fb * kGroup + c] = r.s;
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const GroupRule r = colrule[h][8 * l16 + j];
      const uint32_t w = pack_e4m3x4(apply<MODE>(d[h][0][j], r), apply<MODE>(d[h][1][j], r),
                                     apply<MODE>(d[h][2][j], r), apply<MODE>(d[h][3][j], r));
      *reinterpret_cast<uint32_t*>(tile[h] + tile_at(8 * l16 + j, rq)) = w;
    }
  __syncthreads();
  // 2 x 128 features x 8 pieces of 16 tokens, 4 per lane
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int p = t + kBwThreads * u;
    const int h = p >> 10, c = (p >> 3) & 127, piece = p & 7;
    const v4u o = *reinterpret_cast<const v4u*>(tile[h] + tile_at(c, 4 * piece));
    __builtin_nontemporal_store(
        o, reinterpret_cast<v4u*>(qt + (h * F + (int64_t)fb * kGroup + c) * Mp + tb * kGroup +
                                  16 * piece));
  }
}

hipError_t launch_gated_backward(const void* dh, const void* gu, int64_t M, int64_t F, int act,
                                 int mode, uint8_t* q, float* s, uint8_t* qt, float* st,
                                 hipStream_t stream) {
  const int64_t n_fblk = F / kGroup, tb = (M + kGroup - 1) / kGroup;
  if (n_fblk * tb > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = mode == 0 ? gated_backward_kernel<0> : gated_backward_kernel<1>;
  hipLaunchKernelGGL(kern, dim3((unsigned)(n_fblk * tb)), dim3(kBwThreads), 0, stream,
                     static_cast<const uint16_t*>(dh), static_cast<const uint16_t*>(gu), M, F, act,
                     q, s, qt, st, tb * kGroup, (int)n_fblk);
  return hipGetLastError();
}

}  // namespace fp8q
