// Layer norm over the rows of x[M][N], and its backward pass.
//
//   z = (x - mean) rstd,  y = z weight + bias,  rstd = 1 / sqrt(var + eps);
//   gz = dy weight,  dx = rstd (gz - mean(gz) - z mean(gz z)),
//   dweight = sum over rows of dy z,  dbias = sum over rows of dy.
//
// A row stays in registers (LPR lanes, NV pieces of 8 consecutive elements each):
// it is read once, its variance is taken about its mean in a second pass over
// the registers, and y leaves as E4M3 codes (128 consecutive elements are one DPP
// row of 16 lanes, so a group's maximum costs four instructions), as BF16 or
// FP32, or both: bound by memory.  The codes are those of y in FP32, not of its
// BF16 rounding.
//
// Backward: each workgroup walks rows and keeps its columns' sums of dy z and dy
// in registers; they go to a workspace, one row of it a workgroup, which a second
// kernel adds up in a fixed order (no atomics: the same bits every time).

#include <type_traits>

#include "fp8q.h"
#include "launch.hpp"
#include "quant_rules.hpp"

namespace fp8q {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
// 16 bytes at any element's address: rows of odd N start anywhere
typedef v4u v4u_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

struct Row8 {
  float v[8];
};

// Elements 8c .. 8c+7 of a row of n; those past the row are 0.
template <bool BF16>
__device__ __forceinline__ Row8 load8(const void* row, int c, int n) {
  Row8 r;
  const int i = 8 * c;
  if (i + 8 <= n) {
    if constexpr (BF16) {
      const v4u w = *reinterpret_cast<const v4u_any*>(static_cast<const uint16_t*>(row) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r.v[2 * j] = bf16_lo(w[j]);
        r.v[2 * j + 1] = bf16_hi(w[j]);
      }
    } else {
      const v4f a = *reinterpret_cast<const v4f_any*>(static_cast<const float*>(row) + i);
      const v4f b = *reinterpret_cast<const v4f_any*>(static_cast<const float*>(row) + i + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r.v[j] = a[j];
        r.v[4 + j] = b[j];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r.v[j] = 0.f;
      if (i + j < n) {
        if constexpr (BF16)
          r.v[j] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(row)[i + j] << 16);
        else
          r.v[j] = static_cast<const float*>(row)[i + j];
      }
    }
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ void store8(void* row, int c, int n, const Row8& r) {
  const int i = 8 * c;
  if (i + 8 <= n) {
    if constexpr (BF16) {
      v4u w;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = f32_to_bf16_bits(r.v[2 * j]) | (f32_to_bf16_bits(r.v[2 * j + 1]) << 16);
      *reinterpret_cast<v4u_any*>(static_cast<uint16_t*>(row) + i) = w;
    } else {
      *reinterpret_cast<v4f_any*>(static_cast<float*>(row) + i) =
          v4f{r.v[0], r.v[1], r.v[2], r.v[3]};
      *reinterpret_cast<v4f_any*>(static_cast<float*>(row) + i + 4) =
          v4f{r.v[4], r.v[5], r.v[6], r.v[7]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) {
        if constexpr (BF16)
          static_cast<uint16_t*>(row)[i + j] = (uint16_t)f32_to_bf16_bits(r.v[j]);
        else
          static_cast<float*>(row)[i + j] = r.v[j];
      }
  }
}

template <class T>
__device__ __forceinline__ T* row_at(T* base, int64_t row, int64_t n, bool bf16) {
  return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(base) + row * n * (bf16 ? 2 : 4));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sums of K values over the LPR lanes of a row; every lane gets them.  `red`
// holds K values of each wave; calls alternate between two such places.
template <int LPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*red)[16]) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
  if constexpr (LPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[k][wave] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < LPR / 64; ++w) s += red[k][w];
      v[k] = s;
    }
  }
}

struct NormArgs {
  const void* x;
  const float* weight;
  const float* bias;
  int64_t M;
  int N;
  float eps;
  void* y;
  int y_bf16;
  uint8_t* q;
  float* s;
  int mode;
  float* mean;
  float* rstd;
};

template <int LPR>
constexpr int kRowThreads = LPR < 256 ? 256 : LPR;

template <int MODE>
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t row, int c, const Row8& y) {
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y.v[j]));
  const GroupRule r = group_rule<MODE>(row16_max(amax));
  const v2u o = {pack_e4m3x4(apply<MODE>(y.v[0], r), apply<MODE>(y.v[1], r), apply<MODE>(y.v[2], r),
                             apply<MODE>(y.v[3], r)),
                 pack_e4m3x4(apply<MODE>(y.v[4], r), apply<MODE>(y.v[5], r), apply<MODE>(y.v[6], r),
                             apply<MODE>(y.v[7], r))};
  *reinterpret_cast<v2u*>(a.q + row * a.N + 8 * c) = o;
  if ((threadIdx.x & 15) == 0) a.s[(int64_t)(c >> 4) * a.M + row] = r.s;
}

template <bool X_BF16, int LPR, int NV>
__global__ __launch_bounds__(kRowThreads<LPR>) void layer_norm_kernel(const NormArgs a) {
  __shared__ float red[2][1][16];
  constexpr int RPW = kRowThreads<LPR> / LPR;
  const int l = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / LPR;
  if (RPW > 1 && row >= a.M) return;  // (whole waves, and no barrier follows)
  const int N = a.N;
  const void* x = row_at(a.x, row, N, X_BF16);
  Row8 v[NV];
  float sum[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    v[j] = load8<X_BF16>(x, l + LPR * j, N);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[0] += v[j].v[k];
  }
  row_sum<LPR, 1>(sum, red[0]);
  const float mean = sum[0] / (float)N;
  float sq[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = 8 * (l + LPR * j) + k < N ? v[j].v[k] - mean : 0.f;
      v[j].v[k] = d;
      sq[0] = __builtin_fmaf(d, d, sq[0]);
    }
  row_sum<LPR, 1>(sq, red[1]);
  const float rstd = 1.f / __builtin_sqrtf(sq[0] / (float)N + a.eps);
  if (l == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = l + LPR * j;
    if (8 * c >= N) continue;
    const Row8 w = load8<false>(a.weight, c, N);
    Row8 y;
    if (a.bias) {
      const Row8 b = load8<false>(a.bias, c, N);
#pragma unroll
      for (int k = 0; k < 8; ++k) y.v[k] = __builtin_fmaf(v[j].v[k] * rstd, w.v[k], b.v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) y.v[k] = v[j].v[k] * rstd * w.v[k];
    }
    if (a.q) {
      if (a.mode == 0)
        store_codes<0>(a, row, c, y);
      else
        store_codes<1>(a, row, c, y);
    }
    if (a.y) {
      if (a.y_bf16)
        store8<true>(row_at(a.y, row, N, true), c, N, y);
      else
        store8<false>(row_at(a.y, row, N, false), c, N, y);
    }
  }
}

// ------------------------------------------------------------------ backward
constexpr int kNormBlocks = 256;  // workgroups that walk the rows: one a CU

struct NormBwArgs {
  const void* dy;
  const void* x;
  const float* weight;
  const float* mean;
  const float* rstd;
  int64_t M;
  int N;
  void* dx;
  float* part;  // [workgroups][2][N]
};

template <bool X_BF16, bool DY_BF16, int LPR, int NV>
__global__ __launch_bounds__(kRowThreads<LPR>) void layer_norm_backward_kernel(const NormBwArgs a) {
  __shared__ float red[2][2][16];
  constexpr int RPW = kRowThreads<LPR> / LPR;
  const int l = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int N = a.N;
  const float inv_n = 1.f / (float)N;
  float dw[NV][8], db[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[j][k] = db[j][k] = 0.f;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPW + sub; row < a.M; row += (int64_t)gridDim.x * RPW) {
    const void* x = row_at(a.x, row, N, X_BF16);
    const void* dy = row_at(a.dy, row, N, DY_BF16);
    const float mean = a.mean[row], rstd = a.rstd[row];
    Row8 z[NV], g[NV];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = l + LPR * j;
      z[j] = load8<X_BF16>(x, c, N);
      g[j] = load8<DY_BF16>(dy, c, N);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = l + LPR * j;
      const Row8 w = load8<false>(a.weight, c, N);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float zz = (z[j].v[k] - mean) * rstd;  // (past the row: times a 0 of dy)
        z[j].v[k] = zz;
        dw[j][k] = __builtin_fmaf(g[j].v[k], zz, dw[j][k]);
        db[j][k] += g[j].v[k];
        g[j].v[k] *= w.v[k];
        sum[0] += g[j].v[k];
        sum[1] = __builtin_fmaf(g[j].v[k], zz, sum[1]);
      }
    }
    row_sum<LPR, 2>(sum, red[turn]);
    turn ^= 1;
    const float c2 = sum[0] * inv_n, c1 = sum[1] * inv_n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = l + LPR * j;
      Row8 d;
#pragma unroll
      for (int k = 0; k < 8; ++k) d.v[k] = rstd * (g[j].v[k] - c2 - z[j].v[k] * c1);
      if (8 * c < N) store8<X_BF16>(row_at(a.dx, row, N, X_BF16), c, N, d);
    }
  }
  if constexpr (RPW > 1) {
    // the waves' sums of the same columns, one wave after the other
    __shared__ float part[2][RPW][NV][8][64];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        part[0][sub][j][k][l] = dw[j][k];
        part[1][sub][j][k][l] = db[j][k];
      }
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        for (int s = 1; s < RPW; ++s) {
          dw[j][k] += part[0][s][j][k][l];
          db[j][k] += part[1][s][j][k][l];
        }
  }
  float* out = a.part + (int64_t)blockIdx.x * 2 * N;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = l + LPR * j;
    Row8 w, b;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w.v[k] = dw[j][k];
      b.v[k] = db[j][k];
    }
    if (8 * c < N) {
      store8<false>(out, c, N, w);
      store8<false>(out + N, c, N, b);
    }
  }
}

// Column sums of part[rows][2N]: 64 columns x 4 slices of the rows a workgroup.
__global__ __launch_bounds__(256) void layer_norm_reduce_kernel(const float* __restrict__ part,
                                                                int rows, int N,
                                                                float* __restrict__ dweight,
                                                                float* __restrict__ dbias) {
  __shared__ float red[4][64];
  const int l = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + l;
  const int64_t ld = 2 * (int64_t)N;
  float s = 0.f;
  if (col < ld) {
    const int r0 = (int)((int64_t)rows * slice / 4), r1 = (int)((int64_t)rows * (slice + 1) / 4);
#pragma unroll 8
    for (int r = r0; r < r1; ++r) s += part[r * ld + col];
  }
  red[slice][l] = s;
  __syncthreads();
  if (slice != 0 || col >= ld) return;
  s = red[0][l] + red[1][l] + red[2][l] + red[3][l];
  if (col < N)
    dweight[col] = s;
  else if (dbias)
    dbias[col - N] = s;
}

// ------------------------------------------------------------------ launches
// Lanes of a row and pieces of a lane: the fewest pieces that fit the row.
template <class F>
static hipError_t by_width(int64_t N, F f) {
  const int64_t c = (N + 7) / 8;
  if (c <= 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (c <= 128) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (c <= 256) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (c <= 512) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (c <= 1024) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

hipError_t launch_layer_norm(const void* x, int x_bf16, const float* weight, const float* bias,
                             int64_t M, int64_t N, float eps, void* y, int y_bf16, uint8_t* q,
                             float* s, int mode, float* mean, float* rstd, hipStream_t stream) {
  const NormArgs a = {x, weight, bias, M, (int)N, eps, y, y_bf16, q, s, mode, mean, rstd};
  return by_width(N, [&](auto lpr, auto nv) {
    constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, T = kRowThreads<LPR>;
    const int64_t blocks = (M + T / LPR - 1) / (T / LPR);
    if (blocks > max_blocks(T)) return hipErrorInvalidValue;
    auto kern = x_bf16 ? layer_norm_kernel<true, LPR, NV> : layer_norm_kernel<false, LPR, NV>;
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(T), 0, stream, a);
    return hipGetLastError();
  });
}

static int64_t norm_backward_blocks(int64_t M, int64_t N) {
  const int64_t rpw = N <= 1024 ? 4 : 1;
  const int64_t all = (M + rpw - 1) / rpw;
  return all < kNormBlocks ? all : kNormBlocks;
}

int64_t layer_norm_backward_workspace(int64_t M, int64_t N) {
  return norm_backward_blocks(M, N) * 2 * N * 4;
}

hipError_t launch_layer_norm_backward(const void* dy, int dy_bf16, const void* x, int x_bf16,
                                      const float* weight, const float* mean, const float* rstd,
                                      int64_t M, int64_t N, void* dx, float* dweight, float* dbias,
                                      float* workspace, hipStream_t stream) {
  const NormBwArgs a = {dy, x, weight, mean, rstd, M, (int)N, dx, workspace};
  const int blocks = (int)norm_backward_blocks(M, N);
  const hipError_t e = blocks == 0 ? hipSuccess : by_width(N, [&](auto lpr, auto nv) {
    constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value;
    auto kern = x_bf16 ? (dy_bf16 ? layer_norm_backward_kernel<true, true, LPR, NV>
                                  : layer_norm_backward_kernel<true, false, LPR, NV>)
                       : (dy_bf16 ? layer_norm_backward_kernel<false, true, LPR, NV>
                                  : layer_norm_backward_kernel<false, false, LPR, NV>);
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kRowThreads<LPR>), 0, stream, a);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(layer_norm_reduce_kernel, dim3((unsigned)((2 * N + 63) / 64)), dim3(256), 0,
                     stream, workspace, blocks, (int)N, dweight, dbias);
  return hipGetLastError();
}

}  // namespace fp8q
